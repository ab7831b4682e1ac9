// linear_attention.hip -- causal linear attention with a decay for each head.
//
// Every product of the forward and the backward has one form.  With rows a_t, b_t,
// c_t and a state S (D_a x D_c),
//   out_t = scale (a_t . state),  state = sum over s <= t (s >= t if reversed) of
//           g^|t-s| b_s c_s^T + (decayed initial state)
//   forward:  a = q,   b = k,   c = v                   initial state_in
//   dq:       a = d_o, b = v,   c = k                   initial state_in^T
//   dk:       a = v,   b = d_o, c = q,   reversed       initial d_state_out^T / scale
//   dv:       a = k,   b = q,   c = d_o, reversed       initial d_state_out / scale
// Forward in time the initial state decays before the first token; reversed it does
// not before the last.  d_state_in = g scale (the state of the dv product at token 0).
#include "eq_device.h"
#include "eq_launch.h"

namespace eql {
namespace {

constexpr int kMaxD = 128;   // numbers per head
constexpr int kChunk = 64;   // tokens of one chunk
constexpr float kLog2e = 1.4426950408889634f;

struct Job {
    Heads a, b, c, out;
    int Ha, Hb, Da, Dc;  // heads of a and out, of b and c; numbers per head
    int reverse;
    float scale;
    const float* log_decay;  // min(Ha, Hb) decays
    const float* S0;         // initial and final states [batch][kv][...]: element (i, j)
    float* S1;               // at i sa + j sc
    int sa, sc;
    const int64_t* offsets;
    int64_t batch, T;
    // segments: runs of seg_len tokens (whole chunks) of a sequence, each a
    // workgroup's; part holds the state before each segment (0: one per sequence)
    int64_t seg_len, slots;
    float* part;
    int a_vec, b_vec, c_vec, out_vec;  // whole 16-byte (out: 4-element) pieces
};

__device__ __forceinline__ void sequence(const int64_t* offsets, int64_t batch, int64_t T, int64_t b, int64_t& t0,
                                         int64_t& t1) {
    if (offsets) {
        t0 = offsets[b], t1 = offsets[b + 1];
        t0 = t0 < 0 ? 0 : (t0 > T ? T : t0);
        t1 = t1 < t0 ? t0 : (t1 > T ? T : t1);
    } else {
        const int64_t n = T / batch;
        t0 = b * n, t1 = t0 + n;
    }
}

// A workgroup's part of a sequence.  Sequence b owns the slots from
// offsets[b] / seg_len + b on: at least as many as it has segments, and one if it
// is empty; a slot past its segments is idle.
struct Segment {
    int64_t b, t0, t1;  // sequence, tokens
    bool first, last;   // in time order
    bool idle;
};

__device__ __forceinline__ Segment segment_of(const Job& j, int64_t slot) {
    Segment s;
    int64_t first_slot;
    if (j.seg_len == 0) {
        s.b = slot;
        first_slot = slot;
    } else if (!j.offsets) {
        const int64_t n = j.T / j.batch, per = (n + j.seg_len - 1) / j.seg_len;
        s.b = slot / per;
        first_slot = s.b * per;
    } else {
        int64_t lo = 0, hi = j.batch - 1;  // last b whose first slot is at most `slot`
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            int64_t o = j.offsets[mid];
            o = o < 0 ? 0 : (o > j.T ? j.T : o);
            if (o / j.seg_len + mid <= slot) lo = mid;
            else hi = mid - 1;
        }
        s.b = lo;
        int64_t o = j.offsets[lo];
        o = o < 0 ? 0 : (o > j.T ? j.T : o);
        first_slot = o / j.seg_len + lo;
    }
    int64_t q0, q1;
    sequence(j.offsets, j.batch, j.T, s.b, q0, q1);
    if (j.seg_len == 0) {
        s.t0 = q0, s.t1 = q1;
        s.first = s.last = true;
        s.idle = false;
        return s;
    }
    s.t0 = q0 + (slot - first_slot) * j.seg_len;
    s.t1 = s.t0 + j.seg_len < q1 ? s.t0 + j.seg_len : q1;
    s.first = slot == first_slot;
    s.last = s.t1 == q1;
    s.idle = slot < first_slot || (s.t0 >= q1 && !s.first);
    return s;
}

// exp2(l2 n), n >= 0: 1 at n = 0 even without memory (l2 = -infinity)
__device__ __forceinline__ float power(float l2, int n) {
    return n == 0 ? 1.0f : __builtin_amdgcn_exp2f(l2 * (float)n);
}

// --- matrix-core operands of the three types ----------------------------------------
// A fragment holds, in each lane, KF numbers along the contraction: KS over the four
// lane groups kg = lane / 16, at row (column) lane % 16 of the operand; group kg has
// positions KF kg .. KF kg + KF - 1.

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

template <typename IO>
struct Op {  // __bf16, _Float16
    using F = typename Half<IO>::x8;
    static constexpr int KS = 32, KF = 8, ES = 2;
    // terms in which an fp32 number enters a product without loss of its fp32 accuracy
    static constexpr int TERMS = std::is_same_v<IO, __bf16> ? 3 : 2;
    static __device__ __forceinline__ void mma(f32x4& acc, const F& a, const F& b) {
        if constexpr (std::is_same_v<IO, __bf16>) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
        else acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, acc, 0, 0, 0);
    }
    static __device__ __forceinline__ F row(const char* p) { return *reinterpret_cast<const F*>(p); }
    // Columns of a row-major tile: contraction along its rows row0 + 8 kg + 0..7.  A
    // transposed read takes 4 rows x 4 runs of 4 columns from each group of 16 lanes
    // (lane 4r + u points at row r, run u) and hands lane 4u + v column v of run u.
    // Run u starts at column col0 + step u.
    static __device__ __forceinline__ F column(const char* tile, int pitch, int row0, int col0, int step) {
        const int lane = (int)threadIdx.x & 63, kg = lane >> 4, i = lane & 15;
        const char* p = tile + (row0 + 8 * kg + (i >> 2)) * pitch + (col0 + step * (i & 3)) * 2;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * pitch));
        return __builtin_bit_cast(F, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    static __device__ __forceinline__ float get(const F& f, int e) { return (float)f[e]; }
    // infinities and NaN as 0
    static __device__ __forceinline__ F finite(F f) {
#pragma unroll
        for (int e = 0; e < KF; ++e) f[e] = fabsf((float)f[e]) < __builtin_inff() ? f[e] : (IO)0.0f;
        return f;
    }
    // v (8 numbers) as TERMS fragments, each the rounding of what the ones before left
    template <int N>
    static __device__ __forceinline__ void split(const float (&v)[8], F (&out)[N]) {
        float r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = v[e];
#pragma unroll
        for (int t = 0; t < N; ++t) {
            u32x4 u;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                u[q] = Half<IO>::pack2(r[2 * q], r[2 * q + 1]);
                if (t + 1 < N) {
                    r[2 * q] -= Half<IO>::lo(u[q]);
                    r[2 * q + 1] -= Half<IO>::hi(u[q]);
                }
            }
            out[t] = __builtin_bit_cast(F, u);
        }
    }
    // whether a piece of memory holds an infinity or a NaN
    static __device__ __forceinline__ bool odd(const u32x4& v) {
        constexpr unsigned short top = std::is_same_v<IO, __bf16> ? 0x7f80 : 0x7c00;
        u16x2 m = {0, 0};
#pragma unroll
        for (int q = 0; q < 4; ++q) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[q] & 0x7fff7fffu));
        return m[0] >= top || m[1] >= top;
    }
};

template <>
struct Op<float> {
    using F = f32x4;
    static constexpr int KS = 16, KF = 4, ES = 4, TERMS = 1;
    static __device__ __forceinline__ void mma(f32x4& acc, const F& a, const F& b) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], acc, 0, 0, 0);
    }
    static __device__ __forceinline__ F row(const char* p) { return *reinterpret_cast<const F*>(p); }
    // column lane % 16 of the 16 that the runs name
    static __device__ __forceinline__ F column(const char* tile, int pitch, int row0, int col0, int step) {
        const int lane = (int)threadIdx.x & 63, kg = lane >> 4, i = lane & 15;
        const char* p = tile + (row0 + 4 * kg) * pitch + (col0 + step * (i >> 2) + (i & 3)) * 4;
        F f;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = *reinterpret_cast<const float*>(p + e * pitch);
        return f;
    }
    static __device__ __forceinline__ float get(const F& f, int e) { return f[e]; }
    static __device__ __forceinline__ F finite(F f) {
#pragma unroll
        for (int e = 0; e < KF; ++e) f[e] = fabsf(f[e]) < __builtin_inff() ? f[e] : 0.0f;
        return f;
    }
    template <int N>
    static __device__ __forceinline__ void split(const float (&v)[4], F (&out)[N]) {
        out[0] = F{v[0], v[1], v[2], v[3]};
    }
    static __device__ __forceinline__ bool odd(const u32x4& v) {
        bool b = false;
#pragma unroll
        for (int q = 0; q < 4; ++q) b |= (v[q] & 0x7f800000u) == 0x7f800000u;
        return b;
    }
};

// One 16-byte piece of a row: columns col .. of D, zeros past D.
template <typename IO>
__device__ __forceinline__ u32x4 load_piece(const IO* row, int col, int D, bool vec) {
    constexpr int E = 16 / (int)sizeof(IO);
    u32x4 v = {0u, 0u, 0u, 0u};
    if (col >= D) return v;
    if (vec) return *reinterpret_cast<const u32x4*>(row + col);
    if constexpr (sizeof(IO) == 2) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (col + e < D) v[e >> 1] |= (uint32_t)p[col + e] << (16 * (e & 1));
    } else {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(row);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (col + e < D) v[e] = p[col + e];
    }
    return v;
}

// The kernel's shape: D_a padded to 32 KB, D_c to 16 NW, NW waves; wave w owns
// columns 16 w .. 16 w + 15 of the state and of the output.
template <typename IO_, int KB_, int NW_>
struct Cfg {
    using IO = IO_;
    using O = Op<IO_>;
    static constexpr int ES = O::ES, KB = KB_, NW = NW_, NT = 64 * NW_;
    static constexpr int DA = 32 * KB_, DC = 16 * NW_, NB = DA / 16, NM = DA / O::KS;
    // row pitches: an odd number of 16-byte pieces, so that 16 rows spread over the banks
    static constexpr int PA = DA * ES + 16, PC = DC * ES + 16, PP = kChunk * ES + 16;
    static constexpr int NPA = (kChunk * DA * ES / 16 + NT - 1) / NT, NPC = (kChunk * DC * ES / 16 + NT - 1) / NT;
    static constexpr int OFF_B = kChunk * PA, OFF_C = 2 * kChunk * PA, OFF_P = OFF_C + kChunk * PC;
    static constexpr int OFF_FLAG = OFF_P + kChunk * PP, LDS = OFF_FLAG + 16;
};

// Row of the state that lane group kg holds as element i of block a: such that the
// blocks of one contraction step are, in order, that step's positions of the group.
template <class C>
__device__ __forceinline__ int state_row(int a, int kg, int i) {
    if constexpr (C::ES == 2) return 32 * (a >> 1) + 8 * kg + 4 * (a & 1) + i;
    else return 16 * a + 4 * kg + i;
}
// first column and step of the runs that give those rows as columns of the b tile
template <class C>
__device__ __forceinline__ int state_col0(int a) {
    return C::ES == 2 ? 32 * (a >> 1) + 4 * (a & 1) : 16 * a;
}
constexpr int state_step(int es) { return es == 2 ? 8 : 4; }

// Chunks of 64 tokens, in time order or (reversed) from the end.  Per chunk, and per
// head of b and c that shares the state:
//   1. scores P[t][s] = scale g^|t-s| (a_t . b_s) of the causal half, to LDS in the
//      plan dtype, split over the waves by 16 x 16 blocks;
//   2. wave w, for its 16 columns of out^T: the old state (two terms) times a, decayed
//      per token in fp32, plus c^T P^T;
//   3. the state's 16 columns: S = g^n S + b^T (decayed c), the decayed c in as many
//      terms as keep the state's fp32 accuracy.
// The state never leaves its wave's registers: the accumulator of step 3 is, in its
// lanes, the operand of step 2.  OUT: the whole; else step 3 alone, and the state
// goes to part[slot].
template <class C, bool OUT>
__global__ __launch_bounds__(C::NT) void chunk_kernel(Job j) {
    using IO = typename C::IO;
    using O = typename C::O;
    using F = typename O::F;
    __shared__ __attribute__((aligned(16))) char lds[C::LDS];
    char *const ta = lds, *const tb = lds + C::OFF_B, *const tc = lds + C::OFF_C, *const tp = lds + C::OFF_P;
    volatile int* const flag = reinterpret_cast<volatile int*>(lds + C::OFF_FLAG);

    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kg = lane >> 4, ln = lane & 15;
    const int Hkv = j.Ha < j.Hb ? j.Ha : j.Hb, heads = OUT ? j.Ha : Hkv;
    const int64_t slot = blockIdx.x / heads;
    const int hx = (int)(blockIdx.x % heads);
    const int r = j.Ha > j.Hb ? j.Ha / j.Hb : 1;        // heads of a per state
    const int rb = j.Hb > j.Ha ? j.Hb / j.Ha : 1;       // heads of b and c per state
    const int kv = OUT ? hx / r : hx;
    const Segment seg = segment_of(j, slot);
    if (seg.idle) return;
    const bool final_seg = j.reverse ? seg.first : seg.last, initial_seg = j.reverse ? seg.last : seg.first;
    if (!OUT && final_seg) return;  // no segment comes after it

    const float l2 = j.log_decay[kv] * kLog2e;
    const int n_tok = (int)(seg.t1 - seg.t0), n_chunks = (n_tok + kChunk - 1) / kChunk;
    const bool own = 16 * wave < j.Dc;  // waves past D_c only load and score
    const int dc = 16 * wave + ln;
    const int64_t state_at = (seg.b * Hkv + kv) * (int64_t)j.Da * j.Dc;

    f32x4 S[C::NB];
#pragma unroll
    for (int a = 0; a < C::NB; ++a) S[a] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (OUT && own) {
        if (j.seg_len) {
            const float* p = j.part + ((slot * Hkv + kv) * C::NW + wave) * (int64_t)(C::NB * 256) + lane * 4;
#pragma unroll
            for (int a = 0; a < C::NB; ++a) S[a] = *reinterpret_cast<const f32x4*>(p + a * 256);
        } else if (j.S0) {
            const float s0 = j.reverse && n_tok ? 1.0f / j.scale : 1.0f;
#pragma unroll
            for (int a = 0; a < C::NB; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int da = state_row<C>(a, kg, i);
                    if (da < j.Da && dc < j.Dc) S[a][i] = s0 * j.S0[state_at + (int64_t)da * j.sa + (int64_t)dc * j.sc];
                }
        }
    }

    // decays, the same in every whole chunk: of the scores (within a diagonal block; one
    // block apart; per further block), of the tokens' weights in the state
    float near0[4], near1[4], w0[2][8];
    const float g16 = power(l2, 16);
    const int sgn = j.reverse ? -1 : 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int d = sgn * (ln - (4 * kg + i));  // t - s (s - t reversed) on the diagonal
        near0[i] = d >= 0 ? j.scale * power(l2, d) : 0.0f;
        near1[i] = j.scale * power(l2, 16 + d);
    }
    auto weights = [&](int n, float(&w)[2][8]) {  // token weights of a chunk of n
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // the token of element e: 16-bit fragments hold 32 tokens, fp32 ones 16
                const int s = C::ES == 2 ? 32 * m + 8 * kg + e : 16 * (2 * m + (e >> 2)) + 4 * kg + (e & 3);
                const int d = j.reverse ? s : n - 1 - s;
                w[m][e] = power(l2, d > 0 ? d : 0);
            }
    };
    weights(kChunk, w0);
    if (OUT) {
        for (int i = tid; i < kChunk * C::PP / 16; i += C::NT) reinterpret_cast<u32x4*>(tp)[i] = u32x4{0u, 0u, 0u, 0u};
    }
    if (tid < 2) flag[tid] = 0;
    __syncthreads();

    // loads of one (chunk, head of b and c): pieces tid, tid + NT, ... of each tile
    u32x4 ra[C::NPA], rbv[C::NPA], rc[C::NPC];
    const int total = n_chunks * rb;
    auto chunk_start = [&](int it) {
        const int c = it / rb;
        return seg.t0 + (int64_t)(j.reverse ? n_chunks - 1 - c : c) * kChunk;
    };
    auto load = [&](int it) {
        const int64_t t = chunk_start(it);
        const int hh = it % rb, n = (int)(seg.t1 - t < kChunk ? seg.t1 - t : kChunk);
        const int hb = kv * rb + hh;
        constexpr int E = 16 / C::ES;
        auto tile = [&](const Heads& x, int h, int D, bool vec, auto ppr, auto& reg) {
            constexpr int PPR = decltype(ppr)::value;
#pragma unroll
            for (int k = 0; k < (int)(sizeof(reg) / 16); ++k) {
                const int p = tid + k * C::NT, row = p / PPR, col = (p % PPR) * E;
                reg[k] = u32x4{0u, 0u, 0u, 0u};
                if (row < n) reg[k] = load_piece<IO>((const IO*)x.p + (t + row) * x.ts + h * x.hs, col, D, vec);
            }
        };
        if (OUT && hh == 0) tile(j.a, hx, j.Da, j.a_vec != 0, std::integral_constant<int, C::DA / E>{}, ra);
        tile(j.b, hb, j.Da, j.b_vec != 0, std::integral_constant<int, C::DA / E>{}, rbv);
        tile(j.c, hb, j.Dc, j.c_vec != 0, std::integral_constant<int, C::DC / E>{}, rc);
    };
    auto stage = [&](int it) {
        constexpr int E = 16 / C::ES;
        auto tile = [&](char* to, int pitch, auto ppr, auto& reg) {
            constexpr int PPR = decltype(ppr)::value;
#pragma unroll
            for (int k = 0; k < (int)(sizeof(reg) / 16); ++k) {
                const int p = tid + k * C::NT;
                if (kChunk * PPR % C::NT == 0 || p < kChunk * PPR)
                    *reinterpret_cast<u32x4*>(to + (p / PPR) * pitch + (p % PPR) * 16) = reg[k];
            }
        };
        if (OUT && it % rb == 0) tile(ta, C::PA, std::integral_constant<int, C::DA / E>{}, ra);
        tile(tb, C::PA, std::integral_constant<int, C::DA / E>{}, rbv);
        tile(tc, C::PC, std::integral_constant<int, C::DC / E>{}, rc);
        if constexpr (OUT) {
            bool odd = false;
#pragma unroll
            for (int k = 0; k < C::NPC; ++k) odd |= O::odd(rc[k]);
            if (odd) flag[it & 1] = 1;
        }
    };

    f32x4 acc[4];
    if (total > 0) load(0);
    for (int it = 0; it < total; ++it) {
        const int64_t t = chunk_start(it);
        const int n = (int)(seg.t1 - t < kChunk ? seg.t1 - t : kChunk), nq = (n + 15) / 16;
        const int hh = it % rb;
        stage(it);
        __syncthreads();
        if (it + 1 < total) load(it + 1);

        if constexpr (OUT) {
            // 1. blocks (qb, kb) of the causal half; reversed, whole 32-token steps of keys
            const int nk = j.reverse ? (n + 31) / 32 * 2 : nq;
            int idx = 0;
#pragma unroll
            for (int qb = 0; qb < 4; ++qb)
#pragma unroll
                for (int kb = 0; kb < 4; ++kb) {
                    if (j.reverse ? (kb < qb || kb >= nk || qb >= nq) : (kb > qb || qb >= nq)) continue;
                    if (idx++ % C::NW != wave) continue;
                    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int m = 0; m < C::NM; ++m)
                        O::mma(s, O::row(tb + (16 * kb + ln) * C::PA + (O::KS * m + O::KF * kg) * C::ES),
                               O::row(ta + (16 * qb + ln) * C::PA + (O::KS * m + O::KF * kg) * C::ES));
                    const int d = qb > kb ? qb - kb : kb - qb;
                    float p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int gap = sgn * (ln - (4 * kg + i));
                        if (d == 0) p[i] = gap >= 0 ? s[i] * near0[i] : 0.0f;
                        else p[i] = s[i] * near1[i] * (d == 1 ? 1.0f : (d == 2 ? g16 : g16 * g16));
                    }
                    char* to = tp + (16 * qb + ln) * C::PP + (16 * kb + 4 * kg) * C::ES;
                    if constexpr (C::ES == 2)
                        *reinterpret_cast<u32x2*>(to) = u32x2{Half<IO>::pack2(p[0], p[1]), Half<IO>::pack2(p[2], p[3])};
                    else
                        *reinterpret_cast<f32x4*>(to) = f32x4{p[0], p[1], p[2], p[3]};
                }
            __syncthreads();
            if (tid == 0) flag[(it + 1) & 1] = 0;
        }

        if (own) {
            // the chunk's columns of c: contraction over its tokens
            constexpr int NS = kChunk / O::KS;
            F ct[NS];
#pragma unroll
            for (int m = 0; m < NS; ++m) ct[m] = O::column(tc, C::PC, O::KS * m, 16 * wave, 4);
            // reversed, the initial state belongs to the last token itself: no decay before it
            const int e0 = (j.reverse && initial_seg && it / rb == 0) ? 0 : 1;
            if constexpr (OUT) {
                // 2.
                if (hh == 0) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
                    float norm = 1.0f, inv_norm = 1.0f;  // fp16: the state scaled into its range, by a power of two
                    if constexpr (std::is_same_v<IO, _Float16>) {
                        float mx = 0.0f;
#pragma unroll
                        for (int a = 0; a < C::NB; ++a)
#pragma unroll
                            for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fabsf(S[a][i]));
#pragma unroll
                        for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
                        int ex = 0;
                        if (mx > 0.0f && mx < __builtin_inff()) (void)frexpf(mx, &ex);
                        ex = ex < -100 ? -100 : ex;
                        norm = ldexpf(1.0f, ex);
                        inv_norm = ldexpf(1.0f, -ex);
                    }
#pragma unroll
                    for (int m = 0; m < C::NM; ++m) {
                        constexpr int ST = C::ES == 2 ? 2 : 1;
                        F st[ST];
                        float v[O::KF];
#pragma unroll
                        for (int e = 0; e < O::KF; ++e) v[e] = S[(O::KF * m + e) / 4][e & 3] * inv_norm;
                        O::split(v, st);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (q < nq) {
                                const F at = O::row(ta + (16 * q + ln) * C::PA + (O::KS * m + O::KF * kg) * C::ES);
#pragma unroll
                                for (int x = 0; x < ST; ++x) O::mma(acc[q], st[x], at);
                            }
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int tq = 16 * q + ln, d = (j.reverse ? n - 1 - tq : tq) + e0;
                        acc[q] *= norm * j.scale * power(l2, d > 0 ? d : 0);
                    }
                }
                // An infinity or NaN among the chunk's values: 0 times it must not reach the
                // outputs that do not see it, so the product takes 0 in its place (the other
                // outputs keep their bits) and those that do see it add it one by one.
                const bool odd = flag[it & 1] != 0;
                F cf[NS];
#pragma unroll
                for (int m = 0; m < NS; ++m) cf[m] = odd ? O::finite(ct[m]) : ct[m];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int m = 0; m < NS; ++m) {
                        const bool sees = j.reverse ? O::KS * (m + 1) > 16 * q && O::KS * m < n
                                                    : O::KS * m < 16 * (q + 1);
                        if (q < nq && sees)
                            O::mma(acc[q], cf[m], O::row(tp + (16 * q + ln) * C::PP + (O::KS * m + O::KF * kg) * C::ES));
                    }
                if (odd) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        for (int s = 0; s < n; ++s) {
                            const int tq = 16 * q + ln;
                            if (j.reverse ? s < tq : s > tq) continue;
                            const float p = (float)*reinterpret_cast<const IO*>(tp + tq * C::PP + s * C::ES);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float v = (float)*reinterpret_cast<const IO*>(
                                    tc + s * C::PC + (16 * wave + 4 * kg + i) * C::ES);
                                if (!(fabsf(v) < __builtin_inff())) acc[q][i] = fmaf(p, v, acc[q][i]);
                            }
                        }
                }
                if (hh == rb - 1) {
                    IO* out = (IO*)const_cast<void*>(j.out.p) + hx * j.out.hs;
                    const int c0 = 16 * wave + 4 * kg;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int tq = 16 * q + ln;
                        if (tq >= n) continue;
                        IO* p = out + (t + tq) * j.out.ts + c0;
                        if (j.out_vec && c0 + 3 < j.Dc) {
                            if constexpr (C::ES == 2)
                                *reinterpret_cast<u32x2*>(p) = u32x2{Half<IO>::pack2(acc[q][0], acc[q][1]),
                                                                     Half<IO>::pack2(acc[q][2], acc[q][3])};
                            else
                                *reinterpret_cast<f32x4*>(p) = acc[q];
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (c0 + i < j.Dc) p[i] = (IO)acc[q][i];
                        }
                    }
                }
            }
            // 3.
            if (!OUT || it / rb + 1 < n_chunks || (j.S1 && final_seg && hx % r == 0)) {
                if (hh == 0) {
                    const float carry = power(l2, n - 1 + e0);
#pragma unroll
                    for (int a = 0; a < C::NB; ++a) S[a] *= carry;
                }
                float w[2][8];
                if (n < kChunk) {
                    weights(n, w);
                } else {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[m][e] = w0[m][e];
                }
#pragma unroll
                for (int m = 0; m < NS; ++m) {
                    if (O::KS * m >= n) continue;
                    float v[O::KF];
#pragma unroll
                    for (int e = 0; e < O::KF; ++e) {
                        const int at = O::KF * m + e;
                        v[e] = O::get(ct[m], e) * w[at >> 3][at & 7];
                    }
                    F cw[O::TERMS];
                    O::split(v, cw);
#pragma unroll
                    for (int a = 0; a < C::NB; ++a) {
                        const F bt = O::column(tb, C::PA, O::KS * m, state_col0<C>(a), state_step(C::ES));
#pragma unroll
                        for (int x = 0; x < O::TERMS; ++x) O::mma(S[a], bt, cw[x]);
                    }
                }
            }
        }
        __syncthreads();
    }

    if (!own) return;
    if (!OUT) {
        float* p = j.part + ((slot * Hkv + kv) * C::NW + wave) * (int64_t)(C::NB * 256) + lane * 4;
#pragma unroll
        for (int a = 0; a < C::NB; ++a) *reinterpret_cast<f32x4*>(p + a * 256) = S[a];
    } else if (j.S1 && final_seg && hx % r == 0) {
        const float s1 = j.reverse && n_tok ? power(l2, 1) * j.scale : 1.0f;
#pragma unroll
        for (int a = 0; a < C::NB; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int da = state_row<C>(a, kg, i);
                if (da < j.Da && dc < j.Dc) j.S1[state_at + (int64_t)da * j.sa + (int64_t)dc * j.sc] = s1 * S[a][i];
            }
    }
}

// part[slot]: from each segment's own state to the state before it.  One thread per
// four numbers, along the sequence's segments.
template <class C>
__global__ __launch_bounds__(256) void join_kernel(Job j) {
    constexpr int Q = C::NW * C::NB * 64;  // quads of one state
    const int Hkv = j.Ha < j.Hb ? j.Ha : j.Hb;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t b = id / ((int64_t)Hkv * Q);
    if (b >= j.batch) return;
    const int kv = (int)(id / Q % Hkv), q = (int)(id % Q);
    const int lane = q & 63, a = (q >> 6) % C::NB, wave = (q >> 6) / C::NB;
    const int dc = 16 * wave + (lane & 15);
    if (16 * wave >= j.Dc) return;
    int64_t t0, t1;
    sequence(j.offsets, j.batch, j.T, b, t0, t1);
    const int64_t segs = t1 > t0 ? (t1 - t0 + j.seg_len - 1) / j.seg_len : 1;
    const int64_t slot0 = j.offsets ? t0 / j.seg_len + b : b * segs;
    const float l2 = j.log_decay[kv] * kLog2e;
    f32x4 S = {0.f, 0.f, 0.f, 0.f};
    if (j.S0) {
        const int64_t at = (b * Hkv + kv) * (int64_t)j.Da * j.Dc;
        const float s0 = j.reverse && t1 > t0 ? 1.0f / j.scale : 1.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int da = state_row<C>(a, lane >> 4, i);
            if (da < j.Da && dc < j.Dc) S[i] = s0 * j.S0[at + (int64_t)da * j.sa + (int64_t)dc * j.sc];
        }
    }
    for (int64_t k = 0; k < segs; ++k) {
        const int64_t g = j.reverse ? segs - 1 - k : k;
        float* p = j.part + (((slot0 + g) * Hkv + kv) * (int64_t)Q + q) * 4;
        f32x4 mine = {0.f, 0.f, 0.f, 0.f};
        if (k + 1 < segs) mine = *reinterpret_cast<const f32x4*>(p);
        *reinterpret_cast<f32x4*>(p) = S;
        if (k + 1 == segs) break;
        const int64_t left = t1 - t0 - g * j.seg_len;
        const int64_t n = left < j.seg_len ? left : j.seg_len;
        // reversed, the initial state belongs to the last token itself
        const float carry = power(l2, (int)n - (j.reverse && k == 0 ? 1 : 0));
        S = S * carry + mine;
    }
}

// --- host side ------------------------------------------------------------------------

int padded_a(int Da) { return (Da + 31) / 32; }
int waves_for(int Dc) { return Dc <= 64 ? 4 : 8; }

// Segments: none where the sequences and heads alone give two workgroups per CU;
// otherwise runs of at least four chunks, as many as that takes.
struct Split {
    int64_t seg_len = 0, slots = 0;
};
Split split_for(int64_t T, int64_t batch, int heads, bool ragged) {
    Split s;
    s.slots = batch;
    const int64_t mean = T / batch;
    if (batch * heads >= 512 || mean < 8 * kChunk) return s;
    const int64_t want = (512 + batch * heads - 1) / (batch * heads);
    int64_t chunks = ((mean + kChunk - 1) / kChunk + want - 1) / want;
    chunks = chunks < 4 ? 4 : chunks;
    s.seg_len = chunks * kChunk;
    s.slots = ragged ? T / s.seg_len + batch : batch * ((mean + s.seg_len - 1) / s.seg_len);
    return s;
}

size_t part_bytes(const Split& s, int Hkv, int Da, int Dc) {
    return s.seg_len ? (size_t)s.slots * Hkv * waves_for(Dc) * 16 * padded_a(Da) * 32 * 4 : 0;
}

template <typename IO, int KB, int NW>
hipError_t run_cfg(const Job& j, hipStream_t stream) {
    using C = Cfg<IO, KB, NW>;
    const int Hkv = j.Ha < j.Hb ? j.Ha : j.Hb;
    if (j.slots * j.Ha > 0x7fffffff) return hipErrorNotSupported;
    if (j.seg_len) {
        hipLaunchKernelGGL((chunk_kernel<C, false>), dim3((uint32_t)(j.slots * Hkv)), dim3(C::NT), 0, stream, j);
        const int64_t threads = j.batch * Hkv * (C::NW * C::NB * 64);
        if ((threads + 255) / 256 > 0x7fffffff) return hipErrorNotSupported;
        hipLaunchKernelGGL((join_kernel<C>), dim3((uint32_t)((threads + 255) / 256)), dim3(256), 0, stream, j);
    }
    hipLaunchKernelGGL((chunk_kernel<C, true>), dim3((uint32_t)(j.slots * j.Ha)), dim3(C::NT), 0, stream, j);
    return hipGetLastError();
}

bool vec_ok(const Heads& h, int D, size_t es, size_t piece) {
    return (uintptr_t)h.p % piece == 0 && h.ts * es % piece == 0 && h.hs * es % piece == 0 && D * es % piece == 0;
}

template <typename IO>
hipError_t run(Job j, const MixArgs& a, void* ws, hipStream_t stream) {
    const size_t es = sizeof(IO);
    j.offsets = a.offsets;
    j.batch = a.batch;
    j.T = a.T;
    const Split s = split_for(a.T, a.batch, a.heads, a.offsets != nullptr);
    j.seg_len = s.seg_len;
    j.slots = s.slots;
    j.part = static_cast<float*>(ws);
    j.a_vec = vec_ok(j.a, j.Da, es, 16);
    j.b_vec = vec_ok(j.b, j.Da, es, 16);
    j.c_vec = vec_ok(j.c, j.Dc, es, 16);
    j.out_vec = vec_ok(j.out, 4, es, 4 * es);
    const int kb = padded_a(j.Da);
#define EQL_MIX(KB)                                                    \
    case KB:                                                           \
        if (waves_for(j.Dc) == 4) return run_cfg<IO, KB, 4>(j, stream); \
        else return run_cfg<IO, KB, 8>(j, stream);
    switch (kb) {
        EQL_MIX(1) EQL_MIX(2) EQL_MIX(3) EQL_MIX(4)
        default: return hipErrorNotSupported;
    }
#undef EQL_MIX
}

Job job(const Heads& x, const Heads& y, const Heads& z, const Heads& out, int Ha, int Hb, int Da, int Dc, int reverse,
        const MixArgs& a, const float* S0, float* S1, int sa, int sc) {
    Job j{};
    j.a = x, j.b = y, j.c = z, j.out = out;
    j.Ha = Ha, j.Hb = Hb, j.Da = Da, j.Dc = Dc;
    j.reverse = reverse;
    j.scale = a.scale;
    j.log_decay = a.log_decay;
    j.S0 = S0, j.S1 = S1;
    j.sa = sa, j.sc = sc;
    return j;
}

template <typename IO>
hipError_t forward(const MixArgs& a, void* ws, hipStream_t stream) {
    return run<IO>(job(a.q, a.k, a.v, a.o, a.heads, a.kv_heads, a.D_k, a.D_v, 0, a, a.state_in, a.state_out, a.D_v, 1), a,
                   ws, stream);
}

template <typename IO>
hipError_t backward(const MixArgs& a, void* ws, hipStream_t stream) {
    const Job jobs[3] = {
        job(a.d_o, a.v, a.k, a.dq, a.heads, a.kv_heads, a.D_v, a.D_k, 0, a, a.state_in, nullptr, 1, a.D_v),
        job(a.v, a.d_o, a.q, a.dk, a.kv_heads, a.heads, a.D_v, a.D_k, 1, a, a.d_state_out, nullptr, 1, a.D_v),
        job(a.k, a.q, a.d_o, a.dv, a.kv_heads, a.heads, a.D_k, a.D_v, 1, a, a.d_state_out, a.d_state_in, a.D_v, 1)};
    for (const Job& j : jobs) {
        const hipError_t e = run<IO>(j, a, ws, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

size_t linear_attention_workspace(int, int heads, int kv_heads, int D_k, int D_v, int64_t T, int64_t batch,
                                  bool backward) {
    if (T <= 0 || batch <= 0) return 0;
    // packed sequences need the most slots
    const Split s = split_for(T, batch, heads, true);
    size_t n = part_bytes(s, kv_heads, D_k, D_v);
    if (backward) {
        const size_t m = part_bytes(s, kv_heads, D_v, D_k);
        n = n > m ? n : m;
    }
    return n;
}

hipError_t launch_linear_attention(int io, const MixArgs& a, void* ws, hipStream_t stream) {
    return io == kIoF32 ? forward<float>(a, ws, stream)
                        : (io == kIoBF16 ? forward<__bf16>(a, ws, stream) : forward<_Float16>(a, ws, stream));
}

hipError_t launch_linear_attention_backward(int io, const MixArgs& a, void* ws, hipStream_t stream) {
    return io == kIoF32 ? backward<float>(a, ws, stream)
                        : (io == kIoBF16 ? backward<__bf16>(a, ws, stream) : backward<_Float16>(a, ws, stream));
}

namespace {

// One token.  A workgroup takes one (sequence, kv head): each thread reads, updates
// and writes back four columns (one, where D_v is odd against that) of rows row,
// row + rows, ... of the state, and adds them into the outputs of HB query heads that
// share it; further heads, HB at a time, read the state again.  The state, read and
// written once, is all the traffic that counts; its loads go out U at a time.
template <typename IO, bool VEC, int HB>
__global__ __launch_bounds__(256) void step_kernel(MixArgs a, int cols) {
    constexpr int U = 4, W = VEC ? 4 : 1;  // columns of a thread
    __shared__ float vk[kMaxD], vq[HB][kMaxD], red[HB][256 * W];
    const int64_t b = blockIdx.x / (uint32_t)a.kv_heads;
    const int kv = (int)(blockIdx.x % (uint32_t)a.kv_heads), r = a.heads / a.kv_heads, tid = (int)threadIdx.x;
    const int rows = 256 / cols, row = tid / cols, c = (tid - row * cols) * W;
    const bool on = row < rows;
    using R = std::conditional_t<VEC, f32x4, float>;
    float* S = a.state_out + (int64_t)blockIdx.x * a.D_k * a.D_v + c;
    const float g = power(a.log_decay[kv] * kLog2e, 1);
    R v{};
    if (on) {
        const IO* p = (const IO*)a.v.p + b * a.v.ts + kv * a.v.hs + c;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = (float)p[i];
        } else {
            v = (float)p[0];
        }
    }
    if (tid < a.D_k) vk[tid] = (float)((const IO*)a.k.p)[b * a.k.ts + kv * a.k.hs + tid];
    for (int h0 = 0; h0 < r; h0 += HB) {
        const int nh = r - h0 < HB ? r - h0 : HB;
        const IO* q = (const IO*)a.q.p + b * a.q.ts + (int64_t)(kv * r + h0) * a.q.hs;
        for (int e = tid; e < nh * kMaxD; e += 256) {
            const int h = e / kMaxD, i = e % kMaxD;
            if (i < a.D_k) vq[h][i] = a.scale * (float)q[h * a.q.hs + i];
        }
        __syncthreads();
        R o[HB];
#pragma unroll
        for (int h = 0; h < HB; ++h) o[h] = R{};
        if (on)
            for (int i0 = row; i0 < a.D_k; i0 += U * rows) {
                R s[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i0 + u * rows < a.D_k) s[u] = *reinterpret_cast<const R*>(S + (i0 + u * rows) * a.D_v);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + u * rows;
                    if (i < a.D_k) {
                        if (h0 == 0) {
                            s[u] = s[u] * g + v * vk[i];
                            *reinterpret_cast<R*>(S + i * a.D_v) = s[u];
                        }
#pragma unroll
                        for (int h = 0; h < HB; ++h)
                            if (h < nh) o[h] += s[u] * vq[h][i];
                    }
                }
            }
#pragma unroll
        for (int h = 0; h < HB; ++h) *reinterpret_cast<R*>(red[h] + tid * W) = o[h];
        __syncthreads();
        IO* out = (IO*)const_cast<void*>(a.o.p) + b * a.o.ts + (int64_t)(kv * r + h0) * a.o.hs;
        for (int e = tid; e < nh * a.D_v; e += 256) {
            const int h = e / a.D_v, i = e - h * a.D_v;
            float w = red[h][i];
            for (int k = 1; k < rows; ++k) w += red[h][k * a.D_v + i];
            out[h * a.o.hs + i] = (IO)w;
        }
        __syncthreads();
    }
}

template <typename IO>
hipError_t step(const MixArgs& a, hipStream_t stream) {
    const dim3 grid((uint32_t)(a.batch * a.kv_heads));
    const int r = a.heads / a.kv_heads;
    if (a.D_v % 4 == 0) {
        const int cols = a.D_v / 4;
        if (r == 1) hipLaunchKernelGGL((step_kernel<IO, true, 1>), grid, dim3(256), 0, stream, a, cols);
        else if (r == 2) hipLaunchKernelGGL((step_kernel<IO, true, 2>), grid, dim3(256), 0, stream, a, cols);
        else hipLaunchKernelGGL((step_kernel<IO, true, 4>), grid, dim3(256), 0, stream, a, cols);
    } else {
        hipLaunchKernelGGL((step_kernel<IO, false, 2>), grid, dim3(256), 0, stream, a, a.D_v);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_attention_step(int io, const MixArgs& a, hipStream_t stream) {
    if (a.batch * a.kv_heads > 0x7fffffff) return hipErrorNotSupported;
    return io == kIoF32 ? step<float>(a, stream)
                        : (io == kIoBF16 ? step<__bf16>(a, stream) : step<_Float16>(a, stream));
}

}  // namespace eql
