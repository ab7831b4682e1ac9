// linear_attention.h -- causal linear attention with a decay for each head.
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
#pragma once

#include "cn_fused.h"  // make_rsrc, kOOB
#include "eq_device.h"
#include "eq_launch.h"

namespace eql {
namespace mix {

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
    int out_vec;  // output rows in whole pieces of four
};

// The products of one launch: workgroups first[k] .. first[k + 1] - 1 take jobs[k].
constexpr int kMaxJobs = 3;
struct Jobs {
    Job j[kMaxJobs];
    uint32_t first[kMaxJobs + 1];
    int count;
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

// One 16-byte piece of a row of any alignment: columns col .. of D, zeros past D.
template <typename IO>
__device__ __forceinline__ u32x4 load_piece(const IO* row, int col, int D) {
    constexpr int E = 16 / (int)sizeof(IO);
    u32x4 v = {0u, 0u, 0u, 0u};
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
    static constexpr int DA = 32 * KB_, DC = 16 * NW_, NB = DA / 16, NM = DA / O::KS, NS = kChunk / O::KS;
    // row pitches: an odd number of 16-byte pieces, so that 16 rows spread over the banks
    static constexpr int PA = DA * ES + 16, PC = DC * ES + 16, PP = kChunk * ES + 16;
    static constexpr int E = 16 / ES, PPA = DA / E, PPC = DC / E;  // numbers of a piece; pieces of a row
    static constexpr int NPA = (kChunk * PPA + NT - 1) / NT, NPC = (kChunk * PPC + NT - 1) / NT;
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

__device__ __forceinline__ float uniform(float v) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

// The b (c) tile's pieces of this thread: piece tid + k NT is 16 bytes of row
// (tid + k NT) / PPR.  VEC: rows are whole aligned pieces, read through a buffer
// resource over the chunk's rows, offsets past which read zeros.
template <typename IO, int PPR, int NT, int NP, bool VEC>
struct Loader {
    static constexpr int ES = (int)sizeof(IO), E = 16 / ES;
    uint32_t off[VEC ? NP : 1];
    __device__ __forceinline__ Loader(const Heads& x, int D) {
        if constexpr (VEC) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int p = (int)threadIdx.x + k * NT, row = p / PPR, col = p % PPR * E;
                off[k] = row < kChunk && col < D ? (uint32_t)row * (uint32_t)x.ts * ES + (uint32_t)col * ES : kOOB;
            }
        }
    }
    // rows t .. t + n - 1 of head h
    __device__ __forceinline__ void load(const Heads& x, int64_t t, int64_t h, int n, int D, u32x4 (&r)[NP]) const {
        const IO* base = (const IO*)x.p + t * x.ts + h * x.hs;
        if constexpr (VEC) {
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(base, (uint32_t)(((n - 1) * x.ts + D) * ES));
            if (n == kChunk) {
#pragma unroll
                for (int k = 0; k < NP; ++k) r[k] = __builtin_amdgcn_raw_buffer_load_b128(rs, off[k], 0, 0);
            } else {  // (strides below a row's width: later rows may lie inside the resource)
#pragma unroll
                for (int k = 0; k < NP; ++k) {
                    const int row = ((int)threadIdx.x + k * NT) / PPR;
                    r[k] = __builtin_amdgcn_raw_buffer_load_b128(rs, row < n ? off[k] : kOOB, 0, 0);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int p = (int)threadIdx.x + k * NT, row = p / PPR;
                r[k] = u32x4{0u, 0u, 0u, 0u};
                if (row < n) r[k] = load_piece<IO>(base + row * x.ts, p % PPR * E, D);
            }
        }
    }
    static __device__ __forceinline__ void stage(char* to, int pitch, const u32x4 (&r)[NP]) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int p = (int)threadIdx.x + k * NT;
            if (kChunk * PPR % NT == 0 || p < kChunk * PPR)
                *reinterpret_cast<u32x4*>(to + (p / PPR) * pitch + (p % PPR) * 16) = r[k];
        }
    }
};

// Waves per SIMD that the registers are held to: as many as the LDS allows, except
// where that would spill.
template <class C>
constexpr int kWaves = C::NW == 8 ? 2 : (C::ES == 2 ? (C::KB <= 2 ? 3 : 2) : (C::KB <= 2 ? 2 : 1));

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
template <class C, bool OUT, bool VEC>
__global__ __launch_bounds__(C::NT, kWaves<C>) void chunk_kernel(Jobs jobs) {
    using IO = typename C::IO;
    using O = typename C::O;
    using F = typename O::F;
    constexpr int NS = C::NS, KF = O::KF;
    __shared__ __attribute__((aligned(16))) char lds[C::LDS];
    char *const ta = lds, *const tb = lds + C::OFF_B, *const tc = lds + C::OFF_C, *const tp = lds + C::OFF_P;
    volatile int* const flag = reinterpret_cast<volatile int*>(lds + C::OFF_FLAG);

    // consecutive workgroups (heads of one sequence, which may share b and c) on one XCD
    const uint32_t wg = xcd_remap(blockIdx.x, gridDim.x);
    const int which = wg >= jobs.first[2] ? 2 : (wg >= jobs.first[1] ? 1 : 0);
    const Job j = which == 2 ? jobs.j[2] : (which == 1 ? jobs.j[1] : jobs.j[0]);
    const uint32_t id = wg - jobs.first[which == 2 ? 2 : (which == 1 ? 1 : 0)];

    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kg = lane >> 4, ln = lane & 15;
    const int Hkv = j.Ha < j.Hb ? j.Ha : j.Hb, heads = OUT ? j.Ha : Hkv;
    const int64_t slot = id / (uint32_t)heads;
    const int hx = (int)(id % (uint32_t)heads);
    const int r = j.Ha > j.Hb ? j.Ha / j.Hb : 1;   // heads of a per state
    const int rb = j.Hb > j.Ha ? j.Hb / j.Ha : 1;  // heads of b and c per state
    const int kv = OUT ? hx / r : hx;
    const bool rev = j.reverse != 0;
    const Segment seg = segment_of(j, slot);
    if (seg.idle) return;
    const bool final_seg = rev ? seg.first : seg.last, initial_seg = rev ? seg.last : seg.first;
    if (!OUT && final_seg) return;  // no segment comes after it

    const float l2 = uniform(j.log_decay[kv] * kLog2e);
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
            const float s0 = rev && n_tok ? 1.0f / j.scale : 1.0f;
#pragma unroll
            for (int a = 0; a < C::NB; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int da = state_row<C>(a, kg, i);
                    if (da < j.Da && dc < j.Dc) S[a][i] = s0 * j.S0[state_at + (int64_t)da * j.sa + (int64_t)dc * j.sc];
                }
        }
    }

    // Decays, the same in every whole chunk: of the scores (within a diagonal block, one
    // block apart; g^16 per further block), of the old state at a token (g^16 per block
    // of tokens), of a token's weight in the new state (step m, lane group, element e).
    const int sgn = rev ? -1 : 1;
    float near0[4], near1[4], wb[NS], we[KF];
    const float g16 = uniform(power(l2, 16)), g64 = uniform(power(l2, kChunk));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int d = sgn * (ln - (4 * kg + i));  // t - s (s - t reversed) on the diagonal
        near0[i] = d >= 0 ? j.scale * power(l2, d) : 0.0f;
        near1[i] = j.scale * power(l2, 16 + d);
    }
    const float old = j.scale * power(l2, rev ? 16 - ln : 1 + ln);
#pragma unroll
    for (int m = 0; m < NS; ++m)
        wb[m] = power(l2, rev ? O::KS * m + KF * kg : kChunk - O::KS * m - KF * (kg + 1));
#pragma unroll
    for (int e = 0; e < KF; ++e) we[e] = uniform(power(l2, rev ? e : KF - 1 - e));
    if (OUT) {
        for (int i = tid; i < kChunk * C::PP / 16; i += C::NT) reinterpret_cast<u32x4*>(tp)[i] = u32x4{0u, 0u, 0u, 0u};
    }
    if (tid < 2) flag[tid] = 0;
    __syncthreads();

    u32x4 ra[OUT ? C::NPA : 1], rbv[C::NPA], rc[C::NPC];
    const Loader<IO, C::PPA, C::NT, C::NPA, VEC> la(j.a, j.Da), lb(j.b, j.Da);
    const Loader<IO, C::PPC, C::NT, C::NPC, VEC> lc(j.c, j.Dc);
    const int total = n_chunks * rb;
    auto load = [&](int64_t t, int hh) {  // chunk from t, head hh of those that share the state
        const int n = (int)(seg.t1 - t < kChunk ? seg.t1 - t : kChunk);
        if constexpr (OUT) {
            if (hh == 0) la.load(j.a, t, hx, n, j.Da, ra);
        }
        lb.load(j.b, t, kv * rb + hh, n, j.Da, rbv);
        lc.load(j.c, t, kv * rb + hh, n, j.Dc, rc);
    };

    f32x4 acc[4];
    int64_t t = seg.t0 + (rev ? (int64_t)(n_chunks - 1) * kChunk : 0);
    int hh = 0, left = n_chunks;  // chunks from this one on
    if (total > 0) load(t, 0);
    for (int it = 0; it < total; ++it) {
        const int n = (int)(seg.t1 - t < kChunk ? seg.t1 - t : kChunk), nq = (n + 15) / 16;
        if constexpr (OUT) {
            if (hh == 0) la.stage(ta, C::PA, ra);
        }
        lb.stage(tb, C::PA, rbv);
        lc.stage(tc, C::PC, rc);
        if constexpr (OUT) {
            bool odd = false;
#pragma unroll
            for (int k = 0; k < C::NPC; ++k) odd |= O::odd(rc[k]);
            if (odd) flag[it & 1] = 1;
        }
        __syncthreads();
        if (it + 1 < total) {
            if (hh + 1 < rb) load(t, hh + 1);
            else load(t + sgn * kChunk, 0);
        }

        if constexpr (OUT) {
            // 1. block idx of the lower triangle, row by row; reversed its transpose, and
            // keys in whole 32-token steps
            const int nk = rev ? (n + 31) / 32 * 2 : nq;
            for (int idx = wave; idx < 10; idx += C::NW) {
                const int hi = idx >= 6 ? 3 : (idx >= 3 ? 2 : (idx >= 1 ? 1 : 0));
                const int lo = idx - hi * (hi + 1) / 2;
                const int qb = rev ? lo : hi, kb = rev ? hi : lo;
                if (qb >= nq || kb >= nk) continue;
                f32x4 s = {0.f, 0.f, 0.f, 0.f};
                const char* pb = tb + (16 * kb + ln) * C::PA + KF * kg * C::ES;
                const char* pa = ta + (16 * qb + ln) * C::PA + KF * kg * C::ES;
#pragma unroll
                for (int m = 0; m < C::NM; ++m)
                    O::mma(s, O::row(pb + O::KS * m * C::ES), O::row(pa + O::KS * m * C::ES));
                float p[4];
                if (hi == lo) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = sgn * (ln - (4 * kg + i)) >= 0 ? s[i] * near0[i] : 0.0f;
                } else {
                    const float f = hi - lo == 1 ? 1.0f : (hi - lo == 2 ? g16 : g16 * g16);
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = s[i] * (near1[i] * f);
                }
                char* to = tp + (16 * qb + ln) * C::PP + (16 * kb + 4 * kg) * C::ES;
                if constexpr (C::ES == 2)
                    *reinterpret_cast<u32x2*>(to) = u32x2{Half<IO>::pack2(p[0], p[1]), Half<IO>::pack2(p[2], p[3])};
                else
                    *reinterpret_cast<f32x4*>(to) = f32x4{p[0], p[1], p[2], p[3]};
            }
            __syncthreads();
        }

        if (own) {
            // the chunk's columns of c: contraction over its tokens
            F ct[NS];
#pragma unroll
            for (int m = 0; m < NS; ++m) ct[m] = O::column(tc, C::PC, O::KS * m, 16 * wave, 4);
            // reversed, the initial state belongs to the last token itself: no decay before it
            const int e0 = (rev && initial_seg && left == n_chunks) ? 0 : 1;
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
                        float v[KF];
#pragma unroll
                        for (int e = 0; e < KF; ++e) v[e] = S[(KF * m + e) / 4][e & 3] * inv_norm;
                        O::split(v, st);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (q < nq) {
                                const F at = O::row(ta + (16 * q + ln) * C::PA + (O::KS * m + KF * kg) * C::ES);
#pragma unroll
                                for (int x = 0; x < ST; ++x) O::mma(acc[q], st[x], at);
                            }
                    }
                    if (n == kChunk && e0 == 1) {
                        float f = old * norm;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            acc[rev ? 3 - q : q] *= f;
                            f *= g16;
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int tq = 16 * q + ln, d = (rev ? n - 1 - tq : tq) + e0;
                            acc[q] *= norm * j.scale * power(l2, d > 0 ? d : 0);
                        }
                    }
                }
                // An infinity or NaN among the chunk's values: 0 times it must not reach the
                // outputs that do not see it, so the product takes 0 in its place (the other
                // outputs keep their bits) and those that do see it add it one by one.
                const int odd = __builtin_amdgcn_readfirstlane(flag[it & 1]);
                F cf[NS];
#pragma unroll
                for (int m = 0; m < NS; ++m) cf[m] = ct[m];
                if (odd) {
#pragma unroll
                    for (int m = 0; m < NS; ++m) cf[m] = O::finite(ct[m]);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int m = 0; m < NS; ++m) {
                        const bool sees = rev ? O::KS * (m + 1) > 16 * q && O::KS * m < n : O::KS * m < 16 * (q + 1);
                        if (q < nq && sees)
                            O::mma(acc[q], cf[m], O::row(tp + (16 * q + ln) * C::PP + (O::KS * m + KF * kg) * C::ES));
                    }
                if (odd) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        for (int s = 0; s < n; ++s) {
                            const int tq = 16 * q + ln;
                            if (rev ? s < tq : s > tq) continue;
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
                    const int c0 = 16 * wave + 4 * kg;
                    IO* out = (IO*)const_cast<void*>(j.out.p) + t * j.out.ts + hx * j.out.hs;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int tq = 16 * q + ln;
                        if (tq >= n) continue;
                        IO* p = out + tq * j.out.ts + c0;
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
            if (!OUT || left > 1 || (j.S1 && final_seg && hx % r == 0)) {
                if (hh == 0) {
                    const float carry = n == kChunk && e0 == 1 ? g64 : power(l2, n - 1 + e0);
#pragma unroll
                    for (int a = 0; a < C::NB; ++a) S[a] *= carry;
                }
#pragma unroll
                for (int m = 0; m < NS; ++m) {
                    if (O::KS * m >= n) continue;
                    float v[KF];
                    if (rev || n == kChunk) {
#pragma unroll
                        for (int e = 0; e < KF; ++e) v[e] = O::get(ct[m], e) * (wb[m] * we[e]);
                    } else {
#pragma unroll
                        for (int e = 0; e < KF; ++e) {
                            const int d = n - 1 - (O::KS * m + KF * kg + e);
                            v[e] = O::get(ct[m], e) * power(l2, d > 0 ? d : 0);
                        }
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
        if (tid == 0) flag[it & 1] = 0;  // the next writer comes after the next barrier
        if (++hh == rb) {
            hh = 0;
            t += sgn * kChunk;
            --left;
        }
    }

    if (!own) return;
    if (!OUT) {
        float* p = j.part + ((slot * Hkv + kv) * C::NW + wave) * (int64_t)(C::NB * 256) + lane * 4;
#pragma unroll
        for (int a = 0; a < C::NB; ++a) *reinterpret_cast<f32x4*>(p + a * 256) = S[a];
    } else if (j.S1 && final_seg && hx % r == 0) {
        const float s1 = rev && n_tok ? power(l2, 1) * j.scale : 1.0f;
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
__global__ __launch_bounds__(256) void join_kernel(Jobs jobs) {
    constexpr int Q = C::NW * C::NB * 64;  // quads of one state
    const Job j = blockIdx.y == 2 ? jobs.j[2] : (blockIdx.y == 1 ? jobs.j[1] : jobs.j[0]);
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
    constexpr int U = 8;  // segments in flight
    float* const p = j.part + ((slot0 * Hkv + kv) * (int64_t)Q + q) * 4;
    const int64_t step = (int64_t)Hkv * Q * 4;
    for (int64_t k0 = 0; k0 < segs; k0 += U) {
        f32x4 mine[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = k0 + u, g = j.reverse ? segs - 1 - k : k;
            mine[u] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (k + 1 < segs) mine[u] = *reinterpret_cast<const f32x4*>(p + g * step);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = k0 + u, g = j.reverse ? segs - 1 - k : k;
            if (k >= segs) break;
            *reinterpret_cast<f32x4*>(p + g * step) = S;
            const int64_t rest = t1 - t0 - g * j.seg_len;
            const int64_t n = rest < j.seg_len ? rest : j.seg_len;
            // reversed, the initial state belongs to the last token itself
            S = S * power(l2, (int)n - (j.reverse && k == 0 ? 1 : 0)) + mine[u];
        }
    }
}

// --- host side ------------------------------------------------------------------------

inline int padded_a(int Da) { return (Da + 31) / 32; }
inline int waves_for(int Dc) { return Dc <= 64 ? 4 : 8; }

template <typename IO, int KB, int NW, bool VEC>
hipError_t run_cfg(Jobs& jobs, hipStream_t stream) {
    using C = Cfg<IO, KB, NW>;
    auto grid = [&](bool out) {  // workgroups of each job
        int64_t n = 0;
        for (int k = 0; k <= kMaxJobs; ++k) {
            jobs.first[k] = (uint32_t)n;
            if (k >= jobs.count) continue;
            const Job& j = jobs.j[k];
            n += j.slots * (out || j.Ha < j.Hb ? j.Ha : j.Hb);
            if (n > 0x7fffffff) return (int64_t)0;
        }
        for (int k = jobs.count; k <= kMaxJobs; ++k) jobs.first[k] = 0xffffffffu;  // never reached
        return n;
    };
    if (jobs.j[0].seg_len) {
        const int64_t n = grid(false);
        if (n == 0) return hipErrorNotSupported;
        hipLaunchKernelGGL((chunk_kernel<C, false, VEC>), dim3((uint32_t)n), dim3(C::NT), 0, stream, jobs);
        const Job& j = jobs.j[0];
        const int64_t threads = j.batch * (j.Ha < j.Hb ? j.Ha : j.Hb) * (C::NW * C::NB * 64);
        if ((threads + 255) / 256 > 0x7fffffff) return hipErrorNotSupported;
        hipLaunchKernelGGL((join_kernel<C>), dim3((uint32_t)((threads + 255) / 256), (uint32_t)jobs.count), dim3(256), 0,
                           stream, jobs);
    }
    const int64_t n = grid(true);
    if (n == 0) return hipErrorNotSupported;
    hipLaunchKernelGGL((chunk_kernel<C, true, VEC>), dim3((uint32_t)n), dim3(C::NT), 0, stream, jobs);
    return hipGetLastError();
}

// whole pieces, and offsets within a chunk that fit a buffer resource
inline bool vec_ok(const Heads& h, int D, size_t es) {
    return (uintptr_t)h.p % 16 == 0 && h.ts * es % 16 == 0 && h.hs * es % 16 == 0 && D * es % 16 == 0 &&
           h.ts * es < ((int64_t)1 << 24);
}

// Jobs of one shape (D_a and D_c alike).
template <typename IO>
hipError_t run(Jobs& jobs, hipStream_t stream) {
    const size_t es = sizeof(IO);
    bool vec = true;
    for (int k = 0; k < jobs.count; ++k) {
        Job& j = jobs.j[k];
        vec = vec && vec_ok(j.a, j.Da, es) && vec_ok(j.b, j.Da, es) && vec_ok(j.c, j.Dc, es);
        const size_t p = 4 * es;
        j.out_vec = (uintptr_t)j.out.p % p == 0 && j.out.ts * es % p == 0 && j.out.hs * es % p == 0;
    }
    const int kb = padded_a(jobs.j[0].Da), nw = waves_for(jobs.j[0].Dc);
#define EQL_MIX(KB, NW)                                                     \
    if (kb == KB && nw == NW)                                               \
        return vec ? run_cfg<IO, KB, NW, true>(jobs, stream) : run_cfg<IO, KB, NW, false>(jobs, stream);
    EQL_MIX(1, 4) EQL_MIX(2, 4) EQL_MIX(3, 4) EQL_MIX(4, 4) EQL_MIX(1, 8) EQL_MIX(2, 8) EQL_MIX(3, 8) EQL_MIX(4, 8)
#undef EQL_MIX
    return hipErrorNotSupported;
}

}  // namespace mix
}  // namespace eql
