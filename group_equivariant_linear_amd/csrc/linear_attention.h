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

#include "tiles.h"

namespace eql {
namespace mix {

using namespace tile;

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
    int64_t mean;      // T / batch
    uint32_t per_seq;  // segments of each sequence (no offsets)
    float* part;
    uint32_t wgs;      // workgroups of this launch
    int out_vec;  // rows of out in whole pieces of four
};

// The products of one launch: workgroups first[k] .. first[k + 1] - 1 take jobs[k].
constexpr int kMaxJobs = 3;
struct Jobs {
    Job j[kMaxJobs];
    uint32_t first[kMaxJobs + 1];
    uint32_t base;  // of this launch
    int count;
};

__device__ __forceinline__ int64_t offset_of(const Job& j, int64_t b) {
    const int64_t o = j.offsets[b];
    return o < 0 ? 0 : (o > j.T ? j.T : o);
}

__device__ __forceinline__ void sequence(const Job& j, int64_t b, int64_t& t0, int64_t& t1) {
    if (j.offsets) {
        t0 = offset_of(j, b), t1 = offset_of(j, b + 1);
        t1 = t1 < t0 ? t0 : t1;
    } else {
        t0 = b * j.mean, t1 = t0 + j.mean;
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

__device__ __forceinline__ Segment segment_of(const Job& j, uint32_t slot) {
    Segment s;
    uint32_t first_slot = slot;
    s.b = slot;
    if (j.seg_len && !j.offsets) {
        s.b = slot / j.per_seq;
        first_slot = (uint32_t)s.b * j.per_seq;
    } else if (j.seg_len) {
        uint32_t lo = 0, hi = (uint32_t)j.batch - 1;  // last b whose first slot is at most `slot`
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo + 1) / 2;
            if (offset_of(j, mid) / j.seg_len + mid <= slot) lo = mid;
            else hi = mid - 1;
        }
        s.b = lo;
        first_slot = (uint32_t)(offset_of(j, lo) / j.seg_len) + lo;
    }
    int64_t q0, q1;
    sequence(j, s.b, q0, q1);
    s.t0 = q0, s.t1 = q1;
    s.first = s.last = true;
    s.idle = false;
    if (j.seg_len == 0) return s;
    s.t0 = q0 + (int64_t)(slot - first_slot) * j.seg_len;
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

// The kernel's shape: D_a padded to 32 KB, D_c to 16 NW, NW waves; wave w owns
// columns 16 w .. 16 w + 15 of the state and of the output.
template <typename IO_, int KB_, int NW_, bool OUT_>
struct Cfg {
    using IO = IO_;
    using O = Op<IO_>;
    static constexpr bool OUT = OUT_;
    static constexpr int ES = O::ES, KB = KB_, NW = NW_, NT = 64 * NW_;
    static constexpr int DA = 32 * KB_, NB = DA / 16, NM = DA / O::KS, NS = kChunk / O::KS;
    static constexpr int E = 16 / ES;                                // numbers of a piece
    static constexpr int PA = DA / E, PC = 16 / E, PP = kChunk / E;  // pieces of a row of a and b, c, P
    // a and b of the next chunk load into a second tile while this one is worked on
    // (wide fp32 tiles leave no room for it)
    static constexpr bool TWO = !OUT_ || ES == 2 || KB_ <= 2;
    static constexpr int TILE = kChunk * PA * 16, CTILE = kChunk * PC * 16;
    static constexpr int OFF_B = OUT_ ? (TWO ? 2 : 1) * TILE : 0;
    static constexpr int OFF_C = OFF_B + (TWO ? 2 : 1) * TILE;
    static constexpr int OFF_P = OFF_C + NW * CTILE, LDS = OFF_P + (OUT_ ? kChunk * PP * 16 : 0);
    static constexpr bool ROWS = OUT_ && std::is_same_v<IO_, _Float16>;  // rows of P may carry scales
    // fp16: scores (and with them the outputs until they are stored) times 64, so that
    // ordinary ones lie in the middle of the range
    static constexpr float SCORE = ROWS ? 64.0f : 1.0f;
    // fp16: likewise the states in registers and in `part`
    static constexpr bool COLS = std::is_same_v<IO_, _Float16>;
    static constexpr float STATE = COLS ? 64.0f : 1.0f;
    static constexpr int NPA = (PA + NW - 1) / NW;  // loads of a wave per a or b tile, 64 pieces each
};

// Fragments along the rows of such a tile: rows 16 q + lane % 16, contraction step m
// (pieces 4 m + lane group).  fold() is the same in all blocks q; its high bits permute
// the steps within a run of four.
template <int ES, int P>
struct RowReader {
    static constexpr int N = P / 4 < 4 ? P / 4 : (P % 16 == 0 ? 4 : 2);
    const char* base[N];
    __device__ __forceinline__ void move(int by) {
#pragma unroll
        for (int i = 0; i < N; ++i) base[i] += by;
    }
    __device__ __forceinline__ explicit RowReader(const char* tile) {
        const int lane = (int)threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < N; ++i) base[i] = tile + place<ES, P>(lane & 15, 4 * i + (lane >> 4)) - 64 * i;
    }
    template <typename F>
    __device__ __forceinline__ F get(int q, int m) const {
        return *reinterpret_cast<const F*>(base[m % N] + q * (16 * P * 16) + m * 64);
    }
};

// Fragments along its columns: block a of 16 columns (in the order of state_row),
// contraction over rows KS m + ...
template <class C>
struct ColumnReader {
    static constexpr int P = C::PA, ES = C::ES;
    const char* base[2][C::KB];  // 16-bit types: rows + 0 and + 4, columns from 32 k
    const char* tile;
    __device__ __forceinline__ void move(int by) {
        tile += by;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < C::KB; ++k) base[h][k] += by;
    }
    __device__ __forceinline__ explicit ColumnReader(const char* t) : tile(t) {
        if constexpr (ES == 2) {
            const int lane = (int)threadIdx.x & 63, r = 8 * (lane >> 4) + ((lane & 15) >> 2), u = lane & 3;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < C::KB; ++k) base[h][k] = t + place<ES, P>(r + 4 * h, 4 * k + u);
        }
    }
    __device__ __forceinline__ typename C::O::F get(int a, int m) const {
        if constexpr (ES == 2) {
            const int off = (a & 1) * 8 + m * (32 * P * 16);
            return C::O::column(base[0][a >> 1] + off, base[1][a >> 1] + off);
        } else {
            const int lane = (int)threadIdx.x & 63, kg = lane >> 4, ln = lane & 15;
            typename C::O::F f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = *reinterpret_cast<const float*>(tile + place<ES, P>(16 * m + 4 * kg + e, 4 * a + (ln >> 2)) +
                                                       (ln & 3) * 4);
            return f;
        }
    }
};

// Row of the state that lane group kg holds as element i of block a: such that the
// blocks of one contraction step are, in order, that step's positions of the group.
// (16-bit: run u of block a starts at column 32 (a / 2) + 4 (a % 2) + 8 u of the b tile.)
template <class C>
__device__ __forceinline__ int state_row(int a, int kg, int i) {
    if constexpr (C::ES == 2) return 32 * (a >> 1) + 8 * kg + 4 * (a & 1) + i;
    else return 16 * a + 4 * kg + i;
}

// fp16: a row of decayed scores (times Cfg::SCORE) whose largest is m enters its product as it
// is where no score of it overflows and those that count against the largest are not below
// fp16's normal numbers (2^-8: the floor 2^-25 is 2^-17 of the largest); else times
// range_scale(m).  Whether any row needs it is seen from scores past kRowHigh and from rows whose
// 16 x 16 block on the diagonal has none of kRowLow or more: about one chunk in 5000 of scores
// near 1, whose first rows are one score each there.
constexpr float kRowLow = 0.00390625f, kRowHigh = 32768.0f;
__device__ __forceinline__ float row_scale(float m) {
    return m >= kRowHigh || (m > 0.0f && m < kRowLow) ? range_scale(m) : 1.0f;
}
// Of 16 rows (lane % 16), those for which a lane says yes
__device__ __forceinline__ uint32_t rows_with(bool yes) {
    const uint64_t b = __ballot(yes);
    const uint32_t x = (uint32_t)b | (uint32_t)(b >> 32);
    return (x | x >> 16) & 0xffffu;
}

// fp16: the operands that become two terms (step 2: the state; step 3: the decayed rows of c)
// do so as they are while each column's largest keeps their floor of 2^-24 below 2^-21 of it
// (state) or 2^-27 (rows, before their decays), and none passes the range; else times
// range_scale of that largest.  In units of Cfg::STATE; of c its bits.
constexpr float kColumnLow = 1.0f, kColumnHigh = 32768.0f;
constexpr uint32_t kValueLow = 0x3000, kValueHigh = 0x6000;  // 2^-3, 2^9

// Whether the bits m of a largest |number| are neither 0 nor in low .. high.  That of any lane asks
// for a look at the columns' own, which decide.
__device__ __forceinline__ bool outside(uint32_t m, uint32_t low, uint32_t high) {
    return m - 1 < low - 1 || m > high;
}

// Largest over the four lanes of a column (lane % 16)
template <typename T>
__device__ __forceinline__ T column_max(T v) {
#pragma unroll
    for (int o = 16; o <= 32; o <<= 1) {
        const T w = __shfl_xor(v, o);
        v = w > v ? w : v;
    }
    return v;
}

__device__ __forceinline__ float uniform(float v) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

// Waves per SIMD that the registers are held to.
constexpr int waves_per_simd(int es, int kb, int nw) {
    return es == 4 ? (nw == 8 || kb == 1 ? 2 : 1) : (nw == 8 ? 2 : (kb <= 2 ? 3 : 2));
}
template <class C>
constexpr int kWaves = waves_per_simd(C::ES, C::KB, C::NW);

// Chunks of 64 tokens, in time order or (reversed) from the end.  Per chunk, and per
// head of b and c that shares the state:
//   1. scores P[t][s] = scale g^|t-s| (a_t . b_s) of the causal half, to LDS in the
//      plan dtype, split over the waves by 16 x 16 blocks (fp16: rows that its range does
//      not hold come a second time, times a power of two, which step 4 undoes);
//   2. wave w, for its 16 columns of out^T: the old state (two terms) times a, decayed
//      per token in fp32;
//   3. the state's 16 columns: S = g^n S + b^T (decayed c), the decayed c in three terms
//      (bf16) or two (fp16);
//   4. out^T += c^T P^T, and the rows of out go to memory.
// The state never leaves its wave's registers: the accumulator of step 3 is, in its
// lanes, the operand of step 2.  Two barriers a chunk: the tiles of a and b are there;
// P is there (and the tiles are free).  A wave loads its own columns of c.
// OUT: the whole; else step 3 alone, and the state goes to part[slot].
//
// Memory is the floor (a prompt of 12608 tokens, 12 heads of 64 in bf16 moves 90 MB: 19 us
// at a large copy's 4.7 TB/s), the chunks' own instructions the bound: with the next chunk's
// loads waited for at each barrier it took 32 us, 22 with the loads left out and 22 with the
// arithmetic left out; in flight behind the products, 26.  A chunk is a chain of steps on
// one tile, so other workgroups have to fill its gaps: at 64 tokens three workgroups' tiles
// (two buffers, heads of 64) fit the LDS of a CU.  Measured: bf16 heads of 64 in 26 us for 197
// tokens on three workgroups a CU; f16 heads of 112 (88 KB of LDS, one workgroup a CU) 104 us for
// 1344 tokens on each of 250; fp32 heads of 64, 8 us a chunk, 3.4 of them the fp32 matrix
// instructions' own time.  fp16 takes 3 to 5 percent longer than bf16 for the checks of its range;
// packed training whose every chunk needs scales (gradients of 1e-5) takes 152 us in place of 122.
template <class C, bool VEC>
__global__ __launch_bounds__(C::NT, kWaves<C>) void chunk_kernel(Jobs jobs) {
    using IO = typename C::IO;
    using O = typename C::O;
    using F = typename O::F;
    constexpr bool OUT = C::OUT, TWO = C::TWO;
    constexpr int NS = C::NS, KF = O::KF, ES = C::ES;
    __shared__ __attribute__((aligned(16))) char lds[C::LDS];

    const uint32_t wg = blockIdx.x + jobs.base;
    const int which = wg >= jobs.first[2] ? 2 : (wg >= jobs.first[1] ? 1 : 0);
    const Job j = which == 2 ? jobs.j[2] : (which == 1 ? jobs.j[1] : jobs.j[0]);
    const uint32_t first = jobs.first[which == 2 ? 2 : (which == 1 ? 1 : 0)];
    // consecutive workgroups of a job (heads of one sequence, which may share b and c) on one
    // XCD, and every job on all of them
    const uint32_t id = xcd_remap(wg - first, j.wgs);

    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kg = lane >> 4, ln = lane & 15;
    const int Hkv = j.Ha < j.Hb ? j.Ha : j.Hb, heads = OUT ? j.Ha : Hkv;
    const uint32_t slot = id / (uint32_t)heads;
    const int hx = (int)(id - slot * (uint32_t)heads);
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
    const int total = n_chunks * rb;
    const bool own = 16 * wave < j.Dc;  // waves past D_c only load and score
    const int dc = 16 * wave + ln;
    const int64_t state_at = (seg.b * Hkv + kv) * (int64_t)j.Da * j.Dc;
    const int sgn = rev ? -1 : 1;

    char *const tile_a = lds, *const tile_b = lds + C::OFF_B;
    char *const tc = lds + C::OFF_C + wave * C::CTILE, *const tp = lds + C::OFF_P;
    // fp16, in the quarter of P that step 4 does not read (rows 0 .. 31, tokens 32 .. 63; reversed:
    // rows 32 .. 63, tokens 0 .. 31), 64 bytes of every fourth row: 0 .. 3 the bits of the largest
    // |score| of rows 16 q + lane % 16; 4 + half (of this chunk and the next) word 0, whether the
    // rows have to be looked at.
    auto row_word = [&](int row, int word) {
        return reinterpret_cast<uint32_t*>(tp + (rev ? 32 * C::PP * 16 : 64) + word * 4 + row * (4 * C::PP * 16));
    };
    const Loader<IO, C::PA, C::NPA, true, VEC> la(j.a, j.Da, 0, wave, C::NW), lb(j.b, j.Da, 0, wave, C::NW);
    const Loader<IO, C::PC, C::PC, false, VEC> lc(j.c, j.Dc, 16 * wave, 0, 1);
    auto rows_of = [&](int64_t t) { return (int)(seg.t1 - t < kChunk ? seg.t1 - t : kChunk); };
    auto load_a = [&](int64_t t, int buf) {
        if constexpr (OUT) la.run(j.a, t, hx, rows_of(t), j.Da, 0, wave, C::NW, tile_a + buf * C::TILE);
    };
    auto load_b = [&](int64_t t, int hh, int buf) {
        lb.run(j.b, t, kv * rb + hh, rows_of(t), j.Da, 0, wave, C::NW, tile_b + buf * C::TILE);
    };
    auto load_c = [&](int64_t t, int hh) {
        if (own) lc.run(j.c, t, kv * rb + hh, rows_of(t), j.Dc, 16 * wave, 0, 1, tc);
    };

    int64_t t = seg.t0 + (rev ? (int64_t)(n_chunks - 1) * kChunk : 0);
    if (total > 0) {
        load_a(t, 0);
        load_b(t, 0, 0);
        load_c(t, 0);
    }

    f32x4 S[C::NB];
#pragma unroll
    for (int a = 0; a < C::NB; ++a) S[a] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (OUT && own) {
        if (j.seg_len) {
            const float* p = j.part + (((int64_t)slot * Hkv + kv) * C::NW + wave) * (int64_t)(C::NB * 256) + lane * 4;
#pragma unroll
            for (int a = 0; a < C::NB; ++a) S[a] = *reinterpret_cast<const f32x4*>(p + a * 256);
        } else if (j.S0) {
            const float s0 = n_tok ? (rev ? 1.0f / j.scale : 1.0f) * C::STATE : 1.0f;
#pragma unroll
            for (int a = 0; a < C::NB; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // (rows and columns past the state: any number, then 0)
                    const int da = state_row<C>(a, kg, i);
                    const int ra = da < j.Da ? da : j.Da - 1, rc = dc < j.Dc ? dc : j.Dc - 1;
                    S[a][i] = j.S0[state_at + ra * j.sa + rc * j.sc];
                }
#pragma unroll
            for (int a = 0; a < C::NB; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    S[a][i] = state_row<C>(a, kg, i) < j.Da && dc < j.Dc ? s0 * S[a][i] : 0.0f;
        }
    }

    bool inf_state = false;  // the state may hold an infinity
    if constexpr (OUT && ES == 2) {
        float mx = 0.0f;
#pragma unroll
        for (int a = 0; a < C::NB; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fabsf(S[a][i]));
        inf_state = __any(mx == __builtin_inff());
    }

    // Decays, the same in every whole chunk: of the scores (within a diagonal block, one
    // block apart; g^16 per further block), of the old state at a token (g^16 per block
    // of tokens), of a token's weight in the new state (step m and lane group; element e).
    float near0[4], near1 = 0.0f, wb[NS], we[KF], ge[4];
    const float scale = C::SCORE * j.scale, from_state = C::SCORE / C::STATE * j.scale;  // in what acc holds
    const float g16 = uniform(power(l2, 16)), g64 = uniform(power(l2, kChunk));
    float old = 0.0f;
    if constexpr (OUT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = sgn * (ln - (4 * kg + i));  // t - s (s - t reversed) on the diagonal
            near0[i] = d >= 0 ? scale * power(l2, d) : 0.0f;
        }
        near1 = scale * power(l2, rev ? 16 - ln + 4 * kg : 13 + ln - 4 * kg);  // and ge[i]: g^(16 + d)
        old = from_state * power(l2, rev ? 16 - ln : 1 + ln);
        // blocks of P above (reversed: below) the diagonal that step 4 reads with their neighbours
        for (int i = tid; i < kChunk * C::PP; i += C::NT) reinterpret_cast<u32x4*>(tp)[i] = u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int m = 0; m < NS; ++m)
        wb[m] = C::STATE * power(l2, rev ? O::KS * m + KF * kg : kChunk - O::KS * m - KF * (kg + 1));
    {
        const float g1 = power(l2, 1);
        float up[KF];
        up[0] = 1.0f;
#pragma unroll
        for (int e = 1; e < KF; ++e) up[e] = up[e - 1] * g1;
#pragma unroll
        for (int e = 0; e < KF; ++e) we[e] = uniform(rev ? up[e] : up[KF - 1 - e]);
#pragma unroll
        for (int i = 0; i < 4; ++i) ge[i] = uniform(rev ? up[i] : up[3 - i]);
    }

    RowReader<ES, C::PA> rows_a(tile_a), rows_b(tile_b);
    const RowReader<ES, C::PP> rp(tp);
    ColumnReader<C> cb(tile_b);
    // 16 x 64 tokens of c: its columns of a wave alone, rows of 16 numbers
    const char* const c_lo = ES == 2 ? tc + (8 * kg + (ln >> 2)) * 32 + (ln & 3) * 8 : tc + kg * 256 + ln * 4;

    // the rows of out: element offsets of this lane's four columns at token 16 q + ln
    const uint32_t out_row = (uint32_t)j.out.ts * ES;
    auto out_place = [&](int ln, int kg) { return (uint32_t)ln * out_row + (uint32_t)(16 * wave + 4 * kg) * ES; };
    const uint32_t out_first = out_place(ln, kg);

    f32x4 acc[4];
    int hh = 0, left = n_chunks;  // chunks from this one on
    int ba = 0, bb = 0;           // tiles in use
    int half = 0;                 // fp16: this chunk's of row_word
    bool stored = false;          // four stores went out after this wave's last loads
    for (int it = 0; it < total; ++it) {
        const int n = rows_of(t), nq = (n + 15) / 16;
        const bool last_head = hh + 1 == rb, more = it + 1 < total;
        const int64_t tn = last_head ? t + sgn * kChunk : t;  // of the next iteration
        const int hn = last_head ? 0 : hh + 1;
        // the tiles' loads are older than the last rows' stores, which need not be waited for
        if (stored) asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        stored = false;
        lds_barrier();
        if constexpr (TWO) {
            if (more) {
                if (last_head) load_a(tn, ba ^ 1);
                load_b(tn, hn, bb ^ 1);
            }
        }

        // reversed, the initial state belongs to the last token itself: no decay before it
        const int e0 = (rev && initial_seg && left == n_chunks) ? 0 : 1;
        const bool keep = !OUT || left > 1 || (j.S1 && final_seg && hx % r == 0);  // the state is needed on

        // The chunk's arithmetic, without branches that ordinary numbers take: a whole chunk;
        // part of one; at most 16 tokens.
        auto chunk = [&](auto full_c, auto nq_c) {
            constexpr bool FULL = decltype(full_c)::value;
            constexpr int NQ = decltype(nq_c)::value, NM_T = (16 * NQ + O::KS - 1) / O::KS;  // blocks, steps of tokens
            // (the rare paths compute their indexes where they are: hoisted out of the loop they
            // would take the registers that the whole chunks need)
            int lnp = ln, kgp = kg;
            if constexpr (!FULL) asm volatile("" : "+v"(lnp), "+v"(kgp));
            // the chunk's columns of c, contraction over its tokens
            F ct[NM_T];
            auto column_of_c = [&](int m) {
                F f;
                if constexpr (ES == 2) {
                    f = O::column(c_lo + m * 1024, c_lo + m * 1024 + 128);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] = *reinterpret_cast<const float*>(c_lo + m * 1024 + e * 64);
                }
                return f;
            };
            if (own) {
#pragma unroll
                for (int m = 0; m < NM_T; ++m) ct[m] = column_of_c(m);
            }
            // 1. blocks of the lower triangle, row by row; reversed its transpose, with the keys
            // of a part of a chunk in whole steps of 32
            auto block_of = [&](int idx, int& qb, int& kb) {  // false: past the chunk's end
                const int hi = idx >= 6 ? 3 : (idx >= 3 ? 2 : (idx >= 1 ? 1 : 0));
                const int lo = idx - hi * (hi + 1) / 2;
                qb = rev ? lo : hi, kb = rev ? hi : lo;
                return idx < (NQ == 1 ? 3 : 10) && (FULL || qb < nq);
            };
            auto scores = [&](int qb, int kb, float(&p)[4]) {
                f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int m = 0; m < C::NM; ++m)
                    O::mma(s, rows_b.template get<F>(kb, m), rows_a.template get<F>(qb, m));
                const int apart = rev ? kb - qb : qb - kb;
                const bool diag = apart == 0;
                const float f = near1 * (apart <= 1 ? 1.0f : (apart == 2 ? g16 : g16 * g16));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float w = diag ? near0[i] : f * ge[i];
                    p[i] = diag && w == 0.0f ? 0.0f : s[i] * w;  // (a NaN among the masked scores: 0)
                }
            };
            auto put_scores = [&](int qb, int kb, int ln, int kg, const float(&p)[4]) {
                const int row = 16 * qb + ln;
                if constexpr (ES == 2)
                    *reinterpret_cast<u32x2*>(tp + place<ES, C::PP>(row, 2 * kb + (kg >> 1)) + (kg & 1) * 8) =
                        u32x2{Half<IO>::pack2(p[0], p[1]), Half<IO>::pack2(p[2], p[3])};
                else
                    *reinterpret_cast<f32x4*>(tp + place<ES, C::PP>(row, 4 * kb + kg)) = f32x4{p[0], p[1], p[2], p[3]};
            };
            constexpr int OWN = ((NQ == 1 ? 3 : 10) + C::NW - 1) / C::NW;  // blocks of a wave
            auto largest = [](const float(&p)[4]) {
                return fmaxf(fmaxf(fabsf(p[0]), fabsf(p[1])), fmaxf(fabsf(p[2]), fabsf(p[3])));
            };
            uint32_t small = 0;
            float most = 0.0f;
            if constexpr (OUT) {
#pragma unroll
                for (int k = 0; k < OWN; ++k) {
                    int qb, kb;
                    if (!block_of(wave + k * C::NW, qb, kb)) continue;
                    float p[4];
                    scores(qb, kb, p);
                    if constexpr (C::ROWS) {
                        const float m = largest(p);
                        most = fmaxf(most, m);
                        const uint32_t rows = FULL || n - 16 * qb >= 16 ? 0xffffu : (1u << (n - 16 * qb)) - 1;
                        small |= (qb == kb ? rows : 0u) & ~rows_with(m >= kRowLow);
                    }
                    put_scores(qb, kb, ln, kg, p);
                }
            }
            if constexpr (C::ROWS) {
                if (small || __any(most >= kRowHigh)) [[unlikely]] *row_word(4 + half, 0) = 1;
            }
            if constexpr (C::ROWS) {  // the last chunk's readers are past this chunk's first barrier
                if (wave == 0) {
                    *row_word(kg, ln) = 0;
                    *row_word(4 + (half ^ 1), 0) = 0;
                }
            }
            // the columns of c are in registers: the next chunk's may take their place, unless
            // steps 3 and 4 have to come back to them
            bool odd = false;
            uint32_t top = 0;
            if (own) {
                top = O::top(ct);
                // An infinity or NaN among the chunk's values: the products of steps 3 (where it would
                // be split) and 4 (where rows before it would see 0 times it) take 0 in its place, so
                // that all else keeps its bits, and it joins apart.
                odd = (OUT || ES == 2) && __any(top >= O::kInf);
                if (ES == 2 && odd) {
#pragma unroll
                    for (int m = 0; m < NM_T; ++m) ct[m] = O::finite(ct[m]);
                    top = O::top(ct);
                    inf_state = true;
                }
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                if (more && !odd) load_c(tn, hn);
            }
            // the steps stay apart: mixed, they would not fit the registers
            __builtin_amdgcn_sched_barrier(0);
            if (own) {
                if constexpr (OUT) {
                    // 2.
                    if (hh == 0) {
#pragma unroll
                        for (int q = 0; q < NQ; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
                        float norm = 1.0f;  // of this lane's column
                        bool normed = false;
                        if constexpr (C::COLS) {
                            float mx = 0.0f;
#pragma unroll
                            for (int a = 0; a < C::NB; ++a)
#pragma unroll
                                for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fabsf(S[a][i]));
                            normed = __any(outside(__float_as_uint(mx), __float_as_uint(kColumnLow), __float_as_uint(kColumnHigh)));
                            if (normed) [[unlikely]] {
                                mx = column_max(mx);
                                if (outside(__float_as_uint(mx), __float_as_uint(kColumnLow), __float_as_uint(kColumnHigh)))
                                    norm = range_scale(mx);
                            }
                        }
#pragma unroll
                        for (int m = 0; m < C::NM; ++m) {
                            constexpr int ST = ES == 2 ? 2 : 1;
                            F st[ST], at[NQ];
#pragma unroll
                            for (int q = 0; q < NQ; ++q) at[q] = rows_a.template get<F>(q, m);
                            float v[KF];
#pragma unroll
                            for (int e = 0; e < KF; ++e) v[e] = S[(KF * m + e) / 4][e & 3] * norm;
                            O::split(v, st);
                            // An infinity is its first term (the second would be inf - inf).  The branch also
                            // keeps each step's loads and products together: bf16 packed training takes
                            // 117 us with it, 127 where the compiler mixes the steps.
                            if constexpr (ES == 2) {
                                if (inf_state) [[unlikely]] st[1] = O::finite(st[1]);
                            }
#pragma unroll
                            for (int x = 0; x < ST; ++x)
#pragma unroll
                                for (int q = 0; q < NQ; ++q) O::mma(acc[q], st[x], at[q]);
                            if (m % 2) __builtin_amdgcn_sched_barrier(0);
                        }
                        if (normed) [[unlikely]] {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float back = inverse_of_power(__shfl(norm, 4 * kg + i));
#pragma unroll
                                for (int q = 0; q < NQ; ++q) acc[q][i] *= back;
                            }
                        }
                        if constexpr (FULL) {
                            float d[4];
                            d[0] = (e0 ? old : from_state * power(l2, 15 - ln));
                            d[1] = d[0] * g16, d[2] = d[1] * g16, d[3] = d[2] * g16;
#pragma unroll
                            for (int q = 0; q < 4; ++q) acc[q] *= rev ? d[3 - q] : d[q];
                        } else {
#pragma unroll
                            for (int q = 0; q < NQ; ++q) {
                                const int tq = 16 * q + lnp, d = (rev ? n - 1 - tq : tq) + e0;
                                acc[q] *= from_state * power(l2, d > 0 ? d : 0);
                            }
                        }
                    }
                }
                // 3.
                __builtin_amdgcn_sched_barrier(0);
                if (keep) {
                    float lift = 1.0f;  // of this lane's column of c and of the state
                    bool lifted = false;
                    if constexpr (C::COLS) {
                        lifted = __any(outside(top, kValueLow, kValueHigh));
                        if (lifted) [[unlikely]] {
                            const uint32_t most = column_max(top);
                            if (outside(most, kValueLow, kValueHigh))
                                lift = range_scale(C::STATE * (float)__builtin_bit_cast(_Float16, (uint16_t)most));
                            float mx = 0.0f;  // the state stays finite
#pragma unroll
                            for (int a = 0; a < C::NB; ++a)
#pragma unroll
                                for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fabsf(S[a][i]));
                            const int room = 379 - (int)(__float_as_uint(column_max(mx)) >> 23);
                            lift = fminf(lift, __uint_as_float((uint32_t)(room < 127 ? 127 : (room > 254 ? 254 : room)) << 23));
                        }
                    }
                    if (hh == 0) {
                        const float carry = lift * (FULL ? (e0 ? g64 : power(l2, kChunk - 1)) : power(l2, n - 1 + e0));
#pragma unroll
                        for (int a = 0; a < C::NB; ++a) S[a] *= carry;
                    } else if (lifted) [[unlikely]] {
#pragma unroll
                        for (int a = 0; a < C::NB; ++a) S[a] *= lift;
                    }
#pragma unroll
                    for (int m = 0; m < NM_T; ++m) {
                        float v[KF];
#pragma unroll
                        for (int e = 0; e < KF; ++e) {
                            if constexpr (FULL) {
                                v[e] = O::get(ct[m], e) * we[e] * (C::COLS ? wb[m] * lift : wb[m]);
                            } else {
                                const int s = O::KS * m + KF * kgp + e, d = rev ? s : n - 1 - s;
                                v[e] = O::get(ct[m], e) * power(l2, d > 0 ? d : 0) * (C::STATE * lift);
                            }
                        }
                        F cw[O::TERMS];
                        O::split(v, cw);
#pragma unroll
                        for (int a = 0; a < C::NB; ++a) {
                            const F bt = cb.get(a, m);
#pragma unroll
                            for (int x = 0; x < O::TERMS; ++x) O::mma(S[a], bt, cw[x]);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if (lifted) [[unlikely]] {
#pragma unroll
                        for (int a = 0; a < C::NB; ++a) S[a] *= inverse_of_power(lift);
                    }
                    if (ES == 2 && odd) [[unlikely]] {
                        // what is not finite, as one term and without its decay, which takes nothing off it
                        // (a decay of 0, no memory, would make it NaN: the next chunk's carry does)
#pragma unroll
                        for (int m = 0; m < NM_T; ++m) {
                            const F rest = O::finite(column_of_c(m), true);
#pragma unroll
                            for (int a = 0; a < C::NB; ++a) O::mma(S[a], cb.get(a, m), rest);
                        }
                        // (times the zeros past D_a)
                        int kgo = kg;
                        asm volatile("" : "+v"(kgo));
#pragma unroll
                        for (int a = 0; a < C::NB; ++a)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (state_row<C>(a, kgo, i) >= j.Da) S[a][i] = 0.0f;
                    }
                }
            }
            if constexpr (!OUT && ES == 2) {
                if (odd) {
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    if (more) load_c(tn, hn);
                }
            }
            lds_barrier();  // P is there; the tiles of a and b are free
            if constexpr (!TWO) {
                if (more) {
                    if (last_head) load_a(tn, 0);
                    load_b(tn, hn, 0);
                }
            }
            bool ranged = false;  // rows of P carry scales
            // fp16: the fragments of P that step 4 takes, read along with the flags: whole blocks of
            // rows 0 and 1 (first half of the chunk's tokens), 2 and 3 (second half), and the other
            // half of the two blocks that have one (reversed 0 and 1, else 2 and 3)
            constexpr int NP = !C::ROWS ? 1 : (NQ == 4 ? 6 : 1);
            F pf[NP];
            auto read_p = [&] {
                pf[0] = rp.template get<F>(0, 0);
                if constexpr (NP == 6) {
                    pf[1] = rp.template get<F>(1, 0);
                    pf[2] = rp.template get<F>(2, 1);
                    pf[3] = rp.template get<F>(3, 1);
                    const char* const more = rev ? rp.base[1] + 64 : rp.base[0] + 2 * (16 * C::PP * 16);
                    pf[4] = *reinterpret_cast<const F*>(more);
                    pf[5] = *reinterpret_cast<const F*>(more + 16 * C::PP * 16);
                }
            };
            auto scale_of = [&](int q) { return row_scale(__uint_as_float(*row_word(q, ln))); };
            if constexpr (C::ROWS) {
                const uint32_t look = *row_word(4 + half, 0);
                read_p();
#pragma unroll
                for (int i = 0; i < NP; ++i) asm volatile("" : "+v"(pf[i]));  // here, not past the branch
                ranged = __builtin_amdgcn_readfirstlane(look) != 0;
                if (ranged) [[unlikely]] {
                    float p[OWN][4];
#pragma unroll
                    for (int k = 0; k < OWN; ++k) {
                        int qb, kb;
                        if (!block_of(wave + k * C::NW, qb, kb)) continue;
                        scores(qb, kb, p[k]);
                        atomicMax(row_word(qb, ln), __float_as_uint(largest(p[k])));
                    }
                    lds_barrier();
                    int lns = ln, kgs = kg;
                    asm volatile("" : "+v"(lns), "+v"(kgs));  // (as above)
#pragma unroll
                    for (int k = 0; k < OWN; ++k) {
                        int qb, kb;
                        if (!block_of(wave + k * C::NW, qb, kb)) continue;
                        const float sc = scale_of(qb);
#pragma unroll
                        for (int i = 0; i < 4; ++i) p[k][i] *= sc;
                        put_scores(qb, kb, lns, kgs, p[k]);
                    }
                    if (own) {
#pragma unroll
                        for (int q = 0; q < NQ; ++q) acc[q] *= scale_of(q);
                    }
                    lds_barrier();
                    read_p();
                }
            }
            if constexpr (OUT) {
                if (own) {
                    // 4.  What is not finite among the chunk's values is added one by one by the rows
                    // that see it.
                    if (ES == 4 && odd) {
#pragma unroll
                        for (int m = 0; m < NM_T; ++m) ct[m] = O::finite(ct[m]);
                    }
                    // (P is 0 in the blocks that are not written)
                    if constexpr (NP == 6) {
                        if (!rev) {
                            O::mma(acc[2], ct[0], pf[4]);
                            O::mma(acc[3], ct[0], pf[5]);
                        }
                        O::mma(acc[0], ct[0], pf[0]);
                        O::mma(acc[1], ct[0], pf[1]);
                        O::mma(acc[2], ct[1], pf[2]);
                        O::mma(acc[3], ct[1], pf[3]);
                        if (rev) {
                            O::mma(acc[0], ct[1], pf[4]);
                            O::mma(acc[1], ct[1], pf[5]);
                        }
                    } else if constexpr (C::ROWS) {
                        O::mma(acc[0], ct[0], pf[0]);
                    } else {
#pragma unroll
                        for (int m = 0; m < NM_T; ++m)
#pragma unroll
                            for (int q = 0; q < NQ; ++q) O::mma(acc[q], ct[m], rp.template get<F>(q, m));
                    }
                    if (odd) {
                        int lno = ln, kgo = kg;
                        asm volatile("" : "+v"(lno), "+v"(kgo));
                        for (int s = 0; s < n; ++s)
#pragma unroll
                            for (int q = 0; q < NQ; ++q) {
                                const int tq = 16 * q + lno;
                                if (rev ? s < tq : s > tq) continue;
                                const float p =
                                    (float)*reinterpret_cast<const IO*>(tp + place<ES, C::PP>(tq, s / C::E) + s % C::E * ES);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float v = (float)*reinterpret_cast<const IO*>(tc + (s * 16 + 4 * kgo + i) * ES);
                                    if (!(fabsf(v) < __builtin_inff())) acc[q][i] = fmaf(p, v, acc[q][i]);
                                }
                            }
                        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                        if (more) load_c(tn, hn);
                    }
                    if constexpr (C::ROWS) {
                        if (ranged) [[unlikely]] {
#pragma unroll
                            for (int q = 0; q < NQ; ++q) acc[q] *= inverse_of_power(scale_of(q));
                        }
                    }
                    if (last_head) {
                        if constexpr (C::SCORE != 1.0f) {
#pragma unroll
                            for (int q = 0; q < NQ; ++q) acc[q] *= 1.0f / C::SCORE;
                        }
                        IO* out = (IO*)const_cast<void*>(j.out.p) + t * j.out.ts + hx * j.out.hs;
                        if (j.out_vec) {
                            asm volatile("" ::: "memory");  // the loads above stay older than these
                            __builtin_amdgcn_sched_barrier(0);
                            const __amdgpu_buffer_rsrc_t ro = make_rsrc(out, (uint32_t)(((n - 1) * j.out.ts + j.Dc) * ES));
                            const bool in = 16 * wave + 4 * kg < j.Dc;
                            uint32_t out_at = out_first;
                            if constexpr (C::ROWS) {  // not kept: the fp16 kernels need its register
                                int lno = ln, kgo = kg;
                                asm volatile("" : "+v"(lno), "+v"(kgo));
                                out_at = out_place(lno, kgo);
                            }
#pragma unroll
                            for (int q = 0; q < NQ; ++q) {
                                const uint32_t at = in && (FULL || 16 * q + lnp < n) ? out_at + 16 * q * out_row : kOOB;
                                if constexpr (ES == 2)
                                    __builtin_amdgcn_raw_buffer_store_b64(
                                        u32x2{Half<IO>::pack2(acc[q][0], acc[q][1]), Half<IO>::pack2(acc[q][2], acc[q][3])},
                                        ro, at, 0, 0);
                                else
                                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[q]), ro, at, 0, 0);
                            }
                            stored = NQ == 4;
                        } else {
                            int lno = ln, kgo = kg;
                            asm volatile("" : "+v"(lno), "+v"(kgo));
                            const int c0 = 16 * wave + 4 * kgo;
#pragma unroll
                            for (int q = 0; q < NQ; ++q) {
                                if (16 * q + lno >= n) continue;
                                IO* p = out + (16 * q + lno) * j.out.ts + c0;
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (c0 + i < j.Dc) p[i] = (IO)acc[q][i];
                            }
                        }
                    }
                }
            }
        };
        if (n == kChunk) chunk(std::true_type{}, std::integral_constant<int, 4>{});
        else if (n > 16) chunk(std::false_type{}, std::integral_constant<int, 4>{});
        else chunk(std::false_type{}, std::integral_constant<int, 1>{});
        if constexpr (TWO) {
            const int step_b = bb ? -C::TILE : C::TILE;
            rows_b.move(step_b);
            cb.move(step_b);
            bb ^= 1;
            if (last_head) {
                rows_a.move(ba ? -C::TILE : C::TILE);
                ba ^= 1;
            }
        }
        t = tn;
        hh = hn;
        half ^= 1;
        if (last_head) --left;
    }

    if (!own) return;
    if (!OUT) {
        float* p = j.part + (((int64_t)slot * Hkv + kv) * C::NW + wave) * (int64_t)(C::NB * 256) + lane * 4;
#pragma unroll
        for (int a = 0; a < C::NB; ++a) *reinterpret_cast<f32x4*>(p + a * 256) = S[a];
    } else if (j.S1 && final_seg && hx % r == 0) {
        const float s1 = n_tok ? (rev ? power(l2, 1) * j.scale : 1.0f) * (1.0f / C::STATE) : 1.0f;
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
    sequence(j, b, t0, t1);
    const int64_t segs = t1 > t0 ? (t1 - t0 + j.seg_len - 1) / j.seg_len : 1;
    const int64_t slot0 = j.offsets ? t0 / j.seg_len + b : b * segs;
    const float l2 = j.log_decay[kv] * kLog2e;
    f32x4 S = {0.f, 0.f, 0.f, 0.f};
    if (j.S0) {
        const int64_t at = (b * Hkv + kv) * (int64_t)j.Da * j.Dc;
        const float s0 = t1 > t0 ? (j.reverse ? 1.0f / j.scale : 1.0f) * C::STATE : 1.0f;
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
    using C = Cfg<IO, KB, NW, true>;
    using CS = Cfg<IO, KB, NW, false>;
    auto grid = [&](bool out) {  // workgroups of each job
        int64_t n = 0;
        for (int k = 0; k <= kMaxJobs; ++k) {
            jobs.first[k] = (uint32_t)n;
            if (k >= jobs.count) continue;
            Job& j = jobs.j[k];
            const int64_t w = j.slots * (out || j.Ha < j.Hb ? j.Ha : j.Hb);
            n += w;
            if (n > 0x7fffffff) return (int64_t)0;
            j.wgs = (uint32_t)w;
        }
        for (int k = jobs.count; k <= kMaxJobs; ++k) jobs.first[k] = 0xffffffffu;  // never reached
        return n;
    };
    if (jobs.j[0].seg_len) {
        const int64_t n = grid(false);
        if (n == 0) return hipErrorNotSupported;
        in_pieces(n, C::NT, [&](uint32_t base, uint32_t wgs) {
            jobs.base = base;
            hipLaunchKernelGGL((chunk_kernel<CS, VEC>), dim3(wgs), dim3(C::NT), 0, stream, jobs);
        });
        const Job& j = jobs.j[0];
        const int64_t threads = j.batch * (j.Ha < j.Hb ? j.Ha : j.Hb) * (C::NW * C::NB * 64);
        if (threads > 0x7fffffff) return hipErrorNotSupported;  // (segments are for few sequences)
        hipLaunchKernelGGL((join_kernel<C>), dim3((uint32_t)((threads + 255) / 256), (uint32_t)jobs.count), dim3(256), 0,
                           stream, jobs);
    }
    const int64_t n = grid(true);
    if (n == 0) return hipErrorNotSupported;
    in_pieces(n, C::NT, [&](uint32_t base, uint32_t wgs) {
        jobs.base = base;
        hipLaunchKernelGGL((chunk_kernel<C, VEC>), dim3(wgs), dim3(C::NT), 0, stream, jobs);
    });
    return hipGetLastError();
}

// Jobs of one shape (D_a and D_c alike).
template <typename IO>
hipError_t run(Jobs& jobs, hipStream_t stream) {
    const size_t es = sizeof(IO);
    bool vec = true;
    for (int k = 0; k < jobs.count; ++k) {
        Job& j = jobs.j[k];
        vec = vec && vec_ok(j.a, j.Da, es, 16) && vec_ok(j.b, j.Da, es, 16) && vec_ok(j.c, j.Dc, es, 16);
        j.out_vec = vec_ok(j.out, j.Dc, es, 4 * es);
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
