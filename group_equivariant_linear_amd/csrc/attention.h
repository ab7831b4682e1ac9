// attention.h -- softmax attention on matrix cores: forward, and the gradients from
// recomputed probabilities.
//
//   s_ij = scale q_i . k_j + bias[bucket(p_i - j)],  p_i = i + n_k - n_q
//   P = softmax over the keys that query i sees,  o_i = sum_j P_ij v_j
//   dP = d_o v^T,  dS = P (dP - delta),  delta_i = d_o_i . o_i
//   dq = scale dS k,  dk = scale dS^T q,  dv = P^T d_o,  dbias[b] = sum of dS over bucket b
//
// One wave owns 32 rows (queries, or keys for dk and dv) as columns of its accumulators:
// its scores come as S^T = K Q^T in blocks of 32 x 32, a lane holding 16 numbers of one of
// its rows (lane % 32).  Statistics of a row are then a lane's own (and its partner's, lane
// ^ 32), and the block, packed to the plan's type, is at once the operand of the next
// product: the contraction runs over the numbers in the order in which the lane holds
// them, and the other operand is read from its row-major tile in that order.
#pragma once

#include "tiles.h"

namespace eql {
namespace att {

using namespace tile;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) float lds_float;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kRows = 128;  // rows that a workgroup's four waves own
constexpr int kTile = 64;   // rows of the tiles that they pass over
constexpr int kPad = 96;    // a wave's rows and a tile span fewer distances than this
constexpr float kInf = __builtin_inff();
// Rows whose |lse| passes this are steep: fp32 holds lse, and scores less lse, to 2^-14 and worse, and to no fraction
// from 2^24 on.  dq_kernel finds their largest score again, bit for bit, and probabilities are made from the
// difference to it.  (16 bit: dkv_kernel's accumulators start at lse and are rounded at its size up to 8 times: at this
// one 2^-11 of a probability at most, fp16's own rounding of it and an eighth of bf16's.)
constexpr float kSteepLse = 1024.0f;

template <typename IO>
struct Op32 : Op<IO> {  // __bf16, _Float16
    using F = typename Half<IO>::x8;
    static __device__ __forceinline__ void mma(f32x16& acc, const F& a, const F& b) {
        if constexpr (Op<IO>::BF) acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0);
        else acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, acc, 0, 0, 0);
    }
    static __device__ __forceinline__ F pack(const float* p) {
        u32x4 u;
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = Half<IO>::pack2(p[2 * i], p[2 * i + 1]);
        return __builtin_bit_cast(F, u);
    }
};
template <>
struct Op32<float> : Op<float> {
    using F = f32x4;
    static __device__ __forceinline__ void mma(f32x16& acc, const F& a, const F& b) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], acc, 0, 0, 0);
    }
    static __device__ __forceinline__ F pack(const float* p) { return F{p[0], p[1], p[2], p[3]}; }
};

// Shapes for heads of up to 32 DB numbers.  Lane l: row (column) l % 32, half h = l / 32.
// A step along a row takes two pieces of 16 bytes, one of each half; a step along the
// columns of a tile (over its rows) 2 E rows, which are those of accumulators E t .. E t +
// E - 1 of both halves: row 8 (i / 4) + 4 h + i % 4 of a block belongs to accumulator i.
template <typename IO, int DB_>
struct Shape {
    static constexpr int ES = (int)sizeof(IO), E = 16 / ES, DB = DB_, D = 32 * DB_;
    static constexpr int P = D / E, NS = P / 2, NT = 16 / E;
    static constexpr int TILE = kTile * P * 16;
};
__device__ __forceinline__ constexpr int row_of(int i) { return 8 * (i >> 2) + (i & 3); }  // + 4 h

// Fragments along the rows of a tile: block of 32 rows, step s.
template <class C>
struct RowFrags {
    static constexpr int R = C::P % 16 == 0 ? 8 : (C::P % 8 == 0 ? 4 : 2), N = R < C::NS ? R : C::NS;
    const char* base[N];
    __device__ __forceinline__ explicit RowFrags(const char* t) {
        const int lane = (int)threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < N; ++i) base[i] = t + place<C::ES, C::P>(lane & 31, 2 * i + (lane >> 5));
    }
    template <typename F>
    __device__ __forceinline__ F get(int by, int block, int s) const {
        return *reinterpret_cast<const F*>(base[s % N] + by + block * (32 * C::P * 16) + s / N * (N * 32));
    }
};

// Fragments along its columns: columns 32 cb .. of rows 32 block + 2 E t ..
template <class C, typename O>
struct ColumnFrags {
    static constexpr int R = C::P % 16 == 0 ? 4 : (C::P % 8 == 0 ? 2 : 1), N = R < C::DB ? R : C::DB;
    const char* base[2][N];
    const char* tile;
    __device__ __forceinline__ explicit ColumnFrags(const char* t) : tile(t) {
        if constexpr (C::ES == 2) {
            const int lane = (int)threadIdx.x & 63, u = lane & 3, r = 4 * (lane >> 5) + ((lane & 15) >> 2);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int piece = 4 * k + 2 * ((lane >> 4) & 1) + (u >> 1);
                base[0][k] = t + place<C::ES, C::P>(r, piece) + (u & 1) * 8;
                base[1][k] = t + place<C::ES, C::P>(r + 8, piece) + (u & 1) * 8;
            }
        }
    }
    __device__ __forceinline__ typename O::F get(int by, int block, int t, int cb) const {
        if constexpr (C::ES == 2) {
            const int off = by + cb / N * (N * 64) + (32 * block + 16 * t) * (C::P * 16);
            return O::column(base[0][cb % N] + off, base[1][cb % N] + off);
        } else {
            const int lane = (int)threadIdx.x & 63, h = lane >> 5, ln = lane & 31;
            typename O::F f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = *reinterpret_cast<const float*>(
                    tile + by + place<C::ES, C::P>(32 * block + 8 * t + 4 * h + e, 8 * cb + (ln >> 2)) + (ln & 3) * 4);
            return f;
        }
    }
};

// What the products with finite operands left out of acc: the infinities and NaN of a block of 32 rows
// of a tile.  (A product would spread those in unseen rows as well: 0 times infinity.)  `sees`: the rows
// that the lane's row sees, a bit each.  Of 32 columns, a lane finds the rows of +infinity or NaN in one, or
// (upper half) of -infinity or NaN.  nan: any is a NaN at once (it multiplies factors that may be 0).  Rare,
// and held to few registers; no LDS of its own (4 KB more left one workgroup a CU of two in dq_kernel at 128
// numbers a head, reach 128: 152 us for 111).
template <class C, typename IO>
__device__ __forceinline__ void add_odd_numbers(f32x16 (&acc)[C::DB], const char* tile, uint32_t sees, bool nan) {
    int lane = (int)threadIdx.x & 63;
    asm volatile("" : "+v"(lane)::"memory");  // (addresses are made here, not kept from the kernel's start on)
    const float sign = lane >> 5 ? -1.0f : 1.0f;
    uint32_t met[C::DB] = {};
#pragma unroll 1
    for (int row = 0; row < 32; ++row)
#pragma unroll
        for (int cb = 0; cb < C::DB; ++cb) {
            const int d = 32 * cb + (lane & 31);
            const float x = (float)*reinterpret_cast<const IO*>(tile + place<C::ES, C::P>(row, d / C::E) + d % C::E * C::ES);
            if (!(fabsf(x) < kInf) && (nan || !(x * sign < 0.0f))) met[cb] |= 1u << row;
        }
    const int from = (lane >> 5) * 16;
#pragma unroll
    for (int cb = 0; cb < C::DB; ++cb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i % 4 == 0) asm volatile("" ::: "memory");
            // column row_of(i) + 4 h's lanes
            const int pos = __builtin_amdgcn_ds_bpermute(from + 4 * row_of(i), (int)met[cb]);
            const int neg = __builtin_amdgcn_ds_bpermute(from + 4 * row_of(i) + 128, (int)met[cb]);
            acc[cb][i] += pos & (int)sees ? kInf : 0.0f;
            acc[cb][i] += neg & (int)sees ? -kInf : 0.0f;
        }
    asm volatile("" ::: "memory");
}
// N fragments with these as 0; odd: the largest number met, as O::top has it.
template <typename O, typename F, int N>
__device__ __forceinline__ void take_finite(F (&f)[N], uint32_t& odd) {
    const uint32_t o = O::top(f);
    odd = o > odd ? o : odd;
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = O::finite(f[i]);
}
// Fragments read before such a look that is taken or not: their loads wait together, not one by one.
template <bool ALWAYS>
constexpr int kAtOnce = ALWAYS ? 1 : 2;
// Bits 0 .. last (none below 0, all from 31 on).
__device__ __forceinline__ uint32_t bits_to(int last) { return last >= 31 ? ~0u : (last < 0 ? 0u : (2u << last) - 1u); }
// Bits of the 32 distances from d on, step apart, whose biases in tab are -infinity.
__device__ __forceinline__ uint32_t taken_out_of(const float* tab, int reach, int d, int step) {
    uint32_t out = 0;
#pragma unroll 1
    for (int r = 0; r < 32; ++r, d += step) {
        const int at = d > reach ? reach : (d < -reach ? -reach : d);
        out |= tab[reach + kPad + at] == -kInf ? 1u << r : 0u;
    }
    return out;
}

template <int N>
__device__ __forceinline__ void clear(f32x16 (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = f32x16{};
}

// Rows of one sequence.
struct Seq {
    int64_t q0, k0;  // first tokens
    int n_q, n_k;
};

__device__ __forceinline__ int64_t clamped(const int64_t* offsets, int64_t b, int64_t T) {
    const int64_t o = offsets[b];
    return o < 0 ? 0 : (o > T ? T : o);
}
__device__ __forceinline__ void tokens_of(const int64_t* offsets, int64_t batch, int64_t T, int64_t b, int64_t& t0, int& n) {
    if (offsets) {
        const int64_t e = clamped(offsets, b + 1, T);
        t0 = clamped(offsets, b, T);
        n = e > t0 ? (int)(e - t0) : 0;
    } else {
        n = (int)(T / batch);
        t0 = b * n;
    }
}

// Slot `slot` of runs of kRows tokens: its sequence and first row.  Packed sequence b owns
// the slots from offsets[b] / kRows + b on, at least as many as it has runs.
__device__ __forceinline__ void slot_of(const int64_t* offsets, int64_t batch, int64_t T, uint32_t slot, int64_t& b, int64_t& row) {
    if (!offsets) {
        const int64_t n = T / batch;
        const uint32_t per = (uint32_t)((n + kRows - 1) / kRows);
        b = slot / per;
        row = (int64_t)(slot - (uint32_t)b * per) * kRows;
        return;
    }
    // last b whose first slot is at most `slot`: 64 of them looked at in one load
    const int lane = (int)threadIdx.x & 63;
    int64_t lo = 0, n = batch;
    while (n > 1) {
        const int64_t step = (n + 63) / 64, at = lane * step;
        const bool yes = at < n && clamped(offsets, lo + at, T) / kRows + lo + at <= slot;
        const int last = __popcll(__ballot(yes)) - 1;  // (first slots ascend)
        const int64_t from = (last < 0 ? 0 : last) * step;
        lo += from;
        n = n - from < step ? n - from : step;
    }
    b = lo;
    row = ((int64_t)slot - clamped(offsets, lo, T) / kRows - lo) * kRows;
}

// A workgroup's head and slot.  Short sequences: the slots of all heads in a row, an eighth to
// each XCD, so that those of a sequence find each other's k and v (q and d_o) in its L2.  Long
// ones (dealt): units of a (sequence, head), or a head of packed sequences, go whole to the XCDs as far
// as all get as many, and the slots of those left are dealt to all; the longest slots of a causal unit
// first (falling: the last).  10 heads of 32768 causal tokens took 3500 us in a row (an XCD had
// 1.06 to 1.44 heads' work), 3250 with every head dealt.
struct Place {
    int head;
    uint32_t slot;
};
__device__ __forceinline__ Place place_of(uint32_t base, const Deal& d, bool falling) {
    if (d.units == 0) {
        const uint32_t id = xcd_remap(blockIdx.x, gridDim.x) + base;
        return Place{(int)(id / d.slots), id % d.slots};
    }
    const uint32_t id = blockIdx.x + base, xcd = id % 8, whole = d.units / 8;
    uint32_t k = id / 8, unit, i;
    if (k < whole * d.slots) {
        unit = xcd * whole + k / d.slots;
        i = k % d.slots;
        if (falling) i = d.slots - 1 - i;
    } else {
        const uint32_t per = (d.slots + 7) / 8;
        k -= whole * d.slots;
        unit = 8 * whole + k / per;
        i = k % per;
        i = (falling ? per - 1 - i : i) * 8 + xcd;
        if (i >= d.slots) return Place{-1, 0};
    }
    return Place{(int)(unit / d.per_head), unit % d.per_head * d.slots + i};
}

// Biases (times log2 e) of the distances -(reach + kPad) .. reach + kPad, at distance + reach +
// kPad of `tab`; behind them the least distance of each bucket of one side, and one past the
// reach.  A wave's lanes hold 64 buckets' starts and biases, loaded before all else, and the wave
// writes every 4th (of all: 256 / 64) bucket's distances: no wait between load and store.  (A
// search of each distance's bucket in LDS took 29.2 us for 64 images, this 27.7.)  Ends with its writes not waited for.
// Returns whether one of them is -infinity, alike in all waves: a key at such a distance is not seen, whatever stands there.
__host__ __device__ constexpr int tab_width(int reach) { return 2 * (reach + kPad) + 1; }
__host__ __device__ constexpr int table_words(int reach, int buckets) { return tab_width(reach) + buckets + 1; }
struct BiasLanes {  // of buckets b0 + lane
    int start, next;
    float before, after;
};
// A bias in powers of two; a finite one stays finite (from 2.36e38 on its product is past fp32's largest number).
__device__ __forceinline__ float in_powers(float bias) {
    constexpr float most = 0x1.fffffep127f;
    const float y = kLog2e * bias;
    return fabsf(bias) < kInf ? fminf(fmaxf(y, -most), most) : y;
}
template <typename IO>
__device__ __forceinline__ BiasLanes load_biases(const AttentionArgs& a, const BucketMap& map, int head, int b0 = 0) {
    const int side = a.causal ? a.buckets : a.buckets / 2, b = b0 + ((int)threadIdx.x & 63);
    BiasLanes x{0, 0, 0.0f, 0.0f};
    if (b < side) {
        x.start = map.start[b], x.next = map.start[b + 1];
        const IO* const row = (const IO*)a.bias + (int64_t)head * a.buckets;
        if (a.bias) x.before = in_powers((float)row[b]), x.after = a.causal ? x.before : in_powers((float)row[side + b]);
    }
    return x;
}
template <typename IO, int THREADS = 256>
__device__ __forceinline__ bool fill_biases(float* tab, BiasLanes x, const AttentionArgs& a, const BucketMap& map, int head) {
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int off = a.reach + kPad, side = a.causal ? a.buckets : a.buckets / 2;
    int* const starts = reinterpret_cast<int*>(tab + tab_width(a.reach));
    bool out = false;
    for (int b0 = 0; b0 < side; b0 += 64) {
        if (b0) x = load_biases<IO>(a, map, head, b0);
        if (wave == 0 && b0 + lane < side) starts[b0 + lane] = x.start, starts[b0 + lane + 1] = x.next;
        out |= __any(x.before == -kInf || x.after == -kInf);
        const int n = side - b0 < 64 ? side - b0 : 64;
        for (int b = wave; b < n; b += THREADS / 64) {
            const int from = __builtin_amdgcn_readlane(x.start, b), next = __builtin_amdgcn_readlane(x.next, b);
            const int to = next > a.reach ? off : next - 1;
            const float before = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x.before), b));
            const float after = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x.after), b));
            for (int m = from + lane; m <= to; m += 64) {
                tab[off + m] = before;
                if (m) tab[off - m] = after;
            }
        }
    }
    if (side == 0)
        for (int m = tid; m <= 2 * off; m += THREADS) tab[m] = 0.0f;
    return out;
}

// Scores x of a block in powers of two, with the biases at t[STEP row_of(i)]; a key whose bias takes
// it out has -infinity, whatever its number (and 0 in y).  Returns these, bit i of accumulator i.
template <int STEP>
__device__ __forceinline__ uint32_t biased_or_out(f32x16& x, f32x16& y, float scale, const float* t) {
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float bias = t[STEP * row_of(i)];
        const bool gone = bias == -kInf;
        x[i] = gone ? -kInf : __builtin_fmaf(x[i], scale, bias);
        y[i] = gone ? 0.0f : y[i];
        out |= gone ? 1u << i : 0u;
    }
    return out;
}

// Fragments of 32 rows from memory, the operand of the products over the head's numbers.
template <class C, typename IO, typename F, bool VEC>
__device__ __forceinline__ void load_rows(F (&f)[C::NS], const Heads& x, int64_t t, int64_t head, int n, int D) {
    const int lane = (int)threadIdx.x & 63, row = lane & 31, h = lane >> 5;
    const IO* base = (const IO*)x.p + t * x.ts + head * x.hs;
    if constexpr (VEC) {
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(base, n > 0 ? (uint32_t)(((int64_t)((n < 32 ? n : 32) - 1) * x.ts + D) * C::ES) : 0u);
#pragma unroll
        for (int s = 0; s < C::NS; ++s) {
            const int col = (2 * s + h) * C::E;
            const uint32_t off = col < D && row < n ? (uint32_t)(row * (int)x.ts + col) * C::ES : kOOB;
            f[s] = __builtin_bit_cast(F, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
        }
    } else {
#pragma unroll
        for (int s = 0; s < C::NS; ++s) {
            u32x4 v = {0u, 0u, 0u, 0u};
            if (row < n) v = load_piece<IO>(base + row * x.ts, (2 * s + h) * C::E, D);
            f[s] = __builtin_bit_cast(F, v);
        }
    }
}

// Waits for fragments loaded from memory.  (Otherwise each pass of a loop waits for them at
// their use, and with them for the tiles in flight, which the compiler does not count.)
template <typename F, int N>
__device__ __forceinline__ void arrive(F (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(f[i]));
}

// The numbers of fragments with their signs turned.
template <typename F, int N>
__device__ __forceinline__ void negate(F (&f)[N]) {
    constexpr uint32_t sign = sizeof(f[0][0]) == 2 ? 0x80008000u : 0x80000000u;
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __builtin_bit_cast(F, __builtin_bit_cast(u32x4, f[i]) ^ sign);
}

// The larger of a lane's number and its partner's (lane ^ 32).
__device__ __forceinline__ float half_max(float v) {
    const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
}

// Accumulators of 32 rows to memory, times m, rounded once.
template <class C, typename IO>
__device__ __forceinline__ void store_rows(const f32x16 (&acc)[C::DB], const Heads& x, int64_t t, int64_t head, int n, int D,
                                           float m, int vec) {
    const int lane = (int)threadIdx.x & 63, row = lane & 31, h = lane >> 5;
    if (row >= n) return;
    IO* const p = (IO*)const_cast<void*>(x.p) + (t + row) * x.ts + head * x.hs;
#pragma unroll
    for (int cb = 0; cb < C::DB; ++cb)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int d = 32 * cb + 8 * g + 4 * h;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = m * acc[cb][4 * g + e];
            if (vec) {
                if (d < D) {
                    if constexpr (C::ES == 2)
                        *reinterpret_cast<u32x2*>(p + d) = u32x2{Half<IO>::pack2(v[0], v[1]), Half<IO>::pack2(v[2], v[3])};
                    else *reinterpret_cast<f32x4*>(p + d) = f32x4{v[0], v[1], v[2], v[3]};
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (d + e < D) p[d + e] = (IO)v[e];
            }
        }
}

// The power of two by which a lane's sums of dS times rows are held: fp16 takes dS only near
// the middle of its range.  Starts high and comes down, like a running maximum.
constexpr float kTopScale = 18446744073709551616.0f;  // 2^64

// fp16: probabilities are held times 2^12 (at most 2^15, see kSlack), so that one of 2^-36 of
// the largest still counts.
template <typename IO>
constexpr float kShift = std::is_same_v<IO, _Float16> ? 12.0f : 0.0f;
// How far (in powers of two) a score may pass the running maximum before the sums are scaled
// to a new one.
template <typename IO>
constexpr float kSlack = std::is_same_v<IO, _Float16> ? 3.0f : 8.0f;

__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// 64 numbers of 4 bytes, one from each lane's offset in the resource, to LDS from `to` on.
__device__ __forceinline__ void load_words_to_lds(const u32x4& rsrc, uint32_t offset, const float* to) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)to);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 :
                 : "v"(offset), "s"(rsrc), "s"(at)
                 : "memory");
}

// Two tiles, 64 rows each, pass through LDS; where both fit twice into half of it, the next
// pair's loads are in flight behind the products of this one.
template <class C>
constexpr int kStages = 4 * C::TILE <= 80 * 1024 ? 2 : 1;

// What work on a tile has to look at: every row sees all of it; some of its rows are not
// there (zeros); some are there and not seen, so that no infinity of theirs may be multiplied.
// (UNSEEN kernels look for those: causal ones, and those for rows off 16 bytes, which are one
// for all calls; others with biases do for a head whose biases take keys out: looking at all edges
// took 31.7 us for 64 images, this 28.1.)
constexpr int kWhole = 0, kPartial = 1, kUnseen = 2;
template <int K>
using Kind = std::integral_constant<int, K>;

// `rounds` rounds of n visits to pairs of tiles: load(v, stage) of visit v (counted through
// all rounds), then, when its tiles are there, a(v, stage) for a round's first n_a() visits and
// b(v, stage) for the others; between(r) after round r.  Every wave calls it, and a() and b() have no
// barrier.  start_pass() before it loads the first tiles: early, as the rest of what a
// kernel starts with can be on its way at the same time.  (Loops of their own for a and b: work with
// and without masks in one, by a branch, costs half as many registers again.)
template <class C, typename L>
__device__ __forceinline__ void start_pass(int visits, L&& load) {
    if constexpr (kStages<C> == 2)
        if (visits > 0) load(0, 0);
}
template <class C, typename N, typename L, typename A, typename B, typename R>
__device__ __forceinline__ void pass_over(int rounds, N&& n_a, int visits, L&& load, A&& a, B&& b, R&& between) {
    const int n = rounds * visits;
    int stage = 0, v = 0;
    auto next = [&]() __attribute__((always_inline)) {
        if constexpr (kStages<C> == 2) {
            wait_loads();
            __syncthreads();
            if (v + 1 < n) load(v + 1, stage ^ 1);
        } else {
            __syncthreads();
            load(v, 0);
            wait_loads();
            __syncthreads();
        }
    };
    for (int r = 0; r < rounds; ++r) {
        const int whole = n_a();
        for (int i = 0; i < whole; ++i, ++v, stage ^= kStages<C> - 1) {
            next();
            a(v, stage);
        }
        for (int i = whole; i < visits; ++i, ++v, stage ^= kStages<C> - 1) {
            next();
            b(v, stage);
        }
        between(r);
    }
}
__device__ __forceinline__ int tiles(int rows) { return rows > 0 ? (rows + kTile - 1) / kTile : 0; }

// Waves per SIMD that the registers are held to.
constexpr int forward_waves(int es, int db) { return es == 4 ? (db <= 2 ? 2 : 1) : (db == 1 ? 4 : (db == 2 ? 3 : 2)); }
// alone: no biases, every key seen; at 64 numbers these hold four waves' registers (64 images of 197 tokens, 12 heads:
// training takes 111 us, 115 with three waves).
constexpr int dq_waves(int es, int db, bool alone) {
    return es == 4 ? (db <= 2 ? 2 : 1) : (db == 1 || (db == 2 && alone) ? 4 : (db == 2 ? 3 : 2));
}
constexpr int dkv_waves(int es, int db) { return es == 4 ? 2 : (db == 1 ? 3 : 2); }
// Whether dk and dv are two launches, each with its own accumulators and the scores made twice:
// both at once hold more numbers than 256 registers (at 128 numbers a head 2 x 128 in accumulators
// alone; apart, each takes 124).
constexpr bool dkv_apart(int es, int db) { return es == 4 ? db >= 2 : db >= 4; }

// --- forward --------------------------------------------------------------------------
// A wave's 32 queries pass over the keys once, with the running maximum and sum of each row; a block's
// exponentials lie between the next block's scores and the last one's product, so that the matrix cores have
// work beside them.  10 heads of 32768 causal tokens, 112 numbers each: 3.0 ms, 790 TFLOP/s of the seen pairs,
// bound by the vector instructions of the exponentials and their packing (7 for each matrix instruction; matrix
// cores 47 % busy, vector ALUs 47 %).  64 images of 197 tokens, 12 heads of 64: 28.3 us where 16.3 would move their
// bytes, bound by a workgroup's start and four tiles of 1.5 us in turn.
template <typename IO, int DB, bool VEC, bool BIAS, bool UNSEEN>
__global__ __launch_bounds__(256, forward_waves(sizeof(IO), DB)) void forward_kernel(AttentionArgs a, BucketMap map, uint32_t base) {
    using C = Shape<IO, DB>;
    using O = Op32<IO>;
    using F = typename O::F;
    __shared__ __attribute__((aligned(16))) char lds[kStages<C>][2 * C::TILE];
    extern __shared__ float tab[];  // with biases: fill_biases'
    const Place at = place_of(base, a.deal, true);
    if (at.head < 0) return;
    const int head = at.head, kv = head / (a.heads / a.kv_heads);
    BiasLanes biases;
    if constexpr (BIAS) biases = load_biases<IO>(a, map, head);
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5;
    int64_t b, row0;
    slot_of(a.offsets, a.batch, a.T, at.slot, b, row0);
    Seq s;
    tokens_of(a.offsets, a.batch, a.T, b, s.q0, s.n_q);
    tokens_of(a.kv_offsets, a.batch, a.T_kv, b, s.k0, s.n_k);
    if (row0 < 0 || row0 >= s.n_q) return;
    const int shift = s.n_k - s.n_q, w0 = (int)row0 + 32 * wave, n_rows = s.n_q - w0;
    const int my = w0 + (lane & 31);

    f32x16 acc[DB];
    clear(acc);
    float top = -kInf, total = 0.0f, ref = -kShift<IO>;
    const float scale = fabsf(a.scale) * kLog2e;  // the queries take its sign
    const int last = a.causal ? (my + shift < s.n_k - 1 ? my + shift : s.n_k - 1) : s.n_k - 1;  // last key that it sees
    const int wave_end = a.causal && w0 + 31 + shift < s.n_k - 1 ? w0 + 32 + shift : s.n_k;    // keys that the wave sees
    // keys that some of the workgroup's rows see; tiles that all of them do
    const int end = a.causal && (int)row0 + kRows - 1 + shift < s.n_k - 1 ? (int)row0 + kRows + shift : s.n_k;
    const int all = a.causal && (int)row0 + shift < s.n_k - 1 ? (int)row0 + shift + 1 : s.n_k;
    int whole = all > 0 ? all / kTile : 0;

    constexpr int NP = (C::P + 3) / 4;
    const Loader<IO, C::P, NP, true, VEC> lk(a.k, a.D_k, 0, wave, 4), lv(a.v, a.D_v, 0, wave, 4);
    const RowFrags<C> rows(lds[0]);
    const ColumnFrags<C, O> cols(lds[0] + C::TILE);
    constexpr int S1 = (kStages<C> - 1) * 2 * C::TILE;  // from one stage to the other
    const int n_tiles = tiles(end), blocks = n_rows > 0 && wave_end > 0 ? (wave_end + 31) / 32 : 0;  // blocks that the wave works on
    auto load_k = [&](int t) {
        const int j0 = t * kTile, n = s.n_k - j0 < kTile ? s.n_k - j0 : kTile;
        if (t < n_tiles) lk.run(a.k, s.k0 + j0, kv, n, a.D_k, 0, wave, 4, lds[t & (kStages<C> - 1)]);
    };
    auto load_v = [&](int t) {
        const int j0 = t * kTile, n = s.n_k - j0 < kTile ? s.n_k - j0 : kTile;
        if (t < n_tiles) lv.run(a.v, s.k0 + j0, kv, n, a.D_v, 0, wave, 4, lds[t & (kStages<C> - 1)] + C::TILE);
    };
    if constexpr (kStages<C> == 2) load_k(0), load_v(0);
    F q[C::NS];
    load_rows<C, IO, F, VEC>(q, a.q, s.q0 + w0, head, n_rows, a.D_k);
    bool taken_out = false;  // keys by their biases: then no tile is whole
    if constexpr (BIAS) taken_out = fill_biases<IO>(tab, biases, a, map, head);
    if (taken_out) whole = 0;
    if (a.scale < 0.0f) negate(q);
    arrive(q);

    f32x16 x = {};  // scores of the block at hand
    F p[C::NT];     // probabilities of the one before
    // Scores of block kb of the tile at `by`.
    auto scores = [&](f32x16& y, int kb, int by) __attribute__((always_inline)) {
        y = f32x16{};
#pragma unroll
        for (int st = 0; st < C::NS; ++st) O::mma(y, rows.template get<F>(by, kb, st), q[st]);
    };
    // Block n's probabilities, packed, from its scores in x; between() before the sums are scaled.
    auto probabilities = [&](auto kind, int n, auto&& between) __attribute__((always_inline)) {
        constexpr int K = decltype(kind)::value;
        const int j = 32 * n;
        if constexpr (BIAS) {
            const int from = w0 + shift - j;  // distance of the wave's first row and the block's first key
            const float* t = tab + a.reach + kPad;
            // (the far ones share a value: no other way, which would part the products from it)
            const bool far = from - 31 >= a.reach || from + 31 <= -a.reach;
            t += far ? (from > 0 ? a.reach + 31 : -a.reach) : from + (lane & 31) - 4 * h;
            if (K != kWhole && taken_out) [[unlikely]] {
                f32x16 none{};
                biased_or_out<-1>(x, none, scale, t);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __builtin_fmaf(x[i], scale, t[-row_of(i)]);
            }
        }
        if constexpr (K != kWhole) {
            const int lim = last - j - 4 * h;
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = row_of(i) <= lim ? x[i] : -kInf;
        }
        float mx = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, x[i]);
        mx = half_max(mx);
        if constexpr (!BIAS) mx *= scale;
        const bool grown = mx > top + kSlack<IO>;
        // (a row without scores so far has sums of 0, and none of its terms is counted against -infinity)
        const float now = grown ? mx : top, c = top == -kInf ? 0.0f : __builtin_amdgcn_exp2f(top - now);
        top = now;
        ref = (top == -kInf ? 0.0f : top) - kShift<IO>;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __builtin_amdgcn_exp2f(BIAS ? x[i] - ref : __builtin_fmaf(x[i], scale, -ref));
        between();
#pragma unroll
        for (int t = 0; t < C::NT; ++t) {
            float w[C::E];
#pragma unroll
            for (int e = 0; e < C::E; ++e) w[e] = x[t * C::E + e];
            p[t] = O::pack(w);
        }
        float sum = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) sum += x[i];
        if (__any(grown)) {
            total *= c;
            asm volatile("");  // (rare: not to be computed beside the other way)
#pragma unroll
            for (int cb = 0; cb < DB; ++cb) acc[cb] *= c;
        }
        total += sum;
    };
    // The product of block n's probabilities with v: block kb of the tile at `by`.
    auto product = [&](auto kind, int n, int by, int kb) __attribute__((always_inline)) {
        constexpr int K = decltype(kind)::value;
        uint32_t odd = 0;
#pragma unroll
        for (int t = 0; t < C::NT; ++t)
            static_for<0, (DB + kAtOnce<UNSEEN> - 1) / kAtOnce<UNSEEN>>([&](auto ic) {
                constexpr int c0 = decltype(ic)::value * kAtOnce<UNSEEN>, n = DB - c0 < kAtOnce<UNSEEN> ? DB - c0 : kAtOnce<UNSEEN>;
                F v[n];
#pragma unroll
                for (int c = 0; c < n; ++c) v[c] = cols.get(by, kb, t, c0 + c);
                if (K == kUnseen && (UNSEEN || taken_out)) [[unlikely]] take_finite<O>(v, odd);
#pragma unroll
                for (int c = 0; c < n; ++c) O::mma(acc[c0 + c], v[c], p[t]);
            });
        if (K == kUnseen && __any(odd >= O::kInf)) [[unlikely]] {
            uint32_t sees = bits_to(last - 32 * n);
            if (BIAS && taken_out) sees &= ~taken_out_of(tab, a.reach, my + shift - 32 * n, -1);
            add_odd_numbers<C, IO>(acc, lds[0] + C::TILE + by + kb * (32 * C::P * 16), sees, false);
        }
    };
    using Edge = Kind<UNSEEN || BIAS ? kUnseen : kPartial>;
    if constexpr (kStages<C> == 2) {
        // While a wave makes block n's probabilities, its matrix core has block n + 1's scores and
        // block n - 1's product to make: v follows k by a block, and a tile's v is there one visit
        // later than its k.
        wait_loads();
        __syncthreads();
        load_k(1);
        f32x16 y;
        if (blocks > 0) {
            scores(x, 0, 0);
            scores(y, 1, 0);
            probabilities(Edge{}, 0, [] {});
            x = y;
        }
        auto next = [&](int t) {
            wait_loads();  // k of tile t + 1, v of tile t
            __syncthreads();
            load_k(t + 2), load_v(t + 1);
        };
        auto block = [&](auto kind, int n, int by_k, int by_v, int kb) __attribute__((always_inline)) {
            scores(y, kb, by_k);  // (past the last key: of anything, and not used)
            probabilities(kind, n, [&]() __attribute__((always_inline)) { product(kind, n - 1, by_v, kb); });
            x = y;
        };
        int t = 0;
        for (; t + 1 < whole; ++t) {
            next(t);
            const int by_v = (t & 1) * S1, by_k = S1 - by_v;
            if (blocks > 0) {
                block(Kind<kWhole>{}, 2 * t + 1, by_k, by_v, 0);
                block(Kind<kWhole>{}, 2 * t + 2, by_k, by_v, 1);
            }
        }
        for (; t < n_tiles; ++t) {
            next(t);
            const int by_v = (t & 1) * S1, by_k = S1 - by_v;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const int n = 2 * t + 1 + kb;
                if (n < blocks) block(Edge{}, n, by_k, by_v, kb);
                else if (n == blocks) product(Edge{}, n - 1, by_v, kb);
            }
        }
    } else {
        auto tile = [&](auto kind, int t) __attribute__((always_inline)) {
            __syncthreads();
            load_k(t), load_v(t);
            wait_loads();
            __syncthreads();
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
                if (2 * t + kb < blocks) {
                    scores(x, kb, 0);
                    probabilities(kind, 2 * t + kb, [] {});
                    product(kind, 2 * t + kb, 0, kb);
                }
        };
        int t = 0;
        for (; t < whole; ++t) tile(Kind<kWhole>{}, t);
        for (; t < n_tiles; ++t) tile(Edge{}, t);
    }
    if (n_rows <= 0) return;
    total += __shfl_xor(total, 32);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    store_rows<C, IO>(acc, a.o, s.q0 + w0, head, n_rows, a.D_v, inv, a.out_vec);
    if (a.lse && h == 0 && (lane & 31) < n_rows)
        a.lse[(int64_t)head * a.T + s.q0 + my] =
            total == 0.0f ? -kInf : (ref + __builtin_amdgcn_logf(total)) * kLn2;
}

// --- backward -------------------------------------------------------------------------
// fp16: takes the lane's sums to a scale that holds its numbers x, and returns x's.
template <typename IO, int N, int DB>
__device__ __forceinline__ float hold(const f32x16 (&x)[N], float& f, f32x16 (&acc)[DB]) {
    if constexpr (!std::is_same_v<IO, _Float16>) return 1.0f;
    float m = 0.0f;
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[b][i]));
    m = fmaxf(m, __shfl_xor(m, 32));
    const bool over = m * f > 32768.0f && m < kInf;
    if (__any(over)) {
        const float now = over ? range_scale(m) : f;
        const float c = now * inverse_of_power(f);
        f = now;
#pragma unroll
        for (int cb = 0; cb < DB; ++cb) acc[cb] *= c;
    }
    return f;
}

// Sums of a block of 32 x 32 along its diagonals.  Accumulator i holds row r = row_of(i) (+ 4 h)
// of all 32 columns; turned by r lanes, column c comes to lane c - r, or c - r + 32: the first
// are added to `near` (distance: lane), the others to `wrap` (distance: lane - 32).
__device__ __forceinline__ void add_diagonals(const f32x16& x, float& near, float& wrap) {
    const int lane = (int)threadIdx.x & 31;
    static_for<0, 16>([&](auto ic) {
        constexpr int i = decltype(ic)::value, r = row_of(i);
        float v = x[i];
        if constexpr (r != 0) {
            // swizzle, rotate mode: lane l of each 32 reads lane (l + r) % 32
            v = __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0xc000 | r << 5));
            near += lane < 32 - r ? v : 0.0f;
            wrap += lane < 32 - r ? 0.0f : v;
        } else {
            near += v;
        }
    });
}

// acc += w's 32 rows (of block b) times the columns of the tile at `at`; FINITE and (ALWAYS or) look: odd
// numbers as 0, odd the largest that was met.  fp32 sums a block on its own first: one long chain of roundings
// left dq of 5590 tokens off by a relative 1.5e-6, 0.7e-6 so (and costs 3 % of packed training in fp32).
template <typename C, typename O, bool FINITE, bool ALWAYS, typename Columns, int DB>
__device__ __forceinline__ void add_columns(f32x16 (&acc)[DB], const Columns& columns, int at, int b, const f32x16& w, bool look, uint32_t& odd) {
    using F = typename O::F;
    auto packed = [&](int t) __attribute__((always_inline)) {
        float u[C::E];
#pragma unroll
        for (int e = 0; e < C::E; ++e) u[e] = w[t * C::E + e];
        return O::pack(u);
    };
    if constexpr (C::E == 8) {
#pragma unroll
        for (int t = 0; t < C::NT; ++t) {
            const F f = packed(t);
            static_for<0, (DB + kAtOnce<ALWAYS> - 1) / kAtOnce<ALWAYS>>([&](auto ic) {
                constexpr int c0 = decltype(ic)::value * kAtOnce<ALWAYS>, n = DB - c0 < kAtOnce<ALWAYS> ? DB - c0 : kAtOnce<ALWAYS>;
                F g[n];
#pragma unroll
                for (int c = 0; c < n; ++c) g[c] = columns.get(at, b, t, c0 + c);
                if (FINITE && (ALWAYS || look)) [[unlikely]] take_finite<O>(g, odd);
#pragma unroll
                for (int c = 0; c < n; ++c) O::mma(acc[c0 + c], g[c], f);
            });
        }
    } else {
#pragma unroll
        for (int cb = 0; cb < DB; ++cb) {
            F g[C::NT];
#pragma unroll
            for (int t = 0; t < C::NT; ++t) g[t] = columns.get(at, b, t, cb);
            if (FINITE && (ALWAYS || look)) [[unlikely]] take_finite<O>(g, odd);
            f32x16 sum{};
#pragma unroll
            for (int t = 0; t < C::NT; ++t) O::mma(sum, g[t], packed(t));
            acc[cb] += sum;
        }
    }
}

// Gradients of q and, if wanted, of the biases: a wave owns 32 queries and passes over the
// keys twice.  The first pass makes delta = sum P dP, as what d_o . o leaves of it: o is
// rounded to the plan's type, and delta from it alone is off by that rounding, which dS (a
// difference) shows twofold and the biases' fp32 gradients by 1e-3 of their size.  It also
// takes lse's own rounding out of P (sum P = 1), and leaves both for dkv_kernel.  Steep rows (rare)
// look for their largest score before it, with keys straight from memory, and leave that and 1 / sum P.
// The second makes dS.  Of the biases, dS is summed by distance: along the diagonals of a block in
// registers, then into an array for each half of each wave (its own: read, added to, written);
// distances past the reach share a bucket on either side and are summed in registers.  (In
// packed training on images the kernel took 370 us with one LDS atomic for each of a block's 16
// accumulators, 124 with two for its diagonals, 107 so.)  A workgroup writes the
// sums of its buckets; reduce_kernel joins those of a head.
template <typename IO, int DB, bool VEC, bool BIAS, bool UNSEEN>
__global__ __launch_bounds__(256, dq_waves(sizeof(IO), DB, !BIAS && !UNSEEN)) void dq_kernel(AttentionArgs a, BucketMap map, uint32_t base) {
    using C = Shape<IO, DB>;
    using O = Op32<IO>;
    using F = typename O::F;
    __shared__ __attribute__((aligned(16))) char lds[kStages<C>][2 * C::TILE];
    __shared__ float far_sums[BIAS ? 8 : 1];
    extern __shared__ float tab[];  // with biases: fill_biases', then [8][width] with their gradients
    const Place at = place_of(base, a.deal, true);
    if (at.head < 0) return;
    const int head = at.head, kv = head / (a.heads / a.kv_heads);
    BiasLanes biases;
    if constexpr (BIAS) biases = load_biases<IO>(a, map, head);
    const uint32_t slot = at.slot;
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5;
    int64_t b, row0;
    slot_of(a.offsets, a.batch, a.T, slot, b, row0);
    Seq s;
    tokens_of(a.offsets, a.batch, a.T, b, s.q0, s.n_q);
    tokens_of(a.kv_offsets, a.batch, a.T_kv, b, s.k0, s.n_k);
    const bool idle = row0 < 0 || row0 >= s.n_q;
    if (idle && !(BIAS && a.dbias)) return;
    if (idle) s.n_q = s.n_k = 0, row0 = 0;
    const int shift = s.n_k - s.n_q, w0 = (int)row0 + 32 * wave, n_rows = s.n_q - w0;
    const int my = w0 + (lane & 31);
    const int width = tab_width(a.reach);
    float* const sums = tab + table_words(a.reach, a.buckets);
    f32x16 acc[DB];
    clear(acc);
    float held = kTopScale, far_pos = 0.0f, far_neg = 0.0f;
    const float scale = fabsf(a.scale) * kLog2e;  // the queries take its sign
    const int last = a.causal ? (my + shift < s.n_k - 1 ? my + shift : s.n_k - 1) : s.n_k - 1;
    const int wave_end = a.causal && w0 + 31 + shift < s.n_k - 1 ? w0 + 32 + shift : s.n_k;
    const int end = a.causal && (int)row0 + kRows - 1 + shift < s.n_k - 1 ? (int)row0 + kRows + shift : s.n_k;
    const int all = a.causal && (int)row0 + shift < s.n_k - 1 ? (int)row0 + shift + 1 : s.n_k;
    int whole = all > 0 ? all / kTile : 0;

    constexpr int NP = (C::P + 3) / 4;
    const Loader<IO, C::P, NP, true, VEC> lk(a.k, a.D_k, 0, wave, 4), lv(a.v, a.D_v, 0, wave, 4);
    const RowFrags<C> krows(lds[0]);  // (v's tile lies C::TILE behind k's)
    const ColumnFrags<C, O> kcols(lds[0]);
    auto load = [&](int t, int stage) {
        const int j0 = t * kTile, n = s.n_k - j0 < kTile ? s.n_k - j0 : kTile;
        lk.run(a.k, s.k0 + j0, kv, n, a.D_k, 0, wave, 4, lds[stage]);
        lv.run(a.v, s.k0 + j0, kv, n, a.D_v, 0, wave, 4, lds[stage] + C::TILE);
    };
    const int visits = tiles(end);
    start_pass<C>(visits, load);
    bool taken_out = false;  // keys by their biases: then no tile is whole
    if constexpr (BIAS) {
        taken_out = fill_biases<IO>(tab, biases, a, map, head);
        if (taken_out) whole = 0;
        if (a.dbias)
            for (int x = tid; x < 8 * width; x += 256) sums[x] = 0.0f;
    }

    F q[C::NS], d_o[C::NS];
    load_rows<C, IO, F, VEC>(q, a.q, s.q0 + w0, head, n_rows, a.D_k);
    load_rows<C, IO, F, VEC>(d_o, a.d_o, s.q0 + w0, head, n_rows, a.D_v);
    const bool real = (lane & 31) < n_rows;
    const int64_t row = (int64_t)head * a.T + s.q0 + my;
    // In powers of two.  A row that sees nothing has probabilities of 0.
    float lse = real ? a.lse[row] : kInf, delta = 0.0f, left = 0.0f, ones = 0.0f, inv = 1.0f;
    const bool steep = fabsf(lse) > kSteepLse && fabsf(lse) < kInf, some_steep = __any(steep);
    lse = lse == -kInf ? kInf : lse * kLog2e;
    {
        F o[C::NS];
        load_rows<C, IO, F, VEC>(o, a.o, s.q0 + w0, head, n_rows, a.D_v);
#pragma unroll
        for (int st = 0; st < C::NS; ++st)
#pragma unroll
            for (int e = 0; e < C::E; ++e) delta = __builtin_fmaf(O::get(o[st], e), O::get(d_o[st], e), delta);
        delta += __shfl_xor(delta, 32);
    }
    if (a.scale < 0.0f) negate(q);
    arrive(q), arrive(d_o);
    if constexpr (BIAS) lds_barrier();  // the biases are there
    if (some_steep) [[unlikely]] {
        float top = -kInf;
#pragma unroll 1
        for (int j = 0; j < wave_end; j += 32) {
            F k[C::NS];
            load_rows<C, IO, F, VEC>(k, a.k, s.k0 + j, kv, s.n_k - j, a.D_k);
            f32x16 x{}, none{};
#pragma unroll
            for (int st = 0; st < C::NS; ++st) O::mma(x, k[st], q[st]);
            if constexpr (BIAS) {
                const int from = w0 + shift - j;
                const bool far = from - 31 >= a.reach || from + 31 <= -a.reach;
                biased_or_out<-1>(x, none, scale,
                                  tab + a.reach + kPad + (far ? (from > 0 ? a.reach + 31 : -a.reach) : from + (lane & 31) - 4 * h));
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) top = row_of(i) <= last - j - 4 * h ? fmaxf(top, x[i]) : top;
        }
        top = half_max(top);
        if constexpr (!BIAS) top *= scale;
        if (steep && top > -kInf) lse = top;
    }
    // Probabilities and dP of 32 keys from j on, at block kb of the tiles at `by`; returns the keys taken
    // out (of a block at an edge), bit i of accumulator i.
    auto scores = [&](bool edge, f32x16& x, f32x16& dp, int j, int kb, int by) __attribute__((always_inline)) {
        uint32_t out = 0;
        x = f32x16{}, dp = f32x16{};
#pragma unroll
        for (int st = 0; st < C::NS; ++st) O::mma(x, krows.template get<F>(by, kb, st), q[st]);
#pragma unroll
        for (int st = 0; st < C::NS; ++st) O::mma(dp, krows.template get<F>(by + C::TILE, kb, st), d_o[st]);
        if constexpr (BIAS) {
            const int from = w0 + shift - j;  // distance of the wave's first row and the block's first key
            const float* t = tab + a.reach + kPad;
            const bool far = from - 31 >= a.reach || from + 31 <= -a.reach;
            if (edge && taken_out) [[unlikely]] {
                out = biased_or_out<-1>(x, dp, scale, t + (far ? (from > 0 ? a.reach + 31 : -a.reach) : from + (lane & 31) - 4 * h));
            } else if (far) {
                const float f = t[from > 0 ? a.reach : -a.reach];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __builtin_fmaf(x[i], scale, f);
            } else {
                t += from + (lane & 31) - 4 * h;
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __builtin_fmaf(x[i], scale, t[-row_of(i)]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __builtin_amdgcn_exp2f(x[i] - lse);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], scale, -lse));
        }
        return out;
    };
    auto first = [&](bool edge, int t, int stage) __attribute__((always_inline)) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const int j = t * kTile + 32 * kb;
            if (n_rows <= 0 || j >= wave_end) return;
            f32x16 x, dp;
            scores(edge, x, dp, j, kb, stage * 2 * C::TILE);
            if (edge) {
                const int lim = last - j - 4 * h;
                if (j == 0) {  // a row that sees one key: its dP to the bit, its dS is 0
                    const float one = __shfl(dp[0], lane & 31);
                    delta = last == 0 ? one : delta;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    ones += row_of(i) <= lim ? x[i] : 0.0f;
                    left += row_of(i) <= lim ? x[i] * (dp[i] - delta) : 0.0f;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) ones += x[i], left = __builtin_fmaf(x[i], dp[i] - delta, left);
            }
        }
    };
    pass_over<C>(
        1, [&]() { return whole; }, visits, load, [&](int t, int stage) { first(false, t, stage); },
        [&](int t, int stage) { first(true, t, stage); }, [](int) {});
    __syncthreads();
    start_pass<C>(visits, load);
    ones += __shfl_xor(ones, 32);
    left += __shfl_xor(left, 32);
    if (ones != 0.0f) {
        delta += left / ones;
        if (some_steep) inv = 1.0f / ones;
        else lse += __builtin_amdgcn_logf(ones);
    }
    if (real && h == 0)  // (as dkv_kernel takes them; +infinity: see the others)
        a.row_stats(kRowLse)[row] = some_steep && lse < kInf ? kInf : -lse / scale, a.row_stats(kRowDelta)[row] = -delta;
    if (real && some_steep) a.row_stats(kRowTop)[row] = lse, a.row_stats(kRowInv)[row] = inv;
    if (lane == 0) a.steep()[((int64_t)head * a.slots + slot) * 4 + wave] = some_steep;

    const float delta_inv = delta * inv;
    auto block = [&](auto kind, int j, int kb, int by) __attribute__((always_inline)) {
        constexpr int K = decltype(kind)::value;
        f32x16 x[1], dp;
        const uint32_t out = scores(K != kWhole, x[0], dp, j, kb, by);
        const int lim = last - j - 4 * h;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            // (1 / sum P of steep rows here, as d_bias adds rows up, or, without biases, at the end; else it is 1)
            x[0][i] *= BIAS ? __builtin_fmaf(dp[i], inv, -delta_inv) : dp[i] - delta;
            if constexpr (K != kWhole) x[0][i] = row_of(i) <= lim ? x[0][i] : 0.0f;
        }
        if (BIAS && K != kWhole && taken_out) [[unlikely]] {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[0][i] = out >> i & 1 ? 0.0f : x[0][i];
        }
        if constexpr (BIAS) {
            // (rows past the last query have probabilities of 0 and distances of their own: 0 times a NaN is no term)
            if (a.dbias && n_rows < 32)
#pragma unroll
                for (int i = 0; i < 16; ++i) x[0][i] = real ? x[0][i] : 0.0f;
            const int from = w0 + shift - j;
            if (a.dbias && (from - 31 >= a.reach || from + 31 <= -a.reach)) {
                float t = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) t += x[0][i];
                if (from > 0) far_pos += t;
                else far_neg += t;
            } else if (a.dbias) {
                lds_float* const t = (lds_float*)tab + table_words(a.reach, a.buckets) + (2 * wave + h) * width + a.reach + kPad + from + (lane & 31) - 4 * h;
                float near = t[0], wrap = t[-32];
                add_diagonals(x[0], near, wrap);
                t[0] = near, t[-32] = wrap;
            }
        }
        const float f = hold<IO>(x, held, acc);
        if constexpr (std::is_same_v<IO, _Float16>) x[0] *= f;
        uint32_t odd = 0;
        add_columns<C, O, K == kUnseen, UNSEEN>(acc, kcols, by, kb, x[0], taken_out, odd);
        if (K == kUnseen && __any(odd >= O::kInf)) [[unlikely]] {
            uint32_t sees = bits_to(last - j);
            if (BIAS && taken_out) sees &= ~taken_out_of(tab, a.reach, my + shift - j, -1);
            add_odd_numbers<C, IO>(acc, lds[0] + by + kb * (32 * C::P * 16), sees, true);
        }
    };
    auto second = [&](auto kind, int t, int stage) __attribute__((always_inline)) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
            if (n_rows > 0 && t * kTile + 32 * kb < wave_end) block(kind, t * kTile + 32 * kb, kb, stage * 2 * C::TILE);
    };
    pass_over<C>(
        1, [&]() { return whole; }, visits, load, [&](int t, int stage) { second(Kind<kWhole>{}, t, stage); },
        [&](int t, int stage) { second(Kind<UNSEEN || BIAS ? kUnseen : kPartial>{}, t, stage); }, [](int) {});
    if (n_rows > 0) {
        float m = std::is_same_v<IO, _Float16> ? a.scale * inverse_of_power(held) : a.scale;
        if (!BIAS && some_steep) [[unlikely]] {
            // (the lane's own store, found again: held in registers all along, it left a SIMD 3 waves of 4)
            int own = lane & 31;
            asm volatile("" : "+v"(own));
            if (own < n_rows) m *= *(const volatile float*)(a.row_stats(kRowInv) + (int64_t)head * a.T + s.q0 + w0 + own);
        }
        store_rows<C, IO>(acc, a.dq, s.q0 + w0, head, n_rows, a.D_k, m, a.dq_vec);
    }
    if constexpr (BIAS) {
        if (!a.dbias) return;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            far_pos += __shfl_xor(far_pos, m);
            far_neg += __shfl_xor(far_neg, m);
        }
        if (lane == 0) far_sums[wave] = far_pos, far_sums[4 + wave] = far_neg;
        __syncthreads();
        for (int x = tid; x < width; x += 256) {
            float t = sums[x];
#pragma unroll
            for (int k = 1; k < 8; ++k) t += sums[k * width + x];
            sums[x] = t;
        }
        __syncthreads();
        // a bucket's distances are added up by the lanes of a wave
        const int side = a.causal ? a.buckets : a.buckets / 2;
        const int* const starts = reinterpret_cast<const int*>(tab + width);
        for (int bucket = wave; bucket < a.buckets; bucket += 4) {
            const bool before = bucket < side;  // the key comes before the query (or is its own)
            const int want = before ? bucket : bucket - side;
            int x0 = starts[want];
            const int x1 = want == side - 1 ? a.reach + kPad + 1 : starts[want + 1];
            if (!before && x0 == 0) x0 = 1;  // distance 0 is of the first side
            float t = 0.0f;
            for (int x = x0 + lane; x < x1; x += 64) t += sums[a.reach + kPad + (before ? x : -x)];
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) t += __shfl_xor(t, m);
            if (want == side - 1)
                t += before ? far_sums[0] + far_sums[1] + far_sums[2] + far_sums[3]
                            : far_sums[4] + far_sums[5] + far_sums[6] + far_sums[7];
            if (lane == 0) a.parts[((int64_t)head * a.buckets + bucket) * a.slots + slot] = t;
        }
    }
}

// Gradients of k and v, after dq_kernel: a wave owns 32 keys of a kv head and passes over the
// queries of every head that shares it, in a fixed order; DK and DV: which of the two.  G groups of four waves own the same keys and take
// every G-th tile of queries each; their sums are joined at the end.  (A key of a causal
// sequence is seen by all queries after it: with one group, 512 workgroups that all run at once took as
// long as the longest of them, 817 us for dk of 2 x 8192 tokens.)
template <typename IO, int DB, bool VEC, bool BIAS, bool UNSEEN, int G, bool DK, bool DV>
__global__ __launch_bounds__(256 * G, dkv_waves(sizeof(IO), DB)) void dkv_kernel(AttentionArgs a, BucketMap map, uint32_t base) {
    using C = Shape<IO, DB>;
    using O = Op32<IO>;
    using F = typename O::F;
    __shared__ __attribute__((aligned(16))) char tiles_of[G][kStages<C>][2 * C::TILE];
    __shared__ __attribute__((aligned(16))) float stats_of[G][kStages<C>][2][kTile];  // lse, delta
    extern __shared__ float tab[];
    const Place place = place_of(base, a.kv_deal, false);
    if (place.head < 0) return;
    const int kv = place.head, r = a.heads / a.kv_heads;
    BiasLanes biases;
    if constexpr (BIAS) biases = load_biases<IO>(a, map, kv * r);
    const int tid = (int)threadIdx.x, lane = tid & 63, wave8 = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5;
    const int group = wave8 >> 2, wave = wave8 & 3;
    auto& lds = tiles_of[group];
    auto& stats = stats_of[group];
    int64_t b, row0;
    slot_of(a.kv_offsets, a.batch, a.T_kv, place.slot, b, row0);
    Seq s;
    tokens_of(a.offsets, a.batch, a.T, b, s.q0, s.n_q);
    tokens_of(a.kv_offsets, a.batch, a.T_kv, b, s.k0, s.n_k);
    if (row0 < 0 || row0 >= s.n_k) return;
    const int shift = s.n_k - s.n_q, w0 = (int)row0 + 32 * wave, n_rows = s.n_k - w0;
    const int my = w0 + (lane & 31);

    f32x16 dk[DB], dv[DB];
    clear(dk), clear(dv);
    float held = kTopScale;
    const float scale = fabsf(a.scale) * kLog2e;  // the keys take its sign
    // Tiles of queries from the first that sees one of the workgroup's keys: t_edge .. t_whole - 1
    // see all of them and are visited first, then those before, then the last, if it is not whole.
    const int t_first = a.causal && (int)row0 - shift > 0 ? ((int)row0 - shift) / kTile : 0;
    const int t_all = a.causal && (int)row0 + kRows - 1 - shift > 0 ? tiles((int)row0 + kRows - 1 - shift) : 0;
    const int t_whole = s.n_q / kTile, tail = s.n_q % kTile && t_first <= t_whole ? 1 : 0;
    const int t_edge = t_all < t_whole ? (t_all > t_first ? t_all : t_first) : t_whole;  // edge tiles: t_first .. t_edge - 1
    const int n_whole = t_whole > t_edge ? t_whole - t_edge : 0, n_early = t_edge > t_first ? t_edge - t_first : 0;
    const int n_all = n_whole + n_early + tail, n_visits = (n_all + G - 1) / G;
    auto row_at = [&](int v) {  // of the group's visit v
        int t = G * (v % n_visits) + group;
        t -= n_whole;
        return (t < 0 ? t + n_whole + t_edge : (t < n_early ? t_first + t : t_whole)) * kTile;
    };

    constexpr int NP = (C::P + 3) / 4;
    const Loader<IO, C::P, NP, true, VEC> lq(a.q, a.D_k, 0, wave, 4), lg(a.d_o, a.D_v, 0, wave, 4);
    const RowFrags<C> qrows(lds[0]);  // (d_o's tile lies C::TILE behind q's)
    const ColumnFrags<C, O> qcols(lds[0]);
    auto load = [&](int t, int stage) {
        if (G * (t % n_visits) + group >= n_all) return;
        const int head = kv * r + t / n_visits, i0 = row_at(t), n = s.n_q - i0 < kTile ? s.n_q - i0 : kTile;
        lq.run(a.q, s.q0 + i0, head, n, a.D_k, 0, wave, 4, lds[stage]);
        lg.run(a.d_o, s.q0 + i0, head, n, a.D_v, 0, wave, 4, lds[stage] + C::TILE);
        if (wave < 2) {
            const float* from = a.row_stats(wave ? kRowDelta : kRowLse) + (int64_t)head * a.T + s.q0 + i0;
            load_words_to_lds(resource(from, (uint32_t)n * 4), (uint32_t)lane * 4, stats[stage][wave]);
        }
    };
    start_pass<C>(n_visits, load);
    // Whether some query of the sequence, of any of the heads, is steep: then no tile is whole.  (The marks of four
    // heads' first 64 runs of rows are on their way beside the rest.)
    const int runs = (s.n_q + 31) / 32;
    const int* const marks =
        a.steep() + ((int64_t)kv * r * a.slots + (a.offsets ? s.q0 / kRows + b : b * ((s.n_q + kRows - 1) / kRows))) * 4;
    int mark[4];
#pragma unroll
    for (int hh = 0; hh < 4; ++hh) mark[hh] = hh < r && lane < runs ? marks[(int64_t)hh * a.slots * 4 + lane] : 0;
    F k[C::NS], v[C::NS];
    load_rows<C, IO, F, VEC>(k, a.k, s.k0 + w0, kv, n_rows, a.D_k);
    if constexpr (DK) load_rows<C, IO, F, VEC>(v, a.v, s.k0 + w0, kv, n_rows, a.D_v);
    bool taken_out = false;  // keys by this head's biases: then no tile is whole
    if constexpr (BIAS) taken_out = fill_biases<IO, 256 * G>(tab, biases, a, map, kv * r);
    if (a.scale < 0.0f) negate(k);
    arrive(k);
    if constexpr (DK) arrive(v);
    int some = mark[0] | mark[1] | mark[2] | mark[3];
    for (int hh = 0; hh < r; ++hh)
        for (int i = hh < 4 ? 64 + lane : lane; i < runs; i += 64) some |= marks[(int64_t)hh * a.slots * 4 + i];
    const bool steep = __any(some);
    // Queries q0 .. q0 + 31, at block qb of the tiles at `by`.  In 16 bits their statistics are what the
    // accumulators start from: the products end in (score - lse) / scale and dP - delta.  fp32 adds them
    // behind the products, which would round at lse's size 16 D times (relative 1.2e-6 in dk at D = 48, 4e-7 so),
    // and so do blocks at an edge: dP is then dq_kernel's bit for bit, and a lone key's dS is 0.
    auto block = [&](auto kind, auto of_steep, int q0, int qb, int by, const float (&stat)[2][kTile], int head) __attribute__((always_inline)) {
        constexpr int K = decltype(kind)::value;
        constexpr bool STEEP = decltype(of_steep)::value;  // (from the scores alone, which are dq_kernel's bit for bit)
        const int low = a.causal ? my - shift - q0 : 0, high = s.n_q - 1 - q0;  // rows of the block that see the lane's key
        constexpr bool LATE = sizeof(IO) == 4 || K != kWhole;
        f32x16 x{}, dp{}, p[1], ds[1];
        uint32_t out = 0;
        auto add_stats = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 lse = *reinterpret_cast<const f32x4*>(&stat[0][32 * qb + 8 * g + 4 * h]);
                const f32x4 delta = *reinterpret_cast<const f32x4*>(&stat[1][32 * qb + 8 * g + 4 * h]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (!STEEP) x[4 * g + e] += lse[e];
                    if constexpr (DK) dp[4 * g + e] += delta[e];
                }
            }
        };
        if constexpr (!LATE) add_stats();
#pragma unroll
        for (int st = 0; st < C::NS; ++st) O::mma(x, qrows.template get<F>(by, qb, st), k[st]);
#pragma unroll
        for (int st = 0; st < C::NS; ++st)
            if constexpr (DK) O::mma(dp, qrows.template get<F>(by + C::TILE, qb, st), v[st]);
        if constexpr (LATE) add_stats();
        if constexpr (BIAS) {
            const int from = q0 + shift - w0;  // distance of the block's first row and the wave's first key
            const float* t = tab + a.reach + kPad;
            const bool far = from - 31 >= a.reach || from + 31 <= -a.reach;
            if (K != kWhole && taken_out) [[unlikely]] {
                out = biased_or_out<1>(x, dp, scale, t + (far ? (from > 0 ? a.reach : -a.reach - 31) : from - (lane & 31) + 4 * h));
            } else if (far) {
                const float f = t[from > 0 ? a.reach : -a.reach];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __builtin_fmaf(x[i], scale, f);
            } else {
                t += from - (lane & 31) + 4 * h;
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __builtin_fmaf(x[i], scale, t[row_of(i)]);
            }
        }
        if constexpr (STEEP) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                asm volatile("" ::: "memory");  // (rare: one row's numbers at a time)
                const float l = stat[0][32 * qb + row_of(i) + 4 * h];
                float top = -l * scale, inv = 1.0f;
                if (l == kInf) {
                    const int64_t row = (int64_t)head * a.T + s.q0 + q0 + row_of(i) + 4 * h;
                    top = a.row_stats(kRowTop)[row], inv = a.row_stats(kRowInv)[row];
                }
                p[0][i] = inv * __builtin_amdgcn_exp2f(BIAS ? x[i] - top : __builtin_fmaf(x[i], scale, -top));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) p[0][i] = __builtin_amdgcn_exp2f(BIAS ? x[i] : x[i] * scale);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if constexpr (DK) ds[0][i] = p[0][i] * dp[i];
            if constexpr (K != kWhole) {
                const int at = row_of(i) + 4 * h;
                const bool seen = at >= low && at <= high && !(BIAS && (out >> i & 1));
                p[0][i] = seen ? p[0][i] : 0.0f;
                if constexpr (DK) ds[0][i] = seen ? ds[0][i] : 0.0f;
            }
        }
        if constexpr (DK && std::is_same_v<IO, _Float16>) ds[0] *= hold<IO>(ds, held, dk);
        if constexpr (DV && std::is_same_v<IO, _Float16>) p[0] *= 4096.0f;
        uint32_t odd = 0;
        if constexpr (DV) add_columns<C, O, K == kUnseen, UNSEEN>(dv, qcols, by + C::TILE, qb, p[0], taken_out, odd);
        if constexpr (DK) add_columns<C, O, K == kUnseen, UNSEEN>(dk, qcols, by, qb, ds[0], taken_out, odd);
        if (K == kUnseen && __any(odd >= O::kInf)) [[unlikely]] {
            const char* t = lds[0] + by + qb * (32 * C::P * 16);
            uint32_t sees = bits_to(high) & ~bits_to(low - 1);
            if (BIAS && taken_out) sees &= ~taken_out_of(tab, a.reach, q0 + shift - my, 1);
            if constexpr (DV) add_odd_numbers<C, IO>(dv, t + C::TILE, sees, false);
            if constexpr (DK) add_odd_numbers<C, IO>(dk, t, sees, true);
        }
    };
    auto edge = [&](auto kind, auto of_steep, int t, int stage) __attribute__((always_inline)) {
#pragma unroll
        for (int qb = 0; qb < 2; ++qb) {
            const int q0 = row_at(t) + 32 * qb;
            if (n_rows > 0 && G * (t % n_visits) + group < n_all && q0 < s.n_q && !(a.causal && q0 + 31 + shift < w0))
                block(kind, of_steep, q0, qb, stage * 2 * C::TILE, stats[stage], kv * r + t / n_visits);
        }
    };
    auto between = [&](int hh) {
        if (BIAS && hh + 1 < r) {  // the next head's biases, while its first tiles come
            const BiasLanes next = load_biases<IO>(a, map, kv * r + hh + 1);
            __syncthreads();
            taken_out = fill_biases<IO, 256 * G>(tab, next, a, map, kv * r + hh + 1);
        }
    };
    using Edge = Kind<UNSEEN || BIAS ? kUnseen : kPartial>;
    if (!steep) [[likely]]
        pass_over<C>(
            r, [&]() { return taken_out ? 0 : n_whole / G; }, n_visits, load,
            [&](int t, int stage) {
#pragma unroll
                for (int qb = 0; qb < 2; ++qb)
                    if (n_rows > 0)
                        block(Kind<kWhole>{}, std::false_type{}, row_at(t) + 32 * qb, qb, stage * 2 * C::TILE, stats[stage], 0);
            },
            [&](int t, int stage) { edge(Edge{}, std::false_type{}, t, stage); }, between);
    else
        pass_over<C>(
            r, []() { return 0; }, n_visits, load, [](int, int) {},
            [&](int t, int stage) { edge(Edge{}, std::true_type{}, t, stage); }, between);
    // The other group's sums, in LDS in the accumulators' order, 4 KB for a wave and 32 columns
    // (as many tiles as they are wide hold them).
    static_assert(G == 1 || (DK && DV ? 2 : 1) * DB * 4 * 4096 <= (int)sizeof(tiles_of), "the sums fit the tiles");
    const bool half = std::is_same_v<IO, _Float16>;
    const float mk = half ? a.scale * inverse_of_power(held) : a.scale, mv = half ? 1.0f / 4096.0f : 1.0f;
    float* const other = reinterpret_cast<float*>(tiles_of) + wave * (DB * 1024) + lane;
    auto pass = [&](f32x16 (&acc)[DB], float m, float* to) __attribute__((always_inline)) {
#pragma unroll
        for (int cb = 0; cb < DB; ++cb)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                acc[cb][i] *= m;
                if (G > 1 && group) to[(16 * cb + i) * 64] = acc[cb][i];
            }
    };
    if constexpr (G > 1) __syncthreads();
    if constexpr (DK) pass(dk, mk, other);
    if constexpr (DV) pass(dv, mv, other + (DK ? 4 * DB * 1024 : 0));
    if constexpr (G > 1) __syncthreads();
    if (group || n_rows <= 0) return;
    auto join = [&](f32x16 (&acc)[DB], const float* from) __attribute__((always_inline)) {
#pragma unroll
        for (int cb = 0; cb < DB; ++cb)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if constexpr (G > 1) acc[cb][i] += from[(16 * cb + i) * 64];
    };
    if constexpr (DK) {
        join(dk, other);
        store_rows<C, IO>(dk, a.dk, s.k0 + w0, kv, n_rows, a.D_k, 1.0f, a.dk_vec);
    }
    if constexpr (DV) {
        join(dv, other + (DK ? 4 * DB * 1024 : 0));
        store_rows<C, IO>(dv, a.dv, s.k0 + w0, kv, n_rows, a.D_v, 1.0f, a.dv_vec);
    }
}

// --- host side ------------------------------------------------------------------------
template <typename IO, int DB, bool VEC, bool BIAS, bool UNSEEN>
hipError_t forward_cfg(const AttentionArgs& a, const BucketMap& map, hipStream_t stream) {
    const size_t table = BIAS ? table_words(a.reach, a.buckets) * 4 : 0;
    in_pieces(a.deal.workgroups(a.heads), 256, [&](uint32_t base, uint32_t wgs) {
        hipLaunchKernelGGL((forward_kernel<IO, DB, VEC, BIAS, UNSEEN>), dim3(wgs), dim3(256), table, stream, a, map, base);
    });
    return hipGetLastError();
}

template <typename IO, int DB, bool VEC, bool BIAS, bool UNSEEN, int G>
void dkv_launch(const AttentionArgs& a, const BucketMap& map, size_t table, hipStream_t stream) {
    in_pieces(a.kv_deal.workgroups(a.kv_heads), 256 * G, [&](uint32_t base, uint32_t wgs) {
        const dim3 grid(wgs), threads(256 * G);
        if constexpr (dkv_apart(sizeof(IO), DB)) {
            hipLaunchKernelGGL((dkv_kernel<IO, DB, VEC, BIAS, UNSEEN, G, true, false>), grid, threads, table, stream, a, map, base);
            hipLaunchKernelGGL((dkv_kernel<IO, DB, VEC, BIAS, UNSEEN, G, false, true>), grid, threads, table, stream, a, map, base);
        } else {
            hipLaunchKernelGGL((dkv_kernel<IO, DB, VEC, BIAS, UNSEEN, G, true, true>), grid, threads, table, stream, a, map, base);
        }
    });
}

template <typename IO, int DB, bool VEC, bool BIAS, bool UNSEEN>
hipError_t backward_cfg(const AttentionArgs& a, const BucketMap& map, hipStream_t stream) {
    const size_t table = BIAS ? table_words(a.reach, a.buckets) * 4 : 0, sums = a.dbias ? 8 * tab_width(a.reach) * 4 : 0;
    in_pieces(a.deal.workgroups(a.heads), 256, [&](uint32_t base, uint32_t wgs) {
        hipLaunchKernelGGL((dq_kernel<IO, DB, VEC, BIAS, UNSEEN>), dim3(wgs), dim3(256), table + sums, stream, a, map, base);
    });
    // two groups where a causal key may have thousands of queries; short sequences (64 images of mean 197
    // tokens: 82 us with two groups, 74 with one) have no use for them
    if (a.kv_deal.units) dkv_launch<IO, DB, VEC, BIAS, UNSEEN, 2>(a, map, table, stream);
    else dkv_launch<IO, DB, VEC, BIAS, UNSEEN, 1>(a, map, table, stream);
    return hipGetLastError();
}

// Rows off 16 bytes go number by number, causal or not into the same kernels.  (With biases or without as others do:
// a score that a bias of 0 is added to is rounded at its size, one without only less its maximum.)
#define EQL_ATTENTION(WHAT)                                       \
    const int db = ((a.D_k > a.D_v ? a.D_k : a.D_v) + 31) / 32;   \
    const bool bias = a.bias != nullptr;                          \
    if (db == 1) return EQL_ATTENTION_DB(WHAT, 1);                \
    if (db == 2) return EQL_ATTENTION_DB(WHAT, 2);                \
    if (db == 3) return EQL_ATTENTION_DB(WHAT, 3);                \
    return EQL_ATTENTION_DB(WHAT, 4);
#define EQL_ATTENTION_DB(WHAT, DB)                                                                                            \
    !vec       ? (bias ? WHAT<IO, DB, false, true, true>(a, map, stream) : WHAT<IO, DB, false, false, true>(a, map, stream))  \
    : a.causal ? (bias ? WHAT<IO, DB, true, true, true>(a, map, stream) : WHAT<IO, DB, true, false, true>(a, map, stream))    \
               : (bias ? WHAT<IO, DB, true, true, false>(a, map, stream) : WHAT<IO, DB, true, false, false>(a, map, stream))

template <typename IO>
hipError_t forward(AttentionArgs a, const BucketMap& map, hipStream_t stream) {
    const size_t es = sizeof(IO);
    const bool vec = vec_ok(a.q, a.D_k, es, 16) && vec_ok(a.k, a.D_k, es, 16) && vec_ok(a.v, a.D_v, es, 16);
    a.out_vec = vec_ok(a.o, a.D_v, es, 4 * es);
    EQL_ATTENTION(forward_cfg)
}

template <typename IO>
hipError_t backward(AttentionArgs a, const BucketMap& map, hipStream_t stream) {
    const size_t es = sizeof(IO);
    const bool vec = vec_ok(a.q, a.D_k, es, 16) && vec_ok(a.k, a.D_k, es, 16) && vec_ok(a.v, a.D_v, es, 16) &&
                     vec_ok(a.o, a.D_v, es, 16) && vec_ok(a.d_o, a.D_v, es, 16);
    a.dq_vec = vec_ok(a.dq, a.D_k, es, 4 * es);
    a.dk_vec = vec_ok(a.dk, a.D_k, es, 4 * es);
    a.dv_vec = vec_ok(a.dv, a.D_v, es, 4 * es);
    EQL_ATTENTION(backward_cfg)
}

}  // namespace att
}  // namespace eql
