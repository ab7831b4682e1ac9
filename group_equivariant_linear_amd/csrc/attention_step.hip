// attention_step.hip -- softmax attention of one new token for each of many sequences, over
// keys and values in the blocks of a paged cache.
#include "attention.h"

namespace eql {

namespace {

using namespace tile;
using att::clear;
using att::kInf;
using att::kLn2;
using att::kLog2e;

constexpr int kQueries = 16;     // query heads of one workgroup: the columns of a matrix product
constexpr int kKeys = 32;        // keys of a wave's tile
constexpr int kUnit = 4 * kKeys;  // keys of a workgroup's pass
constexpr int kMaxShared = 2048;  // sequences whose lengths a workgroup sums up
constexpr int kWorkgroups = 1024;  // at most

// A sequence's keys are units of kUnit; an item is one (sequence, kv head, run of kQueries of
// its query heads).  Up to kMaxShared sequences, the units of all items lie in one row that is
// cut evenly over the workgroups (as many as have any), whatever sequences they belong to, so that lengths need not be alike (or known
// on the host).  An item inside one
// workgroup is finished there; of one that spans several, each writes its part, at 2 w + 1 if
// the item starts in w, else at 2 w, and join_kernel takes them in order.  With more sequences
// each item is one workgroup's: their lengths no longer fit beside the tiles, and there are enough
// items to fill the card.  (12 heads on 4 of 128 numbers, bf16: 2048 sequences of 400 keys take 258 us
// cut evenly, 2049 take 224, which need no join; with one of 32768 keys among sequences of 100, 163 and 447.)
struct Grid {
    int groups, items;  // runs of the query heads of a kv head; items of a sequence
    int shared;
    uint32_t wgs;
};
// Waves per SIMD that the registers are held to: workgroups a CU, all of which run at once.
constexpr int step_waves(int es, int db) { return es == 4 ? (db == 1 ? 3 : (db == 2 ? 2 : 1)) : (db == 1 ? 4 : (db == 2 ? 3 : 2)); }
Grid grid_for(int es, int heads, int kv_heads, int D_k, int D_v, int64_t batch) {
    Grid g;
    g.groups = (heads / kv_heads + kQueries - 1) / kQueries;
    g.items = kv_heads * g.groups;
    g.shared = batch <= kMaxShared;
    g.wgs = g.shared ? 256 * step_waves(es, ((D_k > D_v ? D_k : D_v) + 31) / 32) : (uint32_t)(batch * g.items);
    return g;
}
// (64-bit divisions take 150 instructions in a row: 32-bit ones where they do)
__device__ __forceinline__ int64_t divided(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
struct Cut {
    int64_t W, each, more;  // workgroups; units of each; the first `more` take one more
    __device__ __forceinline__ Cut(int64_t units, uint32_t wgs) : W(units < wgs ? units : wgs) {
        each = divided(units, W);
        more = units - each * W;
    }
    __device__ __forceinline__ int64_t first(int64_t w) const { return (w < W ? w : W) * each + (w < more ? w : more); }
    __device__ __forceinline__ int64_t owner(int64_t unit) const {
        const int64_t big = more * (each + 1);
        return unit < big ? divided(unit, each + 1) : more + divided(unit - big, each);
    }
};

__device__ __forceinline__ int length_of(const StepArgs& a, int64_t b) {
    const int n = a.lengths[b];
    const int64_t most = (int64_t)a.max_blocks * a.block_size;
    return n < 0 ? 0 : (n > most ? (int)most : n);
}
// Floats of a part's row of values: whole pieces of four.
__host__ __device__ constexpr int row_floats(int D) { return (D + 3) / 4 * 4; }
// (an empty sequence has one unit, of no keys: its outputs are written too)
__device__ __forceinline__ int units_of(int n) { return n > 0 ? (n + kUnit - 1) / kUnit : 1; }

// One wave takes 32 keys at a time: scores S^T = K Q^T with the keys as rows straight from
// memory, the values through an LDS tile of its own (read back transposed).  The next keys'
// loads go out as soon as these have left their registers, and the blocks of the keys after
// those with them.  Its four waves' sums are joined at the end of an item.  256 sequences of mean
// 2048 tokens: 210 us, the keys and values at 5.0 TB/s (994 with an item to a workgroup); 8 sequences 13.0 us
// and one of 131072 tokens 30.8, of which a workgroup's start and the chain table, keys, values is the most.
template <typename IO, int DB, bool VEC, bool BIAS>
__global__ __launch_bounds__(256, step_waves(sizeof(IO), DB)) void step_kernel(StepArgs a, BucketMap map, Grid g, float* ws, uint32_t base) {
    using O = Op<IO>;
    using F = typename O::F;
    constexpr int ES = O::ES, E = 16 / ES, D = 32 * DB, P = D / E, NB = D / 16, NM = D / O::KS;
    constexpr int NL = kKeys * P / 64;  // loads of a tile of v
    __shared__ __attribute__((aligned(16))) char lds[4][kKeys * P * 16];
    __shared__ float ms[4][kQueries], ls[4][kQueries], all_top[kQueries], all_sum[kQueries];
    __shared__ int wave_units[4], wave_out[4];
    __shared__ __attribute__((aligned(16))) int found[4][2][BIAS ? D : 1];  // columns' keys of +infinity or NaN, of -infinity or NaN
    extern __shared__ int shared[];  // units before each sequence, lengths; an item's biases; the buckets of distances
    const uint32_t wg = blockIdx.x + base;
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), kg = lane >> 4, ln = lane & 15;
    const int r = a.heads / a.kv_heads, nr = r < kQueries ? r : kQueries;
    const float scale = a.scale * kLog2e;
    int* const lengths = shared + a.batch + 1;
    float* const biases = reinterpret_cast<float*>(shared + (g.shared ? 2 * a.batch + 1 : 0));
    uint8_t* const buckets = reinterpret_cast<uint8_t*>(biases + kQueries * a.buckets);

    if (BIAS && a.bias)  // each bucket marks its distances (the step is causal: all past ones are on the first side)
        for (int i = tid; i < a.side; i += 256)
            for (int x = map.start[i]; x < map.start[i + 1]; ++x) buckets[x] = (uint8_t)i;
    int64_t u0, u1;
    if (g.shared) {
        constexpr int N = kMaxShared / 256;
        const int B = (int)a.batch, per = (B + 255) / 256;
        int n[N], sum = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int b = tid * per + i;
            const int len = i < per && b < B ? length_of(a, b) : 0;
            if (i < per && b < B) lengths[b] = len;
            n[i] = i < per && b < B ? units_of(len) : 0;
            sum += n[i];
        }
        int at = sum;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int w = __shfl_up(at, o);
            if (lane >= o) at += w;
        }
        if (lane == 63) wave_units[wave] = at;
        __syncthreads();
        at -= sum;
        for (int w = 0; w < wave; ++w) at += wave_units[w];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int b = tid * per + i;
            if (i < per && b <= B) shared[b] = at;
            at += n[i];
        }
        if (tid == 255 && per * 256 <= B) shared[B] = at;
        __syncthreads();
        if (wg == 0)  // for join_kernel
            for (int b = tid; b <= B; b += 256) reinterpret_cast<int*>(ws)[b] = shared[b];
        const Cut cut((int64_t)shared[B] * g.items, g.wgs);
        u0 = cut.first(wg), u1 = cut.first(wg + 1);
    } else {
        u0 = 0, u1 = 1;
    }
    float* const parts = ws + (g.shared ? (a.batch + 1 + 63) / 64 * 64 : 0);

    while (u0 < u1) {
        int64_t b;
        int item, unit, n, count;
        bool starts = true, ends = true;
        if (g.shared) {
            int lo = 0, hi = (int)a.batch - 1;  // last sequence whose units start at u0 or before
            const int64_t target = divided(u0, g.items);
            // units of sequence b are shared[b] g.items .. shared[b + 1] g.items
            while (lo < hi) {
                const int mid = lo + (hi - lo + 1) / 2;
                if (shared[mid] <= target) lo = mid;
                else hi = mid - 1;
            }
            b = lo;
            n = lengths[lo];
            const int of = units_of(n);
            const int64_t in = u0 - (int64_t)shared[lo] * g.items;
            item = (int)divided(in, of);
            unit = (int)(in - (int64_t)item * of);
            count = u1 - u0 < of - unit ? (int)(u1 - u0) : of - unit;
            starts = unit == 0, ends = unit + count == of;
        } else {
            b = wg / (uint32_t)g.items;
            item = (int)(wg - (uint32_t)b * (uint32_t)g.items);
            n = length_of(a, b);
            unit = 0, count = units_of(n);
        }
        u0 += g.shared ? count : 1;
        const int kv = item / g.groups, group = item - kv * g.groups;
        const int nq = r - group * kQueries < kQueries ? r - group * kQueries : kQueries, head0 = kv * r + group * kQueries;
        const int k0 = unit * kUnit, k1 = n - k0 < count * kUnit ? n : k0 + count * kUnit;

        // Row offsets of a tile's keys, in lanes 0 .. 31 (and again 32 .. 63): -1 where there is none.
        auto block_of = [&](int j0) {
            const int key = j0 + (lane & 31);
            return key < k1 ? a.table[b * a.max_blocks + (uint32_t)key / (uint32_t)a.block_size] : -1;
        };
        u32x4 kreg[2][NM], vreg[NL];
        uint32_t there = 0;  // the tile's keys that are there, a bit each
        const IO* const kp = (const IO*)a.k.p + kv * a.k.hs;
        const IO* const vp = (const IO*)a.v.p + kv * a.v.hs;
        // (a key that is not there reads the cache's first row, and counts for nothing)
        auto at = [&](const Pages& x, int j0, int id) {
            const int64_t in = (uint32_t)(j0 + (lane & 31)) % (uint32_t)a.block_size;
            return id >= 0 && id < a.blocks ? id * x.bs + in * x.ts : (int64_t)0;
        };
        auto load_k = [&](int64_t rows) __attribute__((always_inline)) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const IO* p = kp + __shfl(rows, 16 * kb + ln);
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    const int col = (4 * m + kg) * E;
                    if constexpr (VEC) kreg[kb][m] = *reinterpret_cast<const u32x4*>(p + (col < a.D_k ? col : 0));
                    else kreg[kb][m] = load_piece<IO>(p, col, a.D_k);
                }
            }
        };
        auto load_v = [&](int64_t rows) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int s = 64 * i + lane, col = s % P * E;
                const IO* p = vp + __shfl(rows, s / P);
                if constexpr (VEC) vreg[i] = *reinterpret_cast<const u32x4*>(p + (col < a.D_v ? col : 0));
                else vreg[i] = load_piece<IO>(p, col, a.D_v);
            }
        };

        const int j_first = k0 + wave * kKeys;
        int id = block_of(j_first);
        F q[NM];
        {
            const IO* p = (const IO*)a.q.p + b * a.q.ts + (int64_t)(head0 + (ln < nq ? ln : 0)) * a.q.hs;
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const int col = (4 * m + kg) * E;
                u32x4 v = {0u, 0u, 0u, 0u};
                if (VEC && a.q_vec) {
                    if (ln < nq && col < a.D_k) v = *reinterpret_cast<const u32x4*>(p + col);
                } else {
                    v = load_piece<IO>(p, col, ln < nq ? a.D_k : 0);
                }
                q[m] = __builtin_bit_cast(F, v);
            }
        }
        if (k0 < k1) {  // (else there may be no cache)
            load_k(at(a.k, j_first, id));
            load_v(at(a.v, j_first, id));
        }
        there = (uint32_t)__ballot(id >= 0 && id < a.blocks);
        id = block_of(j_first + kUnit);

        bool out = false;
        if constexpr (BIAS) {
            for (int i = tid; a.bias && i < nq * a.buckets; i += 256) {
                biases[i] = att::in_powers((float)((const IO*)a.bias)[(int64_t)head0 * a.buckets + i]);
                out |= biases[i] == -kInf;
            }
            out = __any(out);
            if (lane == 0) wave_out[wave] = out;
        }
        __syncthreads();
        // Some biases are -infinity: their heads do not see the keys at these distances, whatever stands there.
        const bool taken_out = BIAS && __builtin_amdgcn_readfirstlane(wave_out[0] | wave_out[1] | wave_out[2] | wave_out[3]);

        f32x4 acc[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        float top = -kInf, total = 0.0f;
        char* const tv = lds[wave];
        const float far = BIAS && a.bias ? biases[(ln < nq ? ln : 0) * a.buckets + a.side - 1] : 0.0f;
        for (int j0 = j_first; j0 < k1; j0 += kUnit) {
            f32x4 x[2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                x[kb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    u32x4 v = kreg[kb][m];
                    // (numbers past the row are others': zeros)
                    if (VEC && D != a.D_k && (4 * m + kg) * E >= a.D_k) v = u32x4{0u, 0u, 0u, 0u};
                    O::mma(x[kb], __builtin_bit_cast(F, v), q[m]);
                }
            }
            load_k(at(a.k, j0 + kUnit, id));
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int s = 64 * i + lane, row = s / P, piece = s % P;
                u32x4 v = vreg[i];
                if (VEC && D != a.D_v && piece * E >= a.D_v) v = u32x4{0u, 0u, 0u, 0u};
                if (there != 0xffffffffu && !(there >> row & 1)) v = u32x4{0u, 0u, 0u, 0u};
                *reinterpret_cast<u32x4*>(tv + place<ES, P>(row, piece)) = v;
            }
            load_v(at(a.v, j0 + kUnit, id));
            const uint32_t next = (uint32_t)__ballot(id >= 0 && id < a.blocks);
            id = block_of(j0 + 2 * kUnit);
            if (BIAS && a.bias && n - 1 - (j0 + kKeys - 1) < a.reach) {  // the tile's last key
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        int far_by = n - 1 - (j0 + 16 * kb + 4 * kg + i);
                        far_by = far_by < 0 ? 0 : (far_by < a.reach ? far_by : a.reach);
                        x[kb][i] = __builtin_fmaf(x[kb][i], scale, biases[(ln < nq ? ln : 0) * a.buckets + buckets[far_by]]);
                    }
            } else {
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[kb][i] = __builtin_fmaf(x[kb][i], scale, far);
            }
            uint32_t sees = ~0u;  // keys of the tile, a bit each
            bool odd = false;
            if (taken_out) [[unlikely]] {
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        int far_by = n - 1 - (j0 + 16 * kb + 4 * kg + i);
                        far_by = far_by < 0 ? 0 : (far_by < a.reach ? far_by : a.reach);
                        if (biases[(ln < nq ? ln : 0) * a.buckets + buckets[far_by]] == -kInf)
                            x[kb][i] = -kInf, sees &= ~(1u << (16 * kb + 4 * kg + i));
                    }
                sees &= __shfl_xor(sees, 16);
                sees &= __shfl_xor(sees, 32);
                // (rare) infinities and NaN leave the tile: a product would take them to the heads that do not see
                // them as well, 0 times infinity
                asm volatile("" ::: "memory");
                uint32_t largest = 0;
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    const F f[1] = {*reinterpret_cast<const F*>(tv + (64 * i + lane) * 16)};
                    const uint32_t o = O::top(f);
                    largest = o > largest ? o : largest;
                }
                odd = __any(largest >= O::kInf);
#pragma unroll 1
                for (int d = lane; odd && d < D; d += 64) {
                    uint32_t pos = 0, neg = 0;
#pragma unroll 1
                    for (int row = 0; row < kKeys; ++row) {
                        IO* const y = reinterpret_cast<IO*>(tv + place<ES, P>(row, d / E) + d % E * ES);
                        const float f = (float)*y;
                        if (fabsf(f) < kInf) continue;
                        if (!(f < 0.0f)) pos |= 1u << row;
                        if (!(f > 0.0f)) neg |= 1u << row;
                        *y = (IO)0.0f;
                    }
                    found[wave][0][d] = (int)pos, found[wave][1][d] = (int)neg;
                }
            }
            float mx = -kInf;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (there != 0xffffffffu && !(there >> (16 * kb + 4 * kg + i) & 1)) x[kb][i] = -kInf;
                    mx = fmaxf(mx, x[kb][i]);
                }
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            if (__any(mx > top + att::kSlack<IO>)) {
                const float now = mx > top + att::kSlack<IO> ? mx : top;
                const float c = top == -kInf ? 0.0f : __builtin_amdgcn_exp2f(top - now);
                top = now;
                total *= c;
#pragma unroll
                for (int i = 0; i < NB; ++i) acc[i] *= c;
            }
            const float m = (top == -kInf ? 0.0f : top) - att::kShift<IO>;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[kb][i] = __builtin_amdgcn_exp2f(x[kb][i] - m);
                    total += x[kb][i];
                }
            // (the wave's own tile: its LDS instructions come in order)
            asm volatile("" ::: "memory");
            if constexpr (ES == 2) {
                const u32x4 u = {Half<IO>::pack2(x[0][0], x[0][1]), Half<IO>::pack2(x[0][2], x[0][3]),
                                 Half<IO>::pack2(x[1][0], x[1][1]), Half<IO>::pack2(x[1][2], x[1][3])};
                const F p = __builtin_bit_cast(F, u);
                const int row = 4 * kg + (ln >> 2);
#pragma unroll
                for (int cb = 0; cb < NB; ++cb) {
                    const int piece = 2 * cb + ((lane & 3) >> 1), in = (lane & 1) * 8;
                    O::mma(acc[cb], O::column(tv + place<ES, P>(row, piece) + in, tv + place<ES, P>(row + 16, piece) + in), p);
                }
            } else {
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int cb = 0; cb < NB; ++cb) {
                        F v;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = *reinterpret_cast<const float*>(tv + place<ES, P>(16 * kb + 4 * kg + e, 4 * cb + (ln >> 2)) +
                                                                   (ln & 3) * 4);
                        O::mma(acc[cb], v, x[kb]);
                    }
            }
            if (taken_out && odd) [[unlikely]] {  // and join those that do
#pragma unroll
                for (int cb = 0; cb < NB; ++cb) {
                    asm volatile("" ::: "memory");
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[cb][i] += found[wave][0][16 * cb + 4 * kg + i] & (int)sees ? kInf : 0.0f;
                        acc[cb][i] += found[wave][1][16 * cb + 4 * kg + i] & (int)sees ? -kInf : 0.0f;
                    }
                }
            }
            asm volatile("" ::: "memory");
            there = next;
        }
        total += __shfl_xor(total, 16);
        total += __shfl_xor(total, 32);
        if (kg == 0) ms[wave][ln] = top, ls[wave][ln] = total;
        __syncthreads();
        float all = -kInf;
#pragma unroll
        for (int w = 0; w < 4; ++w) all = fmaxf(all, ms[w][ln]);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float t = ms[w][ln];
            // (a wave whose scores were all NaN has no maximum but a sum)
            sum += ls[w][ln] * (t == all || t == -kInf ? 1.0f : __builtin_amdgcn_exp2f(t - all));
        }
        const float c = top == all || top == -kInf ? 1.0f : __builtin_amdgcn_exp2f(top - all);
        // each wave's sums to LDS (its own tile, which nobody else reads), then joined in order
        float* const mine = reinterpret_cast<float*>(lds[wave]);
        constexpr int kRow = kKeys * P * 16 / 4 / kQueries;  // floats of a query's row: D (16 bit) or 2 D
        static_assert(kRow >= D, "a wave's tile holds its sums");
#pragma unroll
        for (int i = 0; i < NB; ++i) *reinterpret_cast<f32x4*>(mine + ln * kRow + 16 * i + 4 * kg) = acc[i] * c;
        if (tid < kQueries) all_top[tid] = all, all_sum[tid] = sum;  // (lane ln of wave 0)
        __syncthreads();
        const bool whole = starts && ends;
        const int64_t at_part = (int64_t)(2 * wg + (starts ? 1 : 0)) * nr;
        float* const part = parts + 4 * (int64_t)g.wgs * nr + at_part * row_floats(a.D_v);
        for (int e = tid; e < nq * a.D_v; e += 256) {
            const int h = e / a.D_v, d = e - h * a.D_v;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w) v += reinterpret_cast<const float*>(lds[w])[h * kRow + d];
            if (whole) {
                const float s = all_sum[h];
                ((IO*)const_cast<void*>(a.o.p))[b * a.o.ts + (int64_t)(head0 + h) * a.o.hs + d] = (IO)(s == 0.0f ? 0.0f : v / s);
            } else {
                part[h * row_floats(a.D_v) + d] = v;
            }
        }
        if (tid < nq) {
            const float s = all_sum[tid], t = all_top[tid];
            if (!whole) reinterpret_cast<float2*>(parts)[at_part + tid] = float2{t, s};
            else if (a.lse)
                a.lse[(int64_t)(head0 + tid) * a.batch + b] =
                    s == 0.0f ? -kInf : ((t == -kInf ? 0.0f : t) - att::kShift<IO> + __builtin_amdgcn_logf(s)) * kLn2;
        }
        __syncthreads();
    }
}

// Joins the parts of one (sequence, head): a workgroup of kJoin threads, 32 to a part, several
// parts in flight from each.  One sequence of 131072 tokens had 384 parts a head: 7 us on 512
// threads, 71 with a wave that takes one part after the other; 3072 rows of two parts or so
// took 13.7 us on 512 threads, whose waves come in three rounds.
template <typename IO, int kJoin>
__global__ __launch_bounds__(kJoin) void join_kernel(StepArgs a, Grid g, const float* ws, uint32_t base) {
    constexpr int G = kJoin / 32;
    __shared__ float tops[kWorkgroups + 1], sums[G][att::Shape<float, 4>::D], red[kJoin / 64];
    const int tid = (int)threadIdx.x;
    const uint32_t id = blockIdx.x + base;
    const int b = (int)(id / (uint32_t)a.heads), head = (int)(id - (uint32_t)b * (uint32_t)a.heads), r = a.heads / a.kv_heads, kv = head / r;
    const int group = (head - kv * r) / kQueries, h = head - kv * r - group * kQueries, nr = r < kQueries ? r : kQueries;
    const int* const before = reinterpret_cast<const int*>(ws);
    const Cut cut((int64_t)before[a.batch] * g.items, g.wgs);
    const int64_t of = before[b + 1] - before[b];
    const int64_t u = (int64_t)before[b] * g.items + (kv * g.groups + group) * of;
    const int w0 = (int)cut.owner(u), n = (int)cut.owner(u + of - 1) - w0 + 1;
    if (n == 1) return;  // finished there
    const float* const parts = ws + (a.batch + 1 + 63) / 64 * 64;
    auto row = [&](int i) { return (int64_t)(2 * (w0 + i) + (i == 0 ? 1 : 0)) * nr + h; };
    float all = -kInf;
    float2 mine[(kWorkgroups + kJoin - 1) / kJoin];
#pragma unroll
    for (int k = 0; k < (kWorkgroups + kJoin - 1) / kJoin; ++k) {
        const int i = tid + k * kJoin;
        mine[k] = i < n ? reinterpret_cast<const float2*>(parts)[row(i)] : float2{-kInf, 0.0f};
        all = fmaxf(all, mine[k].x);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) all = fmaxf(all, __shfl_xor(all, o));
    if ((tid & 63) == 0) red[tid >> 6] = all;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kJoin / 64; ++k) all = fmaxf(all, red[k]);
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < (kWorkgroups + kJoin - 1) / kJoin; ++k) {
        const float t = mine[k].x, c = t == all || t == -kInf ? 1.0f : __builtin_amdgcn_exp2f(t - all);
        if (tid + k * kJoin < n) tops[tid + k * kJoin] = c;
        sum += c * mine[k].y;
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
    __syncthreads();
    if ((tid & 63) == 0) red[tid >> 6] = sum;
    const float* const values = parts + 4 * (int64_t)g.wgs * nr;
    const int gr = tid / 32, d = (tid & 31) * 4;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    __syncthreads();
    if (d < a.D_v) {
#pragma unroll 8
        for (int i = gr; i < n; i += G) v += *reinterpret_cast<const f32x4*>(values + row(i) * row_floats(a.D_v) + d) * tops[i];
        *reinterpret_cast<f32x4*>(&sums[gr][d]) = v;
    }
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kJoin / 64; ++k) sum += red[k];
    if (tid < a.D_v) {
        float o = 0.0f;
        const int used = n < G ? n : G;
        for (int k = 0; k < used; ++k) o += sums[k][tid];
        ((IO*)const_cast<void*>(a.o.p))[b * a.o.ts + (int64_t)head * a.o.hs + tid] = (IO)(sum == 0.0f ? 0.0f : o / sum);
    }
    if (tid == 0 && a.lse)
        a.lse[(int64_t)head * a.batch + b] =
            sum == 0.0f ? -kInf : ((all == -kInf ? 0.0f : all) - att::kShift<IO> + __builtin_amdgcn_logf(sum)) * kLn2;
}

template <typename IO, int DB, bool VEC, bool BIAS>
hipError_t run_cfg(const StepArgs& a, const BucketMap& map, float* ws, hipStream_t stream) {
    const Grid g = grid_for(sizeof(IO), a.heads, a.kv_heads, a.D_k, a.D_v, a.batch);
    const size_t lds = (g.shared ? (size_t)(2 * a.batch + 1) * 4 : 0) + (a.bias ? (size_t)kQueries * a.buckets * 4 + a.reach + 1 : 0);
    in_pieces(g.wgs, 256, [&](uint32_t base, uint32_t wgs) {
        hipLaunchKernelGGL((step_kernel<IO, DB, VEC, BIAS>), dim3(wgs), dim3(256), lds, stream, a, map, g, ws, base);
    });
    if (g.shared) {
        // many rows: few parts each (on average); few: many
        const bool many = a.batch * g.items >= g.wgs / 8;
        in_pieces(a.batch * a.heads, many ? 128 : 512, [&](uint32_t base, uint32_t rows) {
            if (many) hipLaunchKernelGGL((join_kernel<IO, 128>), dim3(rows), dim3(128), 0, stream, a, g, ws, base);
            else hipLaunchKernelGGL((join_kernel<IO, 512>), dim3(rows), dim3(512), 0, stream, a, g, ws, base);
        });
    }
    return hipGetLastError();
}

template <typename IO>
hipError_t run(StepArgs a, const BucketMap& map, float* ws, hipStream_t stream) {
    const size_t es = sizeof(IO);
    a.q_vec = vec_ok(a.q, a.D_k, es, 16);
    auto vec = [&](const Pages& x, int D) {
        return (uintptr_t)x.p % 16 == 0 && x.bs * es % 16 == 0 && x.ts * es % 16 == 0 && x.hs * es % 16 == 0 && D * es % 16 == 0;
    };
    const bool v = vec(a.k, a.D_k) && vec(a.v, a.D_v);
    const int db = ((a.D_k > a.D_v ? a.D_k : a.D_v) + 31) / 32;
#define EQL_STEP(DB)                                                                                               \
    !v       ? run_cfg<IO, DB, false, true>(a, map, ws, stream)                                                    \
    : a.bias ? run_cfg<IO, DB, true, true>(a, map, ws, stream) : run_cfg<IO, DB, true, false>(a, map, ws, stream)
    if (db == 1) return EQL_STEP(1);
    if (db == 2) return EQL_STEP(2);
    if (db == 3) return EQL_STEP(3);
    return EQL_STEP(4);
#undef EQL_STEP
}

}  // namespace

// Units before each sequence, and two parts of every workgroup.
size_t attention_step_workspace(int io, int heads, int kv_heads, int D_k, int D_v, int64_t batch) {
    if (batch <= 0) return 0;
    const Grid g = grid_for(io == kIoF32 ? 4 : 2, heads, kv_heads, D_k, D_v, batch);
    const int r = heads / kv_heads, nr = r < kQueries ? r : kQueries;
    return g.shared ? ((size_t)(batch + 1 + 63) / 64 * 64 + (size_t)2 * g.wgs * nr * (row_floats(D_v) + 2)) * 4 : 0;
}

hipError_t launch_attention_step(int io, const StepArgs& a, const BucketMap& map, void* ws, hipStream_t stream) {
    if (a.batch * a.kv_heads * ((a.heads / a.kv_heads + kQueries - 1) / kQueries) > 0x7fffffff) return hipErrorNotSupported;
    // (units before each sequence are counted in 32 bits)
    const int64_t most = ((int64_t)a.max_blocks * a.block_size + kUnit - 1) / kUnit;
    if (a.batch <= kMaxShared && a.batch * (most > 0 ? most : 1) > 0x7fffffff) return hipErrorNotSupported;
    float* w = static_cast<float*>(ws);
    return io == kIoF32 ? run<float>(a, map, w, stream)
                        : (io == kIoBF16 ? run<__bf16>(a, map, w, stream) : run<_Float16>(a, map, w, stream));
}

}  // namespace eql
