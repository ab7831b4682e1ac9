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

constexpr int kQueries = 16;  // query heads of one workgroup: the columns of a matrix product
constexpr int kKeys = 32;     // keys of a wave's tile

struct Grid {
    int groups, splits;  // of the query heads of a kv head; of a sequence
};
Grid grid_for(int heads, int kv_heads, int64_t batch) {
    Grid g;
    g.groups = (heads / kv_heads + kQueries - 1) / kQueries;
    const int64_t n = batch * kv_heads * g.groups;
    g.splits = (int)(n >= 1024 ? 1 : (1024 + n - 1) / n);
    g.splits = g.splits > 64 ? 64 : g.splits;
    return g;
}

// Keys of split `split` of a sequence of n: whole tiles of all four waves.
__device__ __forceinline__ void keys_of(int n, int splits, int split, int& k0, int& k1) {
    const int tiles = (n + 4 * kKeys - 1) / (4 * kKeys), per = (tiles + splits - 1) / splits * (4 * kKeys);
    const int64_t a = (int64_t)split * per;
    k0 = a < n ? (int)a : n;
    k1 = a + per < n ? (int)(a + per) : n;
}
__device__ __forceinline__ int length_of(const StepArgs& a, int64_t b) {
    const int n = a.lengths[b];
    const int64_t most = (int64_t)a.max_blocks * a.block_size;
    return n < 0 ? 0 : (n > most ? (int)most : n);
}

// Element offset of a key's row, or -1 where its block is none of the cache's.
__device__ __forceinline__ int64_t row_of_key(const StepArgs& a, const Pages& x, int64_t b, int key, int kv) {
    const int blk = key / a.block_size;
    const int id = a.table[b * a.max_blocks + blk];
    if (id < 0 || id >= a.blocks) return -1;
    return id * x.bs + (int64_t)(key - blk * a.block_size) * x.ts + kv * x.hs;
}

template <typename IO, int DB, bool VEC>
__global__ __launch_bounds__(256) void step_kernel(StepArgs a, BucketMap map, Grid g, float* ws, uint32_t base) {
    using O = Op<IO>;
    using F = typename O::F;
    constexpr int ES = O::ES, E = 16 / ES, D = 32 * DB, P = D / E, NB = D / 16, NM = D / O::KS;
    constexpr int NL = kKeys * P / 64;  // loads of a tile of v
    __shared__ __attribute__((aligned(16))) char lds[4][kKeys * P * 16];
    __shared__ float ms[4][kQueries], ls[4][kQueries], all_top[kQueries], all_sum[kQueries];
    const uint32_t wg = blockIdx.x + base;
    const int split = (int)(wg % (uint32_t)g.splits);
    uint32_t rest = wg / (uint32_t)g.splits;
    const int group = (int)(rest % (uint32_t)g.groups);
    rest /= (uint32_t)g.groups;
    const int kv = (int)(rest % (uint32_t)a.kv_heads);
    const int64_t b = rest / (uint32_t)a.kv_heads;
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6, kg = lane >> 4, ln = lane & 15;
    const int r = a.heads / a.kv_heads, nq = r - group * kQueries < kQueries ? r - group * kQueries : kQueries;
    const int head0 = kv * r + group * kQueries;
    const int n = length_of(a, b);
    int k0, k1;
    keys_of(n, g.splits, split, k0, k1);
    if (k0 >= k1 && !(split == 0 && n == 0)) return;

    F q[NM];
    {
        const IO* p = (const IO*)a.q.p + b * a.q.ts + (int64_t)(head0 + (ln < nq ? ln : 0)) * a.q.hs;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const u32x4 v = load_piece<IO>(p, (4 * m + kg) * E, ln < nq ? a.D_k : 0);
            q[m] = __builtin_bit_cast(F, v);
        }
    }
    f32x4 acc[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    float top = -kInf, total = 0.0f;
    const float scale = a.scale * kLog2e;
    char* const tv = lds[wave];
    for (int j0 = k0 + wave * kKeys; j0 < k1; j0 += 4 * kKeys) {
        f32x4 x[2];
        bool ok[2][4];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const int key = j0 + 16 * kb + ln;
            const int64_t at = key < k1 ? row_of_key(a, a.k, b, key, kv) : -1;
            const IO* p = (const IO*)a.k.p + (at < 0 ? 0 : at);
            x[kb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                u32x4 v = {0u, 0u, 0u, 0u};
                const int col = (4 * m + kg) * E;
                if (at >= 0) {
                    if constexpr (VEC) {
                        if (col < a.D_k) v = *reinterpret_cast<const u32x4*>(p + col);
                    } else {
                        v = load_piece<IO>(p, col, a.D_k);
                    }
                }
                O::mma(x[kb], __builtin_bit_cast(F, v), q[m]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) ok[kb][i] = __shfl((int)(at >= 0), 4 * kg + i) != 0;
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int s = 64 * i + lane, row = s / P, piece = s % P, key = j0 + row, col = piece * E;
            const int64_t at = key < k1 && col < a.D_v ? row_of_key(a, a.v, b, key, kv) : -1;
            u32x4 v = {0u, 0u, 0u, 0u};
            if (at >= 0) {
                const IO* p = (const IO*)a.v.p + at;
                if constexpr (VEC) v = *reinterpret_cast<const u32x4*>(p + col);
                else v = load_piece<IO>(p, col, a.D_v);
            }
            *reinterpret_cast<u32x4*>(tv + place<ES, P>(row, piece)) = v;
        }
        float mx = -kInf;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y = x[kb][i] * scale;
                if (a.bias) {
                    const int far = n - 1 - (j0 + 16 * kb + 4 * kg + i);
                    const int at = map.of[far < 0 ? 0 : (far < a.reach ? far : a.reach)];
                    y += kLog2e * (ln < nq ? (float)((const IO*)a.bias)[(int64_t)(head0 + ln) * a.buckets + at] : 0.0f);
                }
                x[kb][i] = ok[kb][i] ? y : -kInf;
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
        // (the wave's own tile: its writes are there once they are waited for)
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
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
                        v[e] = *reinterpret_cast<const float*>(tv + place<ES, P>(16 * kb + 4 * kg + e, 4 * cb + (ln >> 2)) + (ln & 3) * 4);
                    O::mma(acc[cb], v, x[kb]);
                }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
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
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) mine[ln * kRow + 16 * i + 4 * kg + e] = c * acc[i][e];
    if (tid < kQueries) all_top[tid] = all, all_sum[tid] = sum;  // (lane ln of wave 0)
    __syncthreads();
    const int nr = r < kQueries ? r : kQueries;
    for (int e = tid; e < nq * a.D_v; e += 256) {
        const int h = e / a.D_v, d = e - h * a.D_v;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) v += reinterpret_cast<const float*>(lds[w])[h * kRow + d];
        if (g.splits == 1) {
            const float s = all_sum[h];
            ((IO*)const_cast<void*>(a.o.p))[b * a.o.ts + (int64_t)(head0 + h) * a.o.hs + d] = (IO)(s == 0.0f ? 0.0f : v / s);
        } else {
            ws[((int64_t)wg * nr + h) * (a.D_v + 2) + 2 + d] = v;
        }
    }
    if (tid < nq) {
        const float s = all_sum[tid], t = all_top[tid];
        if (g.splits > 1) {
            float* p = ws + ((int64_t)wg * nr + tid) * (a.D_v + 2);
            p[0] = t, p[1] = s;
        } else if (a.lse) {
            a.lse[(int64_t)(head0 + tid) * a.batch + b] =
                s == 0.0f ? -kInf : ((t == -kInf ? 0.0f : t) - att::kShift<IO> + __builtin_amdgcn_logf(s)) * kLn2;
        }
    }
}

// Joins the splits of one (sequence, head): a wave each.
template <typename IO>
__global__ __launch_bounds__(256) void join_kernel(StepArgs a, Grid g, const float* ws, uint32_t base) {
    const int lane = (int)threadIdx.x & 63;
    const int64_t id = ((int64_t)blockIdx.x + base) * 4 + (threadIdx.x >> 6);
    if (id >= a.batch * a.heads) return;
    const int64_t b = id / a.heads;
    const int head = (int)(id - b * a.heads), r = a.heads / a.kv_heads, kv = head / r, group = (head - kv * r) / kQueries;
    const int h = head - kv * r - group * kQueries, nr = r < kQueries ? r : kQueries;
    const int n = length_of(a, b);
    const float* p = ws + (((b * a.kv_heads + kv) * g.groups + group) * g.splits * nr + h) * (a.D_v + 2);
    const int64_t step = (int64_t)nr * (a.D_v + 2);
    int used = 0;
    for (int s = 0, k0, k1; s < g.splits; ++s) {
        keys_of(n, g.splits, s, k0, k1);
        if (k0 < k1 || (s == 0 && n == 0)) used = s + 1;
    }
    float all = -kInf, sum = 0.0f;
    for (int s = 0; s < used; ++s) all = fmaxf(all, p[s * step]);
    float v0 = 0.0f, v1 = 0.0f;
    for (int s = 0; s < used; ++s) {
        const float t = p[s * step], c = t == all || t == -kInf ? 1.0f : __builtin_amdgcn_exp2f(t - all);
        sum += c * p[s * step + 1];
        if (lane < a.D_v) v0 += c * p[s * step + 2 + lane];
        if (lane + 64 < a.D_v) v1 += c * p[s * step + 2 + lane + 64];
    }
    IO* o = (IO*)const_cast<void*>(a.o.p) + b * a.o.ts + (int64_t)head * a.o.hs;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (lane < a.D_v) o[lane] = (IO)(v0 * inv);
    if (lane + 64 < a.D_v) o[lane + 64] = (IO)(v1 * inv);
    if (lane == 0 && a.lse)
        a.lse[(int64_t)head * a.batch + b] =
            sum == 0.0f ? -kInf : ((all == -kInf ? 0.0f : all) - att::kShift<IO> + __builtin_amdgcn_logf(sum)) * kLn2;
}

template <typename IO, int DB, bool VEC>
hipError_t run_cfg(const StepArgs& a, const BucketMap& map, float* ws, hipStream_t stream) {
    const Grid g = grid_for(a.heads, a.kv_heads, a.batch);
    in_pieces(a.batch * a.kv_heads * g.groups * g.splits, 256, [&](uint32_t base, uint32_t wgs) {
        hipLaunchKernelGGL((step_kernel<IO, DB, VEC>), dim3(wgs), dim3(256), 0, stream, a, map, g, ws, base);
    });
    if (g.splits > 1)
        in_pieces((a.batch * a.heads + 3) / 4, 256, [&](uint32_t base, uint32_t wgs) {
            hipLaunchKernelGGL((join_kernel<IO>), dim3(wgs), dim3(256), 0, stream, a, g, ws, base);
        });
    return hipGetLastError();
}

template <typename IO>
hipError_t run(const StepArgs& a, const BucketMap& map, float* ws, hipStream_t stream) {
    const size_t es = sizeof(IO);
    auto vec = [&](const Pages& x, int D) {
        return (uintptr_t)x.p % 16 == 0 && x.bs * es % 16 == 0 && x.ts * es % 16 == 0 && x.hs * es % 16 == 0 && D * es % 16 == 0;
    };
    const bool v = vec(a.k, a.D_k) && vec(a.v, a.D_v);
    const int db = ((a.D_k > a.D_v ? a.D_k : a.D_v) + 31) / 32;
#define EQL_STEP(DB) v ? run_cfg<IO, DB, true>(a, map, ws, stream) : run_cfg<IO, DB, false>(a, map, ws, stream)
    if (db == 1) return EQL_STEP(1);
    if (db == 2) return EQL_STEP(2);
    if (db == 3) return EQL_STEP(3);
    return EQL_STEP(4);
#undef EQL_STEP
}

}  // namespace

size_t attention_step_workspace(int heads, int kv_heads, int D_v, int64_t batch) {
    if (batch <= 0) return 0;
    const Grid g = grid_for(heads, kv_heads, batch);
    const int r = heads / kv_heads, nr = r < kQueries ? r : kQueries;
    return g.splits == 1 ? 0 : (size_t)batch * kv_heads * g.groups * g.splits * nr * (D_v + 2) * 4;
}

hipError_t launch_attention_step(int io, const StepArgs& a, const BucketMap& map, void* ws, hipStream_t stream) {
    if (a.batch * a.kv_heads * ((a.heads / a.kv_heads + kQueries - 1) / kQueries) > 0x7fffffff) return hipErrorNotSupported;
    float* w = static_cast<float*>(ws);
    return io == kIoF32 ? run<float>(a, map, w, stream)
                        : (io == kIoBF16 ? run<__bf16>(a, map, w, stream) : run<_Float16>(a, map, w, stream));
}

}  // namespace eql
