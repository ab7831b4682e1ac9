// rotary.hip -- rotary positions on regular-representation heads.
//
// Pair (a, b) of channels of every head, for each of the N group elements:
//   a' = m (a cos w - b sin w), b' = m (b cos w + a sin w), w = 2 pi p turns[j].
// The angle's fraction of a turn is taken in fp64, once per (token, pair), and
// shared by every head and group element.
//
// Bound by memory (each number read and written once).  A workgroup takes a run of
// tokens: cos and sin of their pairs go to LDS, then every thread keeps one item of
// a token's row -- a piece of 16 bytes and its partner, or a piece that passes
// through -- from token to token.  12608 tokens, 16 heads of 8 x 8 in bf16 (52 MB):
// 11.9 us, 4.4 TB/s, where items of one number with their own angles took 44; 8 tokens:
// 3.3 us.
#include "eq_device.h"
#include "eq_launch.h"

namespace eql {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxAngles = 1024;  // (token, pair) entries of a workgroup

// p turns less its nearest integer, without the rounding of the product (2^-22 turns
// at the largest positions).
__device__ __forceinline__ float fraction_of_turn(int p, double turns) {
    return (float)fma((double)p, turns, -rint((double)p * turns));
}

// How a row splits into items.
enum Mode {
    kApart,   // the two channels of a pair lie in pieces `dist` numbers apart
    kInside,  // whole pairs lie inside a piece (interleaved, 2 N divides it)
    kSingle   // neither, or rows that no piece fits: items of one number
};

struct Items {
    int turning, passing;  // items of a head that turn, that pass through
    int dist;              // numbers from a pair's first channel to its second
    int per_token;         // items of a token, all heads
    int rows;              // tokens that a workgroup covers at once
    int tokens;            // tokens of a workgroup
};

template <typename IO, int E>
struct Vec {  // E numbers
    using R = std::conditional_t<E == 1, IO, u32x4>;
    static __device__ __forceinline__ void get(const R& r, float (&v)[E]) {
        if constexpr (E == 1) v[0] = (float)r;
        else if constexpr (sizeof(IO) == 4) {
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = __uint_as_float(r[i]);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = i & 1 ? Half<IO>::hi(r[i >> 1]) : Half<IO>::lo(r[i >> 1]);
        }
    }
    static __device__ __forceinline__ R put(const float (&v)[E]) {
        if constexpr (E == 1) return (IO)v[0];
        else if constexpr (sizeof(IO) == 4)
            return u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
        else
            return u32x4{Half<IO>::pack2(v[0], v[1]), Half<IO>::pack2(v[2], v[3]), Half<IO>::pack2(v[4], v[5]),
                         Half<IO>::pack2(v[6], v[7])};
    }
};

template <typename IO, int MODE, int U>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, RotaryFreq f, Items it, uint32_t base) {
    constexpr int E = MODE == kSingle ? 1 : 16 / (int)sizeof(IO);
    using V = Vec<IO, E>;
    using R = typename V::R;
    __shared__ float2 cs[kMaxAngles];
    const int half = a.rot / 2, tid = (int)threadIdx.x;
    const int64_t t0 = (int64_t)(blockIdx.x + base) * it.tokens;
    const int n = (int)(a.T - t0 < it.tokens ? a.T - t0 : it.tokens);
    for (int i = tid; i < n * half; i += kThreads) {
        const int t = i / half;
        const float r = 2.0f * fraction_of_turn(a.positions[t0 + t], f.turns[i - t * half]);
        const float s = f.magnitude * sinpif(r);
        cs[i] = float2{f.magnitude * cospif(r), a.inverse ? -s : s};
    }
    __syncthreads();
    const int row = tid / it.per_token, item = (int)blockIdx.y * kThreads + tid - row * it.per_token;
    if (row >= it.rows || item >= it.per_token) return;
    const int per_head = it.turning + it.passing, h = item / per_head, u = item - h * per_head;
    const bool is_q = h < a.q_heads;
    const Heads& in = is_q ? a.q : a.k;
    const Heads& to = is_q ? a.q_out : a.k_out;
    const int64_t hh = is_q ? h : h - a.q_heads;
    const IO* x = (const IO*)in.p + t0 * in.ts + hh * in.hs;
    IO* y = (IO*)const_cast<void*>(to.p) + t0 * to.ts + hh * to.hs;
    const bool turns = u < it.turning;
    // first number of the item, and its pair
    int e = turns ? u * E : a.rot * a.N + (u - it.turning) * E;
    if (turns && MODE != kInside && a.layout == 1) {  // interleaved: the first channels of the pairs
        const int j = u * E / a.N;
        e = 2 * j * a.N + (u * E - j * a.N);
    }
    int j[E];
    if (turns) {
        if constexpr (MODE == kInside) {
#pragma unroll
            for (int i = 0; i < E; ++i) j[i] = (e + i) / (2 * a.N);
        } else {
            int c = u * E / a.N, r = u * E - c * a.N;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                j[i] = c;
                if (++r == a.N) r = 0, ++c;
            }
        }
    }
    for (int t = row; t < n; t += U * it.rows) {
        R p[U], q[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int tt = t + k * it.rows;
            if (tt < n) {
                p[k] = *reinterpret_cast<const R*>(x + tt * in.ts + e);
                if (MODE != kInside && turns) q[k] = *reinterpret_cast<const R*>(x + tt * in.ts + e + it.dist);
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int tt = t + k * it.rows;
            if (tt >= n) continue;
            if (turns) {
                const float2* w = cs + tt * half;
                float va[E], vb[E];
                V::get(p[k], va);
                if constexpr (MODE == kInside) {
                    // numbers i and i + N of each run of 2 N are a pair
                    auto run = [&](auto nc) {
                        constexpr int N = decltype(nc)::value;
#pragma unroll
                        for (int i = 0; i < E; ++i)
                            if (i % (2 * N) < N) {
                                const float2 c = w[j[i]];
                                const float xa = va[i], xb = va[i + N < E ? i + N : i];
                                vb[i] = xa * c.x - xb * c.y;
                                if (i + N < E) vb[i + N] = xb * c.x + xa * c.y;
                            }
                    };
                    if (a.N == 1) run(std::integral_constant<int, 1>{});
                    else if (a.N == 2) run(std::integral_constant<int, 2>{});
                    else run(std::integral_constant<int, 4>{});
                    p[k] = V::put(vb);
                } else {
                    V::get(q[k], vb);
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const float2 c = w[j[i]];
                        const float xa = va[i], xb = vb[i];
                        va[i] = xa * c.x - xb * c.y;
                        vb[i] = xb * c.x + xa * c.y;
                    }
                    p[k] = V::put(va);
                    *reinterpret_cast<R*>(y + tt * to.ts + e + it.dist) = V::put(vb);
                }
            }
            *reinterpret_cast<R*>(y + tt * to.ts + e) = p[k];
        }
    }
}

bool vec_ok(const Heads& h, size_t es) {
    return ((uintptr_t)h.p & 15u) == 0 && h.ts * es % 16 == 0 && h.hs * es % 16 == 0;
}

template <typename IO, int MODE>
hipError_t launch_mode(const RotaryArgs& a, const RotaryFreq& f, Items it, hipStream_t stream) {
    const int half = a.rot / 2;
    it.per_token = (a.q_heads + a.k_heads) * (it.turning + it.passing);
    it.rows = it.per_token < kThreads ? kThreads / it.per_token : 1;
    const int64_t tiles = (it.per_token + kThreads - 1) / kThreads;
    // four tokens per thread, loaded together, while that leaves two workgroups per CU
    const int most = kMaxAngles / half < 1 ? 1 : kMaxAngles / half;
    const bool four = a.T >= (int64_t)512 * 4 * it.rows && 4 * it.rows <= most;
    if (it.rows > most) it.rows = most;
    it.tokens = four ? 4 * it.rows : it.rows;
    const int64_t wgs = (a.T + it.tokens - 1) / it.tokens;
    if (wgs > 0x7fffffff || tiles > 65535) return hipErrorNotSupported;
    in_pieces(wgs, kThreads, [&](uint32_t base, uint32_t n) {
        const dim3 grid(n, (uint32_t)tiles);
        if (four) hipLaunchKernelGGL((rotary_kernel<IO, MODE, 4>), grid, dim3(kThreads), 0, stream, a, f, it, base);
        else hipLaunchKernelGGL((rotary_kernel<IO, MODE, 1>), grid, dim3(kThreads), 0, stream, a, f, it, base);
    });
    return hipGetLastError();
}

template <typename IO>
hipError_t launch(const RotaryArgs& a, const RotaryFreq& f, hipStream_t stream) {
    constexpr int E = 16 / (int)sizeof(IO);
    const int turn = a.rot / 2 * a.N, pass = (a.d - a.rot) * a.N;  // pairs, and numbers that pass
    Items it{};
    it.dist = a.layout == 0 ? turn : a.N;
    bool vec = vec_ok(a.q, sizeof(IO)) && vec_ok(a.q_out, sizeof(IO)) && pass % E == 0 && a.rot * a.N % E == 0;
    if (a.k_heads) vec = vec && vec_ok(a.k, sizeof(IO)) && vec_ok(a.k_out, sizeof(IO));
    if (vec && (a.layout == 0 ? turn % E == 0 : a.N % E == 0)) {
        it.turning = turn / E;
        it.passing = pass / E;
        return launch_mode<IO, kApart>(a, f, it, stream);
    }
    if (vec && a.layout == 1 && E % (2 * a.N) == 0) {
        it.turning = 2 * turn / E;
        it.passing = pass / E;
        return launch_mode<IO, kInside>(a, f, it, stream);
    }
    it.turning = turn;
    it.passing = pass;
    return launch_mode<IO, kSingle>(a, f, it, stream);
}

}  // namespace

hipError_t launch_rotary(int io, const RotaryArgs& a, const RotaryFreq& f, hipStream_t stream) {
    return io == kIoF32 ? launch<float>(a, f, stream)
                        : (io == kIoBF16 ? launch<__bf16>(a, f, stream) : launch<_Float16>(a, f, stream));
}

}  // namespace eql
