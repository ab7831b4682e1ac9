// rotary.hip -- rotary positions on regular-representation heads.
//
// Pair (a, b) of channels of every head, for each of the N group elements:
//   a' = m (a cos w - b sin w), b' = m (b cos w + a sin w), w = 2 pi p turns[j].
// The angle's fraction of a turn is taken in fp64, once per (token, pair), and
// shared by every head and group element.
#include "eq_device.h"
#include "eq_launch.h"

namespace eql {
namespace {

// p turns less its nearest integer, without the rounding of the product (2^-22 turns
// at the largest positions).
__device__ __forceinline__ float fraction_of_turn(int p, double turns) {
    return (float)fma((double)p, turns, -rint((double)p * turns));
}

// One workgroup per token; cos and sin of the token's pairs in LDS.
template <typename IO>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a, RotaryFreq f) {
    __shared__ float2 cs[kMaxRotaryPairs];
    const int64_t t = blockIdx.x;
    const int half = a.rot / 2;
    for (int j = (int)threadIdx.x; j < half; j += 256) {
        const float r = 2.0f * fraction_of_turn(a.positions[t], f.turns[j]);
        const float s = sinpif(r);
        cs[j] = float2{f.magnitude * cospif(r), f.magnitude * (a.inverse ? -s : s)};
    }
    __syncthreads();
    const int D = a.d * a.N, heads = a.q_heads + a.k_heads;
    for (int e = (int)threadIdx.x; e < heads * D; e += 256) {
        const int h = e / D, r = e % D, c = r / a.N, n = r % a.N;
        const bool is_q = h < a.q_heads;
        const Heads& in = is_q ? a.q : a.k;
        const Heads& to = is_q ? a.q_out : a.k_out;
        const int hh = is_q ? h : h - a.q_heads;
        const IO* x = (const IO*)in.p + t * in.ts + hh * in.hs;
        IO* y = (IO*)const_cast<void*>(to.p) + t * to.ts + hh * to.hs;
        if (c >= a.rot) {
            y[r] = x[r];
            continue;
        }
        const bool first = a.layout == 0 ? c < half : c % 2 == 0;
        if (!first) continue;  // its pair's first channel writes both
        const int j = a.layout == 0 ? c : c / 2;
        const int r2 = (a.layout == 0 ? c + half : c + 1) * a.N + n;
        const float xa = (float)x[r], xb = (float)x[r2];
        y[r] = (IO)(xa * cs[j].x - xb * cs[j].y);
        y[r2] = (IO)(xb * cs[j].x + xa * cs[j].y);
    }
}

}  // namespace

hipError_t launch_rotary(int io, const RotaryArgs& a, const RotaryFreq& f, hipStream_t stream) {
    if (a.T > 0x7fffffff) return hipErrorNotSupported;
    const dim3 grid((uint32_t)a.T);
    if (io == kIoF32) hipLaunchKernelGGL(rotary_kernel<float>, grid, dim3(256), 0, stream, a, f);
    else if (io == kIoBF16) hipLaunchKernelGGL(rotary_kernel<__bf16>, grid, dim3(256), 0, stream, a, f);
    else hipLaunchKernelGGL(rotary_kernel<_Float16>, grid, dim3(256), 0, stream, a, f);
    return hipGetLastError();
}

}  // namespace eql
