// group_norm.hip -- group norm with an activation, channels last, and its gradients.
//
// A slab is one sample's part of one group: its tokens x (C / groups) N numbers,
// contiguous within a token.
#include "activation.h"
#include "eq_device.h"
#include "eq_launch.h"

namespace eql {
namespace {

__device__ __forceinline__ void sample_range(const NormArgs& a, int64_t b, int64_t& t0, int64_t& t1) {
    if (a.offsets) {
        t0 = a.offsets[b], t1 = a.offsets[b + 1];
        t0 = t0 < 0 ? 0 : (t0 > a.T ? a.T : t0);
        t1 = t1 < t0 ? t0 : (t1 > a.T ? a.T : t1);
    } else {
        const int64_t n = a.T / a.batch;
        t0 = b * n, t1 = t0 + n;
    }
}

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return red[0] + red[1] + red[2] + red[3];
}

template <typename IO>
__device__ __forceinline__ float param(const void* p, int c, float none) {
    return p ? (float)((const IO*)p)[c] : none;
}

__device__ __forceinline__ float act_value_of(int act, float v) {
    return act == kActGelu ? act_value<kActGelu>(v) : (act == kActSilu ? act_value<kActSilu>(v) : v);
}
__device__ __forceinline__ float act_slope_of(int act, float v) {
    return act == kActGelu ? act_slope<kActGelu>(v) : (act == kActSilu ? act_slope<kActSilu>(v) : 1.0f);
}

// One workgroup per slab: mean, then squared differences, then the values.
template <typename IO>
__global__ __launch_bounds__(256) void norm_forward_kernel(NormArgs a) {
    __shared__ float red[4];
    const int64_t b = blockIdx.x / a.groups;
    const int g = (int)(blockIdx.x % a.groups), cpg = a.C / a.groups, W = cpg * a.N;
    int64_t t0, t1;
    sample_range(a, b, t0, t1);
    const int64_t n = (t1 - t0) * W;
    const IO* x = (const IO*)a.x + t0 * a.ldx + (int64_t)g * W;
    float s = 0.0f;
    for (int64_t i = threadIdx.x; i < n; i += 256) s += (float)x[i / W * a.ldx + i % W];
    const float inv = n ? 1.0f / (float)n : 0.0f;
    const float mean = block_sum(s, red) * inv;
    float v = 0.0f;
    for (int64_t i = threadIdx.x; i < n; i += 256) {
        const float d = (float)x[i / W * a.ldx + i % W] - mean;
        v = fmaf(d, d, v);
    }
    const float rstd = n ? 1.0f / sqrtf(block_sum(v, red) * inv + a.eps) : 0.0f;
    if (a.stats && threadIdx.x == 0) {
        a.stats[2 * blockIdx.x] = mean;
        a.stats[2 * blockIdx.x + 1] = rstd;
    }
    IO* y = (IO*)a.y + t0 * a.ldy + (int64_t)g * W;
    for (int64_t i = threadIdx.x; i < n; i += 256) {
        const int e = (int)(i % W), c = g * cpg + e / a.N;
        const float xh = ((float)x[i / W * a.ldx + e] - mean) * rstd;
        y[i / W * a.ldy + e] =
            (IO)act_value_of(a.act, fmaf(xh, param<IO>(a.gamma, c, 1.0f), param<IO>(a.beta, c, 0.0f)));
    }
}

// One workgroup per slab: dx.
template <typename IO>
__global__ __launch_bounds__(256) void norm_dx_kernel(NormArgs a) {
    __shared__ float red[4];
    const int64_t b = blockIdx.x / a.groups;
    const int g = (int)(blockIdx.x % a.groups), cpg = a.C / a.groups, W = cpg * a.N;
    int64_t t0, t1;
    sample_range(a, b, t0, t1);
    const int64_t n = (t1 - t0) * W;
    const float mean = a.stats[2 * blockIdx.x], rstd = a.stats[2 * blockIdx.x + 1];
    const IO* x = (const IO*)a.x + t0 * a.ldx + (int64_t)g * W;
    const IO* dy = (const IO*)a.dy + t0 * a.lddy + (int64_t)g * W;
    auto at = [&](int64_t i, float& xh) {
        const int e = (int)(i % W), c = g * cpg + e / a.N;
        xh = ((float)x[i / W * a.ldx + e] - mean) * rstd;
        const float gm = param<IO>(a.gamma, c, 1.0f);
        return (float)dy[i / W * a.lddy + e] * act_slope_of(a.act, fmaf(xh, gm, param<IO>(a.beta, c, 0.0f))) * gm;
    };
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t i = threadIdx.x; i < n; i += 256) {
        float xh;
        const float d = at(i, xh);
        s1 += d;
        s2 = fmaf(d, xh, s2);
    }
    const float inv = n ? 1.0f / (float)n : 0.0f;
    const float m1 = block_sum(s1, red) * inv, m2 = block_sum(s2, red) * inv;
    IO* dx = (IO*)a.dx + t0 * a.lddx + (int64_t)g * W;
    for (int64_t i = threadIdx.x; i < n; i += 256) {
        float xh;
        const float d = at(i, xh);
        dx[i / W * a.lddx + i % W] = (IO)((d - m1 - xh * m2) * rstd);
    }
}

// One workgroup per channel: dgamma, dbeta.
template <typename IO>
__global__ __launch_bounds__(256) void norm_dparam_kernel(NormArgs a) {
    __shared__ float red[4];
    const int c = (int)blockIdx.x, g = c / (a.C / a.groups);
    const float gm = param<IO>(a.gamma, c, 1.0f), be = param<IO>(a.beta, c, 0.0f);
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t b = 0; b < a.batch; ++b) {
        int64_t t0, t1;
        sample_range(a, b, t0, t1);
        const float mean = a.stats[2 * (b * a.groups + g)], rstd = a.stats[2 * (b * a.groups + g) + 1];
        for (int64_t i = threadIdx.x; i < (t1 - t0) * a.N; i += 256) {
            const int64_t t = t0 + i / a.N, e = (int64_t)c * a.N + i % a.N;
            const float xh = ((float)((const IO*)a.x)[t * a.ldx + e] - mean) * rstd;
            const float dz = (float)((const IO*)a.dy)[t * a.lddy + e] * act_slope_of(a.act, fmaf(xh, gm, be));
            s1 += dz;
            s2 = fmaf(dz, xh, s2);
        }
    }
    const float db = block_sum(s1, red), dg = block_sum(s2, red);
    if (threadIdx.x == 0) {
        if (a.dgamma) a.dgamma[c] = dg;
        if (a.dbeta) a.dbeta[c] = db;
    }
}

template <typename IO>
hipError_t forward(const NormArgs& a, hipStream_t stream) {
    if (a.batch * a.groups > 0x7fffffff) return hipErrorNotSupported;
    hipLaunchKernelGGL(norm_forward_kernel<IO>, dim3((uint32_t)(a.batch * a.groups)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <typename IO>
hipError_t backward(const NormArgs& a, hipStream_t stream) {
    if (a.batch * a.groups > 0x7fffffff) return hipErrorNotSupported;
    // dgamma and dbeta first: dx may take dy's place
    if (a.dgamma || a.dbeta)
        hipLaunchKernelGGL(norm_dparam_kernel<IO>, dim3((uint32_t)a.C), dim3(256), 0, stream, a);
    if (a.T > 0)
        hipLaunchKernelGGL(norm_dx_kernel<IO>, dim3((uint32_t)(a.batch * a.groups)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

size_t group_norm_workspace(int, int, int, int, int64_t, int64_t, bool) { return 0; }

hipError_t launch_group_norm(int io, const NormArgs& a, void*, hipStream_t stream) {
    return io == kIoF32 ? forward<float>(a, stream)
                        : (io == kIoBF16 ? forward<__bf16>(a, stream) : forward<_Float16>(a, stream));
}

hipError_t launch_group_norm_backward(int io, const NormArgs& a, void*, hipStream_t stream) {
    return io == kIoF32 ? backward<float>(a, stream)
                        : (io == kIoBF16 ? backward<__bf16>(a, stream) : backward<_Float16>(a, stream));
}

}  // namespace eql
