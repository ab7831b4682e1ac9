// activation.h -- the activations of the operators between the layers, with their
// derivatives, in fp32.
#pragma once

#include "cn_fused.h"  // gelu_erf, GeluCoef

namespace eql {

constexpr int kActNone = 0, kActGelu = 1, kActSilu = 2;

__device__ __forceinline__ float sigmoid(float v) {
    // exp2 overflows to infinity below v = -88, where the reciprocal gives the limit 0
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * (float)-GeluCoef::kLog2e));
}

template <int ACT>
__device__ __forceinline__ float act_value(float v) {
    if constexpr (ACT == kActGelu) return gelu_erf(v);
    else if constexpr (ACT == kActSilu) return v * sigmoid(v);
    else return v;
}

// d act / dv.  GELU: Phi(v) + v phi(v), Phi by the same fitted erfc as the value.
template <int ACT>
__device__ __forceinline__ float act_slope(float v) {
    if constexpr (ACT == kActSilu) {
        const float p = sigmoid(v);
        return p * fmaf(v, 1.0f - p, 1.0f);
    } else if constexpr (ACT == kActGelu) {
        const float a = fabsf(v);
        const float t = __builtin_amdgcn_rcpf(fmaf(a, 0.35355339059327376f, 1.0f));
        float p = GeluCoef::scaled(0);
#pragma unroll
        for (int i = 1; i < 10; ++i) p = fmaf(p, t, GeluCoef::scaled(i));
        const float q = -a * (a * (float)(0.5 * GeluCoef::kLog2e));  // -v^2/2 in powers of two
        const float h = t * __builtin_amdgcn_exp2f(q + p);           // Phi(-|v|)
        const float pdf = 0.3989422804014327f * __builtin_amdgcn_exp2f(q);
        return fmaf(v, pdf, v < 0.0f ? h : 1.0f - h);
    } else {
        return 1.0f;
    }
}

}  // namespace eql
