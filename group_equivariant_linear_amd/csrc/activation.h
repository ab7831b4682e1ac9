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

// d act / dv.  GELU: Phi(v) + v phi(v), Phi(-a) = phi(a) t (b1 + t (b2 + ...)), t = 1 / (1 + 0.2316419 a), for
// a = |v| (Abramowitz and Stegun 26.2.17, absolute error below 7.5e-8): one exponential serves phi and Phi.
template <int ACT>
__device__ __forceinline__ float act_slope(float v) {
    if constexpr (ACT == kActSilu) {
        const float p = sigmoid(v);
        return p * fmaf(v, 1.0f - p, 1.0f);
    } else if constexpr (ACT == kActGelu) {
        const float a = fabsf(v);
        const float t = __builtin_amdgcn_rcpf(fmaf(a, 0.2316419f, 1.0f));
        const float pdf = 0.3989422804014327f * __builtin_amdgcn_exp2f(-a * (a * (float)(0.5 * GeluCoef::kLog2e)));
        float p = 1.330274429f;
        p = fmaf(p, t, -1.821255978f);
        p = fmaf(p, t, 1.781477937f);
        p = fmaf(p, t, -0.356563782f);
        p = fmaf(p, t, 0.319381530f);
        const float tail = p * t;  // Phi(-a) / phi(a)
        return v < 0.0f ? pdf * (tail + v) : fmaf(pdf, v - tail, 1.0f);
    } else {
        return 1.0f;
    }
}

}  // namespace eql
