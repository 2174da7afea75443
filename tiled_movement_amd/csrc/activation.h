// Activations of the gated products, in fp32.
//   SiLU        z s(z),                       s(z) = 1 / (1 + e^-z)
//   GELU        z Phi(z),                     Phi(z) = erfc(-z / sqrt 2) / 2
//   GELU, tanh  z (1 + tanh(q(z))) / 2 = z s(2 q(z)),  q(z) = sqrt(2 / pi) (z + 0.044715 z^3)
// Phi by erfc keeps its digits for z far below zero (relative error z^2 2^-23), where
// 1 + erf(z / sqrt 2) would lose them: 2.7e-4 of the result at -4, all of it from -5.5 on.
// Derivatives take z cut to where they have reached their limits, so that an
// infinite or huge z meets no infinity times zero; NaN stays NaN.
#pragma once

#include <hip/hip_runtime.h>

#include "swz.h"

namespace swz {
namespace act {

__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}
__device__ __forceinline__ float cut(float z, float to) { return z > to ? to : z < -to ? -to : z; }

constexpr float kTwoRoot2OverPi = 1.5957691216057308f, kCube = 0.044715f;

// act(z) and, if DERIV, its derivative.
template <int ACT, bool DERIV>
__device__ __forceinline__ float2 both(float z) {
    if constexpr (ACT == SWZ_ACT_GELU) {
        const float cdf = 0.5f * erfcf(z * -0.7071067811865476f);
        if constexpr (!DERIV) return make_float2(z * cdf, 0.f);
        const float t = cut(z, 20.f);
        const float pdf = 0.3989422804014327f * __builtin_amdgcn_exp2f(-0.7213475204444817f * t * t);
        return make_float2(z * cdf, __builtin_fmaf(t, pdf, cdf));
    } else if constexpr (ACT == SWZ_ACT_GELU_TANH) {
        const float t = cut(z, 20.f), t2 = t * t;  // 2 q(20) = 600: s is 0 or 1
        const float s = sigmoid(kTwoRoot2OverPi * t * __builtin_fmaf(kCube, t2, 1.f));
        if constexpr (!DERIV) return make_float2(z * s, 0.f);
        const float dq = kTwoRoot2OverPi * __builtin_fmaf(3.f * kCube, t2, 1.f);
        return make_float2(z * s, __builtin_fmaf(t * s * (1.f - s), dq, s));
    } else {
        const float s = sigmoid(z);
        if constexpr (!DERIV) return make_float2(z * s, 0.f);
        const float t = cut(z, 200.f);
        return make_float2(z * s, s * __builtin_fmaf(t, 1.f - s, 1.f));
    }
}

}  // namespace act
}  // namespace swz
