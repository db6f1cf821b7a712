// qf8_act.h -- the activations of a gated layer: act(a) = a s, with
//   SiLU  s = sigmoid(a);   GELU (tanh form)  s = (1 + tanh(z / 2)) / 2 = sigmoid(z), z = 2 sqrt(2 / pi) (a + 0.044715 a^3)
//   act'(a) = s + a s (1 - s) z', z' the slope of the sigmoid's argument (SiLU: 1)
// The sigmoid takes the hardware's exp2 and reciprocal (an ulp each). Where the result is rounded to BF16 or FP8, exp2's
// argument is one product: its rounding costs |z| 2^-24 of e^-z, below 2^-17 down to where the sigmoid falls below 2^-126 and
// is 0 (|act| below 2^-119); 2^-9 and 2^-4 are the roundings after it. EXACT (FP32 results): the product's rounding error is
// carried along.
#pragma once
#include "qf8_device.h"
#include "../../include/qf8.h"

namespace qf8 {

template <bool EXACT>
__device__ __forceinline__ float sigmoid(float z) {
    constexpr float kLog2E = 1.44269504088896341f, kRest = (float)(1.4426950408889634074 - (double)kLog2E);
    // 0 or 1 beyond, and no Inf - Inf below; NaN stays
    if constexpr (EXACT) z = z != z ? z : __builtin_amdgcn_fmed3f(z, -200.0f, 200.0f);
    const float t = z * -kLog2E;
    float e = __builtin_amdgcn_exp2f(t);
    if constexpr (EXACT)                              // 2^rest = 1 + rest ln 2, the rest below 2^-17
        e *= __builtin_fmaf(__builtin_fmaf(z, -kRest, __builtin_fmaf(z, -kLog2E, -t)), 0.693147180559945f, 1.0f);
    return __builtin_amdgcn_rcpf(1.0f + e);
}

constexpr float kTwoRootTwoOverPi = 1.59576912160573071f, kCube = 0.044715f;

template <int ACT, bool EXACT>
__device__ __forceinline__ float act(float a) {
    if constexpr (ACT == QF8_ACT_SILU) return a * sigmoid<EXACT>(a);
    else return a * sigmoid<EXACT>(kTwoRootTwoOverPi * __builtin_fmaf(kCube * a * a, a, a));
}
// act(a), and its slope in *d
template <int ACT, bool EXACT>
__device__ __forceinline__ float act_slope(float a, float *d) {
    if constexpr (ACT == QF8_ACT_SILU) {
        const float s = sigmoid<EXACT>(a), y = a * s;
        *d = __builtin_fmaf(y, 1.0f - s, s);
        return y;
    } else {
        const float s = sigmoid<EXACT>(kTwoRootTwoOverPi * __builtin_fmaf(kCube * a * a, a, a)), y = a * s;
        const float c = __builtin_amdgcn_fmed3f(a, -64.0f, 64.0f);     // beyond, s (1 - s) is 0 and a^2 may not be finite
        *d = __builtin_fmaf(c * s * (1.0f - s), kTwoRootTwoOverPi * __builtin_fmaf(3.0f * kCube * c, c, 1.0f), s);
        return y;
    }
}

}  // namespace qf8
