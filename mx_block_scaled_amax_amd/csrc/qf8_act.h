// qf8_act.h -- the activations of a gated layer: act(a) = a s, with
//   SiLU  s = sigmoid(a);   GELU (tanh form)  s = (1 + tanh(z / 2)) / 2 = sigmoid(z), z = 2 sqrt(2 / pi) (a + 0.044715 a^3)
//   act'(a) = s + a s (1 - s) z', z' the slope of the sigmoid's argument (SiLU: 1)
// The sigmoid takes the hardware's exp2 and reciprocal (an ulp each). Where the result is rounded to BF16 or FP8, exp2's
// argument is one product: its rounding costs |z| 2^-24 of e^-z, below 2^-17 down to where the sigmoid falls below 2^-126 and
// is 0 (|act| below 2^-119); 2^-9 and 2^-4 are the roundings after it. EXACT (FP32 results): z and exp2's argument go in two
// parts, and 1 - s is e^-z s, so s and 1 - s are within 2^-21 of themselves. us of FP32 to FP32, 8192 x 2048, z in one
// part / this: GELU 34.1 / 35.4, its gradients 62.1 / 64.8.
#pragma once
#include "qf8_device.h"
#include "../../include/qf8.h"

namespace qf8 {

struct Sigmoid {
    float s, rest;               // sigmoid(z), and 1 - that
};
// of z + more; more (EXACT): what z's own rounding left.
template <bool EXACT>
__device__ __forceinline__ Sigmoid sigmoid(float z, float more = 0.0f) {
    constexpr float kLog2E = 1.44269504088896341f, kRest = (float)(1.4426950408889634074 - (double)kLog2E);
    // 0 or 1 beyond, and no Inf - Inf below; NaN stays
    if constexpr (EXACT) z = z != z ? z : __builtin_amdgcn_fmed3f(z, -200.0f, 200.0f);
    const float t = z * -kLog2E;
    float e = __builtin_amdgcn_exp2f(t);
    if constexpr (EXACT)                              // 2^rest = 1 + rest ln 2, the rest below 2^-14
        e *= __builtin_fmaf(__builtin_fmaf(more, -kLog2E, __builtin_fmaf(z, -kRest, __builtin_fmaf(z, -kLog2E, -t))), 0.693147180559945f, 1.0f);
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    if constexpr (EXACT) return {s, s == 0.0f ? 1.0f : e * s};
    else return {s, 1.0f - s};
}

constexpr double kTwoRootTwoOverPi64 = 1.59576912160573071176, kCube64 = 0.044715;
constexpr float kTwoRootTwoOverPi = (float)kTwoRootTwoOverPi64, kCube = (float)kCube64;

// GELU's sigmoid: z = k (a + m a^3) = (k a) (1 + m a^2), EXACT with what each step's rounding, and the constants', left.
template <bool EXACT>
__device__ __forceinline__ Sigmoid gelu_sigmoid(float a) {
#pragma clang fp contract(off)       // v is the rounded sum of the rounded u
    if constexpr (!EXACT) return sigmoid<false>(kTwoRootTwoOverPi * __builtin_fmaf(kCube * a * a, a, a));
    constexpr float kRest = (float)(kTwoRootTwoOverPi64 - (double)kTwoRootTwoOverPi), kCubeRest = (float)(kCube64 - (double)kCube);
    a = a != a ? a : __builtin_amdgcn_fmed3f(a, -64.0f, 64.0f);      // 0 or 1 beyond
    const float q = a * a, q2 = __builtin_fmaf(a, a, -q);
    const float u = kCube * q, u2 = __builtin_fmaf(kCube, q, -u) + __builtin_fmaf(kCube, q2, kCubeRest * q);
    const float v = 1.0f + u, one = v - u, v2 = u2 + ((1.0f - one) + (u - (v - one)));
    const float w = kTwoRootTwoOverPi * a, w2 = __builtin_fmaf(kTwoRootTwoOverPi, a, -w) + kRest * a;
    const float z = w * v;
    return sigmoid<true>(z, __builtin_fmaf(w, v, -z) + __builtin_fmaf(w, v2, w2 * v));
}

template <int ACT, bool EXACT>
__device__ __forceinline__ float act(float a) {
    if constexpr (ACT == QF8_ACT_SILU) return a * sigmoid<EXACT>(a).s;
    else return a * gelu_sigmoid<EXACT>(a).s;
}
// act(a), and its slope in *d
template <int ACT, bool EXACT>
__device__ __forceinline__ float act_slope(float a, float *d) {
    if constexpr (ACT == QF8_ACT_SILU) {
        const Sigmoid g = sigmoid<EXACT>(a);
        const float y = a * g.s;
        *d = __builtin_fmaf(y, g.rest, g.s);
        return y;
    } else {
        const Sigmoid g = gelu_sigmoid<EXACT>(a);
        const float c = __builtin_amdgcn_fmed3f(a, -64.0f, 64.0f);     // beyond, s (1 - s) is 0 and a^2 may not be finite
        *d = __builtin_fmaf(c * g.s * g.rest, kTwoRootTwoOverPi * __builtin_fmaf(3.0f * kCube * c, c, 1.0f), g.s);
        return a * g.s;
    }
}

}  // namespace qf8
