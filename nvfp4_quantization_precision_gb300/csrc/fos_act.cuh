// fos_act.cuh -- the activations of the product's epilogue and their
// derivatives, in fp32.
//
//   relu       max(v, 0)
//   gelu       v * (1 + erf(v / sqrt 2)) / 2
//   gelu_tanh  v * (1 + tanh(u)) / 2 = v * s(2u),  u = sqrt(2/pi) (v + 0.044715 v^3)
//   silu       v * s(v),  s(z) = 1 / (1 + exp(-z))
//
// gelu_tanh is written with s(2u): one exponential and one reciprocal, and no
// cancellation of 1 + tanh(u) on the negative side.
#pragma once

#include "fos_device.cuh"

namespace fos {

enum class Act : int { NONE = 0, RELU = 1, GELU = 2, GELU_TANH = 3, SILU = 4 };

// 1 / (1 + exp(-z)): the reciprocal approximation and one Newton step (the
// step is skipped where the sum has overflowed and the reciprocal is 0).
__device__ __forceinline__ float sigmoid(float z) {
    const float x = fadd(1.0f, expf(-z));
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    const float e = __fmaf_rn(-x, r, 1.0f);
    return x < kFltMax ? __fmaf_rn(e, r, r) : r;
}

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float k2Sqrt2OverPi = 1.5957691216057308f;  // 2 sqrt(2 / pi)

template <Act A>
__device__ __forceinline__ float act_value(float v) {
    if constexpr (A == Act::RELU) return v < 0.0f ? 0.0f : v;
    if constexpr (A == Act::GELU) return fmul(fmul(0.5f, v), fadd(1.0f, erff(fmul(v, kSqrtHalf))));
    if constexpr (A == Act::GELU_TANH) {
        const float u2 = fmul(k2Sqrt2OverPi, __fmaf_rn(fmul(0.044715f, fmul(v, v)), v, v));
        return fmul(v, sigmoid(u2));
    }
    if constexpr (A == Act::SILU) return fmul(v, sigmoid(v));
    return v;
}

template <Act A>
__device__ __forceinline__ float act_slope(float p) {
    if constexpr (A == Act::RELU) return p > 0.0f ? 1.0f : 0.0f;
    if constexpr (A == Act::GELU) {
        const float phi = fmul(kInvSqrt2Pi, expf(fmul(fmul(-0.5f, p), p)));
        return __fmaf_rn(p, phi, fmul(0.5f, fadd(1.0f, erff(fmul(p, kSqrtHalf)))));
    }
    if constexpr (A == Act::GELU_TANH) {
        const float p2 = fmul(p, p);
        const float s = sigmoid(fmul(k2Sqrt2OverPi, __fmaf_rn(fmul(0.044715f, p2), p, p)));
        const float du = fmul(k2Sqrt2OverPi, __fmaf_rn(0.134145f, p2, 1.0f));
        return __fmaf_rn(fmul(p, du), fmul(s, __fsub_rn(1.0f, s)), s);
    }
    if constexpr (A == Act::SILU) {
        const float s = sigmoid(p);
        return fmul(s, __fmaf_rn(p, __fsub_rn(1.0f, s), 1.0f));
    }
    return 1.0f;
}

}  // namespace fos
