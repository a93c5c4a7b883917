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

// The epilogue's form of v * s(z), s(z) = 1 / (1 + 2^(-z log2 e)), for z = v (silu)
// and z = 2u (gelu_tanh): the hardware's approximations of 2^x (2 ulp, and the
// argument's rounding, a relative |z| 2^-24) and of the reciprocal (1 ulp).
// That is a relative error of a few 2^-24 where s is not negligible, below
// every stored type's rounding but fp32's, at 5 and 7 instructions instead of
// 18 and 20 with expf and a refined reciprocal: 32 columns of gelu_tanh took
// 1800 cycles of the product's epilogue that way.  A zero or infinite sum ends
// in the right limit (2^x = inf gives s = 0).
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kNegLog2e = -1.4426950408889634f;
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float k2Sqrt2OverPi = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// 1 - Phi(|x|) = q(t) exp(-x^2 / 2), t = 1 / (1 + p |x| / sqrt 2): Abramowitz and
// Stegun, Handbook of Mathematical Functions, 7.1.26 (erf within 1.5e-7), with
// q half their polynomial.  Written on |x|, it has no cancellation on the
// negative side.
constexpr float kErfP = 0.3275911f;
__device__ __forceinline__ float half_erf_poly(float t) {
    float q = __fmaf_rn(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f);
    q = __fmaf_rn(t, q, 0.5f * 1.421413741f);
    q = __fmaf_rn(t, q, 0.5f * -0.284496736f);
    q = __fmaf_rn(t, q, 0.5f * 0.254829592f);
    return fmul(t, q);
}

// Values of kN elements in place, step by step over groups of eight so that
// eight independent chains are in flight.
template <Act A, int kN>
__device__ __forceinline__ void act_values(float (&v)[kN]) {
    constexpr int kG = kN < 8 ? kN : 8;
#pragma unroll
    for (int g = 0; g < kN; g += kG) {
        float t[kG];
#pragma unroll
        for (int i = 0; i < kG; ++i) {
            const float x = v[g + i];
            if constexpr (A == Act::RELU) t[i] = x < 0.0f ? 0.0f : x;
            if constexpr (A == Act::GELU) t[i] = rcp(__fmaf_rn(fabsf(x), kErfP * kSqrtHalf, 1.0f));
            if constexpr (A == Act::GELU_TANH)
                t[i] = fmul(x, __fmaf_rn(kNegLog2e * k2Sqrt2OverPi * 0.044715f, fmul(x, x),
                                         kNegLog2e * k2Sqrt2OverPi));
            if constexpr (A == Act::SILU) t[i] = fmul(x, kNegLog2e);
        }
        if constexpr (A == Act::GELU_TANH || A == Act::SILU) {
#pragma unroll
            for (int i = 0; i < kG; ++i) t[i] = ex2(t[i]);
#pragma unroll
            for (int i = 0; i < kG; ++i) t[i] = rcp(fadd(1.0f, t[i]));
        }
        if constexpr (A == Act::GELU) {
            float e[kG];
#pragma unroll
            for (int i = 0; i < kG; ++i)
                e[i] = ex2(fmul(fmul(v[g + i], v[g + i]), 0.5f * kNegLog2e));
#pragma unroll
            for (int i = 0; i < kG; ++i) t[i] = fmul(half_erf_poly(t[i]), e[i]);
        }
#pragma unroll
        for (int i = 0; i < kG; ++i) {
            if constexpr (A == Act::RELU) v[g + i] = t[i];
            if constexpr (A == Act::GELU) {
                const float x = v[g + i];  // max(x, 0) - |x| (1 - Phi(|x|))
                v[g + i] = x > kFltMax ? x : __fmaf_rn(-fabsf(x), t[i], fmaxf(x, 0.0f));
            }
            if constexpr (A == Act::GELU_TANH || A == Act::SILU) v[g + i] = fmul(v[g + i], t[i]);
        }
    }
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
