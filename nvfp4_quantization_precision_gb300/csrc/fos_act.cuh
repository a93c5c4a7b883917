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

#include "fos_block8.cuh"

namespace fos {

enum class Act : int { NONE = 0, RELU = 1, GELU = 2, GELU_TANH = 3, SILU = 4 };

// The epilogue's form of v * s(z), s(z) = 1 / (1 + 2^(-z log2 e)), for z = v (silu)
// and z = 2u (gelu_tanh): the hardware's approximations of 2^x (relative error
// 2^-22) and of the reciprocal (2^-23), at 5 and 7 instructions instead of 18 and 20
// with expf and a refined reciprocal: 32 columns of gelu_tanh took 1800 cycles of the
// product's epilogue that way.  The rounding of the argument adds a relative error
// that grows in the negative tail, and there is one of the result:
//   silu       (9 + |z|) 2^-24, up to 2^-17 at z = -87, where a result is below 2^-118
//              and the next ones are 0.  Beneath a 16-bit output's own rounding (2^-11,
//              2^-8); for 32-bit outputs silu_values takes a closer form.
//   gelu_tanh  (9 + 3.5 |z|) 2^-24, for every output: v = -10 gives |z| = 87 and the
//              range's end.  (1 + tanh(u), the formula as it stands, has no correct
//              digit below v = -6.)
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
constexpr float kNegLog2eLo = -1.9259630e-8f;  // what kNegLog2e rounds off
constexpr float kLn2 = 0.69314718f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float k2Sqrt2OverPi = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// 1 - Phi(|x|) = q(t) exp(-x^2 / 2) with t = 1 / (1 + 0.28 |x|) and q a polynomial
// without constant term, fitted by a Lawson iteration of weighted least squares.
// Written on |x|, it has no cancellation on the negative side, where gelu is |x| times
// it.  Two of them:
//   degree 6, nearest in absolute distance over x = 0 .. 9: 3e-8 (4e-8 evaluated in
//     fp32); of the tail itself 5e-6 at 3, 1e-4 at 6, 1e-3 at 9, 4e-3 at 14.  For 16-bit
//     data, whose rounding (2^-11 down to 1e-8, that is x = 6; 2^-8) lies above.
//   degree 9, nearest in relative distance over x = 0 .. 14.4, where the product
//     leaves fp32's range: 6e-8, evaluated in fp32 4e-7; with the rounded argument
//     of the exponential the tail is within (15 + 1.25 x^2) 2^-24 of itself.  For
//     32-bit data; with 16-bit ones it would take an 8192 x 14336 gradient from 139
//     to 145 us and a product of that size with gelu from 351 to 361.
constexpr float kTailT = 0.28f;
template <bool kFine>
__host__ __device__ constexpr int tail_degree() { return kFine ? 9 : 6; }
// Coefficient of t^(i + 1).
template <bool kFine>
__host__ __device__ constexpr float tail_coef(int i) {
    if constexpr (kFine) {
        constexpr float c[9] = {0.11168936f, 0.11195968f, 0.10117771f, 0.09112499f, 0.055468258f,
                                0.017690117f, 0.07250024f, -0.08466628f, 0.023055973f};
        return c[i];
    } else {
        constexpr float c[6] = {0.116520897f, 0.0674960166f, 0.268912017f,
                                -0.236995801f, 0.389875442f, -0.105808601f};
        return c[i];
    }
}
template <bool kFine>
__device__ __forceinline__ float tail_poly(float t) {
    constexpr int kD = tail_degree<kFine>();
    float q = tail_coef<kFine>(kD - 1);
#pragma unroll
    for (int i = kD - 2; i >= 0; --i) q = __fmaf_rn(t, q, tail_coef<kFine>(i));
    return fmul(t, q);
}
template <bool kFine>
__device__ __forceinline__ uint64_t tail_poly2(uint64_t t) {
    constexpr int kD = tail_degree<kFine>();
    uint64_t q = pk(tail_coef<kFine>(kD - 1), tail_coef<kFine>(kD - 1));
#pragma unroll
    for (int i = kD - 2; i >= 0; --i)
        q = fma2(t, q, pk(tail_coef<kFine>(i), tail_coef<kFine>(i)));
    return mul2(t, q);
}

// silu for 32-bit outputs, kN elements in place: the argument's rounding put back to
// first order, 2^(t + lo) = 2^t (1 + lo ln 2), within 10 * 2^-24 of the result.  For
// |v| > 80, where 1 + exp(-v) is 1 or exp(-v) in fp32: v exp(v), by halves because
// exp(v) leaves fp32's range before the product does (at -87 and -92).
template <int kN>
__device__ __forceinline__ void silu_values(float (&v)[kN]) {
    float y[kN], most = 0.0f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const float x = v[i], t = fmul(x, kNegLog2e);
        const float lo = __fmaf_rn(x, kNegLog2eLo, __fmaf_rn(x, kNegLog2e, -t));
        y[i] = fmul(x, rcp(__fmaf_rn(ex2(t), __fmaf_rn(lo, kLn2, 1.0f), 1.0f)));
        most = fmaxf(most, fabsf(x));
    }
    if (most > 80.0f) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const float x = v[i], h = expf(0.5f * x);
            if (x > 80.0f) y[i] = x;
            if (x < -80.0f) y[i] = fmul(fmul(x, h), h);
        }
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = y[i];
}

// Values of kN elements in place, step by step over groups of eight so that
// eight independent chains are in flight.  kFine: for 32-bit outputs.
template <Act A, bool kFine, int kN>
__device__ __forceinline__ void act_values(float (&v)[kN]) {
    constexpr int kG = kN < 8 ? kN : 8;
#pragma unroll
    for (int g = 0; g < kN; g += kG) {
        float t[kG];
#pragma unroll
        for (int i = 0; i < kG; ++i) {
            const float x = v[g + i];
            if constexpr (A == Act::RELU) t[i] = x < 0.0f ? 0.0f : x;
            if constexpr (A == Act::GELU) t[i] = rcp(__fmaf_rn(fabsf(x), kTailT, 1.0f));
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
            for (int i = 0; i < kG; ++i) t[i] = fmul(tail_poly<kFine>(t[i]), e[i]);
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

__device__ __forceinline__ uint64_t pk1(float a) { return pk(a, a); }
__device__ __forceinline__ uint64_t ex2_2(uint64_t x) {
    float a, b;
    upk(x, a, b);
    return pk(ex2(a), ex2(b));
}
__device__ __forceinline__ uint64_t rcp_2(uint64_t x) {
    float a, b;
    upk(x, a, b);
    return pk(rcp(a), rcp(b));
}

// Derivatives of two elements, on packed pairs:
//   silu       s (1 + p (1 - s))
//   gelu_tanh  s + p u2' s (1 - s),  s = s(u2), u2 = 2 sqrt(2/pi) (p + 0.044715 p^3)
//   gelu       Phi(p) + p phi(p)
// For every finite p, up to the type's largest; infinities end in inf * 0 = NaN, as
// these forms do (relu: 1 and 0).  kFine: for 32-bit data.
template <Act A, bool kFine>
__device__ __forceinline__ uint64_t act_slope2(uint64_t p) {
    if constexpr (A == Act::RELU) {
        float a, b;
        upk(p, a, b);
        return pk(a > 0.0f ? 1.0f : 0.0f, b > 0.0f ? 1.0f : 0.0f);
    }
    if constexpr (A == Act::SILU) {
        const uint64_t s = rcp_2(add2(ex2_2(mul2(p, pk1(kNegLog2e))), pk1(1.0f)));
        return mul2(s, fma2(p, sub2(pk1(1.0f), s), pk1(1.0f)));
    }
    if constexpr (A == Act::GELU_TANH) {
        // p^2 no larger than 512, past which s is 0 or 1: p s (1 - s) u2' then has no
        // factor that overflows, and the one that vanishes comes first
        const uint64_t pp = mul2(p, p);
        float a, b;
        upk(pp, a, b);
        const uint64_t p2 = pk(fminf(a, 512.0f), fminf(b, 512.0f));
        const uint64_t z = mul2(p, fma2(p2, pk1(kNegLog2e * k2Sqrt2OverPi * 0.044715f),
                                        pk1(kNegLog2e * k2Sqrt2OverPi)));
        const uint64_t s = rcp_2(add2(ex2_2(z), pk1(1.0f)));
        const uint64_t du = fma2(p2, pk1(k2Sqrt2OverPi * 0.134145f), pk1(k2Sqrt2OverPi));
        return fma2(mul2(p, mul2(s, sub2(pk1(1.0f), s))), du, s);
    }
    if constexpr (A == Act::GELU) {
        float a, b;
        upk(p, a, b);
        const uint64_t t = rcp_2(fma2(pk(fabsf(a), fabsf(b)), pk1(kTailT), pk1(1.0f)));
        const uint64_t e = ex2_2(mul2(mul2(p, p), pk1(0.5f * kNegLog2e)));
        // Phi(-|p|) as it is for negative p, where the slope is small: by way of
        // Phi - 1/2 an 8192 x 14336 gradient takes 135 instead of 139 us, but as many
        // of its codes as a plain form's differ from the exact ones, not 60 % of them
        const uint64_t tail = mul2(tail_poly2<kFine>(t), e);
        float ta, tb, ua, ub;
        upk(tail, ta, tb);
        upk(sub2(pk1(1.0f), tail), ua, ub);
        const uint64_t cdf = pk(a < 0.0f ? ta : ua, b < 0.0f ? tb : ub);
        return fma2(mul2(p, pk1(kInvSqrt2Pi)), e, cdf);
    }
    return pk1(1.0f);
}

}  // namespace fos
