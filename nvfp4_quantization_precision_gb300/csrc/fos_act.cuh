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
//   silu       (9 + 1.3 |z|) 2^-24, up to 2^-17 at z = -87, where a result is below 2^-118
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

// 1 - Phi(|x|) = q(s) exp(-x^2 / 2) with s = |x| / (1 + c |x|) and q a polynomial whose
// constant term is 1/2, fitted by a Lawson iteration of weighted least squares.  Written
// on |x|, it has no cancellation on the negative side, where gelu is |x| times it;
// in s, which is 0 with x, the reciprocal's rounding vanishes where q is large (a
// polynomial in 1 / (1 + c |x|) is off by 4e-8 root mean square over 0 .. 1, this by 1.2e-8).
// Two of them, their errors evaluated in fp32:
//   degree 6, c = 0.38, fitted within 8e-9 in all and of the tail itself, as it is
//     evaluated, 1.3e-6 to 3, 6e-5 to 6, 3e-4 to 9, 3e-3 to 14.  For 16-bit data,
//     whose rounding (2^-11 down to 1e-8, that is x = 6; 2^-8) lies above.
//   degree 9, c = 0.45, for 32-bit data: 1.8e-6 of the tail itself to 14.4, where the
//     product leaves fp32's range.
// Either way the exponential adds its own error, 4 * 2^-24, and its argument's, 1.25 x^2
// 2^-24.
template <bool kFine>
__host__ __device__ constexpr int tail_degree() { return kFine ? 9 : 6; }
template <bool kFine>
__host__ __device__ constexpr float tail_c() { return kFine ? 0.45f : 0.38f; }
// Coefficient of s^(i + 1).
template <bool kFine>
__host__ __device__ constexpr float tail_coef(int i) {
    if constexpr (kFine) {
        constexpr float c[9] = {-0.3989421f, 0.07047819f, 0.011195586f, -0.0013211702f, -0.0013286442f,
                                0.00042060253f, -0.00041844323f, 0.0002011633f, -0.000029093711f};
        return c[i];
    } else {
        constexpr float c[6] = {-0.3989426f, 0.0984082f, -0.0006266588f,
                                -0.002581888f, -0.00040525946f, 0.00016812574f};
        return c[i];
    }
}
template <bool kFine>
__device__ __forceinline__ float tail_poly(float s) {
    constexpr int kD = tail_degree<kFine>();
    float q = tail_coef<kFine>(kD - 1);
#pragma unroll
    for (int i = kD - 2; i >= 0; --i) q = __fmaf_rn(s, q, tail_coef<kFine>(i));
    return __fmaf_rn(s, q, 0.5f);
}
template <bool kFine>
__device__ __forceinline__ uint64_t tail_poly2(uint64_t s) {
    constexpr int kD = tail_degree<kFine>();
    uint64_t q = pk(tail_coef<kFine>(kD - 1), tail_coef<kFine>(kD - 1));
#pragma unroll
    for (int i = kD - 2; i >= 0; --i)
        q = fma2(s, q, pk(tail_coef<kFine>(i), tail_coef<kFine>(i)));
    return fma2(s, q, pk(0.5f, 0.5f));
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
            if constexpr (A == Act::GELU)
                t[i] = fmul(fabsf(x), rcp(__fmaf_rn(fabsf(x), tail_c<kFine>(), 1.0f)));
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
//   gelu       Phi(p) + p phi(p), Phi(-p) = q exp(-p^2 / 2)
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
        // (1 - s as E s, like below, halves the error from p = 3 on, but the roundings of s no
        // longer cancel below: of 123 M codes of fp16 gradients 194 instead of 153 differ
        // from the exact ones, and 8192 x 14336 takes 123.7 instead of 121.8 us)
        const uint64_t s = rcp_2(add2(ex2_2(mul2(p, pk1(kNegLog2e))), pk1(1.0f)));
        return mul2(s, fma2(p, sub2(pk1(1.0f), s), pk1(1.0f)));
    }
    if constexpr (A == Act::GELU_TANH) {
        // 1 - s as E s, E = exp(-u2), without the cancellation (which for p = 2 .. 6 leaves
        // an error of 3.6e-7 instead of 6e-8).  For u2 and its derivative p is held within
        // 16, where E is 0, and -10.05, where E is finite and its reciprocal 0: no
        // factor overflows, and the one that vanishes meets p first.
        float a, b;
        upk(p, a, b);
        const uint64_t x = pk(fmaxf(fminf(a, 16.0f), -10.05f), fmaxf(fminf(b, 16.0f), -10.05f));
        const uint64_t x2 = mul2(x, x);
        const uint64_t e = ex2_2(mul2(x, fma2(x2, pk1(kNegLog2e * k2Sqrt2OverPi * 0.044715f),
                                              pk1(kNegLog2e * k2Sqrt2OverPi))));
        const uint64_t s = rcp_2(add2(e, pk1(1.0f)));
        const uint64_t du = fma2(x2, pk1(k2Sqrt2OverPi * 0.134145f), pk1(k2Sqrt2OverPi));
        return fma2(mul2(p, mul2(mul2(e, s), s)), du, s);
    }
    if constexpr (A == Act::GELU) {
        // the negative side's slope exp(-p^2 / 2) (q - |p| / sqrt(2 pi)), the positive
        // side's 1 minus that
        float a, b;
        upk(p, a, b);
        const uint64_t x = pk(fabsf(a), fabsf(b));
        const uint64_t t = mul2(x, rcp_2(fma2(x, pk1(tail_c<kFine>()), pk1(1.0f))));
        const uint64_t e = ex2_2(mul2(mul2(p, p), pk1(0.5f * kNegLog2e)));
        const uint64_t neg = mul2(fma2(x, pk1(-kInvSqrt2Pi), tail_poly2<kFine>(t)), e);
        float na, nb, ua, ub;
        upk(neg, na, nb);
        upk(sub2(pk1(1.0f), neg), ua, ub);
        return pk(a < 0.0f ? na : ua, b < 0.0f ? nb : ub);
    }
    return pk1(1.0f);
}

}  // namespace fos
