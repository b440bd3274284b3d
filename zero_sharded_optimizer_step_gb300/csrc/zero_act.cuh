// The activations of linear layers and their slopes, in fp32.
//
// Exponentials and reciprocals are the hardware's, a few units in the last place off
// and 0 instead of subnormal: a value or slope below 2^-118 may come out as 0.
// The exponential's argument is rounded too, so that its relative error grows with it: in
// the negative tails, where values are small, by tens of units.  Measured against 64 bits
// (values, in units of 2^-23 of themselves): above -1 at most 5; GELU 24 down to -6,
// 48 to -9, 94 to -12.9; by tanh 33 to -6, 90 to -9; SiLU 9 to -20, 33 to -87.  Slopes the
// same of their terms, at most 3e-7 in all.
//
// Differences of nearly equal numbers are avoided: p (1 - p) of a logistic p is
// e / (1 + e)^2, and the normal distribution function is made from its small side.
#pragma once

#include <type_traits>

#include <cuda_runtime.h>

namespace zgb {

enum Act : int32_t { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

namespace act {

constexpr float kTwoA = 1.5957691216057308f;          // 2 sqrt(2 / pi)
constexpr float kCube = 0.044715f;

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float power_of_2(float v)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v));
    return e;
}

__device__ __forceinline__ float exp_of(float v) { return power_of_2(__fmul_rn(v, kLog2e)); }

__device__ __forceinline__ float inverse(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// p = 1 / (1 + 2^-u).  Where the power overflows it is 0.
__device__ __forceinline__ float logistic(float u)
{
    return inverse(__fadd_rn(1.0f, power_of_2(-u)));
}

// p and q = p (1 - p).
__device__ __forceinline__ void logistic2(float u, float &p, float &q)
{
    const float e = power_of_2(-fabsf(u)), r = inverse(__fadd_rn(1.0f, e)), s = __fmul_rn(e, r);
    p = u < 0.0f ? s : r;
    q = __fmul_rn(s, r);
}

// The normal distribution function.  With x = |v| / sqrt(2) and t = 1 / (1 + x / 2),
// log(erfc(x) exp(x^2) / t) is smooth over all of 0 < t <= 1 (the form of the complementary
// error function in Numerical Recipes, chapter 6): a polynomial of degree
// 9 in t, with coefficients fitted here for the least largest error (7.4e-8, x up to
// 10.5), stands for it.  The tail is a product and not a difference, and keeps a relative
// precision: that of the exponential of g - v^2 / 2.  (Measured against the CUDA library's
// normcdff: the forward pass of a 6400 x 1600 layer over 8192 tokens 211 -> 102 us.)
__device__ __forceinline__ float normal(float v)
{
    const float t = inverse(__fmaf_rn(0.35355339059327373f, fabsf(v), 1.0f));
    float g = 0.14575070142745972f;
    g = __fmaf_rn(g, t, -0.6855512261390686f);
    g = __fmaf_rn(g, t, 1.1685633659362793f);
    g = __fmaf_rn(g, t, -0.7131166458129883f);
    g = __fmaf_rn(g, t, -0.06524422019720078f);
    g = __fmaf_rn(g, t, -0.007393619976937771f);
    g = __fmaf_rn(g, t, 0.037811607122421265f);
    g = __fmaf_rn(g, t, 0.3859069049358368f);
    g = __fmaf_rn(g, t, 0.9987261295318604f);
    g = __fmaf_rn(g, t, -1.2654529809951782f);
    const float x2 = __fmul_rn(0.5f, __fmul_rn(v, v));
    const float q = __fmul_rn(__fmul_rn(0.5f, t), exp_of(__fsub_rn(g, x2)));
    return v < 0.0f ? q : __fsub_rn(1.0f, q);
}

// (1 + tanh(a (v + c v^3))) / 2 is the logistic of this, for 2 to its power.
__device__ __forceinline__ float tanh_arg(float v, float v2)
{
    return __fmul_rn(v, __fmaf_rn(kTwoA * kLog2e * kCube, v2, kTwoA * kLog2e));
}

__device__ __forceinline__ float value(float v, int32_t kind)
{
    switch (kind) {
    case kActRelu: return v < 0.0f ? 0.0f : v;
    case kActGelu: return __fmul_rn(v, normal(v));
    case kActGeluTanh: return __fmul_rn(v, logistic(tanh_arg(v, __fmul_rn(v, v))));
    case kActSilu: return __fmul_rn(v, logistic(__fmul_rn(v, kLog2e)));
    default: return v;
    }
}

// The activation and its slope.
__device__ __forceinline__ void both(float v, int32_t kind, float &y, float &slope)
{
    float p, q;
    switch (kind) {
    case kActRelu:
        y = v < 0.0f ? 0.0f : v;
        slope = v <= 0.0f ? 0.0f : 1.0f;
        return;
    case kActGelu: {
        p = normal(v);
        q = __fmul_rn(0.3989422804014327f, exp_of(__fmul_rn(-0.5f, __fmul_rn(v, v))));
        y = __fmul_rn(v, p);
        slope = __fmaf_rn(v, q, p);
        return;
    }
    case kActGeluTanh: {
        const float v2 = __fmul_rn(v, v);
        logistic2(tanh_arg(v, v2), p, q);
        y = __fmul_rn(v, p);
        // q is 0 long before v^2 is held back, which keeps 0 times an overflow out
        slope = __fmaf_rn(__fmul_rn(v, q), __fmaf_rn(3.0f * kCube * kTwoA, fminf(v2, 1e9f), kTwoA), p);
        return;
    }
    case kActSilu:
        logistic2(__fmul_rn(v, kLog2e), p, q);
        y = __fmul_rn(v, p);
        slope = __fmaf_rn(v, q, p);
        return;
    default:
        y = v;
        slope = 1.0f;
    }
}

// f(kind) with the activation's kind as a constant: one switch around the loop over
// a thread's elements, instead of one in it.
template <class F> __device__ __forceinline__ void with_kind(int32_t kind, F f)
{
    switch (kind) {
    case kActRelu: f(std::integral_constant<int32_t, kActRelu>{}); break;
    case kActGelu: f(std::integral_constant<int32_t, kActGelu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int32_t, kActGeluTanh>{}); break;
    case kActSilu: f(std::integral_constant<int32_t, kActSilu>{}); break;
    default: f(std::integral_constant<int32_t, kActNone>{});
    }
}

}  // namespace act
}  // namespace zgb
