// The activations of linear layers and their slopes, in fp32.
//
// The exponentials and quotients are CUDA's fast ones (a few units in the last
// place), the normal distribution function its accurate one.  Differences of
// nearly equal numbers are avoided: p (1 - p) of a logistic p is e / (1 + e)^2.
#pragma once

#include <type_traits>

#include <cuda_runtime.h>

namespace zgb {

enum Act : int32_t { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

namespace act {

constexpr float kTwoA = 1.5957691216057308f;          // 2 sqrt(2 / pi)
constexpr float kCube = 0.044715f;

// 1 / (1 + exp(-v)).  Where exp(-v) overflows the quotient is 0.
__device__ __forceinline__ float logistic(float v)
{
    return __fdividef(1.0f, __fadd_rn(1.0f, __expf(-v)));
}

// p = 1 / (1 + exp(-v)) and q = p (1 - p).
__device__ __forceinline__ void logistic2(float v, float &p, float &q)
{
    const float e = __expf(-fabsf(v)), r = __fdividef(1.0f, __fadd_rn(1.0f, e));
    p = v < 0.0f ? __fmul_rn(e, r) : r;
    q = __fmul_rn(__fmul_rn(e, r), r);
}

__device__ __forceinline__ float tanh_arg(float v)     // twice tanh's argument
{
    return __fmul_rn(__fmul_rn(kTwoA, v), __fmaf_rn(kCube, __fmul_rn(v, v), 1.0f));
}

__device__ __forceinline__ float value(float v, int32_t kind)
{
    switch (kind) {
    case kActRelu: return v < 0.0f ? 0.0f : v;
    case kActGelu: return __fmul_rn(v, normcdff(v));
    case kActGeluTanh: return __fmul_rn(v, logistic(tanh_arg(v)));
    case kActSilu: return __fmul_rn(v, logistic(v));
    default: return v;
    }
}

// The activation and its slope.  Far from 0 a slope's second term is 0 times
// a number that may have overflowed: it is left out there.
__device__ __forceinline__ void both(float v, int32_t kind, float &y, float &slope)
{
    float p, q;
    switch (kind) {
    case kActRelu:
        y = v < 0.0f ? 0.0f : v;
        slope = v <= 0.0f ? 0.0f : 1.0f;
        return;
    case kActGelu: {
        p = normcdff(v);
        q = __fmul_rn(0.3989422804014327f, __expf(__fmul_rn(-0.5f, __fmul_rn(v, v))));
        y = __fmul_rn(v, p);
        slope = q == 0.0f ? p : __fmaf_rn(v, q, p);
        return;
    }
    case kActGeluTanh:
        logistic2(tanh_arg(v), p, q);
        y = __fmul_rn(v, p);
        slope = q == 0.0f ? p
                          : __fmaf_rn(__fmul_rn(__fmul_rn(v, q), kTwoA),
                                      __fmaf_rn(3.0f * kCube, __fmul_rn(v, v), 1.0f), p);
        return;
    case kActSilu:
        logistic2(v, p, q);
        y = __fmul_rn(v, p);
        slope = q == 0.0f ? p : __fmaf_rn(v, q, p);
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
