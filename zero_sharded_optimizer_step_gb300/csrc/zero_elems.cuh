// Elements of the three types as floats, E (8, 2 or 1) at a time.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "zero_internal.h"

namespace zgb {
namespace elems {

template <int DT> struct El;
template <> struct El<F32> { using T = float; };
template <> struct El<BF16> { using T = __nv_bfloat16; };
template <> struct El<F16> { using T = __half; };

template <int DT>
__device__ __forceinline__ void widen2(uint32_t w, float &lo, float &hi)
{
    static_assert(DT != F32, "16-bit types only");
    if constexpr (DT == BF16) {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xffff0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        lo = f.x;
        hi = f.y;
    }
}

template <int DT> __device__ __forceinline__ uint32_t narrow2(float lo, float hi)
{
    static_assert(DT != F32, "16-bit types only");
    if constexpr (DT == BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <int DT> __device__ __forceinline__ float load1(const void *p, int64_t i)
{
    if constexpr (DT == F32) return static_cast<const float *>(p)[i];
    else if constexpr (DT == BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    else return __half2float(static_cast<const __half *>(p)[i]);
}

template <int DT> __device__ __forceinline__ void store1(void *p, int64_t i, float x)
{
    if constexpr (DT == F32) static_cast<float *>(p)[i] = x;
    else if constexpr (DT == BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
    else static_cast<__half *>(p)[i] = __float2half_rn(x);
}

// E elements as they lie in memory.
template <int DT, int E> struct Raw {
    static constexpr int kWords = DT == F32 ? E : (E + 1) / 2;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const void *base, int64_t i)
    {
        using T = typename El<DT>::T;
        const T *p = static_cast<const T *>(base) + i;
        if constexpr (E == 1 && DT != F32) {
            w[0] = *reinterpret_cast<const unsigned short *>(p);
        } else if constexpr (kWords == 1) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else if constexpr (kWords == 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x;
            w[1] = v.y;
        } else {
#pragma unroll
            for (int h = 0; h < kWords / 4; ++h) {
                const uint4 v = reinterpret_cast<const uint4 *>(p)[h];
                w[4 * h] = v.x;
                w[4 * h + 1] = v.y;
                w[4 * h + 2] = v.z;
                w[4 * h + 3] = v.w;
            }
        }
    }

    __device__ __forceinline__ void store(void *base, int64_t i) const
    {
        using T = typename El<DT>::T;
        T *p = static_cast<T *>(base) + i;
        if constexpr (E == 1 && DT != F32) {
            *reinterpret_cast<unsigned short *>(p) = (unsigned short)w[0];
        } else if constexpr (kWords == 1) {
            *reinterpret_cast<uint32_t *>(p) = w[0];
        } else if constexpr (kWords == 2) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int h = 0; h < kWords / 4; ++h)
                reinterpret_cast<uint4 *>(p)[h] =
                    make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
        }
    }

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }

    __device__ __forceinline__ void get(float (&f)[E]) const
    {
        if constexpr (DT == F32) {
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] = __uint_as_float(w[i]);
        } else if constexpr (E == 1) {
            float hi;
            widen2<DT>(w[0], f[0], hi);
        } else {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) widen2<DT>(w[i], f[2 * i], f[2 * i + 1]);
        }
    }

    __device__ __forceinline__ void set(const float (&f)[E])
    {
        if constexpr (DT == F32) {
#pragma unroll
            for (int i = 0; i < E; ++i) w[i] = __float_as_uint(f[i]);
        } else if constexpr (E == 1) {
            w[0] = narrow2<DT>(f[0], 0.0f);
        } else {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) w[i] = narrow2<DT>(f[2 * i], f[2 * i + 1]);
        }
    }
};

}  // namespace elems
}  // namespace zgb
