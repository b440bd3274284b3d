// Rows kept in 8 bits: e4m3 elements with a power-of-two scale (E8M0) for every
// 32 of a row.  The scale is the smallest that keeps the block within e4m3's
// largest value, 448 = 1.75 * 2^8, so that nothing saturates.
//
// A matrix of R rows by C columns is R rows of `pitch` codes (C rounded up to
// whole blocks), then R rows of pitch / 32 scale exponents.
#pragma once

#include <cuda_fp8.h>

#include "zero_elems.cuh"

namespace zgb {
namespace pack8 {

constexpr int kBlock = 32;

__host__ __device__ inline int64_t pitch(int64_t cols) { return (cols + kBlock - 1) / kBlock * kBlock; }

// The bits of |x|: their order is that of the magnitudes, NaN last.
__device__ __forceinline__ uint32_t magnitude(float x)
{
    return __float_as_uint(x) & 0x7fffffffu;
}

// The scale's exponent + 127 for a block whose largest magnitude has these bits;
// 255, the NaN scale, where an element is infinite or NaN.
__device__ __forceinline__ uint32_t exponent(uint32_t top)
{
    if (top >= 0x7f800000u) return 255;
    const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u);
    return e < 0 ? 0 : (uint32_t)e;
}

__device__ __forceinline__ float down(uint32_t e)        // 2^-(e - 127)
{
    return __uint_as_float((254u - (e < 254 ? e : 254)) << 23);
}

__device__ __forceinline__ float up(uint32_t e)          // 2^(e - 127), or NaN
{
    return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7fc00000u : e << 23);
}

// Two codes, the first in the low byte.  (A product with a power of two
// is exact unless it is far below the smallest code.)
__device__ __forceinline__ uint32_t codes2(float a, float b, float d)
{
    return __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(a, d), __fmul_rn(b, d)), __NV_SATFINITE,
                                    __NV_E4M3);
}

__device__ __forceinline__ uint32_t codes4(const float *v, float d)
{
    return codes2(v[0], v[1], d) | codes2(v[2], v[3], d) << 16;
}

template <int DT> __device__ __forceinline__ float most()
{
    return DT == F32 ? 3.4028234663852886e38f : DT == BF16 ? 3.3895313892515355e38f : 65504.0f;
}

// The values of eight codes of a block with the scale exponent e, none larger than the
// type's largest: rounding up to a code must not make an infinity of a finite
// element.  Only blocks whose scale times 448 is beyond that are looked at.
template <int DT>
__device__ __forceinline__ void values8(uint2 c, uint32_t e, float (&v)[8])
{
    const float u = up(e);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const uint32_t two = (h < 2 ? c.x : c.y) >> (16 * (h & 1));
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r));
        v[2 * h] = __fmul_rn(f.x, u);
        v[2 * h + 1] = __fmul_rn(f.y, u);
    }
    if (e >= (DT == F16 ? 127 + 8 : 127 + 119)) {        // 448 * 2^8 > 65504, 448 * 2^119 > 2^127
#pragma unroll
        for (int i = 0; i < 8; ++i)                      // (a comparison: NaN stays NaN)
            v[i] = fabsf(v[i]) > most<DT>() ? copysignf(most<DT>(), v[i]) : v[i];
    }
}

// A matrix in 8 bits.
struct View {
    unsigned char *codes, *scales;
    int64_t wide;                                        // codes of a row
};

__host__ __device__ inline View view(unsigned char *q, int64_t rows, int64_t cols)
{
    const int64_t p = pitch(cols);
    return {q, q ? q + rows * p : nullptr, p};
}

// A warp's lanes hold 32 consecutive elements of row r from column j0 (whole
// blocks): packs them.  All lanes take part; those past the row hold 0.
__device__ __forceinline__ void put_lane(const View &q, int64_t r, int64_t j0, float v)
{
    const uint32_t e = exponent(__reduce_max_sync(0xffffffffu, magnitude(v)));
    const int lane = threadIdx.x & 31;
    q.codes[r * q.wide + j0 + lane] = (unsigned char)codes2(v, 0.0f, down(e));
    if (lane == 0) q.scales[r * (q.wide / kBlock) + j0 / kBlock] = (unsigned char)e;
}

// A thread holds them.
__device__ __forceinline__ void put_thread(const View &q, int64_t r, int64_t j0,
                                           const float (&v)[32])
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = max(top, magnitude(v[i]));
    const uint32_t e = exponent(top);
    const float d = down(e);
    uint4 *p = reinterpret_cast<uint4 *>(q.codes + r * q.wide + j0);
#pragma unroll
    for (int h = 0; h < 2; ++h)
        p[h] = make_uint4(codes4(v + 16 * h, d), codes4(v + 16 * h + 4, d),
                          codes4(v + 16 * h + 8, d), codes4(v + 16 * h + 12, d));
    q.scales[r * (q.wide / kBlock) + j0 / kBlock] = (unsigned char)e;
}

// Four neighbouring lanes hold them, 8 each: lane l's from column 8 l on of the
// warp's 256 (j: this lane's first column, below the pitch where `in`).
__device__ __forceinline__ void put_eight(const View &q, int64_t r, int64_t j, bool in,
                                          const float (&v)[8])
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, magnitude(v[i]));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (!in) return;
    const uint32_t e = exponent(top);
    const float d = down(e);
    *reinterpret_cast<uint2 *>(q.codes + r * q.wide + j) = make_uint2(codes4(v, d),
                                                                      codes4(v + 4, d));
    if ((threadIdx.x & 3) == 0) q.scales[r * (q.wide / kBlock) + j / kBlock] = (unsigned char)e;
}

}  // namespace pack8
}  // namespace zgb
