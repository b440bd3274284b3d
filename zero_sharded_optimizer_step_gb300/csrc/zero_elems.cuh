// Elements of the three types as floats, one at a time or 8 of a matrix's row.
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

// ---- rows of a matrix, 8 consecutive elements a lane
//
// Rows that all begin on a boundary of 8 elements (VEC: 16 bytes, fp32 32) are
// read and written whole.  Others (ANY) go through the 16-byte pieces that
// their elements lie in: a lane reads the two pieces around its 16 bytes and shifts
// them together, and writes the one piece that its own and its neighbour's
// elements make up.  Single elements move only at the ends of a row's part.

// A matrix as its bytes: nothing outside is read.
struct Span {
    const char *lo, *hi;

    // Whether the pieces around `bytes` bytes from byte `at` lie inside.
    __device__ __forceinline__ bool around(int64_t at, int64_t bytes) const
    {
        return at >= 16 && at + bytes + 16 <= hi - lo;
    }
};

// 16 bytes from byte o (even, 0 .. 16) of a and b side by side.
__device__ __forceinline__ uint4 join_pieces(uint4 a, uint4 b, uint32_t o)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (o & 16) return b;
    if (o & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (o & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (o & 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes at p, two at a time; bytes outside the matrix are 0.
__device__ __forceinline__ uint4 load_piecemeal(const char *p, const Span &m)
{
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (p + 2 * i >= m.lo && p + 2 * i + 2 <= m.hi)
            w[i >> 1] |= (uint32_t)*reinterpret_cast<const unsigned short *>(p + 2 * i)
                         << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight consecutive elements as they lie in memory.
template <int DT> struct Raw {
    static constexpr int kSize = DT == F32 ? 4 : 2;
    static constexpr int kPieces = DT == F32 ? 2 : 1;
    uint4 v[kPieces];

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int h = 0; h < kPieces; ++h) v[h] = make_uint4(0, 0, 0, 0);
    }

    // VEC: element i of base begins a boundary of 8 elements.
    __device__ __forceinline__ void load(const void *base, int64_t i)
    {
        const char *p = static_cast<const char *>(base) + i * kSize;
        if constexpr (DT == F32) {
            const ulonglong4_32a u = *reinterpret_cast<const ulonglong4_32a *>(p);
            v[0] = make_uint4((uint32_t)u.x, (uint32_t)(u.x >> 32), (uint32_t)u.y,
                              (uint32_t)(u.y >> 32));
            v[1] = make_uint4((uint32_t)u.z, (uint32_t)(u.z >> 32), (uint32_t)u.w,
                              (uint32_t)(u.w >> 32));
        } else {
            v[0] = *reinterpret_cast<const uint4 *>(p);
        }
    }

    __device__ __forceinline__ void store(void *base, int64_t i) const
    {
        char *p = static_cast<char *>(base) + i * kSize;
        if constexpr (DT == F32) {
            ulonglong4_32a u;
            u.x = v[0].x | (unsigned long long)v[0].y << 32;
            u.y = v[0].z | (unsigned long long)v[0].w << 32;
            u.z = v[1].x | (unsigned long long)v[1].y << 32;
            u.w = v[1].z | (unsigned long long)v[1].w << 32;
            *reinterpret_cast<ulonglong4_32a *>(p) = u;
        } else {
            *reinterpret_cast<uint4 *>(p) = v[0];
        }
    }

    // ANY, by the whole warp: lane l's elements go to 8 * l and on from element i;
    // the first `valid` elements of the warp's 256 are written.
    __device__ __forceinline__ void store_any(void *base, int64_t i, int valid) const
    {
        constexpr int kLane = 16 * kPieces, kPart = 32 * kLane;
        char *start = static_cast<char *>(base) + i * kSize;
        const int lane = threadIdx.x & 31;
        const int o = (int)((uintptr_t)start & 15u), bytes = valid * kSize;
        uint4 before;
        before.x = __shfl_up_sync(0xffffffffu, v[kPieces - 1].x, 1);
        before.y = __shfl_up_sync(0xffffffffu, v[kPieces - 1].y, 1);
        before.z = __shfl_up_sync(0xffffffffu, v[kPieces - 1].z, 1);
        before.w = __shfl_up_sync(0xffffffffu, v[kPieces - 1].w, 1);
#pragma unroll
        for (int h = 0; h < kPieces; ++h) {
            const int at = lane * kLane + 16 * h - o;     // of the aligned piece, in the part
            const uint4 p = join_pieces(h ? v[h - 1] : before, v[h], 16 - o);
            if (at >= 0 && at + 16 <= bytes) *reinterpret_cast<uint4 *>(start + at) = p;
        }
        // the elements before the first whole piece and after the last one, at most
        // 16 / kSize of either: an element a lane, fetched from the lane that has it
        const int head = o ? (16 - o < bytes ? 16 - o : bytes) : 0;
        const int body = (bytes - head) & ~15, tail = bytes - head - body;
        constexpr int kMost = 16 / kSize;
        const int at = lane < kMost ? lane * kSize : head + body + (lane - kMost) * kSize;
        const bool mine = lane < kMost ? at < head : lane < 2 * kMost && at < head + body + tail;
        const int from = at < kPart ? at / kLane : 0, word = (at % kLane) / 4;
        uint32_t x = 0;
#pragma unroll
        for (int h = 0; h < kPieces; ++h) {
            const uint32_t w0 = __shfl_sync(0xffffffffu, v[h].x, from);
            const uint32_t w1 = __shfl_sync(0xffffffffu, v[h].y, from);
            const uint32_t w2 = __shfl_sync(0xffffffffu, v[h].z, from);
            const uint32_t w3 = __shfl_sync(0xffffffffu, v[h].w, from);
            if (word / 4 == h) x = word % 4 == 0 ? w0 : word % 4 == 1 ? w1 : word % 4 == 2 ? w2 : w3;
        }
        if (mine) {
            if constexpr (kSize == 4) *reinterpret_cast<uint32_t *>(start + at) = x;
            else *reinterpret_cast<unsigned short *>(start + at) =
                     (unsigned short)(at & 2 ? x >> 16 : x);
        }
    }

    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        if constexpr (DT == F32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f[4 * h] = __uint_as_float(v[h].x);
                f[4 * h + 1] = __uint_as_float(v[h].y);
                f[4 * h + 2] = __uint_as_float(v[h].z);
                f[4 * h + 3] = __uint_as_float(v[h].w);
            }
        } else {
            widen2<DT>(v[0].x, f[0], f[1]);
            widen2<DT>(v[0].y, f[2], f[3]);
            widen2<DT>(v[0].z, f[4], f[5]);
            widen2<DT>(v[0].w, f[6], f[7]);
        }
    }

    __device__ __forceinline__ void set(const float (&f)[8])
    {
        if constexpr (DT == F32) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                v[h] = make_uint4(__float_as_uint(f[4 * h]), __float_as_uint(f[4 * h + 1]),
                                  __float_as_uint(f[4 * h + 2]), __float_as_uint(f[4 * h + 3]));
        } else {
            v[0] = make_uint4(narrow2<DT>(f[0], f[1]), narrow2<DT>(f[2], f[3]),
                              narrow2<DT>(f[4], f[5]), narrow2<DT>(f[6], f[7]));
        }
    }

    // Zeroes the elements from the `keep`-th on.
    __device__ __forceinline__ void cut(int keep)
    {
        if (keep >= 8) return;
        if constexpr (DT == F32) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint4 &u = v[e >> 2];
                if (e >= keep) ((e & 3) == 0 ? u.x : (e & 3) == 1 ? u.y : (e & 3) == 2 ? u.z : u.w) = 0;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t &u = e == 0 ? v[0].x : e == 1 ? v[0].y : e == 2 ? v[0].z : v[0].w;
                u = 2 * e >= keep ? 0u : 2 * e + 1 >= keep ? u & 0xffffu : u;
            }
        }
    }
};

// ANY: the elements from element i on, whatever their boundary; those outside
// the matrix are 0.  The pieces are asked for first and put together later, so
// that several rows' are on their way at once.  `inside` (the same for the
// whole warp): all pieces lie in the matrix.
template <int DT> struct Pieces {
    static constexpr int kPieces = Raw<DT>::kPieces;
    uint4 w[kPieces + 1];
    uint32_t o;

    __device__ __forceinline__ void ask(const void *base, int64_t i, const Span &m, bool inside)
    {
        const char *p = static_cast<const char *>(base) + i * Raw<DT>::kSize;
        o = (uint32_t)(uintptr_t)p & 15u;
        if (inside) {
#pragma unroll
            for (int h = 0; h <= kPieces; ++h) {
                w[h] = make_uint4(0, 0, 0, 0);
                if (h < kPieces || o) w[h] = *reinterpret_cast<const uint4 *>(p - o + 16 * h);
            }
        } else {                 // already put together
            o = 0;
#pragma unroll
            for (int h = 0; h < kPieces; ++h) w[h] = load_piecemeal(p + 16 * h, m);
            w[kPieces] = make_uint4(0, 0, 0, 0);
        }
    }

    __device__ __forceinline__ Raw<DT> take() const
    {
        Raw<DT> r;
#pragma unroll
        for (int h = 0; h < kPieces; ++h) r.v[h] = join_pieces(w[h], w[h + 1], o);
        return r;
    }
};

// 8 elements of a row, either way.
template <int DT, bool VEC> struct Eight;
template <int DT> struct Eight<DT, true> {
    Raw<DT> r;
    __device__ __forceinline__ void ask(const void *base, int64_t i, const Span &, bool)
    {
        r.load(base, i);
    }
    __device__ __forceinline__ Raw<DT> take() const { return r; }
};
template <int DT> struct Eight<DT, false> : Pieces<DT> {};

}  // namespace elems
}  // namespace zgb
