// Eight consecutive columns of a matrix's row as floats, for kernels whose
// warps take 256 columns of a row at a time, and sums over a row.
#pragma once

#include "zero_elems.cuh"

namespace zgb {
namespace rows {

// A matrix that is read: element (r, c) at r * stride + c.
struct In {
    const void *p;
    int64_t stride;
    elems::Span span;
};

inline In in(const void *p, int64_t rows, int64_t cols, int64_t stride, int32_t dt)
{
    const char *b = static_cast<const char *>(p);
    const int64_t bytes = rows > 0 ? ((rows - 1) * stride + cols) * elem_size(dt) : 0;
    return {p, stride, {b, b ? b + bytes : b}};
}

// A lane's eight of a warp's 256 columns from c0 on: asked for first, taken later.
// Columns past `cols` are 0.
template <int DT, bool VEC> struct Eight {
    elems::Eight<DT, VEC> e;
    int keep;

    __device__ __forceinline__ void ask(const In &m, int64_t r, int64_t c0, int64_t cols)
    {
        const int64_t c = c0 + 8 * (threadIdx.x & 31);
        keep = cols - c < 8 ? (cols > c ? (int)(cols - c) : 0) : 8;
        const int64_t at = r * m.stride + c0;
        if constexpr (VEC) {
            if (keep > 0) e.ask(m.p, at + 8 * (threadIdx.x & 31), m.span, true);
            else e.r.zero();
        } else {
            constexpr int size = elems::Raw<DT>::kSize;
            // bytes from the first whole piece of the matrix on
            const int64_t off = static_cast<const char *>(m.p) + at * size - m.span.lo;
            e.ask(m.p, at + 8 * (threadIdx.x & 31), m.span, m.span.around(off, 256 * size));
        }
    }

    __device__ __forceinline__ void take(float (&f)[8]) const
    {
        elems::Raw<DT> r = e.take();
        if (!VEC) r.cut(keep);
        r.get(f);
    }
};

// Stores the lane's eight of columns c0 .. c0 + 256 (those below cols).
template <int DT, bool VEC>
__device__ __forceinline__ void put(void *p, int64_t stride, int64_t r, int64_t c0, int64_t cols,
                                    const float (&f)[8])
{
    elems::Raw<DT> v;
    v.set(f);
    if constexpr (VEC) {
        const int64_t c = c0 + 8 * (threadIdx.x & 31);
        if (c < cols) v.store(p, r * stride + c);
    } else if (c0 < cols) {
        v.store_any(p, r * stride + c0, cols - c0 < 256 ? (int)(cols - c0) : 256);
    }
}

// Run w of a matrix whose rows have `runs` runs of 256 columns: its row and first column.
__device__ __forceinline__ void run_at(int64_t w, int64_t runs, int64_t &r, int64_t &c0)
{
    if (w < 0x80000000ll && runs < 0x80000000ll) r = (uint32_t)w / (uint32_t)runs;
    else r = w / runs;
    c0 = (w - r * runs) * 256;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

}  // namespace rows

// Column sums: partial rows [parts][cols] in fp32, added up in their order, into
// out (DT), or added to it.
cudaError_t launch_column_sums(int32_t dt, const float *parts, int64_t n_parts, int64_t cols,
                               void *out, bool accumulate, cudaStream_t s);

}  // namespace zgb
