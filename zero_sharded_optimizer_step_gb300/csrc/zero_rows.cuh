// Eight columns of a matrix's row as floats, for kernels whose warps take 256
// columns of a row at a time, and sums over a row.
//
// Rows that all begin on a boundary of 8 elements (VEC) are read and written eight
// consecutive elements a lane.  Others go an element a lane, 32 consecutive
// ones at a time, so that a warp's accesses are consecutive whatever their boundary.
// (Putting the eights together from aligned pieces, as the embedding does, took
// three to eight times as long here: 8192 x 4099 in bf16 through the norm 162 us,
// its gradient 406.)
#pragma once

#include "zero_elems.cuh"
#include "zero_pack8.cuh"

namespace zgb {
namespace rows {

// A matrix that is read: element (r, c) at r * stride + c.
struct In {
    const void *p;
    int64_t stride;
};

// The column of a lane's element e, after the warp's first.
template <bool VEC> __device__ __forceinline__ int column(int e)
{
    const int lane = threadIdx.x & 31;
    return VEC ? lane * 8 + e : e * 32 + lane;
}

// A lane's eight of a warp's 256 columns from c0 on: asked for first, taken later.
// Columns past `cols` are 0.
template <int DT, bool VEC> struct Eight;
template <int DT> struct Eight<DT, true> {
    elems::Raw<DT> v;

    __device__ __forceinline__ void ask(const In &m, int64_t r, int64_t c0, int64_t cols)
    {
        const int64_t at = r * m.stride + c0;            // the same for the warp
        if (c0 + column<true>(0) < cols) v.load(m.p, at + column<true>(0));
        else v.zero();
    }
    __device__ __forceinline__ void take(float (&f)[8]) const { v.get(f); }
};

template <int DT> struct Eight<DT, false> {
    using T = typename elems::El<DT>::T;
    T v[8];

    __device__ __forceinline__ void ask(const In &m, int64_t r, int64_t c0, int64_t cols)
    {
        const T *p = static_cast<const T *>(m.p) + (r * m.stride + c0) + column<false>(0);
        const int left = (cols - c0 < 256 ? (int)(cols - c0) : 256) - column<false>(0);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 32 * e < left ? p[32 * e] : T(0.0f);
    }
    __device__ __forceinline__ void take(float (&f)[8]) const
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = elems::load1<DT>(v, e);
    }
};

// Stores the lane's eight of columns c0 .. c0 + 256 (those below cols).
template <int DT, bool VEC>
__device__ __forceinline__ void put(void *p, int64_t stride, int64_t r, int64_t c0, int64_t cols,
                                    const float (&f)[8])
{
    const int64_t c = c0 + column<VEC>(0);
    if constexpr (VEC) {
        elems::Raw<DT> v;
        v.set(f);
        if (c < cols) v.store(p, r * stride + c);
    } else {
        const int left = cols - c < 256 ? (int)(cols - c) : 256;
        void *at = static_cast<typename elems::El<DT>::T *>(p) + r * stride + c;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (32 * e < left) elems::store1<DT>(at, 32 * e, f[e]);
    }
}

// Run w of a matrix whose rows have `runs` runs of 256 columns: its row and first column.
__device__ __forceinline__ void run_at(int64_t w, int64_t runs, int64_t &r, int64_t &c0)
{
    if (w < 0x80000000ll && runs < 0x80000000ll) r = (uint32_t)w / (uint32_t)runs;
    else r = w / runs;
    c0 = (w - r * runs) * 256;
}

inline In in(const void *p, int64_t stride) { return {p, stride}; }

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

// A warp's 256 values from a lane's eight consecutive ones to its every thirty-second,
// or back, through its own shared memory.
template <bool BACK> __device__ __forceinline__ void turn(float *shared, float (&f)[8])
{
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e) shared[column<!BACK>(e)] = f[e];
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = shared[column<BACK>(e)];
}

// Packs the lane's eight of row r from column c0 on; columns past the row are 0.
// `shared`: 256 floats of the warp's own where rows are off their boundaries.
template <bool VEC>
__device__ __forceinline__ void pack(const pack8::View &q, int64_t r, int64_t c0, float *shared,
                                     float (&f)[8])
{
    if constexpr (!VEC) turn<true>(shared, f);
    const int64_t c = c0 + column<true>(0);
    pack8::put_eight(q, r, c, c < q.wide, f);
}

// A row's eight in 8 bits, asked for and taken (`shared` as pack's).
template <int DT, bool VEC> struct Packed {
    uint2 codes;
    uint32_t scale;

    __device__ __forceinline__ void ask(const pack8::View &q, int64_t r, int64_t c0)
    {
        const int64_t c = c0 + column<true>(0);
        codes = make_uint2(0, 0);
        scale = 0;
        if (c < q.wide) {
            codes = *reinterpret_cast<const uint2 *>(q.codes + r * q.wide + c);
            scale = q.scales[r * (q.wide / pack8::kBlock) + c / pack8::kBlock];
        }
    }
    __device__ __forceinline__ void take(float *shared, float (&f)[8]) const
    {
        pack8::values8<DT>(codes, scale, f);
        if constexpr (!VEC) turn<false>(shared, f);
    }
};

}  // namespace rows

// Column sums: partial rows [parts][cols] in fp32, added up in their order, into
// out (DT), or added to it.
cudaError_t launch_column_sums(int32_t dt, const float *parts, int64_t n_parts, int64_t cols,
                               void *out, bool accumulate, cudaStream_t s);

}  // namespace zgb
