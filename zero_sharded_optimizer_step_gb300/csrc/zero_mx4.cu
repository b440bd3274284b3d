// Microscaled 4-bit matrices (OCP MX, MXFP4: 4-bit E2M1 elements, one power
// of two per block of 32): quantisation along the rows, along the columns, or
// both from one read, and back to values.
//
// A block's shared exponent is floor(log2(max |x|)) - 2 (2 is the exponent
// of E2M1's largest power of two), held biased by 127 and not below 0; an
// element is x / 2^exponent rounded to the nearest of +-{0, .5, 1, 1.5, 2, 3,
// 4, 6}, ties to the even code, larger ones to 6.  The division is by a power
// of two whose reciprocal is a normal number, so it is one exact (or, for
// elements far below the block's largest, correctly rounded) multiplication.
// A block that holds an infinity or NaN gets the scale 255 (NaN): every
// product with it is NaN.
//
// What bounds it: memory (2 bytes in, 17/32 out an element and direction) for
// one direction, for both from one read the ALU beside it (14 instructions an
// element).  Measured for 8192 x 11008 bf16: both ways 54 us (5.1 TB/s), rows
// alone 42, back to values 35 (6.4 TB/s); fp32 both ways 85 us (5.4 TB/s).
#include "zero_elems.cuh"
#include "zero_ops.h"

namespace zgb {
namespace {

// The scale byte of a block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t block_scale(uint32_t top)
{
    const uint32_t e = top >> 23;
    return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}

// 2^-(scale - 127); for the NaN scale any number does.
__device__ __forceinline__ float block_inverse(uint32_t scale)
{
    return __uint_as_float((254u - (scale < 253u ? scale : 253u)) << 23);
}

// Eight floats to E2M1 codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8])
{
    uint32_t r;
    asm("{\n .reg .b8 p, q, r, s;\n"
        " cvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 r, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 s, %8, %7;\n"
        " mov.b32 %0, {p, q, r, s};\n}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float inv)
{
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(x[i], inv);
    return codes8(y);
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t top_of(const float (&x)[8])
{
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, magnitude(x[i]));
    return t;
}

__device__ __forceinline__ int64_t scale_at(int row, int block)
{
    return kMxCodes + (block >> 2) * 512 + (row & 31) * 16 + (row >> 5) * 4 + (block & 3);
}

template <int DT> __device__ __forceinline__ elems::Span span_of(const MxQuantArgs &a)
{
    const char *lo = static_cast<const char *>(a.x);
    return {lo, lo + ((a.rows - 1) * a.stride + a.cols) * elems::Raw<DT>::kSize};
}

// A lane's 8 of the 256 columns from c0 of a row: asked for, and later taken,
// with zeros where the matrix has none.
template <int DT, bool VEC>
__device__ __forceinline__ void ask8(const MxQuantArgs &a, const elems::Span &m, int64_t row,
                                     int64_t c0, elems::Eight<DT, VEC> &r)
{
    constexpr int kSize = elems::Raw<DT>::kSize;
    const int64_t c = c0 + (threadIdx.x & 31) * 8;
    if constexpr (VEC && DT != F32) {
        r.r.zero();
        if (row < a.rows && c < a.cols) r.r.load(a.x, row * a.stride + c);
    } else {      // fp32: 34 us against 40 of a predicated load, for 8192 x 4096 both ways
        const int64_t from = (row < a.rows ? row : 0) * a.stride;
        r.ask(a.x, from + (VEC && c >= a.cols ? a.cols - 8 : c), m,
              m.around((from + c0) * kSize, kMxCols * kSize));
    }
}

template <int DT, bool VEC>
__device__ __forceinline__ elems::Raw<DT> take8(const MxQuantArgs &a, int64_t row, int64_t c0,
                                                const elems::Eight<DT, VEC> &r)
{
    elems::Raw<DT> v = r.take();
    if (VEC && DT != F32) return v;
    const int64_t left = row < a.rows ? a.cols - c0 - (threadIdx.x & 31) * 8 : 0;
    v.cut(left >= 8 ? 8 : left > 0 ? (int)left : 0);
    return v;
}

template <int DT, bool VEC>
__device__ __forceinline__ elems::Raw<DT> load8(const MxQuantArgs &a, int64_t row, int64_t c0)
{
    elems::Eight<DT, VEC> r;
    ask8<DT, VEC>(a, span_of<DT>(a), row, c0, r);
    return take8<DT, VEC>(a, row, c0, r);
}

// ---- 16-bit types, two elements a word

// The larger of a's elements and of b's magnitudes; NaN where one is.
template <int DT> __device__ __forceinline__ uint32_t top2(uint32_t a, uint32_t b)
{
    if constexpr (DT == BF16) {
        const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a),
                                             __habs2(*reinterpret_cast<__nv_bfloat162 *>(&b)));
        return *reinterpret_cast<const uint32_t *>(&m);
    } else {
        const __half2 m = __hmax2_nan(*reinterpret_cast<__half2 *>(&a),
                                      __habs2(*reinterpret_cast<__half2 *>(&b)));
        return *reinterpret_cast<const uint32_t *>(&m);
    }
}

// The scale byte of a block whose largest magnitude has these 15 bits.
template <int DT> __device__ __forceinline__ uint32_t block_scale16(uint32_t top)
{
    if constexpr (DT == BF16) return block_scale(top << 16);
    float lo, hi;
    elems::widen2<F16>(top, lo, hi);
    return block_scale(__float_as_uint(lo));
}

// A word's elements times their blocks' 2^-exponent.  Of bf16 the product is
// taken two at a time: it is exact, or below every threshold of the rounding.
template <int DT>
__device__ __forceinline__ void scaled2(uint32_t w, float inv_lo, float inv_hi, float &lo,
                                        float &hi)
{
    if constexpr (DT == BF16) {
        const uint32_t inv = (__float_as_uint(inv_hi) & 0xffff0000u) | (__float_as_uint(inv_lo) >> 16);
        const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&inv));
        elems::widen2<BF16>(*reinterpret_cast<const uint32_t *>(&y), lo, hi);
    } else {
        elems::widen2<DT>(w, lo, hi);
        lo = __fmul_rn(lo, inv_lo);
        hi = __fmul_rn(hi, inv_hi);
    }
}

// A warp's row of 256 columns of a record, 8 elements a lane, a block over 4
// lanes: the codes, and the scales (four blocks' are one word).
template <int DT>
__device__ __forceinline__ void put_row16(unsigned char *rec, int r, uint4 v)
{
    const int lane = threadIdx.x & 31;
    uint32_t top = top2<DT>(top2<DT>(top2<DT>(top2<DT>(0, v.x), v.y), v.z), v.w);
    top = top2<DT>(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = top2<DT>(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t scale = block_scale16<DT>(max(top & 0xffffu, top >> 16));
    const float inv = block_inverse(scale);
    float y[8];
    scaled2<DT>(v.x, inv, inv, y[0], y[1]);
    scaled2<DT>(v.y, inv, inv, y[2], y[3]);
    scaled2<DT>(v.z, inv, inv, y[4], y[5]);
    scaled2<DT>(v.w, inv, inv, y[6], y[7]);
    uint32_t w = scale << (8 * ((lane >> 2) & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    w |= __shfl_xor_sync(0xffffffffu, w, 8);
    if (!rec) return;
    *reinterpret_cast<uint32_t *>(rec + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) +
                                  (lane & 3) * 4) = codes8(y);
    if ((lane & 15) == 0) *reinterpret_cast<uint32_t *>(rec + scale_at(r, lane >> 2)) = w;
}

// Few rows: a warp a row.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
mx4_rows16_kernel(const __grid_constant__ MxQuantArgs a, int64_t kt)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t task = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t row = task / kt, t = task - row * kt;
    if (row >= a.rows) return;
    put_row16<DT>(a.q + ((row / kMxRows) * kt + t) * kMxRecord, (int)(row % kMxRows),
                  load8<DT, VEC>(a, row, t * kMxCols).v[0]);
}

// Either direction, or both from one read: a block takes 64 rows by 256
// columns through shared memory.  For q a thread takes 32 columns of a row, a
// block of the matrix, twice; for qt 32 rows of two neighbouring columns, two blocks
// of its transpose: neither needs another thread's elements for its scale.
// Past the matrix's last row the transpose gets zeros, up to the end of its
// record.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
mx4_both16_kernel(const __grid_constant__ MxQuantArgs a, int64_t kt, int64_t ktt)
{
    __shared__ __align__(16) uint32_t strip[64][kMxCols / 2];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t ct = blockIdx.x % kt, r0 = (blockIdx.x / kt) * 64, c0 = ct * kMxCols;
    {
        const elems::Span m = span_of<DT>(a);
        elems::Eight<DT, VEC> v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) ask8<DT, VEC>(a, m, r0 + warp * 8 + j, c0, v[j]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4 *>(&strip[warp * 8 + j][lane * 4]) =
                take8<DT, VEC>(a, r0 + warp * 8 + j, c0, v[j]).v[0];
    }
    __syncthreads();
    if (a.q) {
        unsigned char *rec = a.q + ((r0 / kMxRows) * kt + ct) * kMxRecord;
        // a thread's four 16-byte pieces start at another one in every second
        // thread, so that eight threads' reads fall into different banks
        const int blk = threadIdx.x & 7, turn = blk >> 1;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int sr = half * 32 + (threadIdx.x >> 3);
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = *reinterpret_cast<const uint4 *>(
                    &strip[sr][blk * 16 + ((j + turn) & 3) * 4]);
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                top = top2<DT>(top2<DT>(top2<DT>(top2<DT>(top, v[j].x), v[j].y), v[j].z), v[j].w);
            const uint32_t scale = block_scale16<DT>(max(top & 0xffffu, top >> 16));
            const float inv = block_inverse(scale);
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float y[8];
                scaled2<DT>(v[j].x, inv, inv, y[0], y[1]);
                scaled2<DT>(v[j].y, inv, inv, y[2], y[3]);
                scaled2<DT>(v[j].z, inv, inv, y[4], y[5]);
                scaled2<DT>(v[j].w, inv, inv, y[6], y[7]);
                w[j] = codes8(y);
            }
            // w[j] is piece (j + turn) & 3: turn them back
            const uint32_t u0 = turn & 1 ? w[3] : w[0], u1 = turn & 1 ? w[0] : w[1];
            const uint32_t u2 = turn & 1 ? w[1] : w[2], u3 = turn & 1 ? w[2] : w[3];
            const uint4 out = turn & 2 ? make_uint4(u2, u3, u0, u1) : make_uint4(u0, u1, u2, u3);
            if (r0 + sr < a.rows) {
                const int r = (int)(r0 % kMxRows) + sr;
                *reinterpret_cast<uint4 *>(rec + r * 128 + ((blk ^ (r & 7)) << 4)) = out;
                rec[scale_at(r, blk)] = (unsigned char)scale;
            }
        }
    }
    const int pair = threadIdx.x & 127, half = threadIdx.x >> 7;
    const int64_t col = c0 + 2 * pair;
    if (!a.qt || col >= a.cols) return;
    uint32_t w[32], top = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        w[i] = strip[half * 32 + i][pair];
        top = top2<DT>(top, w[i]);
    }
    const uint32_t s0 = block_scale16<DT>(top & 0xffffu), s1 = block_scale16<DT>(top >> 16);
    const float inv0 = block_inverse(s0), inv1 = block_inverse(s1);
    uint32_t q0[4], q1[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float y0[8], y1[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) scaled2<DT>(w[g * 8 + i], inv0, inv1, y0[i], y1[i]);
        q0[g] = codes8(y0);
        q1[g] = codes8(y1);
    }
    unsigned char *rec = a.qt + ((col / kMxRows) * ktt + r0 / kMxCols) * kMxRecord;
    const int r = (int)(col % kMxRows), blk = (int)(r0 % kMxCols) / 32 + half;
    *reinterpret_cast<uint4 *>(rec + r * 128 + ((blk ^ (r & 7)) << 4)) =
        make_uint4(q0[0], q0[1], q0[2], q0[3]);
    rec[scale_at(r, blk)] = (unsigned char)s0;
    if (col + 1 >= a.cols) return;
    *reinterpret_cast<uint4 *>(rec + (r + 1) * 128 + ((blk ^ ((r + 1) & 7)) << 4)) =
        make_uint4(q1[0], q1[1], q1[2], q1[3]);
    rec[scale_at(r + 1, blk)] = (unsigned char)s1;
}

// ---- fp32

// A warp quantises one row's 256 columns of a record: 8 elements a lane, a
// block over 4 lanes.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
mx4_rows_kernel(const __grid_constant__ MxQuantArgs a, int64_t kt)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t task = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t row = task / kt, t = task - row * kt;
    if (row >= a.rows) return;
    float x[8];
    load8<DT, VEC>(a, row, t * kMxCols).get(x);
    uint32_t top = top_of(x);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t scale = block_scale(top);
    unsigned char *rec = a.q + ((row / kMxRows) * kt + t) * kMxRecord;
    const int r = (int)(row % kMxRows);
    *reinterpret_cast<uint32_t *>(rec + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) +
                                  (lane & 3) * 4) = codes8(x, block_inverse(scale));
    // four blocks' scales are one word
    uint32_t w = scale << (8 * ((lane >> 2) & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    w |= __shfl_xor_sync(0xffffffffu, w, 8);
    if ((lane & 15) == 0) *reinterpret_cast<uint32_t *>(rec + scale_at(r, lane >> 2)) = w;
}

// Both directions from one read: a block takes 128 rows by 256 columns,
// 32 rows at a time.  The rows are quantised from the registers that they
// were read into; through shared memory every thread then takes one column,
// whose 32 elements are a block of the transpose.  Past the matrix's last
// row the transpose gets zeros, up to the end of its record.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
mx4_both_kernel(const __grid_constant__ MxQuantArgs a, int64_t kt, int64_t ktt)
{
    static_assert(DT == F32, "16-bit types take mx4_both16_kernel");
    __shared__ __align__(16) float strip[32][kMxCols + 8];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t ct = blockIdx.x % kt, r0 = (blockIdx.x / kt) * 128;
    const int64_t c0 = ct * kMxCols;
    const int64_t col = c0 + threadIdx.x;
    unsigned char *rect = nullptr;
    if (a.qt && col < a.cols)
        rect = a.qt + ((col / kMxRows) * ktt + r0 / kMxCols) * kMxRecord;
    const int tr = (int)(col % kMxRows);
    const int tb0 = (int)(r0 % kMxCols) / 32;     // first block of the record's columns
    uint32_t tscales = 0;
    const elems::Span m = span_of<DT>(a);
    for (int s = 0; s < 4; ++s) {
        float x[4][8];
        {
            elems::Eight<DT, VEC> v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                ask8<DT, VEC>(a, m, r0 + s * 32 + warp * 4 + j, c0, v[j]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                take8<DT, VEC>(a, r0 + s * 32 + warp * 4 + j, c0, v[j]).get(x[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float4 *to = reinterpret_cast<float4 *>(&strip[warp * 4 + j][lane * 8]);
            to[0] = make_float4(x[j][0], x[j][1], x[j][2], x[j][3]);
            to[1] = make_float4(x[j][4], x[j][5], x[j][6], x[j][7]);
            const int64_t row = r0 + s * 32 + warp * 4 + j;
            uint32_t top = top_of(x[j]);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const uint32_t scale = block_scale(top);
            uint32_t w = scale << (8 * ((lane >> 2) & 3));
            w |= __shfl_xor_sync(0xffffffffu, w, 4);
            w |= __shfl_xor_sync(0xffffffffu, w, 8);
            if (a.q && row < a.rows) {
                unsigned char *rec = a.q + ((row / kMxRows) * kt + ct) * kMxRecord;
                const int r = (int)(row % kMxRows);
                *reinterpret_cast<uint32_t *>(rec + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) +
                                              (lane & 3) * 4) =
                    codes8(x[j], block_inverse(scale));
                if ((lane & 15) == 0)
                    *reinterpret_cast<uint32_t *>(rec + scale_at(r, lane >> 2)) = w;
            }
        }
        __syncthreads();
        if (rect) {
            float y[4][8];
            uint32_t top = 0;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[g][e] = strip[g * 8 + e][threadIdx.x];
                top = max(top, top_of(y[g]));
            }
            const uint32_t scale = block_scale(top);
            const float inv = block_inverse(scale);
            uint4 w;
            w.x = codes8(y[0], inv);
            w.y = codes8(y[1], inv);
            w.z = codes8(y[2], inv);
            w.w = codes8(y[3], inv);
            *reinterpret_cast<uint4 *>(rect + tr * 128 + (((tb0 + s) ^ (tr & 7)) << 4)) = w;
            tscales |= scale << (8 * s);
        }
        __syncthreads();
    }
    if (rect) *reinterpret_cast<uint32_t *>(rect + scale_at(tr, tb0)) = tscales;
}

template <int DT, bool VEC> cudaError_t quant_go(const MxQuantArgs &a, int sms, cudaStream_t s)
{
    const int64_t kt = (a.cols + kMxCols - 1) / kMxCols;
    const int64_t ktt = (a.rows + kMxCols - 1) / kMxCols;
    const int64_t limit = 0x7fffffff;
    if (!a.qt && (DT == F32 || a.rows * kt < (int64_t)sms * 32)) {
        const int64_t warps = a.rows * kt;
        // one warp a block for few: 2.2 us a pass among others either way up to 1024
        // warps, then slower (256 rows of 4096: 4.9 us against 2.2)
        const int threads = warps <= 1024 ? 32 : kThreads;
        const int64_t blocks = (warps * 32 + threads - 1) / threads;
        if (blocks > limit) return cudaErrorInvalidValue;
        const dim3 grid((unsigned)blocks), block((unsigned)threads);
        if constexpr (DT == F32)
            return launch_dependent(mx4_rows_kernel<DT, VEC>, grid, block, 0, s, a, kt);
        else
            return launch_dependent(mx4_rows16_kernel<DT, VEC>, grid, block, 0, s, a, kt);
    }
    const int64_t blocks = kt * ktt * (DT == F32 ? 2 : 4);
    if (blocks > limit) return cudaErrorInvalidValue;
    if constexpr (DT == F32)
        return launch_dependent(mx4_both_kernel<DT, VEC>, dim3((unsigned)blocks), dim3(kThreads), 0,
                                s, a, kt, ktt);
    else
        return launch_dependent(mx4_both16_kernel<DT, VEC>, dim3((unsigned)blocks), dim3(kThreads),
                                0, s, a, kt, ktt);
}

template <int DT> cudaError_t quant_pick(const MxQuantArgs &a, int sms, cudaStream_t s)
{
    return rows_aligned(a.x, a.stride, DT, a.cols) ? quant_go<DT, true>(a, sms, s)
                                                   : quant_go<DT, false>(a, sms, s);
}

// ---------------------------------------------------------------- to values

// Four bytes of codes, 8 elements, times 2^(scale - 127).
__device__ __forceinline__ void values8(uint32_t w, uint32_t scale, float (&f)[8])
{
    // 2^-127 is subnormal, so the exponent's field cannot hold it; 255 is NaN
    const float s = scale == 255u ? __uint_as_float(0x7fffffffu)
                    : scale == 0u ? __uint_as_float(0x00400000u)
                                  : __uint_as_float(scale << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("{\n .reg .b8 b;\n cvt.u8.u32 b, %1;\n cvt.rn.f16x2.e2m1x2 %0, b;\n}"
            : "=r"(h) : "r"((w >> (8 * i)) & 255u));
        float lo, hi;
        elems::widen2<F16>(h, lo, hi);
        f[2 * i] = __fmul_rn(lo, s);
        f[2 * i + 1] = __fmul_rn(hi, s);
    }
}

// A warp takes R rows' 256 columns of a record, all read before any is
// written; 8 elements of a row a lane.  R divides 128.
template <int DT, bool VEC, int R>
__global__ void __launch_bounds__(kThreads)
mx4_values_kernel(const __grid_constant__ MxDequantArgs a, int64_t kt)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t task = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t row0 = task / kt * R, t = task % kt;
    const int64_t c = t * kMxCols;
    if (row0 >= a.rows) return;
    const unsigned char *rec = a.q + ((row0 / kMxRows) * kt + t) * kMxRecord;
    const int r0 = (int)(row0 % kMxRows);
    uint32_t w[R], scale[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const int r = r0 + j;
        if (row0 + j < a.rows) {
            w[j] = *reinterpret_cast<const uint32_t *>(
                rec + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
            scale[j] = rec[scale_at(r, lane >> 2)];
        }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
        if (row0 + j >= a.rows) break;
        float f[8];
        values8(w[j], scale[j], f);
        const int64_t at = (row0 + j) * a.stride + c;
        elems::Raw<DT> o;
        o.set(f);
        if (!VEC) o.store_any(a.out, at, a.cols - c < kMxCols ? (int)(a.cols - c) : kMxCols);
        else if (c + lane * 8 < a.cols) o.store(a.out, at + lane * 8);
    }
}

template <int DT, bool VEC> cudaError_t dequant_go(const MxDequantArgs &a, int sms, cudaStream_t s)
{
    const int64_t kt = (a.cols + kMxCols - 1) / kMxCols;
    // an fp32 row is long enough to keep its warp busy: 27 us against 34 of four
    // rows for 8192 x 4096
    const bool many = DT != F32 && a.rows * kt >= (int64_t)sms * 64;
    const int64_t warps = (many ? (a.rows + 3) / 4 : a.rows) * kt;
    const int threads = warps <= 1024 ? 32 : kThreads;
    const int64_t blocks = (warps * 32 + threads - 1) / threads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block((unsigned)threads);
    return many ? launch_dependent(mx4_values_kernel<DT, VEC, 4>, grid, block, 0, s, a, kt)
                : launch_dependent(mx4_values_kernel<DT, VEC, 1>, grid, block, 0, s, a, kt);
}

template <int DT> cudaError_t dequant_pick(const MxDequantArgs &a, int sms, cudaStream_t s)
{
    return rows_aligned(a.out, a.stride, DT, a.cols) ? dequant_go<DT, true>(a, sms, s)
                                                     : dequant_go<DT, false>(a, sms, s);
}

}  // namespace

cudaError_t launch_mx4_quantize(int32_t dt, const MxQuantArgs &a, int sms, cudaStream_t s)
{
    if (a.rows <= 0 || a.cols <= 0 || (!a.q && !a.qt)) return cudaSuccess;
    return dt == F32 ? quant_pick<F32>(a, sms, s)
                     : dt == BF16 ? quant_pick<BF16>(a, sms, s) : quant_pick<F16>(a, sms, s);
}

cudaError_t launch_mx4_dequantize(int32_t dt, const MxDequantArgs &a, int sms, cudaStream_t s)
{
    if (a.rows <= 0 || a.cols <= 0) return cudaSuccess;
    return dt == F32 ? dequant_pick<F32>(a, sms, s) : dt == BF16 ? dequant_pick<BF16>(a, sms, s)
                                                            : dequant_pick<F16>(a, sms, s);
}

}  // namespace zgb
