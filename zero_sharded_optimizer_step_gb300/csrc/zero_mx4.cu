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

// Two floats to two E2M1 codes, `lo` in the low half of the byte.
__device__ __forceinline__ uint32_t codes2(float lo, float hi)
{
    uint32_t r;
    asm("{\n .reg .b8 b;\n cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n cvt.u32.u8 %0, b;\n}"
        : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float inv)
{
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w |= codes2(__fmul_rn(x[2 * i], inv), __fmul_rn(x[2 * i + 1], inv)) << (8 * i);
    return w;
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

// 8 consecutive elements from column c of a row, zeros past the row's end.
template <int DT, int E>
__device__ __forceinline__ void load8(const void *x, int64_t at, int64_t c, int64_t cols,
                                      float (&f)[8])
{
    if constexpr (E == 8) {
        elems::Raw<DT, 8> r;
        r.zero();
        if (c < cols) r.load(x, at + c);
        r.get(f);
    } else {
#pragma unroll
        for (int j = 0; j < 8 / E; ++j) {
            elems::Raw<DT, E> r;
            float g[E];
            r.zero();
            if (c + j * E < cols) r.load(x, at + c + j * E);
            r.get(g);
#pragma unroll
            for (int e = 0; e < E; ++e) f[j * E + e] = g[e];
        }
    }
}

// A warp quantises one row's 256 columns of a record: 8 elements a lane, a
// block over 4 lanes.
template <int DT, int E>
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
    load8<DT, E>(a.x, row * a.stride, t * kMxCols + lane * 8, a.cols, x);
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
template <int DT, int E>
__global__ void __launch_bounds__(kThreads)
mx4_both_kernel(const __grid_constant__ MxQuantArgs a, int64_t kt, int64_t ktt)
{
    using T = typename elems::El<DT>::T;
    __shared__ __align__(16) T strip[32][kMxCols + 8];
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
    for (int s = 0; s < 4; ++s) {
        float x[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t row = r0 + s * 32 + warp * 4 + j;
            if (row < a.rows) {
                load8<DT, E>(a.x, row * a.stride, c0 + lane * 8, a.cols, x[j]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[j][e] = 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            elems::Raw<DT, 8> raw;
            raw.set(x[j]);
            raw.store(&strip[warp * 4 + j][0], lane * 8);
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
                    y[g][e] = elems::load1<DT>(&strip[g * 8 + e][0], threadIdx.x);
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

template <int DT, int E> cudaError_t quant_go(const MxQuantArgs &a, cudaStream_t s)
{
    const int64_t kt = (a.cols + kMxCols - 1) / kMxCols;
    if (!a.qt) {
        const int64_t warps = a.rows * kt;
        const int threads = warps <= 1024 ? 32 : kThreads;
        const int64_t blocks = (warps * 32 + threads - 1) / threads;
        if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
        return launch_dependent(mx4_rows_kernel<DT, E>, dim3((unsigned)blocks),
                                dim3((unsigned)threads), 0, s, a, kt);
    }
    const int64_t ktt = (a.rows + kMxCols - 1) / kMxCols;
    const int64_t blocks = kt * ktt * 2;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_dependent(mx4_both_kernel<DT, E>, dim3((unsigned)blocks), dim3(kThreads), 0, s,
                            a, kt, ktt);
}

template <int DT> cudaError_t quant_pick(const MxQuantArgs &a, cudaStream_t s)
{
    const int e = row_access(a.x, a.stride, DT == F32 ? 4 : 2, a.cols);
    return e == 8 ? quant_go<DT, 8>(a, s) : e == 2 ? quant_go<DT, 2>(a, s) : quant_go<DT, 1>(a, s);
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

template <int DT, int E>
__global__ void __launch_bounds__(kThreads)
mx4_values_kernel(const __grid_constant__ MxDequantArgs a, int64_t kt)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t task = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t row = task / kt, t = task - row * kt;
    if (row >= a.rows) return;
    const unsigned char *rec = a.q + ((row / kMxRows) * kt + t) * kMxRecord;
    const int r = (int)(row % kMxRows);
    const int64_t c = t * kMxCols + lane * 8;
    if (c >= a.cols) return;
    const uint32_t w = *reinterpret_cast<const uint32_t *>(
        rec + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
    float f[8];
    values8(w, rec[scale_at(r, lane >> 2)], f);
#pragma unroll
    for (int j = 0; j < 8 / E; ++j) {
        if (c + j * E >= a.cols) break;
        elems::Raw<DT, E> o;
        float g[E];
#pragma unroll
        for (int e = 0; e < E; ++e) g[e] = f[j * E + e];
        o.set(g);
        o.store(a.out, row * a.stride + c + j * E);
    }
}

template <int DT, int E> cudaError_t dequant_go(const MxDequantArgs &a, cudaStream_t s)
{
    const int64_t kt = (a.cols + kMxCols - 1) / kMxCols;
    const int64_t warps = a.rows * kt;
    const int threads = warps <= 1024 ? 32 : kThreads;
    const int64_t blocks = (warps * 32 + threads - 1) / threads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_dependent(mx4_values_kernel<DT, E>, dim3((unsigned)blocks),
                            dim3((unsigned)threads), 0, s, a, kt);
}

template <int DT> cudaError_t dequant_pick(const MxDequantArgs &a, cudaStream_t s)
{
    const int e = row_access(a.out, a.stride, DT == F32 ? 4 : 2, a.cols);
    return e == 8 ? dequant_go<DT, 8>(a, s)
                  : e == 2 ? dequant_go<DT, 2>(a, s) : dequant_go<DT, 1>(a, s);
}

}  // namespace

cudaError_t launch_mx4_quantize(int32_t dt, const MxQuantArgs &a, int, cudaStream_t s)
{
    if (a.rows <= 0 || a.cols <= 0 || (!a.q && !a.qt)) return cudaSuccess;
    return dt == F32 ? quant_pick<F32>(a, s) : dt == BF16 ? quant_pick<BF16>(a, s)
                                                          : quant_pick<F16>(a, s);
}

cudaError_t launch_mx4_dequantize(int32_t dt, const MxDequantArgs &a, cudaStream_t s)
{
    if (a.rows <= 0 || a.cols <= 0) return cudaSuccess;
    return dt == F32 ? dequant_pick<F32>(a, s) : dt == BF16 ? dequant_pick<BF16>(a, s)
                                                            : dequant_pick<F16>(a, s);
}

}  // namespace zgb
