// Internal interface between the training operators' C ABI (zero_ops_abi.cu)
// and their kernels (zero_embed.cu, zero_dropout.cu, zero_mx4.cu,
// zero_mx4_matmul.cu).  Element types are the DType codes of
// zero_internal.h; every launcher returns a cudaError_t and launches on `s`.
#pragma once

#include <atomic>

#include "zero_internal.h"

namespace zgb {

// Lets `kernel` use so much dynamic shared memory, once a device: `done` has a
// bit for each (of the first 64).
inline cudaError_t allow_shared(const void *kernel, int bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Whether all rows of a matrix begin on a boundary of 8 elements and hold whole
// eights (zero_elems.cuh: VEC).
inline bool rows_aligned(const void *p, int64_t stride, int32_t dt, int64_t width)
{
    const int b = 8 * elem_size(dt);
    return ((uintptr_t)p % (uintptr_t)b) == 0 && stride % 8 == 0 && width % 8 == 0;
}

// ---- embedding

struct TokenArgs {
    const void *ids;
    int32_t wide;        // 64-bit ids, else 32-bit
    int64_t n;
    int64_t pad;         // this id names no row
    int64_t rows;        // ids outside [0, rows) name no row either
};

struct EmbedArgs {
    TokenArgs tok;
    const void *table;
    int64_t dim, table_stride, out_stride;
    float scale;
    void *out;
    unsigned long long *bad;     // += ids outside the table that are not `pad`, -1 always (or null)
};
cudaError_t launch_embed(int32_t dt, const EmbedArgs &a, cudaStream_t s);

struct EmbedGradArgs {
    TokenArgs tok;
    const void *dy;
    int64_t dim, dy_stride, grad_stride;
    float scale;
    void *grad;
    int32_t accumulate;
    // workspace (embed_grad_layout)
    uint32_t *key[2], *idx[2];   // ids and positions, the sort's two sides
    uint32_t *hist;              // [pass][sort blocks][256]
    uint32_t *n_runs;            // runs of one id that pass the end of a chunk
    uint32_t *runs;              // the chunk each begins in
    float *part;                 // [chunk][2][columns rounded up to 256]
};
// Places the workspace's arrays from `base` on (may be null) and returns
// their bytes.
int64_t embed_grad_layout(EmbedGradArgs &a, char *base);
cudaError_t launch_embed_grad(int32_t ydt, int32_t gdt, const EmbedGradArgs &a, int sms,
                              cudaStream_t s);

// ---- dropout

struct DropoutArgs {
    const void *x, *residual;
    void *out;
    int64_t n;
    uint32_t threshold;             // keep where the word >= threshold
    int32_t all;                    // p = 1: drop everything
    float up;                       // 1 / (1 - p)
    uint32_t key0[10], key1[10];    // the rounds' keys
    uint32_t off0, off1;
    // What the first two rounds make of the offset alone, for counters below
    // 2^32 (zero_dropout.cu)
    uint32_t pre[4];
    unsigned long long first;       // counter of element 0 (first element / 4)
};
cudaError_t launch_dropout(int32_t dt, const DropoutArgs &a, cudaStream_t s);

// ---- microscaled 4-bit matrices
//
// A matrix of R rows by C columns is ceil(R/128) by ceil(C/256) records,
// row-major, each of kMxRecord bytes: 128 rows of 128 bytes of codes (column
// 2b in the low and 2b + 1 in the high half of byte b; the 16-byte piece p
// of row r lies at piece p ^ (r & 7)), then 1024 bytes of scale exponents,
// the one of row r and block b (of 32 columns) at
// (b / 4) * 512 + (r % 32) * 16 + (r / 32) * 4 + b % 4.
constexpr int kMxRows = 128, kMxCols = 256, kMxBlock = 32;
constexpr int kMxCodes = kMxRows * kMxCols / 2;
constexpr int kMxScales = kMxRows * kMxCols / kMxBlock;
constexpr int kMxRecord = kMxCodes + kMxScales;

struct MxQuantArgs {
    const void *x;
    int64_t rows, cols, stride;
    unsigned char *q, *qt;       // either may be null
};
cudaError_t launch_mx4_quantize(int32_t dt, const MxQuantArgs &a, int sms, cudaStream_t s);

struct MxDequantArgs {
    const unsigned char *q;
    int64_t rows, cols, stride;
    void *out;
};
cudaError_t launch_mx4_dequantize(int32_t dt, const MxDequantArgs &a, int sms, cudaStream_t s);

struct MxMatmulArgs {
    const unsigned char *a, *b;  // [m, k] and [n, k]
    int64_t m, n, k;
    float alpha;
    int32_t accumulate;
    void *out;                   // [m, n]
    int64_t stride;
};
cudaError_t launch_mx4_matmul(int32_t dt, const MxMatmulArgs &a, int sms, cudaStream_t s);
cudaError_t mx4_timeouts(unsigned int *count);

}  // namespace zgb
