// Internal interface between the training operators' C ABI (zero_ops_abi.cu)
// and their kernels (zero_embed.cu, zero_dropout.cu, zero_mx4.cu,
// zero_mx4_matmul.cu, zero_matmul.cu, zero_norm.cu, zero_activation.cu).  Element
// types are the DType codes of zero_internal.h; every launcher returns a
// cudaError_t and launches on `s`.
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

// ---- products of 16-bit matrices
//
// out = act(A B^T (+ A2 B2^T) + bias) + residual, or, gated, act(A B^T) * (A B2^T).
struct ProductArgs {
    const void *a, *b, *a2, *b2;           // a2, b2 may be null; gated: b2 alone is given
    int64_t a_stride, b_stride, a2_stride, b2_stride;
    int32_t a_cols, b_cols;                // the matrix lies as its transpose, k by m or n
    int32_t gated, act;                    // act: zero_act.cuh
    int64_t m, n, k;
    const void *bias, *residual;           // [n] of the operands' type, [m, n] of the result's
    int64_t residual_stride;
    // what the backward pass needs: the sums with the bias in the operands' type, or
    // packed (zero_pack8.cuh); kept2 the gated block's second ones
    void *kept, *kept2;
    int64_t kept_stride;
    unsigned char *kept_q, *kept2_q;
    void *out;                             // [m, n]
    int64_t stride;
};
// Bytes for the operands whose rows are not on 16-byte boundaries.
int64_t product_workspace(const ProductArgs &a);
cudaError_t launch_product(int32_t dt, int32_t odt, ProductArgs a, void *workspace, int sms,
                           cudaStream_t s);
cudaError_t matmul_timeouts(unsigned int *count);

// ---- the norm (dt of all matrices and the weight; gradients of wdt)
struct NormArgs {
    const void *x, *residual, *weight;     // residual may be null
    int64_t rows, dim, x_stride, residual_stride;
    float eps;
    void *sum, *y;                         // either may be null
    int64_t sum_stride, y_stride;
    unsigned char *q;                      // y packed, or null
    float *rstd;                           // [rows], or null
};
cudaError_t launch_norm(int32_t dt, const NormArgs &a, int sms, cudaStream_t s);

struct NormGradArgs {
    const void *dy, *ds, *sum, *weight;    // ds may be null
    const float *rstd;
    int64_t rows, dim, dy_stride, ds_stride, sum_stride;
    void *dx, *dweight;                    // dweight may be null
    int64_t dx_stride;
    int32_t accumulate;                    // dweight
};
int64_t norm_grad_workspace(int64_t rows, int64_t dim);
cudaError_t launch_norm_grad(int32_t dt, int32_t wdt, const NormGradArgs &a, float *workspace,
                             cudaStream_t s);

// ---- through activations; z, g, u in the type or packed (one of the two is given)
struct ActGradArgs {
    const void *dy, *kept;
    unsigned char *kept_q;
    int64_t rows, cols, dy_stride, kept_stride;
    int32_t act;
    void *dz, *dbias;                      // either may be null
    int64_t dz_stride;
    int32_t accumulate;                    // dbias
};
int64_t activation_grad_workspace(int64_t rows, int64_t cols);
cudaError_t launch_activation_grad(int32_t dt, int32_t bdt, const ActGradArgs &a, float *workspace,
                                   cudaStream_t s);

struct GatedGradArgs {
    const void *dh, *gate, *up;
    unsigned char *gate_q, *up_q;
    int64_t rows, cols, dh_stride, kept_stride;
    int32_t act;
    void *dgate, *dup, *h;                 // h may be null
    int64_t grad_stride, h_stride;
};
cudaError_t launch_gated_grad(int32_t dt, const GatedGradArgs &a, cudaStream_t s);

// ---- rows in 8 bits (zero_pack8.cuh)
int64_t pack8_bytes(int64_t rows, int64_t cols);
cudaError_t launch_pack8(int32_t dt, const void *x, int64_t rows, int64_t cols, int64_t stride,
                         unsigned char *q, cudaStream_t s);
cudaError_t launch_unpack8(int32_t dt, const unsigned char *q, int64_t rows, int64_t cols,
                           void *out, int64_t stride, cudaStream_t s);

}  // namespace zgb
