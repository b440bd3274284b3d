// The root-mean-square norm with the residual's addition, and its gradient.
//
//   s = T(x + r), rstd = 1 / sqrt(mean of s^2 + eps), y = s rstd w
//   dx = ds + rstd (w dy - n mean(w dy n)), dw = sum over rows of dy n, n = s rstd
//
// A row's elements stay in registers between the sum and the result, so that
// every matrix is read or written once.  One to eight warps share a row; sums
// are in fp32, in an order that depends on the sizes alone.
//
// What bounds it: memory.  16384 x 4096 in bf16 with a residual, both ways: 1.07 GB in
// 170 us, 6.3 TB/s.  Few rows are a launch's time: 333 x 1600 5.2 us.
#include "zero_ops.h"
#include "zero_pack8.cuh"
#include "zero_rows.cuh"

namespace zgb {
namespace {

constexpr int kWarps = kThreads / 32;

struct Norm {
    rows::In x, residual, w;
    int64_t n, dim;
    float eps;
    void *sum, *y;
    int64_t sum_stride, y_stride;
    unsigned char *q;
    float *rstd;
};

// The sum over the W warps of a row, the same in all of them.
template <int W> __device__ __forceinline__ float row_sum(float v, float *shared)
{
    v = rows::warp_sum(v);
    if constexpr (W == 1) return v;
    const int warp = threadIdx.x >> 5;
    __syncthreads();                             // the sum before has been read
    if ((threadIdx.x & 31) == 0) shared[warp] = v;
    __syncthreads();
    const int first = warp / W * W;
    v = shared[first];
#pragma unroll
    for (int i = 1; i < W; ++i) v = __fadd_rn(v, shared[first + i]);
    return v;
}

// 1 / sqrt(v) in two floats: the nearest one, and what it is off by, from v r^2 - 1,
// whose first terms are exact.  An element's product with the weight is exact too (16-bit
// types), so that the norm is off by little more than its last rounding: what is
// packed goes to the code that it should but next to a border.
struct Rstd {
    float hi, lo;
};

__device__ __forceinline__ Rstd rstd_of(float squares, int64_t dim, float eps)
{
    const float v = __fadd_rn(__fdiv_rn(squares, (float)dim), eps);
    const float r = __frcp_rn(__fsqrt_rn(v)), t = __fmul_rn(v, r);
    const float off = __fmaf_rn(-__fmaf_rn(v, r, -t), r, __fmaf_rn(-t, r, 1.0f));
    const float lo = __fmul_rn(__fmul_rn(0.5f, r), off);
    return {r, fabsf(lo) < r ? lo : 0.0f};       // (v of 0, infinity or NaN: r alone says it)
}

// x + r rounded to the type, as it is kept.
template <int DT, bool VEC>
__device__ __forceinline__ void total(bool add, const rows::Eight<DT, VEC> &x,
                                      const rows::Eight<DT, VEC> &r, float (&s)[8])
{
    x.take(s);
    if (add) {
        float f[8];
        r.take(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = __fadd_rn(s[e], f[e]);
        elems::Raw<DT> v;
        v.set(s);
        v.get(s);
    }
}

template <int DT, bool VEC>
__device__ __forceinline__ void finish(const Norm &a, int64_t row, int64_t c0, Rstd rstd,
                                       const rows::Eight<DT, VEC> &weight, float *turned,
                                       float (&s)[8])
{
    float w[8];
    weight.take(w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float p = __fmul_rn(s[e], w[e]);
        s[e] = __fmaf_rn(p, rstd.hi, __fmul_rn(p, rstd.lo));
    }
    if (a.y) rows::put<DT, VEC>(a.y, a.y_stride, row, c0, a.dim, s);
    if (!a.q) return;
#pragma unroll
    for (int e = 0; e < 8; ++e)                  // (0 times a NaN or infinite rstd is not 0)
        if (c0 + rows::column<VEC>(e) >= a.dim) s[e] = 0.0f;
    rows::pack<VEC>(pack8::view(a.q, a.n, a.dim), row, c0, turned, s);
}

// Rows of up to W * G * 256 elements.
template <int DT, int W, int G, bool VEC>
__global__ void __launch_bounds__(kThreads)
norm_kernel(const __grid_constant__ Norm a)
{
    constexpr bool kCut = !VEC || G == 4;        // wide steps: runs past the row are left out
    __shared__ float shared[kWarps], turned[VEC ? 1 : kWarps][256];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * (kWarps / W) + warp / W;
    const int64_t first = (int64_t)(warp % W) * 256;         // and every W-th run
    const bool live = row < a.n;
    rows::Eight<DT, VEC> x[G], r[G], w[G];
    if (live) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (kCut && first + g * (W * 256) >= a.dim) break;       // no run of the row's left
            x[g].ask(a.x, row, first + g * (W * 256), a.dim);
            if (a.residual.p) r[g].ask(a.residual, row, first + g * (W * 256), a.dim);
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (kCut && first + g * (W * 256) >= a.dim) break;
            w[g].ask(a.w, 0, first + g * (W * 256), a.dim);
        }
    }
    float s[G][8], squares = 0.0f;
    if (live) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (kCut && first + g * (W * 256) >= a.dim) break;
            total<DT, VEC>(a.residual.p != nullptr, x[g], r[g], s[g]);
            if (a.sum)
                rows::put<DT, VEC>(a.sum, a.sum_stride, row, first + g * (W * 256), a.dim, s[g]);
#pragma unroll
            for (int e = 0; e < 8; ++e) squares = __fmaf_rn(s[g][e], s[g][e], squares);
        }
    }
    const Rstd rstd = rstd_of(row_sum<W>(squares, shared), a.dim, a.eps);
    if (!live) return;
    if (a.rstd && warp % W == 0 && (threadIdx.x & 31) == 0) a.rstd[row] = rstd.hi;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        if (kCut && first + g * (W * 256) >= a.dim) break;
        finish<DT, VEC>(a, row, first + g * (W * 256), rstd, w[g], turned[VEC ? 0 : warp], s[g]);
    }
}

// Longer rows, a block each: the elements are read again for the result, from L2 as far
// as the rows at work at one time fit there.  (4096 x 16384 in bf16 49 us, 40 of them the
// bytes of one reading; 4096 x 12000 41 and 29.)
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
norm_long_kernel(const __grid_constant__ Norm a)
{
    __shared__ float shared[kWarps], turned[VEC ? 1 : kWarps][256];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x, first = (int64_t)(threadIdx.x >> 5) * 256;
    float squares = 0.0f, s[8];
    rows::Eight<DT, VEC> x, r, w;
    for (int64_t c0 = first; c0 < a.dim; c0 += kWarps * 256) {
        x.ask(a.x, row, c0, a.dim);
        if (a.residual.p) r.ask(a.residual, row, c0, a.dim);
        total<DT, VEC>(a.residual.p != nullptr, x, r, s);
        // (sum may be residual: its rows are read again below from there)
        if (a.sum) rows::put<DT, VEC>(a.sum, a.sum_stride, row, c0, a.dim, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) squares = __fmaf_rn(s[e], s[e], squares);
    }
    const Rstd rstd = rstd_of(row_sum<kWarps>(squares, shared), a.dim, a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd.hi;
    __syncwarp();
    const bool again = !a.sum && a.residual.p;   // the sum was not stored: it is made again
    const rows::In from = a.sum ? rows::In{a.sum, a.sum_stride} : a.x;
    for (int64_t c0 = first; c0 < a.dim; c0 += kWarps * 256) {
        x.ask(from, row, c0, a.dim);
        if (again) r.ask(a.residual, row, c0, a.dim);
        w.ask(a.w, 0, c0, a.dim);
        total<DT, VEC>(again, x, r, s);
        finish<DT, VEC>(a, row, c0, rstd, w, turned[VEC ? 0 : threadIdx.x >> 5], s);
    }
}

template <int DT, int W, int G, bool VEC> cudaError_t norm_go(const Norm &a, cudaStream_t s)
{
    const int64_t blocks = (a.n + kWarps / W - 1) / (kWarps / W);
    return launch_dependent(norm_kernel<DT, W, G, VEC>, dim3((unsigned)blocks), dim3(kThreads), 0,
                            s, a);
}

// Rows that a warp holds go a warp each, as long as that fills the SMs; few or
// longer ones a block each.
template <int DT, bool VEC> cudaError_t norm_pick(const Norm &a, int sms, cudaStream_t s)
{
    if (a.dim > 8192)
        return launch_dependent(norm_long_kernel<DT, VEC>, dim3((unsigned)a.n), dim3(kThreads), 0,
                                s, a);
    if (a.n >= (int64_t)sms * 16) {
        if (a.dim <= 256) return norm_go<DT, 1, 1, VEC>(a, s);
        if (a.dim <= 1024) return norm_go<DT, 1, 4, VEC>(a, s);
        if (a.dim <= 4096 && a.dim > 2048) return norm_go<DT, 4, 4, VEC>(a, s);
    }
    if (a.dim <= 2048) return norm_go<DT, 8, 1, VEC>(a, s);
    if (a.dim <= 4096) return norm_go<DT, 8, 2, VEC>(a, s);
    return norm_go<DT, 8, 4, VEC>(a, s);
}

// ----------------------------------------------------------------- the gradient

struct NormGrad {
    rows::In dy, ds, s, w;
    const float *rstd;
    int64_t n, dim;
    void *dx;
    int64_t dx_stride;
    float *parts;                                // [blocks][dim], or null
};

// Whether runs past the row are left out step by step: fp32 rows gain (8192 x 4096 112 to
// 91 us), 16-bit ones lose by the branches (16384 x 4096 both ways 167 to 195).
template <int DT> constexpr bool kCut = DT == F32;

// A row's three matrices, a thread's share.
template <int DT, int W, int G, bool VEC> struct GradRow {
    rows::Eight<DT, VEC> dy[G], s[G], ds[G];
    float rstd;

    __device__ __forceinline__ void ask(const NormGrad &a, int64_t row, int64_t first)
    {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (kCut<DT> && first + g * (W * 256) >= a.dim) break;       // no run of the row's left
            dy[g].ask(a.dy, row, first + g * (W * 256), a.dim);
            s[g].ask(a.s, row, first + g * (W * 256), a.dim);
            if (a.ds.p) ds[g].ask(a.ds, row, first + g * (W * 256), a.dim);
        }
        rstd = a.rstd[row];
    }
};

// Groups of W warps stride over the rows, the next row on its way while one is worked
// on (without that, both ways of 16384 x 4096 took 195 us for 167); a thread adds up
// its columns' part of dw in registers, and the block's groups join theirs at the end.
template <int DT, int W, int G, bool VEC>
__global__ void __launch_bounds__(W > 8 ? W * 32 : kThreads)
norm_grad_kernel(const __grid_constant__ NormGrad a)
{
    constexpr int kAll = W > 8 ? W : 8, kGroups = kAll / W;
    __shared__ float shared[2][kAll];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = warp / W;
    const int64_t first = (int64_t)(warp % W) * 256;         // and every W-th run
    const float inv_dim = __fdiv_rn(1.0f, (float)a.dim);
    float dw[G][8];
    rows::Eight<DT, VEC> we[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        we[g].ask(a.w, 0, first + g * (W * 256), a.dim);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[g][e] = 0.0f;
    }
    const int64_t step = (int64_t)gridDim.x * kGroups;
    int64_t row = (int64_t)blockIdx.x * kGroups + group;
    GradRow<DT, W, G, VEC> now, next;
    if (row < a.n) now.ask(a, row, first);
    for (int turn = 0; row < a.n; row += step, turn ^= 1) {
        if (row + step < a.n) next.ask(a, row + step, first);
        const float rstd = now.rstd;
        float share = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (kCut<DT> && first + g * (W * 256) >= a.dim) break;
            float dy[8], n[8], w[8];
            now.dy[g].take(dy);
            now.s[g].take(n);
            we[g].take(w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                n[e] = __fmul_rn(n[e], rstd);
                dw[g][e] = __fmaf_rn(dy[e], n[e], dw[g][e]);
                share = __fmaf_rn(__fmul_rn(dy[e], w[e]), n[e], share);
            }
        }
        share = rows::warp_sum(share);
        if constexpr (W > 1) {
            // (two rows' sums in turn: one barrier of the group a row is enough)
            if (lane == 0) shared[turn][warp] = share;
            __syncwarp();                        // (the barrier wants it converged)
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(W * 32) : "memory");
            share = shared[turn][group * W];
#pragma unroll
            for (int i = 1; i < W; ++i) share = __fadd_rn(share, shared[turn][group * W + i]);
        }
        share = __fmul_rn(share, inv_dim);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (kCut<DT> && first + g * (W * 256) >= a.dim) break;
            float dy[8], n[8], w[8], d[8];
            now.dy[g].take(dy);
            now.s[g].take(n);
            we[g].take(w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                n[e] = __fmul_rn(n[e], rstd);
                d[e] = __fmul_rn(rstd, __fmaf_rn(-n[e], share, __fmul_rn(dy[e], w[e])));
            }
            if (a.ds.p) {
                float f[8];
                now.ds[g].take(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = __fadd_rn(d[e], f[e]);
            }
            rows::put<DT, VEC>(a.dx, a.dx_stride, row, first + g * (W * 256), a.dim, d);
        }
        now = next;
    }
    if (!a.parts) return;
    float *part = a.parts + (int64_t)blockIdx.x * a.dim;
    if constexpr (kGroups == 1) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t c = first + g * (W * 256) + rows::column<VEC>(e);
                if (c < a.dim) part[c] = dw[g][e];
            }
    } else {
        __shared__ float joined[kGroups * W * G * 256];
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                joined[group * (W * G * 256) + (int)first + g * (W * 256) + rows::column<VEC>(e)] = dw[g][e];
        __syncthreads();
        for (int c = threadIdx.x; c < a.dim; c += kThreads) {
            float v = joined[c];
#pragma unroll
            for (int i = 1; i < kGroups; ++i) v = __fadd_rn(v, joined[i * (W * G * 256) + c]);
            part[c] = v;
        }
    }
}

// Rows of more than 8192 elements: dx by a block a row, which reads it twice ...
// (4096 x 16384 in bf16, both kernels, 130 us, 60 of them the bytes of one reading)
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
norm_grad_long_kernel(const __grid_constant__ NormGrad a)
{
    __shared__ float shared[kWarps];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x, first = (int64_t)(threadIdx.x >> 5) * 256;
    const float rstd = a.rstd[row];
    float share = 0.0f;
    rows::Eight<DT, VEC> dye, se, we, dse;
    float dy[8], n[8], w[8], d[8];
    for (int64_t c0 = first; c0 < a.dim; c0 += kWarps * 256) {
        dye.ask(a.dy, row, c0, a.dim);
        se.ask(a.s, row, c0, a.dim);
        we.ask(a.w, 0, c0, a.dim);
        dye.take(dy);
        se.take(n);
        we.take(w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            share = __fmaf_rn(__fmul_rn(dy[e], w[e]), __fmul_rn(n[e], rstd), share);
    }
    share = __fdiv_rn(row_sum<kWarps>(share, shared), (float)a.dim);
    for (int64_t c0 = first; c0 < a.dim; c0 += kWarps * 256) {
        dye.ask(a.dy, row, c0, a.dim);
        se.ask(a.s, row, c0, a.dim);
        we.ask(a.w, 0, c0, a.dim);
        if (a.ds.p) dse.ask(a.ds, row, c0, a.dim);
        dye.take(dy);
        se.take(n);
        we.take(w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            n[e] = __fmul_rn(n[e], rstd);
            d[e] = __fmul_rn(rstd, __fmaf_rn(-n[e], share, __fmul_rn(dy[e], w[e])));
        }
        if (a.ds.p) {
            dse.take(w);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = __fadd_rn(d[e], w[e]);
        }
        rows::put<DT, VEC>(a.dx, a.dx_stride, row, c0, a.dim, d);
    }
}

// ... and dw by strips of 256 columns, a share of the rows each block.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
norm_grad_strips_kernel(const __grid_constant__ NormGrad a)
{
    __shared__ float joined[kWarps][256];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5;
    const int64_t c0 = (int64_t)blockIdx.x * 256;
    float dw[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int64_t r = (int64_t)blockIdx.y * kWarps + warp; r < a.n; r += (int64_t)gridDim.y * kWarps) {
        rows::Eight<DT, VEC> dye, se;
        float dy[8], n[8];
        dye.ask(a.dy, r, c0, a.dim);
        se.ask(a.s, r, c0, a.dim);
        const float rstd = a.rstd[r];
        dye.take(dy);
        se.take(n);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] = __fmaf_rn(dy[e], __fmul_rn(n[e], rstd), dw[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) joined[warp][rows::column<VEC>(e)] = dw[e];
    __syncthreads();
    const int64_t c = c0 + threadIdx.x;
    if (c < a.dim) {
        float v = joined[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) v = __fadd_rn(v, joined[i][threadIdx.x]);
        a.parts[(int64_t)blockIdx.y * a.dim + c] = v;
    }
}

constexpr int kMostBlocks = 304;                 // two on each of 152 SMs
constexpr int kStripParts = 16;

// Warps that share a row of this width, 512 elements each (768 alone in a warp).
int row_warps(int64_t dim)
{
    return dim <= 768 ? 1 : dim <= 1024 ? 2 : dim <= 2048 ? 4 : dim <= 4096 ? 8 : 16;
}

template <int DT, int W, int G, bool VEC>
cudaError_t grad_go(const NormGrad &a, int64_t parts, cudaStream_t s)
{
    return launch_dependent(norm_grad_kernel<DT, W, G, VEC>, dim3((unsigned)parts),
                            dim3(W > 8 ? W * 32 : kThreads), 0, s, a);
}

template <int DT, bool VEC>
cudaError_t grad_pick(const NormGrad &a, int64_t parts, cudaStream_t s)
{
    if (a.dim > 8192) {
        cudaError_t e = launch_dependent(norm_grad_long_kernel<DT, VEC>, dim3((unsigned)a.n),
                                         dim3(kThreads), 0, s, a);
        if (e != cudaSuccess || !a.parts) return e;
        return launch_dependent(norm_grad_strips_kernel<DT, VEC>,
                                dim3((unsigned)((a.dim + 255) / 256), (unsigned)parts),
                                dim3(kThreads), 0, s, a);
    }
    if (a.dim <= 256) return grad_go<DT, 1, 1, VEC>(a, parts, s);
    if (a.dim <= 512) return grad_go<DT, 1, 2, VEC>(a, parts, s);
    if (a.dim <= 768) return grad_go<DT, 1, 3, VEC>(a, parts, s);
    if (a.dim <= 1024) return grad_go<DT, 2, 2, VEC>(a, parts, s);
    if (a.dim <= 2048) return grad_go<DT, 4, 2, VEC>(a, parts, s);
    if (a.dim <= 4096) return grad_go<DT, 8, 2, VEC>(a, parts, s);
    return grad_go<DT, 16, 2, VEC>(a, parts, s);
}

int64_t norm_parts(int64_t n, int64_t dim)
{
    if (dim > 8192) return (n + 7) / 8 < kStripParts ? (n + 7) / 8 : kStripParts;
    const int64_t warps = row_warps(dim), groups = warps < kWarps ? kWarps / warps : 1;
    const int64_t blocks = (n + groups - 1) / groups;
    return blocks < kMostBlocks ? blocks : kMostBlocks;
}

}  // namespace

cudaError_t launch_norm(int32_t dt, const NormArgs &a, int sms, cudaStream_t s)
{
    if (a.rows <= 0 || a.dim <= 0) return cudaSuccess;
    Norm n = {rows::in(a.x, a.x_stride),
              rows::in(a.residual, a.residual_stride),
              rows::in(a.weight, a.dim),
              a.rows, a.dim, a.eps, a.sum, a.y, a.sum_stride, a.y_stride, a.q, a.rstd};
    const bool vec = rows_aligned(a.x, a.x_stride, dt, a.dim) &&
                     rows_aligned(a.weight, 0, dt, a.dim) &&
                     (!a.residual || rows_aligned(a.residual, a.residual_stride, dt, a.dim)) &&
                     (!a.sum || rows_aligned(a.sum, a.sum_stride, dt, a.dim)) &&
                     (!a.y || rows_aligned(a.y, a.y_stride, dt, a.dim));
    auto go = [&](auto t) {
        constexpr int DT = decltype(t)::value;
        return vec ? norm_pick<DT, true>(n, sms, s) : norm_pick<DT, false>(n, sms, s);
    };
    return dt == F32 ? go(std::integral_constant<int, F32>{})
           : dt == BF16 ? go(std::integral_constant<int, BF16>{})
                        : go(std::integral_constant<int, F16>{});
}

int64_t norm_grad_workspace(int64_t rows, int64_t dim)
{
    return norm_parts(rows, dim) * dim * 4;
}

cudaError_t launch_norm_grad(int32_t dt, int32_t wdt, const NormGradArgs &a, float *workspace,
                             cudaStream_t s)
{
    if (a.dim <= 0) return cudaSuccess;
    const int64_t parts = norm_parts(a.rows, a.dim);
    if (a.rows > 0) {
        NormGrad n = {rows::in(a.dy, a.dy_stride),
                      rows::in(a.ds, a.ds_stride),
                      rows::in(a.sum, a.sum_stride),
                      rows::in(a.weight, a.dim),
                      a.rstd, a.rows, a.dim, a.dx, a.dx_stride, a.dweight ? workspace : nullptr};
        const bool vec = rows_aligned(a.dy, a.dy_stride, dt, a.dim) &&
                         rows_aligned(a.sum, a.sum_stride, dt, a.dim) &&
                         rows_aligned(a.weight, 0, dt, a.dim) &&
                         (!a.ds || rows_aligned(a.ds, a.ds_stride, dt, a.dim)) &&
                         rows_aligned(a.dx, a.dx_stride, dt, a.dim);
        auto go = [&](auto t) {
            constexpr int DT = decltype(t)::value;
            return vec ? grad_pick<DT, true>(n, parts, s) : grad_pick<DT, false>(n, parts, s);
        };
        const cudaError_t e = dt == F32 ? go(std::integral_constant<int, F32>{})
                              : dt == BF16 ? go(std::integral_constant<int, BF16>{})
                                           : go(std::integral_constant<int, F16>{});
        if (e != cudaSuccess) return e;
    }
    if (!a.dweight) return cudaSuccess;
    return launch_column_sums(wdt, workspace, parts, a.dim, a.dweight, a.accumulate, s);
}

}  // namespace zgb
