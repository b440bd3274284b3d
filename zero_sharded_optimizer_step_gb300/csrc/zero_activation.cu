// What a layer's backward pass does element by element: the gradients through
// an activation and through a gated block's product, the bias's gradient, and
// rows kept in 8 bits.
//
//   dz = dy act'(z), db = sum over rows of dz
//   dg = dh u act'(g), du = dh act(g), h = act(g) u again for what it feeds
//
// z, g and u are read in the type or in 8 bits, straight from what the forward
// pass kept.  Every matrix is read or written once, 256 columns of a row a warp.
//
// What bounds it: memory, where values are in the type (the gated gradient of 8192 x
// 11008 131 us, 902 MB at 6.9 TB/s; 6400 columns through RELU with the bias's
// 58, 315 MB at 5.4); else the instructions: GELU's normal
// distribution function (76 us), taking values out of 8 bits (135) and packing them (54 for
// 8192 x 11008, 273 MB).
#include "zero_act.cuh"
#include "zero_ops.h"
#include "zero_pack8.cuh"
#include "zero_rows.cuh"
#include "zero_tensor.cuh"

namespace zgb {
namespace {

constexpr int kWarps = kThreads / 32;

// Values kept in the type or in 8 bits.
template <int DT, bool VEC, bool PACKED> struct Kept {
    rows::Eight<DT, VEC> e;
    __device__ __forceinline__ void ask(const rows::In &m, const pack8::View &, int64_t r,
                                        int64_t c0, int64_t cols)
    {
        e.ask(m, r, c0, cols);
    }
    __device__ __forceinline__ void take(float *, float (&f)[8]) const { e.take(f); }
};
template <int DT, bool VEC> struct Kept<DT, VEC, true> {
    rows::Packed<DT, VEC> e;
    __device__ __forceinline__ void ask(const rows::In &, const pack8::View &q, int64_t r,
                                        int64_t c0, int64_t)
    {
        e.ask(q, r, c0);
    }
    __device__ __forceinline__ void take(float *shared, float (&f)[8]) const
    {
        e.take(shared, f);
    }
};

// ------------------------------------------------------- through an activation

struct ActGrad {
    rows::In dy, z;
    pack8::View q;
    int64_t n, cols;
    int32_t act;
    void *dz;
    int64_t dz_stride;
    float *parts;                                // [gridDim.y][cols], or null
    void *dbias;                                 // ONE: the sums go here at once
    int32_t bias_dtype, accumulate;
};

__device__ __forceinline__ void put_sum(void *out, int32_t dt, int64_t c, float v, bool accumulate)
{
    if (dt == F32) elems::store1<F32>(out, c, accumulate ? __fadd_rn(elems::load1<F32>(out, c), v) : v);
    else if (dt == BF16)
        elems::store1<BF16>(out, c, accumulate ? __fadd_rn(elems::load1<BF16>(out, c), v) : v);
    else elems::store1<F16>(out, c, accumulate ? __fadd_rn(elems::load1<F16>(out, c), v) : v);
}

// A block takes a strip of 256 columns and every gridDim.y-th eight of its rows.
// ONE: a strip's blocks are a cluster, whose first block adds up the sums of all through
// distributed shared memory, in their order; otherwise a second kernel does.
template <int DT, bool VEC, bool PACKED, bool ONE>
__global__ void __launch_bounds__(kThreads, VEC ? 4 : 1)
activation_grad_kernel(const __grid_constant__ ActGrad a)
{
    __shared__ float joined[kWarps][256];        // (until the end, room to turn values)
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5;
    const int64_t c0 = (int64_t)blockIdx.x * 256, step = (int64_t)gridDim.y * kWarps;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    constexpr int U = DT == F32 ? 1 : 2;         // rows on their way together
    for (int64_t r0 = (int64_t)blockIdx.y * kWarps + warp; r0 < a.n; r0 += U * step) {
        rows::Eight<DT, VEC> dye[U];
        Kept<DT, VEC, PACKED> ze[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * step;
            if (r >= a.n) break;
            dye[u].ask(a.dy, r, c0, a.cols);
            if (a.act != kActNone) ze[u].ask(a.z, a.q, r, c0, a.cols);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * step;
            if (r >= a.n) break;
            float d[8];
            dye[u].take(d);
            if (a.act != kActNone) {
                float z[8];
                ze[u].take(joined[warp], z);
                act::with_kind(a.act, [&](auto kind) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float y, slope;
                        act::both(z[e], decltype(kind)::value, y, slope);
                        d[e] = __fmul_rn(d[e], slope);
                    }
                });
            }
            if (a.dz) rows::put<DT, VEC>(a.dz, a.dz_stride, r, c0, a.cols, d);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = __fadd_rn(sum[e], d[e]);
        }
    }
    if (!a.parts && !a.dbias) return;
    __syncwarp();                                // all lanes have read what was turned there
#pragma unroll
    for (int e = 0; e < 8; ++e) joined[warp][rows::column<VEC>(e)] = sum[e];
    __syncthreads();
    const int64_t c = c0 + threadIdx.x;
    float v = joined[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) v = __fadd_rn(v, joined[i][threadIdx.x]);
    if constexpr (ONE) {
        __shared__ float total[256];
        total[threadIdx.x] = v;
        cluster_sync();
        if (blockIdx.y == 0) {
            for (uint32_t p = 1; p < gridDim.y; ++p)
                v = __fadd_rn(v, load_peer(saddr(&total[threadIdx.x]), p));
            if (c < a.cols) put_sum(a.dbias, a.bias_dtype, c, v, a.accumulate != 0);
        }
        cluster_sync();                          // the first block has read them
    } else {
        if (c < a.cols) a.parts[(int64_t)blockIdx.y * a.cols + c] = v;
    }
}

constexpr int64_t kBlocks = 152 * 8;             // about eight a SM
constexpr int64_t kOneRows = 256;

int64_t act_parts(int64_t n, int64_t cols)
{
    const int64_t strips = (cols + 255) / 256, most = (n + kWarps - 1) / kWarps;
    int64_t parts = (kBlocks + strips - 1) / strips;
    parts = parts < most ? parts : most;
    // with few rows eight blocks, a cluster, can do it in one launch
    if (n <= kOneRows) parts = most < 8 ? most : 8;
    return parts < 1 ? 1 : parts < 65535 ? parts : 65535;
}

// ----------------------------------------------------- through a gated product

struct GatedGrad {
    rows::In dh, g, u;
    pack8::View gq, uq;
    int64_t n, cols, runs;
    int32_t act;
    void *dg, *du, *h;
    int64_t grad_stride, h_stride;
};

// Runs of 256 columns that a warp asks for together, so that enough bytes are on their way.
template <int DT> constexpr int kRuns = DT == F32 ? 1 : 2;

template <int DT, bool VEC, bool PACKED>
__global__ void __launch_bounds__(kThreads)
gated_grad_kernel(const __grid_constant__ GatedGrad a)
{
    constexpr int U = kRuns<DT>;
    __shared__ float turned[PACKED && !VEC ? kWarps : 1][256];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5;
    const int64_t w = ((int64_t)blockIdx.x * kWarps + warp) * U;
    int64_t r[U], c0[U];
    rows::Eight<DT, VEC> dhe[U];
    Kept<DT, VEC, PACKED> ge[U], ue[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        rows::run_at(w + k, a.runs, r[k], c0[k]);
        if (r[k] >= a.n) break;
        dhe[k].ask(a.dh, r[k], c0[k], a.cols);
        ge[k].ask(a.g, a.gq, r[k], c0[k], a.cols);
        ue[k].ask(a.u, a.uq, r[k], c0[k], a.cols);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (r[k] >= a.n) break;
        float dh[8], g[8], u[8], f[8], d[8];
        dhe[k].take(dh);
        ge[k].take(turned[PACKED && !VEC ? warp : 0], g);
        ue[k].take(turned[PACKED && !VEC ? warp : 0], u);
        act::with_kind(a.act, [&](auto kind) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float slope;
                act::both(g[e], decltype(kind)::value, f[e], slope);
                d[e] = __fmul_rn(__fmul_rn(dh[e], u[e]), slope);
                dh[e] = __fmul_rn(dh[e], f[e]);
                f[e] = __fmul_rn(f[e], u[e]);
            }
        });
        rows::put<DT, VEC>(a.dg, a.grad_stride, r[k], c0[k], a.cols, d);
        rows::put<DT, VEC>(a.du, a.grad_stride, r[k], c0[k], a.cols, dh);
        if (a.h) rows::put<DT, VEC>(a.h, a.h_stride, r[k], c0[k], a.cols, f);
    }
}

// -------------------------------------------------------------- rows in 8 bits

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
pack8_kernel(const __grid_constant__ rows::In x, const __grid_constant__ pack8::View q,
             int64_t n, int64_t cols, int64_t runs)
{
    constexpr int U = kRuns<DT>;
    __shared__ float turned[VEC ? 1 : kWarps][256];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5;
    const int64_t w = ((int64_t)blockIdx.x * kWarps + warp) * U;
    int64_t r[U], c0[U];
    rows::Eight<DT, VEC> e[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        rows::run_at(w + k, runs, r[k], c0[k]);
        if (r[k] < n) e[k].ask(x, r[k], c0[k], cols);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (r[k] >= n) break;
        float f[8];
        e[k].take(f);
        rows::pack<VEC>(q, r[k], c0[k], turned[VEC ? 0 : warp], f);
    }
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
unpack8_kernel(const __grid_constant__ pack8::View q, int64_t n, int64_t cols, int64_t runs,
               void *out, int64_t stride)
{
    constexpr int U = kRuns<DT>;
    __shared__ float turned[VEC ? 1 : kWarps][256];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5;
    const int64_t w = ((int64_t)blockIdx.x * kWarps + warp) * U;
    int64_t r[U], c0[U];
    rows::Packed<DT, VEC> e[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        rows::run_at(w + k, runs, r[k], c0[k]);
        if (r[k] < n) e[k].ask(q, r[k], c0[k]);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (r[k] >= n) break;
        float f[8];
        e[k].take(turned[VEC ? 0 : warp], f);
        rows::put<DT, VEC>(out, stride, r[k], c0[k], cols, f);
    }
}

// ----------------------------------------------------------------- column sums

// A block takes 32 columns, its warps (up to 32) every so many of the partial rows,
// in order.
template <int DT>
__global__ void __launch_bounds__(1024)
column_sums_kernel(const float *parts, int64_t n_parts, int64_t cols, void *out, int accumulate)
{
    __shared__ float joined[32][32];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < cols) {
        constexpr int U = 8;
        for (int64_t p = warp; p < n_parts; p += U * warps) {
            float f[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                f[u] = p + u * warps < n_parts ? parts[(p + u * warps) * cols + c] : 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) v = __fadd_rn(v, f[u]);
        }
    }
    joined[warp][lane] = v;
    __syncthreads();
    if (warp || c >= cols) return;
    for (int i = 1; i < warps; ++i) v = __fadd_rn(v, joined[i][lane]);
    if (accumulate) v = __fadd_rn(elems::load1<DT>(out, c), v);
    elems::store1<DT>(out, c, v);
}

template <class F> cudaError_t by_type(int32_t dt, F f)
{
    return dt == F32 ? f(std::integral_constant<int, F32>{})
           : dt == BF16 ? f(std::integral_constant<int, BF16>{})
                        : f(std::integral_constant<int, F16>{});
}

// Blocks for so many runs of 256 columns; 0 where there are too many.
unsigned run_blocks(int32_t dt, int64_t n, int64_t runs)
{
    const int64_t of = kWarps * (dt == F32 ? kRuns<F32> : kRuns<BF16>);
    const int64_t blocks = (n * runs + of - 1) / of;
    return blocks > 0x7fffffff ? 0 : (unsigned)blocks;
}

}  // namespace

cudaError_t launch_column_sums(int32_t dt, const float *parts, int64_t n_parts, int64_t cols,
                               void *out, bool accumulate, cudaStream_t s)
{
    const int64_t eights = (n_parts + 7) / 8, warps = eights < 4 ? 4 : eights < 32 ? eights : 32;
    return by_type(dt, [&](auto t) {
        return launch_dependent(column_sums_kernel<decltype(t)::value>,
                                dim3((unsigned)((cols + 31) / 32)), dim3((unsigned)warps * 32), 0,
                                s, parts, n_parts, cols, out, accumulate ? 1 : 0);
    });
}

int64_t activation_grad_workspace(int64_t rows, int64_t cols)
{
    return act_parts(rows, cols) * cols * 4;
}

cudaError_t launch_activation_grad(int32_t dt, int32_t bdt, const ActGradArgs &a, float *workspace,
                                   cudaStream_t s)
{
    if (a.cols <= 0) return cudaSuccess;
    const int64_t parts = act_parts(a.rows, a.cols);
    if (a.rows > 0) {
        const bool one = a.dbias && a.rows <= kOneRows;
        ActGrad g = {rows::in(a.dy, a.dy_stride),
                     rows::in(a.kept, a.kept_stride),
                     pack8::view(a.kept_q, a.rows, a.cols), a.rows, a.cols, a.act, a.dz,
                     a.dz_stride, a.dbias && !one ? workspace : nullptr,
                     one ? a.dbias : nullptr, bdt, a.accumulate};
        const bool vec = rows_aligned(a.dy, a.dy_stride, dt, a.cols) &&
                         (!a.kept || rows_aligned(a.kept, a.kept_stride, dt, a.cols)) &&
                         (!a.dz || rows_aligned(a.dz, a.dz_stride, dt, a.cols));
        const dim3 grid((unsigned)((a.cols + 255) / 256), (unsigned)parts);
        const cudaError_t e = by_type(dt, [&](auto t) {
            constexpr int DT = decltype(t)::value;
            auto pick = [&](auto joined) {
                constexpr bool ONE = decltype(joined)::value;
                return a.kept_q ? (vec ? activation_grad_kernel<DT, true, true, ONE>
                                       : activation_grad_kernel<DT, false, true, ONE>)
                                : (vec ? activation_grad_kernel<DT, true, false, ONE>
                                       : activation_grad_kernel<DT, false, false, ONE>);
            };
            if (!one) return launch_dependent(pick(std::false_type{}), grid, dim3(kThreads), 0, s, g);
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = grid;
            cfg.blockDim = dim3(kThreads);
            cfg.stream = s;
            cudaLaunchAttribute attr[2];
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            attr[1].id = cudaLaunchAttributeClusterDimension;
            attr[1].val.clusterDim.x = 1;
            attr[1].val.clusterDim.y = (unsigned)parts;
            attr[1].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 2;
            return cudaLaunchKernelEx(&cfg, pick(std::true_type{}), g);
        });
        if (e != cudaSuccess || one) return e;
    }
    if (!a.dbias) return cudaSuccess;
    return launch_column_sums(bdt, workspace, a.rows > 0 ? parts : 0, a.cols, a.dbias,
                              a.accumulate, s);
}

cudaError_t launch_gated_grad(int32_t dt, const GatedGradArgs &a, cudaStream_t s)
{
    if (a.rows <= 0 || a.cols <= 0) return cudaSuccess;
    const int64_t runs = (a.cols + 255) / 256;
    GatedGrad g = {rows::in(a.dh, a.dh_stride),
                   rows::in(a.gate, a.kept_stride),
                   rows::in(a.up, a.kept_stride),
                   pack8::view(a.gate_q, a.rows, a.cols), pack8::view(a.up_q, a.rows, a.cols),
                   a.rows, a.cols, runs, a.act, a.dgate, a.dup, a.h, a.grad_stride, a.h_stride};
    const bool vec = rows_aligned(a.dh, a.dh_stride, dt, a.cols) &&
                     (!a.gate || (rows_aligned(a.gate, a.kept_stride, dt, a.cols) &&
                                  rows_aligned(a.up, a.kept_stride, dt, a.cols))) &&
                     rows_aligned(a.dgate, a.grad_stride, dt, a.cols) &&
                     rows_aligned(a.dup, a.grad_stride, dt, a.cols) &&
                     (!a.h || rows_aligned(a.h, a.h_stride, dt, a.cols));
    const unsigned blocks = run_blocks(dt, a.rows, runs);
    if (!blocks) return cudaErrorInvalidValue;
    return by_type(dt, [&](auto t) {
        constexpr int DT = decltype(t)::value;
        auto k = a.gate_q ? (vec ? gated_grad_kernel<DT, true, true>
                                 : gated_grad_kernel<DT, false, true>)
                          : (vec ? gated_grad_kernel<DT, true, false>
                                 : gated_grad_kernel<DT, false, false>);
        return launch_dependent(k, dim3(blocks), dim3(kThreads), 0, s, g);
    });
}

int64_t pack8_bytes(int64_t rows, int64_t cols)
{
    return rows * (pack8::pitch(cols) + pack8::pitch(cols) / pack8::kBlock);
}

cudaError_t launch_pack8(int32_t dt, const void *x, int64_t rows, int64_t cols, int64_t stride,
                         unsigned char *q, cudaStream_t s)
{
    if (rows <= 0 || cols <= 0) return cudaSuccess;
    const int64_t runs = (cols + 255) / 256;
    const unsigned blocks = run_blocks(dt, rows, runs);
    if (!blocks) return cudaErrorInvalidValue;
    const rows::In in = rows::in(x, stride);
    const bool vec = rows_aligned(x, stride, dt, cols);
    return by_type(dt, [&](auto t) {
        constexpr int DT = decltype(t)::value;
        return launch_dependent(vec ? pack8_kernel<DT, true> : pack8_kernel<DT, false>,
                                dim3(blocks), dim3(kThreads), 0, s, in,
                                pack8::view(q, rows, cols), rows, cols, runs);
    });
}

cudaError_t launch_unpack8(int32_t dt, const unsigned char *q, int64_t rows, int64_t cols,
                           void *out, int64_t stride, cudaStream_t s)
{
    if (rows <= 0 || cols <= 0) return cudaSuccess;
    const int64_t runs = (cols + 255) / 256;
    const unsigned blocks = run_blocks(dt, rows, runs);
    if (!blocks) return cudaErrorInvalidValue;
    const bool vec = rows_aligned(out, stride, dt, cols);
    return by_type(dt, [&](auto t) {
        constexpr int DT = decltype(t)::value;
        return launch_dependent(vec ? unpack8_kernel<DT, true> : unpack8_kernel<DT, false>,
                                dim3(blocks), dim3(kThreads), 0, s,
                                pack8::view(const_cast<unsigned char *>(q), rows, cols), rows,
                                cols, runs, out, stride);
    });
}

}  // namespace zgb
