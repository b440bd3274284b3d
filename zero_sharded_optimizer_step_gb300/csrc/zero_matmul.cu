// Products of 16-bit matrices on the tensor cores with what surrounds them in a
// linear layer:
//
//   z[i, j] = sum over c of A[i, c] B[j, c] (+ of A2[i, c] B2[j, c]) + bias[j]
//   out[i, j] = act(z[i, j]) (+ residual[i, j])
//
// and the gated block's first half, out = act(A B^T) * (A B2^T).  Either
// operand may lie as its transpose: both orders are ones in which the tensor
// cores read shared memory, so a layer's three products (y = x W^T, dx = dz W,
// dW = dz^T x) need no transposed copy.  Products of two 16-bit numbers are exact in the
// fp32 sums; bias, activation, residual follow in fp32, and the
// result is rounded once.  What the backward pass needs of z is stored beside it,
// rounded to the type or packed to 8 bits from the fp32 sum.
//
// Tensor copies (TMA) bring blocks of 64 columns c into shared memory, 128-byte lines
// swizzled; what lies outside a matrix arrives as zeros.  They need 16-byte
// boundaries: an operand whose rows are not on them is first copied to a
// workspace whose rows are.
#include <atomic>

#include <cuda.h>

#include "zero_act.cuh"
#include "zero_elems.cuh"
#include "zero_ops.h"
#include "zero_pack8.cuh"
#include "zero_product_sizes.h"
#include "zero_rows.cuh"
#include "zero_tensor.cuh"

namespace zgb {
namespace {

using namespace product;

__device__ unsigned int g_matmul_timeouts;

// An operand's stage as the tensor cores read it.  Rows of c lie as lines of 128
// bytes (64 c), eight lines a swizzle atom; the transpose as chunks of 64
// rows of the operand, each 64 lines (one c each) of 128 bytes.
struct Layout {
    uint64_t desc;                               // without the address
    uint32_t step;                               // 16 c further, in units of 16 bytes
};

__device__ __forceinline__ Layout layout_of(int32_t cols)
{
    const uint64_t fixed = ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
    return cols ? Layout{fixed | ((uint64_t)(kDepth * kLine >> 4) << 16), 16 * kLine >> 4}
                : Layout{fixed | (1ull << 16), 32 >> 4};
}

__device__ __forceinline__ uint64_t at(const Layout &l, uint32_t addr)
{
    return l.desc | ((addr & 0x3ffffu) >> 4);
}

// fp32 sums of 16-bit products, M lanes by N columns.
template <int DT> __device__ __forceinline__ uint32_t shape_desc(int32_t a_cols, int32_t b_cols)
{
    constexpr uint32_t t = DT == BF16 ? 1u : 0u;
    return (1u << 4) | (t << 7) | (t << 10) | ((uint32_t)(a_cols != 0) << 15) |
           ((uint32_t)(b_cols != 0) << 16);
}

__device__ __forceinline__ void mma1(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                     uint32_t add)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a),
                 "l"(b), "r"(idesc), "r"(add) : "memory");
}

__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                     uint32_t add)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a),
                 "l"(b), "r"(idesc), "r"(add) : "memory");
}

// A box of `map` from (x, y) into this block's shared memory, signalled here.
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap *map, int32_t x,
                                         int32_t y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile"
                 ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}

// The same, signalled at `bar` of the pair's first block.
__device__ __forceinline__ void tensor_load(uint32_t dst, const CUtensorMap *map, int32_t x,
                                            int32_t y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
                 ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}

// ---------------------------------------------------------------- the results

// Column j of row i, by a whole warp with 32 consecutive columns from a multiple
// of 32 on; `in`: the column is one of the result's.  Every pointer that is
// given is written or read by whole runs of the warp.
template <int DT, int ODT, bool GATED>
__device__ __forceinline__ void finish_lane(const ProductArgs &a, int64_t i, int64_t j, bool in,
                                            float acc, float acc2, float bias)
{
    const float z = __fadd_rn(acc, bias);
    if (a.kept && in) elems::store1<DT>(a.kept, i * a.kept_stride + j, z);
    if (a.kept_q)
        pack8::put_lane(pack8::view(a.kept_q, a.m, a.n), i, j - (threadIdx.x & 31), in ? z : 0.0f);
    float y = act::value(z, a.act);
    if constexpr (GATED) {
        if (a.kept2 && in) elems::store1<DT>(a.kept2, i * a.kept_stride + j, acc2);
        if (a.kept2_q)
            pack8::put_lane(pack8::view(a.kept2_q, a.m, a.n), i, j - (threadIdx.x & 31),
                            in ? acc2 : 0.0f);
        y = __fmul_rn(y, acc2);
    }
    if (in) {
        if (a.residual) y = __fadd_rn(y, elems::load1<ODT>(a.residual, i * a.residual_stride + j));
        elems::store1<ODT>(a.out, i * a.stride + j, y);
    }
}

// The activation of an array.
template <int U, int N> __device__ __forceinline__ void activate(float (&z)[U][N], int32_t kind)
{
    if (kind == kActNone) return;
    act::with_kind(kind, [&](auto k) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < N; ++e) z[u][e] = act::value(z[u][e], decltype(k)::value);
    });
}

// What is added to 32 columns of a row, on 32-byte boundaries: asked for before the sums
// are there.  (The residual may be the result's own place: a thread's elements are its own.)
template <int DT, int ODT, bool GATED> struct Beside {
    elems::Raw<DT> bias[4];
    elems::Raw<ODT> residual[4];

    __device__ __forceinline__ void ask(const ProductArgs &a, int64_t i, int64_t j)
    {
        if constexpr (!GATED) {
            if (a.bias) {
#pragma unroll
                for (int u = 0; u < 4; ++u) bias[u].load(a.bias, j + 8 * u);
            }
            if (a.residual) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    residual[u].load(a.residual, i * a.residual_stride + j + 8 * u);
            }
        }
    }
};

template <class R> __device__ __forceinline__ void add_run(const R (&r)[4], float (&z)[32])
{
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        float f[8];
        r[u].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[8 * u + e] = __fadd_rn(z[8 * u + e], f[e]);
    }
}

// 16 columns of a row on 32-byte boundaries.
template <int DT> __device__ __forceinline__ void store_run(void *p, int64_t at, const float *f)
{
    using T = typename elems::El<DT>::T;
#pragma unroll
    for (int u = 0; u < (DT == F32 ? 2 : 1); ++u) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (DT == F32) w[e] = __float_as_uint(f[8 * u + e]);
            else w[e] = elems::narrow2<DT>(f[2 * e], f[2 * e + 1]);
        }
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(
                         static_cast<T *>(p) + at + 8 * u),
                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                     "r"(w[7]) : "memory");
    }
}

// 32 columns of row i from j on, all the result's, by one thread.  z holds the
// sums, z2 the second ones of a gated block.
template <int DT, int ODT, bool GATED>
__device__ __forceinline__ void finish_run(const ProductArgs &a, int64_t i, int64_t j,
                                           const Beside<DT, ODT, GATED> &beside, float (&z)[32],
                                           float (&z2)[32])
{
    if constexpr (!GATED) {
        if (a.bias) add_run(beside.bias, z);
    }
    if (a.kept) {
        store_run<DT>(a.kept, i * a.kept_stride + j, z);
        store_run<DT>(a.kept, i * a.kept_stride + j + 16, z + 16);
        if constexpr (GATED) {
            store_run<DT>(a.kept2, i * a.kept_stride + j, z2);
            store_run<DT>(a.kept2, i * a.kept_stride + j + 16, z2 + 16);
        }
    }
    if (a.kept_q) {
        pack8::put_thread(pack8::view(a.kept_q, a.m, a.n), i, j, z);
        if constexpr (GATED) pack8::put_thread(pack8::view(a.kept2_q, a.m, a.n), i, j, z2);
    }
    activate(reinterpret_cast<float(&)[1][32]>(z), a.act);
    if constexpr (GATED) {
#pragma unroll
        for (int e = 0; e < 32; ++e) z[e] = __fmul_rn(z[e], z2[e]);
    } else {
        if (a.residual) add_run(beside.residual, z);
    }
    store_run<ODT>(a.out, i * a.stride + j, z);
    store_run<ODT>(a.out, i * a.stride + j + 16, z + 16);
}

// Rows off the boundaries, and ragged ends: 32 rows by 32 columns, a row a lane,
// change places with a row a step through the warp's shared memory (`staged`, 32 by
// kStagePad floats), so that its accesses are consecutive.

// v into rows i0 .. i0 + rows of p from column j on; `in`: column j + lane is the matrix's.
template <int DT>
__device__ __forceinline__ void store_turned(void *p, int64_t stride, int64_t i0, int rows,
                                             int64_t j, bool in, float *staged,
                                             const float (&v)[32])
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 32; ++e) staged[lane * kStagePad + e] = v[e];
    __syncwarp();
    using T = typename elems::El<DT>::T;
    T *to = static_cast<T *>(p) + i0 * stride + j + lane;
#pragma unroll 4
    for (int e = 0; e < rows; ++e, to += stride)
        if (in) elems::store1<DT>(to, 0, staged[e * kStagePad + lane]);
}

// The same the other way, added to v.
template <int DT>
__device__ __forceinline__ void add_turned(const void *p, int64_t stride, int64_t i0, int rows,
                                           int64_t j, bool in, float *staged, float (&v)[32])
{
    const int lane = threadIdx.x & 31;
    using T = typename elems::El<DT>::T;
    const T *from = static_cast<const T *>(p) + i0 * stride + j + lane;
    __syncwarp();
#pragma unroll 4
    for (int e = 0; e < rows; ++e, from += stride)
        staged[e * kStagePad + lane] = in ? elems::load1<DT>(from, 0) : 0.0f;
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = __fadd_rn(v[e], staged[lane * kStagePad + e]);
}

// 32 columns from j on of 32 rows from i0 on (those below `end`), a row a lane.
template <int DT, int ODT, bool GATED>
__device__ __forceinline__ void finish_rows(const ProductArgs &a, bool vec, float *staged,
                                            int64_t i0, int64_t end, int64_t j,
                                            const Beside<DT, ODT, GATED> &beside, float (&z)[32],
                                            float (&z2)[32])
{
    const int lane = threadIdx.x & 31;
    if (j >= a.n || i0 >= end) return;
    if (vec && j + 32 <= a.n) {
        if (i0 + lane < end) finish_run<DT, ODT, GATED>(a, i0 + lane, j, beside, z, z2);
        return;
    }
    const bool in = j + lane < a.n;
    const int rows = end - i0 < 32 ? (int)(end - i0) : 32;
    if (a.bias) {
        const float bias = in ? elems::load1<DT>(a.bias, j + lane) : 0.0f;
#pragma unroll
        for (int e = 0; e < 32; ++e)
            z[e] = __fadd_rn(z[e], __shfl_sync(0xffffffffu, bias, e));
    }
    if (a.kept) {
        store_turned<DT>(a.kept, a.kept_stride, i0, rows, j, in, staged, z);
        if constexpr (GATED)
            store_turned<DT>(a.kept2, a.kept_stride, i0, rows, j, in, staged, z2);
    }
    if (a.kept_q) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (j + e >= a.n) z[e] = z2[e] = 0.0f;
        if (i0 + lane < end) {
            pack8::put_thread(pack8::view(a.kept_q, a.m, a.n), i0 + lane, j, z);
            if constexpr (GATED)
                pack8::put_thread(pack8::view(a.kept2_q, a.m, a.n), i0 + lane, j, z2);
        }
    }
    activate(reinterpret_cast<float(&)[1][32]>(z), a.act);
    if constexpr (GATED) {
#pragma unroll
        for (int e = 0; e < 32; ++e) z[e] = __fmul_rn(z[e], z2[e]);
    }
    if (a.residual) add_turned<ODT>(a.residual, a.residual_stride, i0, rows, j, in, staged, z);
    store_turned<ODT>(a.out, a.stride, i0, rows, j, in, staged, z);
    __syncwarp();
}

// ------------------------------------------------------------------- one row
//
// The weights' bytes are all there is: a warp reads four rows of B (of both, in a
// gated block) in the memory's own order, 512 bytes of each at a time, multiplies in
// fp32 and adds up over its lanes.  A block makes 32 columns of the result; KS warps
// share a row's length where the blocks are few.  No copy engine and no tensor
// memory to set up, and rows need no boundary.
//
// Measured: 2 x 11008 x 4096 29 us (6.2 TB/s), through the tensor cores 33; 6400 x 1600
// 6.0 (in L2 4.1), tensor cores 7.5; 4096 x 11008 with KS = 4 16.5, KS = 2 19.6, tensor
// cores 18.2.  (Four rows of A this way took 2 x 11008 x 4096 46 us, for the arithmetic.)
template <int DT, int ODT, bool GATED, int KS, bool VEC>
__global__ void __launch_bounds__(256 * KS)
matvec_kernel(const __grid_constant__ ProductArgs a, const __grid_constant__ rows::In x,
              const __grid_constant__ rows::In w, const __grid_constant__ rows::In w2)
{
    constexpr int kWeights = GATED ? 2 : 1, R = 4;
    __shared__ float part[kWeights][KS][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, share = warp / 8;
    const int64_t j0 = (int64_t)blockIdx.x * 32, first = j0 + (warp % 8) * R;
    pdl_wait();
    pdl_launch_dependents();
    float acc[kWeights][R] = {};
#pragma unroll 2
    for (int64_t c0 = share * 256; c0 < a.k; c0 += KS * 256) {
        if (VEC && c0 + 8 * lane >= a.k) break;          // nothing left for this lane
        rows::Eight<DT, VEC> we[kWeights][R], xe;
#pragma unroll
        for (int g = 0; g < kWeights; ++g)
#pragma unroll
            for (int r = 0; r < R; ++r) {    // (the last row again past the end: not written)
                const int64_t row = first + r < a.n ? first + r : a.n - 1;
                if constexpr (VEC)
                    we[g][r].v.load(g ? w2.p : w.p,
                                    row * (g ? w2.stride : w.stride) + c0 + 8 * lane);
                else
                    we[g][r].ask(g ? w2 : w, row, c0, a.k);
            }
        if constexpr (VEC) xe.v.load(x.p, c0 + 8 * lane);
        else xe.ask(x, 0, c0, a.k);
        float xv[8];
        xe.take(xv);
#pragma unroll
        for (int g = 0; g < kWeights; ++g)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float f[8];
                we[g][r].take(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[g][r] = __fmaf_rn(f[e], xv[e], acc[g][r]);
            }
    }
    __syncwarp();
#pragma unroll
    for (int g = 0; g < kWeights; ++g)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float v = rows::warp_sum(acc[g][r]);
            if (lane == 0) part[g][share][(warp % 8) * R + r] = v;
        }
    __syncthreads();
    if (warp) return;
    float z[2] = {0.0f, 0.0f};
#pragma unroll
    for (int g = 0; g < kWeights; ++g) {
        z[g] = part[g][0][lane];
#pragma unroll
        for (int s = 1; s < KS; ++s) z[g] = __fadd_rn(z[g], part[g][s][lane]);
    }
    const int64_t j = j0 + lane;
    const float bias = a.bias && j < a.n ? elems::load1<DT>(a.bias, j) : 0.0f;
    finish_lane<DT, ODT, GATED>(a, 0, j, j < a.n, z[0], z[1], bias);
}

// ------------------------------------------------- few rows, or few tiles
//
// The accumulator's 128 lanes are 128 rows of B (128 consecutive columns of
// the result, so that a warp's stores are contiguous), its columns up to 128 rows of
// A (256 in pick()'s wide tiles): with few tokens the tile is as narrow as they are,
// and the product reads the weights once.  A gated block's lanes are 64 rows of B and
// the same 64 of B2.  One warp issues the copies, one the products, eight write.  With fewer tiles
// than SMs the columns c are split over a cluster of up to 8 blocks, whose partial sums
// join through distributed shared memory in the blocks' order.
//
// What bounds it: the weights' bytes.  77 rows gated, 2 x 11008 x 4096 values of
// weights, took 35.8 us (180 MB at 5.0 TB/s) in its 172 tiles before matmul_mid_kernel
// had them; with 128 rows of either weight a tile, in two accumulators, 37.1.
struct OneArgs {
    CUtensorMap a, b, b2, a2;
    int64_t kt1, kt, tiles_n;            // stages of the first pair of operands, of both
    int32_t splits, stages;
    int32_t nt, wide;                    // rows of A in a tile, a multiple of 16; of B
    int32_t span;                        // an accumulator's columns in shared memory
    int32_t vec;                         // runs of columns lie on their boundaries
};

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---- joining a split
//
// Every block of a split has partial sums of the whole tile, rows of 128 columns of the
// result (kPitch floats apart; of a gated block 64 and their 64 second ones) in its
// shared memory.  The rows are shared out; each block sends every other
// one's share there by one bulk copy and adds up what it receives in the blocks' order.

struct Split {
    static constexpr int pitch = kPitch;
    int rows, span, splits;
    uint32_t rank;

    __device__ __forceinline__ int first(uint32_t q) const { return rows * (int)q / splits; }
    __device__ __forceinline__ int share() const { return (span + splits - 1) / splits; }
    // where block q's sums for this block arrive, behind its own
    __device__ __forceinline__ int slot(uint32_t q) const
    {
        return (span + (int)q * share()) * pitch;
    }
    __device__ __forceinline__ uint32_t bytes(uint32_t q) const
    {
        return (uint32_t)((first(q + 1) - first(q)) * pitch * 4);
    }
    // by one thread, before the first cluster_arrive()
    __device__ __forceinline__ void expect(uint32_t bar) const
    {
        bar_init(bar, 1);
        bar_expect(bar, (uint32_t)(splits - 1) * bytes(rank));
    }
};

// By one thread, once every block's sums and barrier are there.
__device__ __forceinline__ void send_shares(const Split &t, const float *part, uint32_t bar)
{
    for (int d = 1; d < t.splits; ++d) {
        const uint32_t q = (t.rank + d) % t.splits, bytes = t.bytes(q);
        if (!bytes) continue;
        asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes"
                     " [%0], [%1], %2, [%3];" ::"r"(peer_addr(saddr(part + t.slot(t.rank)), q)),
                     "r"(saddr(part + t.first(q) * t.pitch)), "r"(bytes), "r"(peer_addr(bar, q))
                     : "memory");
    }
}

// 32 columns from c on of row r, which is in this block's share, added up.
__device__ __forceinline__ void sum32(const Split &t, const float *part, int r, int c,
                                      float (&z)[32])
{
    const float *own = part + r * kPitch + c;
    const float *in = part + t.slot(0) + (r - t.first(t.rank)) * kPitch + c;
    const int step = t.slot(1) - t.slot(0);
    const float4 *first = reinterpret_cast<const float4 *>(t.rank == 0 ? own : in);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float4 f = first[e];
        z[4 * e] = f.x, z[4 * e + 1] = f.y, z[4 * e + 2] = f.z, z[4 * e + 3] = f.w;
    }
    in += step;
#pragma unroll 1
    for (int q = 1; q < t.splits; ++q, in += step) {
        const float4 *v = reinterpret_cast<const float4 *>((uint32_t)q == t.rank ? own : in);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float4 f = v[e];
            z[4 * e] = __fadd_rn(z[4 * e], f.x);
            z[4 * e + 1] = __fadd_rn(z[4 * e + 1], f.y);
            z[4 * e + 2] = __fadd_rn(z[4 * e + 2], f.z);
            z[4 * e + 3] = __fadd_rn(z[4 * e + 3], f.w);
        }
    }
}

// Writes the result of this block's share of the rows: the warps take 32 rows by 32
// columns in turn, a row a lane.  (Four columns of a row a lane, a row a warp,
// took 550 clocks a row: it is the instructions that count here.)
template <int DT, int ODT, bool GATED>
__device__ __forceinline__ bool join(const ProductArgs &a, const Split &t, float *part,
                                     uint32_t bar, bool vec, int64_t i0, int64_t j0)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int from = t.first(t.rank), end = t.first(t.rank + 1);
    float *staged = part + split_floats(t.span, t.splits) + warp * 32 * kStagePad;
    constexpr int kAcross = GATED ? 2 : 4;
#pragma unroll 1
    for (int item = warp; item < (end - from + 31) / 32 * kAcross; item += kOneThreads / 32) {
        const int r0 = from + item / kAcross * 32, c = item % kAcross * 32;
        const int r = r0 + lane < end ? r0 + lane : end - 1;
        Beside<DT, ODT, GATED> beside;
        if (vec && j0 + c + 32 <= a.n) beside.ask(a, i0 + r, j0 + c);
        if (t.splits > 1 && !bar_wait(bar, 0)) return false;
        float z[32], z2[32];
        sum32(t, part, r, c, z);
        if constexpr (GATED) sum32(t, part, r, 64 + c, z2);
        finish_rows<DT, ODT, GATED>(a, vec, staged, i0 + r0, i0 + end, j0 + c, beside, z,
                                          z2);
    }
    return true;
}

// The end of a tile whose sums lie in shared memory: sends and receives the shares
// and writes the result.  The whole block comes here, after cluster_arrive() where its
// ring was free for what the others send; `failed` blocks take part in the barriers
// alone.
template <int DT, int ODT, bool GATED>
__device__ __forceinline__ void settle(const ProductArgs &a, const Split &t, float *part,
                                       uint32_t bar, const uint32_t &failed, bool vec, int64_t i0,
                                       int64_t j0)
{
    if (t.splits > 1) {
        // what the copies read was written by this block's threads
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        cluster_wait();
        if (threadIdx.x == 0 && !failed) send_shares(t, part, bar);
        __syncwarp();
    } else {
        __syncthreads();
    }
    if (failed) {
        if (t.splits > 1) bar_wait(bar, 0);      // what is on its way lands before the block ends
    } else if (!join<DT, ODT, GATED>(a, t, part, bar, vec, i0, j0) && (threadIdx.x & 31) == 0) {
        atomicAdd(&g_matmul_timeouts, 1u);
    }
    if (t.splits > 1) cluster_meet();       // the peers have received what this block sent
}

template <int DT, int ODT, bool GATED>
__global__ void __launch_bounds__(kOneThreads, kMostBlocks)
matmul_kernel(const __grid_constant__ ProductArgs a, const __grid_constant__ OneArgs g)
{
    using Tl = Tile;
    constexpr int kAcross = GATED ? 64 : 128;                // columns of the result
    const int stage = Tl::stage(g.nt);
    const uint32_t columns = Tl::tmem(g.nt);
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t bars[2 * Tl::kStages + 2];
    __shared__ uint32_t tmem_base, failed;
    const uint32_t ring = saddr(dyn) + ((1024 - (saddr(dyn) & 1023)) & 1023);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = g.splits > 1 ? cluster_rank() : 0;
    const int64_t tile = blockIdx.x / g.splits;
    const int64_t tn = tile % g.tiles_n, tm = tile / g.tiles_n;
    const int64_t k0 = g.kt * rank / g.splits, k1 = g.kt * (rank + 1) / g.splits;
    const int rounds = (int)(k1 - k0);
    const uint32_t done_bar = saddr(&bars[2 * Tl::kStages]), join_bar = done_bar + 8;
    auto full = [&](int s) { return saddr(&bars[s]); };
    auto empty = [&](int s) { return saddr(&bars[Tl::kStages + s]); };

    const int64_t i0 = tm * g.nt;
    const int cols = (int)(a.m - i0 < g.nt ? a.m - i0 : g.nt);
    const Split split = {cols, g.span, g.splits, rank};

    bool ok = true;
    if (warp == kOneWarps) {                                         // the copies
        const bool one = elect_one();
        if (one) {
            for (int s = 0; s < Tl::kStages; ++s) {
                bar_init(full(s), 1);
                bar_init(empty(s), 1);
            }
            bar_init(done_bar, 1);
            split.expect(join_bar);
            failed = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        if (one && g.kt > 0) {
            prefetch_map(&g.a);
            prefetch_map(&g.b);
        }
        __syncwarp();
        pdl_wait();
        const int32_t jx = (int32_t)(tn * kAcross), ix = (int32_t)(tm * g.nt);
        auto load = [&](int it, int s) {
            const int64_t kt = k0 + it;
            const bool second = kt >= g.kt1;
            const int32_t c = (int32_t)((second ? kt - g.kt1 : kt) * kDepth);
            const uint32_t st = ring + s * stage;
            bar_expect(full(s), (uint32_t)stage);
            if constexpr (GATED) {
                box_load(st, &g.b, c, jx, full(s));
                box_load(st + kHalf / 2, &g.b2, c, jx, full(s));
            } else {
                const CUtensorMap *b = second ? &g.b2 : &g.b;
                if (a.b_cols) {
                    box_load(st, b, jx, c, full(s));
                    box_load(st + kHalf / 2, b, jx + 64, c, full(s));
                } else {
                    box_load(st, b, c, jx, full(s));
                }
            }
            const CUtensorMap *map = second ? &g.a2 : &g.a;
            box_load(st + kHalf, map, c, ix, full(s));
        };
        // the first stages' copies need not wait for the other warps
        const int ahead = rounds < g.stages ? rounds : g.stages;
        for (int it = 0; it < ahead; ++it)
            if (one) load(it, it);
        __syncthreads();
        int s = 0;
        uint32_t phase = 0;
        for (int it = ahead; it < rounds; ++it) {
            ok = bar_wait(empty(s), phase);
            if (!ok) break;
            if (one) load(it, s);
            __syncwarp();
            if (++s == g.stages) s = 0, phase ^= 1;
        }
    } else if (warp == kOneWarps + 1) {                                  // the products
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         saddr(&tmem_base)), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncthreads();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const bool one = elect_one();
        const uint32_t tmem = tmem_base;
        const Layout lb = layout_of(a.b_cols), la = layout_of(0);
        const uint32_t desc = shape_desc<DT>(a.b_cols, 0) | ((uint32_t)(g.nt >> 3) << 17) |
                              ((128u >> 4) << 24);
        int s = 0;
        uint32_t phase = 0;
        for (int it = 0; it < rounds; ++it) {
            ok = bar_wait(full(s), phase);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (one) {
                const uint32_t st = ring + s * stage;
                const uint64_t db = at(lb, st), da = at(la, st + kHalf);
                // columns past k are zeros: their products are left out
                const int64_t kt = k0 + it;
                const int64_t left = a.k - (kt >= g.kt1 ? kt - g.kt1 : kt) * kDepth;
                const int steps = left >= kDepth ? 4 : (int)((left + 15) / 16);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q >= steps) break;
                    mma1(tmem, db + q * lb.step, da + q * la.step, desc, it > 0 || q > 0);
                }
                commit(empty(s));
            }
            __syncwarp();
            if (++s == g.stages) s = 0, phase ^= 1;
        }
        if (ok && one) commit(done_bar);
        __syncwarp();
    } else {                                                 // the results
        pdl_wait();
        __syncthreads();
        pdl_launch_dependents();
        ok = bar_wait(done_bar, 0);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    }
    if (!ok) {
        if (lane == 0) atomicAdd(&g_matmul_timeouts, 1u);
        failed = 1;
    }
    if (g.splits > 1) cluster_arrive();                      // the ring is free
    // The sums go where the stages were, [column][lane]: all copies have landed and
    // all products have read them.  From there the block writes the result.
    float *part = reinterpret_cast<float *>(dyn + (ring - saddr(dyn)));
    if (warp < kOneWarps && ok) {
        const uint32_t lanes = tmem_base + ((uint32_t)(warp % 4 * 32) << 16);
#pragma unroll 1
        for (int c = warp / 4 * 16; c < g.nt; c += kOneWarps / 4 * 16) {
            float v[16];
            load16(lanes + c, v);
            float *to = part + c * kPitch + warp % 4 * 32 + lane;
#pragma unroll
            for (int e = 0; e < 16; ++e) to[e * kPitch] = g.kt == 0 ? 0.0f : v[e];   // empty sums
        }
    }
    settle<DT, ODT, GATED>(a, split, part, join_bar, failed, g.vec != 0, i0,
                                          tn * kAcross);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (failed && threadIdx.x == 0)       // copies still in flight land before the block ends
        for (int s = 0; s < g.stages; ++s) bar_wait_alone(full(s), 0), bar_wait_alone(full(s), 1);
    __syncthreads();
    if (warp == kOneWarps + 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(columns));
    }
}

// ------------------------------------------------------ some rows, few tiles
//
// Products of more than 64 rows that are too small for the pairs: tiles of 128
// by 128 (128 by 64 where there is little to do but to begin and to end), a block each
// or, split along c, a cluster of blocks.  Both operands in either order.  A whole
// block's warps write the result from the tensor memory, a row a lane.
//
// What bounds it: the shared memory, which takes in and gives out 32 KB a stage: 437
// clocks against the 256 of its products.  256 x 4096 x 4096: 14 us.
//
// A gated block's tile has up to 128 rows of A in the lanes, as many rows of A in a stage as
// there are, and `wide` rows of either weight, whose sums are the accumulator's columns
// beside one another: tiles of 64, 96 or 128, so that each SM has one.
template <int DT, int ODT, bool GATED>
__global__ void __launch_bounds__(kOneThreads, GATED ? 1 : 2)
matmul_mid_kernel(const __grid_constant__ ProductArgs a, const __grid_constant__ OneArgs g)
{
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t bars[2 * kMidStages + 2];
    __shared__ uint32_t tmem_base, failed;
    const uint32_t ring = saddr(dyn) + ((1024 - (saddr(dyn) & 1023)) & 1023);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = g.splits > 1 ? cluster_rank() : 0;
    const int64_t tile = blockIdx.x / g.splits;
    const int64_t tn = tile % g.tiles_n, tm = tile / g.tiles_n;
    const int64_t k0 = g.kt * rank / g.splits, k1 = g.kt * (rank + 1) / g.splits;
    const int rounds = (int)(k1 - k0);
    const uint32_t done_bar = saddr(&bars[2 * kMidStages]), join_bar = done_bar + 8;
    auto full = [&](int s) { return saddr(&bars[s]); };
    auto empty = [&](int s) { return saddr(&bars[kMidStages + s]); };

    const int64_t i0 = tm * 128, j0 = tn * g.wide;
    const int stage = GATED ? mid_gated_stage(g.nt, g.wide) : mid_stage(g.wide);
    const int b_at = GATED ? g.nt * kLine : kHalf;       // B in a stage
    constexpr uint32_t kColumns = GATED ? 256 : 128;     // of tensor memory
    const int rows = (int)(a.m - i0 < 128 ? a.m - i0 : 128);
    const Split split = {rows, 128, g.splits, rank};

    bool ok = true;
    if (warp == kOneWarps) {                                         // the copies
        const bool one = elect_one();
        if (one) {
            for (int s = 0; s < kMidStages; ++s) {
                bar_init(full(s), 1);
                bar_init(empty(s), 1);
            }
            bar_init(done_bar, 1);
            split.expect(join_bar);
            failed = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            prefetch_map(&g.a);
            prefetch_map(&g.b);
        }
        __syncwarp();
        pdl_wait();
        const int32_t ix = (int32_t)i0, jx = (int32_t)j0;
        auto half = [&](uint32_t to, const CUtensorMap *map, int32_t cols, int32_t x, int32_t c,
                        int rows, uint32_t bar) {
            if (cols) {
                box_load(to, map, x, c, bar);
                if (rows > 64) box_load(to + kHalf / 2, map, x + 64, c, bar);
            } else {
                box_load(to, map, c, x, bar);
            }
        };
        auto load = [&](int it, int s) {
            const int64_t kt = k0 + it;
            const bool second = kt >= g.kt1;
            const int32_t c = (int32_t)((second ? kt - g.kt1 : kt) * kDepth);
            const uint32_t st = ring + s * stage;
            bar_expect(full(s), (uint32_t)stage);
            if constexpr (GATED) {
                box_load(st, &g.a, c, ix, full(s));
                box_load(st + b_at, &g.b, c, jx, full(s));
                box_load(st + b_at + g.wide * kLine, &g.b2, c, jx, full(s));
                return;
            }
            half(st, second ? &g.a2 : &g.a, a.a_cols, ix, c, 128, full(s));
            half(st + kHalf, second ? &g.b2 : &g.b, a.b_cols, jx, c, g.wide, full(s));
        };
        const int ahead = rounds < g.stages ? rounds : g.stages;
        for (int it = 0; it < ahead; ++it)
            if (one) load(it, it);
        __syncthreads();
        int s = 0;
        uint32_t phase = 0;
        for (int it = ahead; it < rounds; ++it) {
            ok = bar_wait(empty(s), phase);
            if (!ok) break;
            if (one) load(it, s);
            __syncwarp();
            if (++s == g.stages) s = 0, phase ^= 1;
        }
    } else if (warp == kOneWarps + 1) {                                  // the products
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         saddr(&tmem_base)), "r"(kColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncthreads();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const bool one = elect_one();
        const uint32_t tmem = tmem_base;
        const Layout la = layout_of(a.a_cols), lb = layout_of(a.b_cols);
        // (a gated block's lanes past its rows of A hold what follows them, which nothing reads)
        const uint32_t desc = shape_desc<DT>(a.a_cols, a.b_cols) |
                              ((uint32_t)((GATED ? 2 : 1) * g.wide >> 3) << 17) |
                              ((128u >> 4) << 24);
        int s = 0;
        uint32_t phase = 0;
        for (int it = 0; it < rounds; ++it) {
            ok = bar_wait(full(s), phase);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (one) {
                const uint64_t da = at(la, ring + s * stage);
                const uint64_t db = at(lb, ring + s * stage + b_at);
                const int64_t kt = k0 + it;
                const int64_t left = a.k - (kt >= g.kt1 ? kt - g.kt1 : kt) * kDepth;
                const int steps = left >= kDepth ? 4 : (int)((left + 15) / 16);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q >= steps) break;
                    mma1(tmem, da + q * la.step, db + q * lb.step, desc, it > 0 || q > 0);
                }
                commit(empty(s));
            }
            __syncwarp();
            if (++s == g.stages) s = 0, phase ^= 1;
        }
        if (ok && one) commit(done_bar);
        __syncwarp();
    } else {                                                 // the results
        pdl_wait();
        __syncthreads();
        pdl_launch_dependents();
        ok = bar_wait(done_bar, 0);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    }
    if (!ok) {
        if (lane == 0) atomicAdd(&g_matmul_timeouts, 1u);
        failed = 1;
    }
    if (g.splits > 1) cluster_arrive();                      // the ring is free
    // all copies have landed and all products have read them: the stages' place is free
    float *part = reinterpret_cast<float *>(dyn + (ring - saddr(dyn)));
    const int row = warp % 4 * 32;
    const uint32_t lanes = tmem_base + ((uint32_t)row << 16);
    if (g.splits == 1) {
        if (warp < kOneWarps && ok && i0 + row < a.m) {
            float *staged = part + warp * 32 * kStagePad;
#pragma unroll 1
            for (int c = warp / 4 * 32; c < g.wide; c += kOneWarps / 4 * 32) {
                Beside<DT, ODT, GATED> beside;
                if (g.vec && j0 + c + 32 <= a.n && i0 + row + lane < a.m)
                    beside.ask(a, i0 + row + lane, j0 + c);
                uint32_t r[32], r2[32];
                load32(lanes + c, r);
                if constexpr (GATED) load32(lanes + g.wide + c, r2);
                float z[32], z2[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    z[e] = __uint_as_float(r[e]);
                    z2[e] = GATED ? __uint_as_float(r2[e]) : 0.0f;
                }
                finish_rows<DT, ODT, GATED>(a, g.vec != 0, staged, i0 + row, a.m, j0 + c,
                                                  beside, z, z2);
            }
        }
    } else if constexpr (!GATED) {
        if (warp < kOneWarps && ok) {
#pragma unroll 1
            for (int c = warp / 4 * 16; c < 128; c += kOneWarps / 4 * 16) {
                float v[16];
                load16(lanes + c, v);
                float4 *to = reinterpret_cast<float4 *>(part + (row + lane) * kPitch + c);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    to[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            }
        }
        settle<DT, ODT, false>(a, split, part, join_bar, failed, g.vec != 0, i0, j0);
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (failed && threadIdx.x == 0)       // copies still in flight land before the block ends
        for (int s = 0; s < g.stages; ++s) bar_wait_alone(full(s), 0), bar_wait_alone(full(s), 1);
    __syncthreads();
    if (warp == kOneWarps + 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(kColumns));
    }
}

// ------------------------------------------------------------ the pair kernel
//
// Large products: two SMs share a tile of 256 rows of A by 256 rows of B, so that
// either reads only its own 128 rows of both.  The first block's MMA
// warp issues for both (cta_group::2), and both blocks' copies arrive at its
// barriers.  Lanes are rows of A, so that a thread holds consecutive columns of a
// row of the result.  A gated tile has 128 columns of the result: the first block
// brings the gate's weights, the second the other ones, and the accumulator's
// columns are 128 sums of either.
//
// The blocks are persistent, with two accumulators of 256 columns (all of the
// tensor memory): eight warps write one tile's result, in 32 columns at a time,
// while the next tile's products run.
//
// What bounds it: the tensor cores, and in long runs the power limit.  8192 x 8192 x 8192
// 560 us in all orders (1.96 PFLOP/s); a gated 8192 x 11008 x 4096 716 us, and the
// gradient of its input from two pairs 766 (2.0 and 1.93).
constexpr int kPairStages = 6;
constexpr int kPairStage = 2 * kHalf;
constexpr int kPairWarps = 8;                            // of results
constexpr int kPairThreads = (kPairWarps + 2) * 32;
constexpr int kPairStaged = kPairWarps * 32 * kStagePad * 4;
constexpr int kPairSmem = kPairStages * kPairStage + kPairStaged + 1024;
static_assert(kPairSmem <= kSmemBlock, "one block's shared memory");

struct PairArgs {
    CUtensorMap a, b, b2, a2;
    int64_t kt1, kt;                     // stages of the first pair of operands, of both
    int64_t tiles_n, tiles_m;
    int32_t half;                        // rows of B that either block brings, at most 128
    int32_t cut;                         // parts of a tile from tile `whole` on
    int64_t whole, steps;                // steps: whole tiles and parts
    int32_t vec;                         // finish_run's boundaries hold
};

// Step t of the sweep: bands of 8 tiles of rows of A (16 of a gated block), so that
// the blocks at work at one time share both operands in L2 (8192 x 8192 x 8192 at the
// power limit: bands of 4, 8, 16, 32 660, 648, 663, 698 us; a gated 11008 x 4096 over
// 8192 rows 909, 881, 863, 939).  The tiles of the last, unfilled turn
// go in `cut` parts, so that all pairs share them.  Rows from row0 on; `half` rows of
// B in either block, from row first + rank * half on (a gated block's from first
// on in both); columns of the result from first on.  The last tile of a row is as
// narrow as what is left, in steps of 32 columns.
struct PairTile {
    int64_t row0, first;
    int half;                            // 0: nothing left for this part
};

template <bool GATED>
__device__ __forceinline__ PairTile pair_tile(const PairArgs &g, int64_t n, int64_t t)
{
    int64_t tile = t;
    int part = 0, half = g.half;
    if (t >= g.whole) {
        tile = g.whole + (t - g.whole) / g.cut;
        part = (int)((t - g.whole) % g.cut);
        half /= g.cut;
    }
    constexpr int kBand = GATED ? 16 : 8;
    const int64_t band = tile / (kBand * g.tiles_n), in = tile - band * kBand * g.tiles_n;
    const int64_t rest = g.tiles_m - band * kBand, wide = rest < kBand ? rest : kBand;
    const int64_t tn = in / wide, tm = band * kBand + in - tn * wide;
    const int across = GATED ? 1 : 2;
    PairTile p;
    p.row0 = tm * 256;
    p.first = (tn * g.half + part * half) * across;
    const int64_t left = n - p.first;
    if (left < across * half) {
        if constexpr (GATED) half = left <= 0 ? 0 : (int)((left + 15) / 16 * 16);
        else half = left <= 0 ? 0 : (int)((left + 31) / 32 * 16);
    }
    p.half = half;
    return p;
}

template <int DT, int ODT, bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads)
matmul_pair_kernel(const __grid_constant__ ProductArgs a, const __grid_constant__ PairArgs g)
{
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t bars[2 * kPairStages + 4];
    __shared__ uint32_t tmem_base, failed;
    const uint32_t ring = saddr(dyn) + ((1024 - (saddr(dyn) & 1023)) & 1023);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int64_t step = gridDim.x / 2;
    auto full = [&](int s) { return saddr(&bars[s]); };                     // the first block's
    auto empty = [&](int s) { return saddr(&bars[kPairStages + s]); };
    auto done = [&](int b) { return saddr(&bars[2 * kPairStages + b]); };
    auto drained = [&](int b) { return saddr(&bars[2 * kPairStages + 2 + b]); };  // the first's

    if (warp == kPairWarps) {
        if (lane == 0) {
            for (int s = 0; s < 2 * kPairStages + 2; ++s) bar_init(saddr(&bars[s]), 1);
            for (int b = 0; b < 2; ++b) bar_init(drained(b), 2 * kPairWarps);
            failed = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
    } else if (warp == kPairWarps + 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         saddr(&tmem_base)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync();             // both blocks' barriers and tensor memory are there
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_base;
    pdl_wait();
    pdl_launch_dependents();

    bool ok = true;
    if (warp == kPairWarps) {                                // the copies
        const bool one = elect_one();
        // (the transpose comes in chunks of 64 rows)
        const int brought = (a.b_cols ? (g.half + 63) / 64 * 64 : g.half) * kLine;
        int s = 0;
        uint32_t phase = 1;                                  // the stages start empty
        for (int64_t t = blockIdx.x / 2; t < g.steps && ok; t += step) {
            const PairTile p = pair_tile<GATED>(g, a.n, t);
            if (p.half == 0) continue;
            const int32_t ix = (int32_t)(p.row0 + rank * 128);
            const int32_t jx = (int32_t)(p.first + (GATED ? 0 : rank * p.half));
            for (int64_t kt = 0; kt < g.kt; ++kt) {
                ok = bar_wait(empty(s), phase);
                if (!ok) break;
                if (one) {
                    const bool second = kt >= g.kt1;
                    const int32_t c = (int32_t)((second ? kt - g.kt1 : kt) * kDepth);
                    const CUtensorMap *ma = second ? &g.a2 : &g.a;
                    const CUtensorMap *mb = (GATED ? rank != 0 : second) ? &g.b2 : &g.b;
                    const uint32_t st = ring + s * kPairStage, bar = peer_addr(full(s), 0);
                    if (rank == 0) bar_expect(full(s), (uint32_t)(2 * (kHalf + brought)));
                    if (a.a_cols) {
                        tensor_load(st, ma, ix, c, bar);
                        tensor_load(st + kHalf / 2, ma, ix + 64, c, bar);
                    } else {
                        tensor_load(st, ma, c, ix, bar);
                    }
                    if (a.b_cols) {
                        tensor_load(st + kHalf, mb, jx, c, bar);
                        if (g.half > 64)
                            tensor_load(st + kHalf + kHalf / 2, mb, jx + 64, c, bar);
                    } else {
                        tensor_load(st + kHalf, mb, c, jx, bar);
                    }
                }
                __syncwarp();
                if (++s == kPairStages) s = 0, phase ^= 1;
            }
        }
    } else if (warp == kPairWarps + 1) {                     // the products
        if (rank == 0) {
            const bool one = elect_one();
            const Layout la = layout_of(a.a_cols), lb = layout_of(a.b_cols);
            const uint32_t shape = shape_desc<DT>(a.a_cols, a.b_cols) | ((256u >> 4) << 24);
            const int last_steps = (int)((a.k - (g.kt1 - 1) * kDepth + 15) / 16);
            int s = 0;
            uint32_t phase = 0, i = 0, drained_phase = 1;    // the accumulators start drained
            for (int64_t t = blockIdx.x / 2; t < g.steps && ok; t += step) {
                const PairTile p = pair_tile<GATED>(g, a.n, t);
                if (p.half == 0) continue;
                const uint32_t desc = shape | ((uint32_t)(2 * p.half) >> 3 << 17);
                const uint32_t acc = tmem + i * 256;
                ok = bar_wait(drained((int)i), drained_phase);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                for (int64_t kt = 0; kt < g.kt; ++kt) {
                    ok = bar_wait(full(s), phase);
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    if (one) {
                        const uint64_t da = at(la, ring + s * kPairStage);
                        const uint64_t db = at(lb, ring + s * kPairStage + kHalf);
                        const int steps = kt == g.kt1 - 1 || kt == g.kt - 1 ? last_steps : 4;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (q >= steps) break;
                            mma2(acc, da + q * la.step, db + q * lb.step, desc, kt > 0 || q > 0);
                        }
                        commit2(empty(s));
                        if (kt == g.kt - 1) commit2(done((int)i));
                    }
                    __syncwarp();
                    if (++s == kPairStages) s = 0, phase ^= 1;
                }
                i ^= 1;
                if (i == 0) drained_phase ^= 1;
            }
        }
    } else {                                                 // the results
        const int part = warp & 3, turn = warp >> 2;
        const uint32_t lanes = (uint32_t)(part * 32) << 16;
        float *staged = reinterpret_cast<float *>(dyn + (ring - saddr(dyn)) +
                                                  kPairStages * kPairStage) +
                        warp * 32 * kStagePad;
        uint32_t b = 0, done_phase = 0;
        for (int64_t t = blockIdx.x / 2; t < g.steps; t += step) {
            const PairTile p = pair_tile<GATED>(g, a.n, t);
            if (p.half == 0) continue;
            ok = bar_wait(done((int)b), done_phase);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const int half = p.half;
            const int64_t i0 = p.row0 + rank * 128 + part * 32, j0 = p.first;
            const int wide = GATED ? half : 2 * half;        // columns of the result
#pragma unroll 1
            for (int c = turn * 32; c < wide; c += 64) {
                const uint32_t from = tmem + lanes + b * 256 + c;
                Beside<DT, ODT, GATED> beside;
                if (g.vec && j0 + c + 32 <= a.n && i0 + lane < a.m)
                    beside.ask(a, i0 + lane, j0 + c);
                uint32_t r[32], r2[32];
                load32(from, r);
                if constexpr (GATED) load32(from + half, r2);
                float z[32], z2[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    z[e] = __uint_as_float(r[e]);
                    z2[e] = GATED ? __uint_as_float(r2[e]) : 0.0f;
                }
                finish_rows<DT, ODT, GATED>(a, g.vec != 0, staged, i0, a.m, j0 + c, beside, z,
                                                   z2);
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) arrive_first(drained((int)b));
            b ^= 1;
            if (b == 0) done_phase ^= 1;
        }
    }
    if (!ok) {
        if (lane == 0) atomicAdd(&g_matmul_timeouts, 1u);
        failed = 1;
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    // copies still in flight land before either block ends
    if (failed && threadIdx.x == 0 && rank == 0)
        for (int s = 0; s < kPairStages; ++s) bar_wait_alone(full(s), 0), bar_wait_alone(full(s), 1);
    __syncthreads();
    cluster_sync();             // nothing of either block is still in use by the other
    if (warp == kPairWarps + 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(512u));
    }
}

// ------------------------------------------------------- rows onto boundaries
//
// A matrix whose rows do not begin on 16-byte boundaries, copied to one whose
// rows do: a warp takes twice 256 elements, a lane one of 32 consecutive at a time.
__global__ void __launch_bounds__(kThreads)
align_rows_kernel(const uint16_t *from, int64_t rows, int64_t cols, int64_t stride, uint16_t *to,
                  int64_t to_stride, int64_t runs)
{
    constexpr int U = 2;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t w = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * U;
    uint16_t v[U][8];
    int64_t r[U], c0[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        rows::run_at(w + k, runs, r[k], c0[k]);
        c0[k] += threadIdx.x & 31;
        const uint16_t *p = from + r[k] * stride + c0[k];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[k][e] = r[k] < rows && c0[k] + 32 * e < cols ? p[32 * e] : (uint16_t)0;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        uint16_t *p = to + r[k] * to_stride + c0[k];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (r[k] < rows && c0[k] + 32 * e < cols) p[32 * e] = v[k][e];
    }
}

cudaError_t align_rows(const void *from, int64_t rows, int64_t cols, int64_t stride, void *to,
                       int64_t to_stride, cudaStream_t s)
{
    const int64_t runs = (cols + 255) / 256, blocks = (rows * runs + 15) / 16;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_dependent(align_rows_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s,
                            static_cast<const uint16_t *>(from), rows, cols, stride,
                            static_cast<uint16_t *>(to), to_stride, runs);
}

// ------------------------------------------------------------------- the host

using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                            const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                            const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encoder(Encode &f)
{
    static std::atomic<Encode> known{nullptr};
    f = known.load(std::memory_order_relaxed);
    if (f) return cudaSuccess;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                     cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (!p || found != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
    f = reinterpret_cast<Encode>(p);
    known.store(f, std::memory_order_relaxed);
    return cudaSuccess;
}

// `rows` rows of k elements, or (cols) their transpose; boxes of 64 c by
// `box` rows, or of 64 rows by 64 c.
cudaError_t operand_map(CUtensorMap *map, const void *p, int64_t rows, int64_t k, int64_t stride,
                        int32_t cols, int box)
{
    Encode f;
    const cudaError_t e = encoder(f);
    if (e != cudaSuccess) return e;
    const cuuint64_t dims[2] = {(cuuint64_t)(cols ? rows : k), (cuuint64_t)(cols ? k : rows)};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t boxes[2] = {64, (cuuint32_t)(cols ? 64 : box)}, one[2] = {1, 1};
    const CUresult r = f(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(p), dims,
                         strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The maps of one call's operands, `rows_a` rows of A and `rows_b` of B a box.
template <class G>
cudaError_t operand_maps(const ProductArgs &a, G &g, int rows_a, int rows_b)
{
    if (a.k == 0) return cudaSuccess;                   // nothing is read
    cudaError_t e = operand_map(&g.a, a.a, a.m, a.k, a.a_stride, a.a_cols, rows_a);
    if (e == cudaSuccess) e = operand_map(&g.b, a.b, a.n, a.k, a.b_stride, a.b_cols, rows_b);
    if (e == cudaSuccess && a.b2)
        e = operand_map(&g.b2, a.b2, a.n, a.k, a.b2_stride, a.b_cols, rows_b);
    if (e == cudaSuccess && a.a2)
        e = operand_map(&g.a2, a.a2, a.m, a.k, a.a2_stride, a.a_cols, rows_a);
    return e;
}

// Whether runs of 32 bytes of a row of everything that is written beside the
// result, and of what is added, lie on their boundaries.
template <int ODT> bool in_runs(const ProductArgs &a)
{
    constexpr int kOut = ODT == F32 ? 4 : 2;
    auto rows = [](const void *p, int64_t stride, int es) {
        return !p || ((uintptr_t)p % 32 == 0 && stride * es % 32 == 0);
    };
    return rows(a.out, a.stride, kOut) && rows(a.residual, a.residual_stride, kOut) &&
           rows(a.kept, a.kept_stride, 2) && rows(a.kept2, a.kept_stride, 2) &&
           ((uintptr_t)a.bias & 15) == 0;
}

template <int DT, int ODT, bool GATED>
cudaError_t pair_go(const ProductArgs &a, int sms, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    cudaError_t e =
        allow_shared(reinterpret_cast<const void *>(matmul_pair_kernel<DT, ODT, GATED>),
                     kSmemBlock, done);
    if (e != cudaSuccess) return e;
    PairArgs g;
    const PairShape t = pair_shape(a.m, a.n, sms, GATED);
    g.half = t.half, g.cut = t.cut;
    g.tiles_m = t.tiles_m, g.tiles_n = t.tiles_n;
    g.whole = t.whole, g.steps = t.steps;
    e = operand_maps(a, g, 128, g.half);
    if (e != cudaSuccess) return e;
    g.kt1 = (a.k + kDepth - 1) / kDepth;
    g.kt = a.a2 ? 2 * g.kt1 : g.kt1;
    g.vec = in_runs<ODT>(a);
    const int64_t pairs = g.steps < sms / 2 ? g.steps : sms / 2;
    return launch_dependent(matmul_pair_kernel<DT, ODT, GATED>, dim3((unsigned)(2 * pairs)),
                            dim3(kPairThreads), kSmemBlock, s, a, g);
}

// A launch in clusters of `splits` blocks.
struct Clusters {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    Clusters(int64_t blocks, int splits, int smem, cudaStream_t s)
    {
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3(kOneThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)splits;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
    }
};

// Clusters of a kernel's blocks that find a place at once on the current device, through
// what is known of it.
auto clusters_of(const void *kernel, Room &room)
{
    return [kernel, &room](int splits, int stages, int smem) {
        int device = -1;
        if (cudaGetDevice(&device) != cudaSuccess) device = -1;
        return room.of(device, splits, stages, smem, [&](int n, int bytes, int &found) {
            Clusters c(n, n, bytes, nullptr);
            const bool answered =
                cudaOccupancyMaxActiveClusters(&found, kernel, &c.cfg) == cudaSuccess;
            if (!answered) cudaGetLastError();
            return answered;
        });
    };
}

int64_t stages_of(const ProductArgs &a)
{
    return (a.k + kDepth - 1) / kDepth * (a.a2 ? 2 : 1);
}

template <int ODT> bool needs_staging(const ProductArgs &a)       // finish_rows does
{
    return !in_runs<ODT>(a) || a.n % 32;
}

// (The device's answer on room depends on what a kernel is allowed: asked first.)
template <int DT, int ODT, bool GATED> cudaError_t allow_one()
{
    static std::atomic<uint64_t> done{0};
    return allow_shared(reinterpret_cast<const void *>(matmul_kernel<DT, ODT, GATED>), kSmemBlock,
                        done);
}

template <int DT, int ODT> cudaError_t allow_mid()
{
    static std::atomic<uint64_t> done{0};
    return allow_shared(reinterpret_cast<const void *>(matmul_mid_kernel<DT, ODT, false>),
                        kSmemBlock, done);
}

// matmul_kernel with `tiles_m` tiles of rows of A, as equal as multiples of 16 can be.
template <int DT, int ODT, bool GATED>
Cut one_cut(const ProductArgs &a, int64_t tiles_m, int nt, int sms)
{
    constexpr int kAcross = GATED ? 64 : 128;
    static Room room[2][16];                          // for each width of a tile
    const bool staged = needs_staging<ODT>(a);
    const auto place = clusters_of(reinterpret_cast<const void *>(matmul_kernel<DT, ODT, GATED>),
                                   room[staged][nt / 16 - 1]);
    return choose_split(stages_of(a), (a.n + kAcross - 1) / kAcross * tiles_m, sms, Tile::most(nt),
                        kMostBlocks, [&](int stages, int splits) {
                            return Tile::smem(stages, nt, splits, staged);
                        }, place);
}

template <int DT, int ODT, bool GATED>
cudaError_t one_go(const ProductArgs &a, int64_t tiles_m, int sms, cudaStream_t s)
{
    using Tl = Tile;
    constexpr int kAcross = GATED ? 64 : 128;
    const auto kernel = matmul_kernel<DT, ODT, GATED>;
    cudaError_t e = allow_one<DT, ODT, GATED>();
    if (e != cudaSuccess) return e;
    OneArgs g;
    g.nt = g.span = width(a.m, tiles_m);
    e = operand_maps(a, g, g.nt, kAcross);
    if (e != cudaSuccess) return e;
    g.kt1 = (a.k + kDepth - 1) / kDepth;
    g.kt = stages_of(a);
    g.tiles_n = (a.n + kAcross - 1) / kAcross;
    g.vec = in_runs<ODT>(a);
    const Cut cut = one_cut<DT, ODT, GATED>(a, tiles_m, g.nt, sms);
    g.splits = cut.splits, g.stages = cut.stages;
    const int64_t blocks = g.tiles_n * tiles_m * g.splits;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    Clusters c(blocks, g.splits, Tl::smem(g.stages, g.nt, g.splits, needs_staging<ODT>(a)), s);
    return cudaLaunchKernelEx(&c.cfg, kernel, a, g);
}

// matmul_mid_kernel: tiles of 128 by 128, or, `wide`, 64.
template <int DT, int ODT> Cut mid_cut(const ProductArgs &a, int wide, int sms)
{
    static Room room[2];
    const bool staged = needs_staging<ODT>(a);
    const int64_t kt = stages_of(a);
    if (wide < 128) return {1, kt < kMidStages ? (int)kt : kMidStages, 0};
    const auto place = clusters_of(reinterpret_cast<const void *>(matmul_mid_kernel<DT, ODT, false>),
                                   room[staged]);
    return choose_split(kt, (a.n + wide - 1) / wide * ((a.m + 127) / 128), sms, kMidStages, 2,
                        [&](int stages, int splits) {
                            return mid_smem(stages, wide, splits, staged);
                        }, place);
}

// (100 x 256 by 64 columns c: with 64 columns of the result a block 2.7 us, with 128 3.1)
int mid_width(const ProductArgs &a, int sms)
{
    return stages_of(a) <= 16 && (a.n + 63) / 64 * ((a.m + 127) / 128) <= sms ? 64 : 128;
}

template <int DT, int ODT> cudaError_t mid_go(const ProductArgs &a, int sms, cudaStream_t s)
{
    const auto kernel = matmul_mid_kernel<DT, ODT, false>;
    cudaError_t e = allow_mid<DT, ODT>();
    if (e != cudaSuccess) return e;
    OneArgs g;
    g.kt1 = (a.k + kDepth - 1) / kDepth;
    g.kt = stages_of(a);
    g.wide = mid_width(a, sms);
    e = operand_maps(a, g, 128, g.wide);
    if (e != cudaSuccess) return e;
    g.tiles_n = (a.n + g.wide - 1) / g.wide;
    g.vec = in_runs<ODT>(a);
    g.nt = g.span = 128;
    const Cut cut = mid_cut<DT, ODT>(a, g.wide, sms);
    g.splits = cut.splits, g.stages = cut.stages;
    const int64_t blocks = g.tiles_n * ((a.m + 127) / 128) * g.splits;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    Clusters c(blocks, g.splits, mid_smem(g.stages, g.wide, g.splits, needs_staging<ODT>(a)), s);
    return cudaLaunchKernelEx(&c.cfg, kernel, a, g);
}

// A gated block in one tile a SM, rows of A in the lanes.
template <int DT> cudaError_t mid_gated_go(const ProductArgs &a, int wide, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    const auto kernel = matmul_mid_kernel<DT, DT, true>;
    cudaError_t e = allow_shared(reinterpret_cast<const void *>(kernel), kSmemBlock, done);
    if (e != cudaSuccess) return e;
    OneArgs g;
    g.nt = a.m < 128 ? width(a.m, 1) : 128;
    g.wide = wide;
    e = operand_maps(a, g, g.nt, wide);
    if (e != cudaSuccess) return e;
    g.kt = g.kt1 = stages_of(a);
    g.tiles_n = (a.n + wide - 1) / wide;
    g.vec = in_runs<DT>(a);
    g.splits = 1;
    g.span = 128;
    const int most = (kSmemBlock - 1024) / mid_gated_stage(g.nt, wide);
    g.stages = most < kMidStages ? most : kMidStages;
    if (g.kt < g.stages) g.stages = (int)g.kt;
    Clusters c(g.tiles_n * ((a.m + 127) / 128), 1, mid_gated_smem(g.stages, g.nt, wide), s);
    return cudaLaunchKernelEx(&c.cfg, kernel, a, g);
}

// Whether matvec_kernel takes the product.
bool one_row(const ProductArgs &a)
{
    return a.m == 1 && a.k > 0 && !a.a_cols && !a.b_cols && !a.a2;
}

template <int DT, int ODT, bool GATED>
cudaError_t matvec_go(const ProductArgs &a, int sms, cudaStream_t s)
{
    const rows::In x = rows::in(a.a, a.a_stride);
    const rows::In w = rows::in(a.b, a.b_stride);
    const rows::In w2 = rows::in(a.b2, a.b2_stride);
    const bool vec = rows_aligned(a.a, 0, DT, a.k) && rows_aligned(a.b, a.b_stride, DT, a.k) &&
                     (!a.b2 || rows_aligned(a.b2, a.b2_stride, DT, a.k));
    const int64_t blocks = (a.n + 31) / 32;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    // warps that read 20 rows' strides at once on every SM, as long as a row is long
    // enough to share
    const int64_t strides = blocks * 8 * (GATED ? 2 : 1), want = (int64_t)sms * 20;
    const int ks = strides >= want || a.k <= 512 ? 1 : strides * 2 >= want || a.k <= 1024 ? 2 : 4;
    auto go = [&](auto k, int threads) {
        return launch_dependent(k, dim3((unsigned)blocks), dim3(threads), 0, s, a, x, w, w2);
    };
    if (!vec) return ks == 1 ? go(matvec_kernel<DT, ODT, GATED, 1, false>, 256)
                             : go(matvec_kernel<DT, ODT, GATED, 2, false>, 512);
    return ks == 1 ? go(matvec_kernel<DT, ODT, GATED, 1, true>, 256)
           : ks == 2 ? go(matvec_kernel<DT, ODT, GATED, 2, true>, 512)
                     : go(matvec_kernel<DT, ODT, GATED, 4, true>, 1024);
}

template <int DT, int ODT, bool GATED>
cudaError_t pick(const ProductArgs &a, int sms, cudaStream_t s)
{
    if (one_row(a)) return matvec_go<DT, ODT, GATED>(a, sms, s);
    // Few rows, or no more tiles of 128 by 128 than SMs: the single blocks, whose
    // columns c can be split.  Beyond that the pairs.
    const int64_t tiles = ((a.n + 127) / 128) * ((a.m + 127) / 128);
    if (a.k > 0 && a.m > 64 && tiles > sms) return pair_go<DT, ODT, GATED>(a, sms, s);
    if constexpr (!GATED) {
        if (a.k > 0 && a.m > 128 && !a.a_cols && mid_width(a, sms) == 128) {
            // Tiles of up to 256 rows of A by 128 of B, where they leave clearly less to
            // the fullest SM, a stage's time being that of its rows: 384 x 4096 x 4096
            // 18.2 us in tiles of 128 by 128, 16.6 in tiles of 192; 333 x 1600 x 6400
            // 13.9 and 13.6.  With 5% less to do they are behind (1024 x 1024 x 4096, 3
            // blocks a tile for 2: 13.2 us and 14.5).
            cudaError_t e = allow_one<DT, ODT, false>();
            if (e == cudaSuccess) e = allow_mid<DT, ODT>();
            if (e != cudaSuccess) return e;
            const int64_t few = (a.m + 255) / 256;
            int64_t best = 0, least = mid_cut<DT, ODT>(a, 128, sms).least * 256 / 8 * 7;
            for (int64_t tiles_m = few; tiles_m < few + 3; ++tiles_m) {
                const int nt = width(a.m, tiles_m);
                const Cut c = one_cut<DT, ODT, false>(a, tiles_m, nt, sms);
                if (c.stages < 1 || c.least * (128 + nt) >= least) continue;
                least = c.least * (128 + nt);
                best = tiles_m;
            }
            if (best) return one_go<DT, ODT, false>(a, best, sms, s);
        }
        if (a.k > 0 && (a.m > 64 || a.a_cols)) return mid_go<DT, ODT>(a, sms, s);
    } else if (a.k > 0) {
        // One tile a SM, as narrow as that allows, against tiles of 64 that may be split
        // or be two on some SMs: by the bytes of the fullest SM.  (2 x 11008 x 4096, 115
        // tiles of 96 and 172 of 64: 16 rows 31.4 us and 34.8, 77 rows 32.5 and 34.4; 256
        // rows of 2 x 6400 x 1600 12.3 and 15.5.)
        const int64_t tiles_m = (a.m + 127) / 128;
        int wide = 64;
        while (wide < 128 && (a.n + wide - 1) / wide * tiles_m > sms) wide += 32;
        const int nt = a.m < 128 ? width(a.m, 1) : 128, one = width(a.m, tiles_m);
        const cudaError_t e = allow_one<DT, ODT, true>();
        if (e != cudaSuccess) return e;
        if ((a.n + wide - 1) / wide * tiles_m <= sms &&
            stages_of(a) * (nt + 2 * wide) * 8 <
                one_cut<DT, ODT, true>(a, tiles_m, one, sms).least * (128 + one) * 7)
            return mid_gated_go<DT>(a, wide, s);
    }
    return one_go<DT, ODT, GATED>(a, (a.m + 127) / 128, sms, s);
}

// An operand's place in the workspace, if it needs one: bytes.
struct Place {
    int64_t rows, cols, stride;                       // as it lies
    int64_t bytes() const
    {
        return (rows * ((cols + 7) / 8 * 8) * 2 + 127) / 128 * 128;
    }
};

bool on_boundaries(const void *p, int64_t rows, int64_t stride)
{
    return ((uintptr_t)p & 15) == 0 && (rows <= 1 || stride % 8 == 0);
}

}  // namespace

int64_t product_workspace(const ProductArgs &a)
{
    if (one_row(a)) return 0;
    int64_t need = 0;
    auto add = [&](const void *p, int64_t rows, int32_t cols, int64_t stride) {
        const Place at = cols ? Place{a.k, rows, stride} : Place{rows, a.k, stride};
        if (p && !on_boundaries(p, at.rows, stride)) need += at.bytes();
    };
    add(a.a, a.m, a.a_cols, a.a_stride);
    add(a.b, a.n, a.b_cols, a.b_stride);
    add(a.a2, a.m, a.a_cols, a.a2_stride);
    add(a.b2, a.n, a.b_cols, a.b2_stride);
    return need;
}

cudaError_t launch_product(int32_t dt, int32_t odt, ProductArgs a, void *workspace, int sms,
                           cudaStream_t s)
{
    if (a.m <= 0 || a.n <= 0) return cudaSuccess;
    if (a.k > 0 && !one_row(a)) {
        char *room = static_cast<char *>(workspace);
        cudaError_t e = cudaSuccess;
        auto settle = [&](const void *&p, int64_t rows, int32_t cols, int64_t &stride) {
            if (!p || e != cudaSuccess) return;
            const Place at = cols ? Place{a.k, rows, stride} : Place{rows, a.k, stride};
            if (!on_boundaries(p, at.rows, stride)) {
                const int64_t to = (at.cols + 7) / 8 * 8;
                e = align_rows(p, at.rows, at.cols, stride, room, to, s);
                p = room;
                stride = to;
                room += at.bytes();
            } else if (at.rows <= 1) {
                stride = (at.cols + 7) / 8 * 8;       // of no use, but it has to be a stride
            }
        };
        settle(a.a, a.m, a.a_cols, a.a_stride);
        settle(a.b, a.n, a.b_cols, a.b_stride);
        settle(a.a2, a.m, a.a_cols, a.a2_stride);
        settle(a.b2, a.n, a.b_cols, a.b2_stride);
        if (e != cudaSuccess) return e;
    }
    if (a.gated)
        return dt == BF16 ? pick<BF16, BF16, true>(a, sms, s) : pick<F16, F16, true>(a, sms, s);
    if (dt == BF16)
        return odt == F32 ? pick<BF16, F32, false>(a, sms, s) : pick<BF16, BF16, false>(a, sms, s);
    return odt == F32 ? pick<F16, F32, false>(a, sms, s) : pick<F16, F16, false>(a, sms, s);
}

cudaError_t matmul_timeouts(unsigned int *count)
{
    // the copy alone would not wait for streams that do not synchronise with the
    // default one
    const cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return e;
    return cudaMemcpyFromSymbol(count, g_matmul_timeouts, sizeof(unsigned int));
}

}  // namespace zgb
