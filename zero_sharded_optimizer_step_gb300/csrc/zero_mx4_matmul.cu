// Product of two microscaled 4-bit matrices on the tensor cores:
//
//   out[i, j] (+)= alpha * sum over c of A[i, c] * B[j, c]
//
// A is [m, k] and B [n, k], both as zero_mx4_quantize lays them out.  The
// 128 lanes of an accumulator tile are 128 rows of B (128 consecutive columns
// of the result, so that a warp's stores are contiguous without going through
// shared memory) and its columns NT rows of A: with few tokens the tile is
// as narrow as they are, and the product reads the weights once.
//
// A record of 128 rows by 256 columns lies in memory as the tensor core wants
// it in shared memory (128-byte rows, 16-byte pieces exchanged by the row's
// low bits; then the scale exponents in the order in which tcgen05.cp spreads
// them over the lanes), so one bulk copy brings it in.  tcgen05.mma of kind
// mxf4 multiplies 64 columns at a time and applies the scales; the sums stay
// in 32 bits in tensor memory.
//
// A block has one warp that issues the copies, one that issues the
// products, and four that write the result.  With fewer tiles than SMs the columns
// of A and B are split over a cluster of up to 8 blocks, whose partial sums
// join through distributed shared memory in the blocks' order.
//
// Every wait on a barrier is bounded; one that runs out is counted and ends
// the block without a store.
//
// What bounds it: with few rows of A the bytes of B and the latency of a launch
// (one row by 11008 x 4096: 6.7 us for 24 MB; 768 x 768: 2.5 us), with many the
// tensor cores, whose rate for this kind is 16,384 multiply-adds a clock and SM
// (measured: 128 clocks for 128 x 256 x 64).  Large products take the pair
// kernel: 8192^3 in 149 us, 7.4 PFLOP/s, the tensor pipe 84% busy.
#include <atomic>

#include <cuda.h>

#include "zero_elems.cuh"
#include "zero_ops.h"
#include "zero_tensor.cuh"

namespace zgb {
namespace {

__device__ unsigned int g_mx4_timeouts;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

__device__ __forceinline__ uint64_t scale_desc(uint32_t addr)       // 16-byte rows, as they lie
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}

__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                 : "memory");
}

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t sa, uint32_t sb, uint32_t add)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X"
                 " [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
                 "r"(sa), "r"(sb), "r"(add) : "memory");
}

template <int NT> struct Tile {
    static_assert(NT <= 128, "a record of A at most");
    static constexpr int kACodes = NT * 128;                // A's codes of a stage
    static constexpr int kStage = kMxRecord + kACodes + kMxScales;
    // the accumulator, 8 columns of B's scales, 8 of A's
    static constexpr int kTmemUsed = NT + 16;
    static constexpr int kTmem = kTmemUsed <= 32 ? 32 : kTmemUsed <= 64 ? 64
                                 : kTmemUsed <= 128 ? 128 : 256;
    static constexpr int kStages = kSmemBlock / kStage < 6 ? (kSmemBlock - 1024) / kStage : 6;
    static constexpr int kPart = NT * 128 * 4;              // a split's partial sums
    // Shared memory of a block, for so many stages.  A block's share of it is
    // at least its share of the tensor memory, so that no block on an
    // SM waits for tensor memory that another one holds: two that wait for
    // their cluster peers so would wait forever.
    static constexpr int smem(int stages)
    {
        const int ring = stages * kStage > kPart ? stages * kStage : kPart;
        const int share = (kSmemSm / (512 / kTmem) + 127) / 128 * 128;
        return ring + 1024 > share ? ring + 1024 : share;
    }
    static_assert(kStage % 1024 == 0, "stages start on the swizzle's boundary");
};

constexpr int kMmThreads = 192;

struct MxSplit {
    int64_t kt, tiles_n;
    int32_t splits, stages;
};

// Element e of v, `stride` elements apart from `p` on, for the first `valid`
// of them, times alpha and, where the call says so, added to what is there.
template <int DT, int E>
__device__ __forceinline__ void put_run(const MxMatmulArgs &a, int64_t at, int64_t stride,
                                        const float (&v)[E], int valid)
{
    float f[E];
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = __fmul_rn(v[e], a.alpha);
    if (a.accumulate) {
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = e < valid ? elems::load1<DT>(a.out, at + e * stride) : 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = __fadd_rn(o[e], f[e]);
    }
    using T = typename elems::El<DT>::T;
    T *p = static_cast<T *>(a.out) + at;
    if (valid >= E) {
#pragma unroll
        for (int e = 0; e < E; ++e) elems::store1<DT>(p + e * stride, 0, f[e]);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e < valid) elems::store1<DT>(p + e * stride, 0, f[e]);
    }
}

// Adds up the SP splits' partial sums, [column][lane] in every block's shared
// memory, in the blocks' order, and writes them.  The blocks and threads take
// four lanes of a column each in turn; 8 loads are in flight a thread, so that
// the peers' latency is paid once for them.
template <int DT, int SP>
__device__ __forceinline__ void join(const MxMatmulArgs &a, const float *part, uint32_t rank,
                                     int64_t i0, int64_t j0, int cols)
{
    constexpr int U = 8 / SP;
    for (int first = (int)rank * 128 + threadIdx.x; first < cols * 32; first += U * SP * 128) {
        float4 v[U][SP];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = first + u * SP * 128;
#pragma unroll
            for (int q = 0; q < SP; ++q)
                if (at < cols * 32) v[u][q] = load_peer4(saddr(part + at * 4), q);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = first + u * SP * 128;
            if (at >= cols * 32) break;
            float4 sum = v[u][0];
#pragma unroll
            for (int q = 1; q < SP; ++q) {
                sum.x = __fadd_rn(sum.x, v[u][q].x);
                sum.y = __fadd_rn(sum.y, v[u][q].y);
                sum.z = __fadd_rn(sum.z, v[u][q].z);
                sum.w = __fadd_rn(sum.w, v[u][q].w);
            }
            const int64_t i = i0 + (at >> 5), j = j0 + (at & 31) * 4;
            const float w[4] = {sum.x, sum.y, sum.z, sum.w};
            const int64_t left = a.n - j;
            put_run<DT, 4>(a, i * a.stride + j, 1, w, left < 4 ? (int)left : 4);
        }
    }
}

template <int DT, int NT>
__global__ void __launch_bounds__(kMmThreads)
mx4_matmul_kernel(const __grid_constant__ MxMatmulArgs a, const __grid_constant__ MxSplit sp)
{
    using Tl = Tile<NT>;
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t bars[2 * Tl::kStages + 1];
    __shared__ uint32_t tmem_base, failed;
    const uint32_t ring = saddr(dyn) + ((1024 - (saddr(dyn) & 1023)) & 1023);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = sp.splits > 1 ? cluster_rank() : 0;
    const int64_t tile = blockIdx.x / sp.splits;
    const int64_t tn = tile % sp.tiles_n, tm = tile / sp.tiles_n;
    const int64_t k0 = sp.kt * rank / sp.splits, k1 = sp.kt * (rank + 1) / sp.splits;
    const int rounds = (int)(k1 - k0);
    const uint32_t done_bar = saddr(&bars[2 * Tl::kStages]);
    auto full = [&](int s) { return saddr(&bars[s]); };
    auto empty = [&](int s) { return saddr(&bars[Tl::kStages + s]); };

    bool ok = true;
    if (warp == 4) {                                         // the copies
        const bool one = elect_one();
        if (one) {
            for (int s = 0; s < Tl::kStages; ++s) {
                bar_init(full(s), 1);
                bar_init(empty(s), 1);
            }
            bar_init(done_bar, 1);
            failed = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncwarp();
        pdl_wait();
        // a single tile holds all rows of A when it is narrower than a record
        const unsigned char *ra = a.a + (tm * sp.kt + k0) * kMxRecord;
        const unsigned char *rb = a.b + (tn * sp.kt + k0) * kMxRecord;
        constexpr uint32_t bytes = kMxRecord + Tl::kACodes + kMxScales;
        // the first stages' copies need not wait for the other warps
        const int ahead = rounds < sp.stages ? rounds : sp.stages;
        for (int it = 0; it < ahead; ++it, ra += kMxRecord, rb += kMxRecord)
            if (one) {
                const uint32_t st = ring + it * Tl::kStage;
                bar_expect(full(it), bytes);
                bulk_load(st, rb, kMxRecord, full(it));
                bulk_load(st + kMxRecord, ra, Tl::kACodes, full(it));
                bulk_load(st + kMxRecord + Tl::kACodes, ra + kMxCodes, kMxScales, full(it));
            }
        __syncthreads();
        int s = 0;
        uint32_t phase = 0;
        for (int it = ahead; it < rounds; ++it, ra += kMxRecord, rb += kMxRecord) {
            ok = bar_wait(empty(s), phase);
            if (!ok) break;
            if (one) {
                const uint32_t st = ring + s * Tl::kStage;
                bar_expect(full(s), bytes);
                bulk_load(st, rb, kMxRecord, full(s));
                bulk_load(st + kMxRecord, ra, Tl::kACodes, full(s));
                bulk_load(st + kMxRecord + Tl::kACodes, ra + kMxCodes, kMxScales, full(s));
            }
            __syncwarp();
            if (++s == sp.stages) s = 0, phase ^= 1;
        }
    } else if (warp == 5) {                                  // the scales and the products
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         saddr(&tmem_base)), "r"((uint32_t)Tl::kTmem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncthreads();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const bool one = elect_one();
        const uint32_t tmem = tmem_base, sb = tmem + NT, sa = sb + 8;
        constexpr uint32_t desc = (1u << 7) | (1u << 10) | ((uint32_t)(NT >> 3) << 17) |
                                  (1u << 23) | (1u << 27);
        int s = 0;
        uint32_t phase = 0;
        for (int it = 0; it < rounds; ++it) {
            ok = bar_wait(full(s), phase);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (one) {
                const uint32_t st = ring + s * Tl::kStage;
                const uint64_t db = operand_desc(st), da = db + (kMxRecord >> 4);
                const uint64_t qb = scale_desc(st + kMxCodes);
                const uint64_t qa = scale_desc(st + kMxRecord + Tl::kACodes);
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    copy_scales(sb + 4 * g, qb + g * (512 >> 4));
                    copy_scales(sa + 4 * g, qa + g * (512 >> 4));
                }
                // the record's columns past k are zeros: their products are left out
                const int64_t left = a.k - (k0 + it) * kMxCols;
                const int steps = left >= kMxCols ? 4 : (int)((left + 63) / 64);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j >= steps) break;
                    const uint32_t id = (j & 1) * 2;         // which half of the scale words
                    mma(tmem, db + j * 2, da + j * 2, desc | (id << 4) | (id << 29),
                        sb + 4 * (j >> 1), sa + 4 * (j >> 1), it > 0 || j > 0);
                }
                commit(empty(s));
            }
            __syncwarp();
            if (++s == sp.stages) s = 0, phase ^= 1;
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
        if (lane == 0) atomicAdd(&g_mx4_timeouts, 1u);
        failed = 1;
    }
    const int64_t j = tn * kMxRows + warp * 32 + lane;       // this thread's column of the result
    const int64_t i0 = tm * NT;
    const int cols = (int)(a.m - i0 < NT ? a.m - i0 : NT);
    const uint32_t lanes = tmem_base + ((uint32_t)(warp * 32) << 16);
    if (sp.splits == 1) {
        if (warp < 4 && ok) {
#pragma unroll 1
            for (int c = 0; c < cols; c += 16) {
                float v[16];
                load16(lanes + c, v);
                if (sp.kt == 0) {                            // an empty sum
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = 0.0f;
                }
                if (j < a.n) put_run<DT, 16>(a, (i0 + c) * a.stride + j, a.stride, v, cols - c);
            }
        }
    } else {
        // partial sums [column][lane] where the stages were: all copies have
        // landed and all products have read them
        float *part = reinterpret_cast<float *>(dyn + (ring - saddr(dyn)));
        if (warp < 4 && ok) {
#pragma unroll 1
            for (int c = 0; c < cols; c += 16) {
                float v[16];
                load16(lanes + c, v);
#pragma unroll
                for (int e = 0; e < 16; ++e) part[(c + e) * 128 + warp * 32 + lane] = v[e];
            }
        }
        cluster_sync();
        if (warp < 4 && ok) {
            if (sp.splits == 2) join<DT, 2>(a, part, rank, i0, tn * kMxRows, cols);
            else if (sp.splits == 4) join<DT, 4>(a, part, rank, i0, tn * kMxRows, cols);
            else join<DT, 8>(a, part, rank, i0, tn * kMxRows, cols);
        }
        cluster_sync();       // the peers have read this block's shared memory
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (failed && threadIdx.x == 0)       // copies still in flight land before the block ends
        for (int s = 0; s < sp.stages; ++s) bar_wait_alone(full(s), 0), bar_wait_alone(full(s), 1);
    __syncthreads();
    if (warp == 5) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"((uint32_t)Tl::kTmem));
    }
}

// ------------------------------------------------------------ the pair kernel
//
// Large products: two SMs share a tile of 256 lanes (rows of B) by 256 columns
// (rows of A), so that either reads only its own 128 rows of both operands.
// The first block's MMA warp issues for both (cta_group::2), and both blocks'
// copies arrive at its barriers: a record is a tensor of 136 rows of 128 bytes
// to the copy engine, because only tensor copies may signal the other block.
//
// The scales have a warp of their own, which copies them up to three stages
// ahead into one of four sets of columns.  A thread that issues both the copies and the
// products stands at its next barrier until the copies are done, and
// the tensor cores run dry: 177 clocks a product of 256 x 256 x 64, against
// 134 with two warps and 128 for the products alone.
//
// The blocks are persistent.  The accumulators of consecutive tiles lie at
// columns 0 and 160 of the tensor memory (of 512, 96 hold the scales): they
// overlap in 96 columns, which the result warps read first, so that the next
// tile's products start as soon as those are out and run while the other
// 160 are read, converted and stored.
constexpr int kPairStages = 6;
constexpr int kPairStage = kMxRecord + kMxCodes + 2 * kMxScales;
constexpr int kPairSmem = kPairStages * kPairStage + 1024;
constexpr int kPairThreads = 224;
constexpr int kOverlap = 96;
constexpr int kSets = 4;                                 // of scales in tensor memory
constexpr uint32_t kPairAcc = 256 - kOverlap;            // the upper accumulator
constexpr uint32_t kPairScales = 2 * 256 - kOverlap;     // a set: 8 columns for B, 16 for A
static_assert(kPairSmem <= kSmemBlock, "one block's shared memory");
static_assert(kPairScales + kSets * 24 <= 512, "the tensor memory's columns");

constexpr int kMxLines = kMxRecord / 128;               // 128-byte lines of a record

struct MxPair {
    CUtensorMap lanes, codes, scales;               // boxes of 136, 128 and 8 lines
    int64_t kt, tiles_n, tiles_m, recs_n, recs_m;   // 256 and 128 rows of the lanes' operand
};                                                  // (n) and of the columns' (m)


// Rows y, y + 1, ... of the record rows that `map` describes (its box's height
// of them), into this block, signalled at `bar` of the first one.
__device__ __forceinline__ void tensor_load(uint32_t dst, const CUtensorMap *map, int32_t y,
                                            uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
                 ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(map), "r"(0), "r"(y), "r"(bar) : "memory");
}

__device__ __forceinline__ void copy_scales2(uint32_t tmem, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                 : "memory");
}

__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                     uint32_t sa, uint32_t sb, uint32_t add)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
                 " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X"
                 " [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
                 "r"(sa), "r"(sb), "r"(add) : "memory");
}

__device__ __forceinline__ void commit2_first(uint32_t bar)       // at the issuing block alone
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::
                     "r"(bar) : "memory");
}

// Tile t of the sweep: bands of 8 tiles of rows of A, so that the blocks at work
// at one time share both operands' records in L2.
__device__ __forceinline__ void pair_tile(const MxPair &g, int64_t t, int64_t &tn, int64_t &tm)
{
    const int64_t band = t / (8 * g.tiles_n), in = t - band * 8 * g.tiles_n;
    const int64_t wide = g.tiles_m - band * 8 < 8 ? g.tiles_m - band * 8 : 8;
    tn = in / wide;
    tm = band * 8 + in - tn * wide;
}

// Stages that the pair `first` of every `step` goes through.
__device__ __forceinline__ int64_t pair_stages(const MxPair &g, int64_t first, int64_t step)
{
    const int64_t tiles = g.tiles_n * g.tiles_m;
    return first < tiles ? ((tiles - 1 - first) / step + 1) * g.kt : 0;
}

// 32 consecutive columns of row i of the result, from column j on, 32 bytes a
// store: `out` and its rows lie on 32-byte boundaries.
template <int DT>
__device__ __forceinline__ void put_row32(const MxMatmulArgs &a, int64_t i, int64_t j,
                                          const uint32_t (&r)[32])
{
    constexpr int kPer = DT == F32 ? 8 : 16;                 // elements of 32 bytes
    const int64_t at = i * a.stride + j;
#pragma unroll
    for (int h = 0; h < 32 / kPer; ++h) {
        if (j + (h + 1) * kPer > a.n) {                      // the row's ragged end
            float v[kPer];
#pragma unroll
            for (int e = 0; e < kPer; ++e) v[e] = __uint_as_float(r[h * kPer + e]);
            const int64_t left = a.n - (j + h * kPer);
            put_run<DT, kPer>(a, at + h * kPer, 1, v, left < 0 ? 0 : (int)left);
            continue;
        }
        float f[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) f[e] = __fmul_rn(__uint_as_float(r[h * kPer + e]), a.alpha);
        if (a.accumulate) {
            float o[8];
#pragma unroll
            for (int u = 0; u < kPer / 8; ++u) {
                elems::Raw<DT> old;
                old.load(a.out, at + h * kPer + u * 8);
                old.get(o);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[u * 8 + e] = __fadd_rn(o[e], f[u * 8 + e]);
            }
        }
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (DT == F32) w[e] = __float_as_uint(f[e]);
            else w[e] = elems::narrow2<DT>(f[2 * e], f[2 * e + 1]);
        }
        using T = typename elems::El<DT>::T;
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(
                         static_cast<T *>(a.out) + at + h * kPer),
                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                     "r"(w[7]) : "memory");
    }
}

// The tile's lanes are rows of the operand `lanes`, its columns rows of the
// operand `cols`.  WIDE: lanes = A, so that a thread holds consecutive
// columns of a row of the result and stores them 32 bytes at a time.  A result
// that is not aligned for that has lanes = B, so that a warp's stores are
// consecutive whatever their alignment.
template <int DT, bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads)
mx4_pair_kernel(const __grid_constant__ MxMatmulArgs a, const __grid_constant__ MxPair g)
{
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t bars[2 * kPairStages + 3 + kSets];
    __shared__ uint32_t tmem_base, failed;
    const uint32_t ring = saddr(dyn) + ((1024 - (saddr(dyn) & 1023)) & 1023);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int64_t tiles = g.tiles_n * g.tiles_m, step = gridDim.x / 2;
    auto full = [&](int s) { return saddr(&bars[s]); };                     // the first block's
    auto empty = [&](int s) { return saddr(&bars[kPairStages + s]); };
    auto done = [&](int b) { return saddr(&bars[2 * kPairStages + b]); };
    auto scaled = [&](int b) { return saddr(&bars[2 * kPairStages + 2 + b]); };  // the first block's
    const uint32_t drained = saddr(&bars[2 * kPairStages + 2 + kSets]);             // the first block's

    if (warp == 4) {
        if (lane == 0) {
            for (int s = 0; s < 2 * kPairStages + 2 + kSets; ++s) bar_init(saddr(&bars[s]), 1);
            bar_init(drained, 8);
            failed = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
    } else if (warp == 5) {
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
    if (warp == 4) {                                         // the copies
        const bool one = elect_one();
        int s = 0;
        uint32_t phase = 1;                                  // the stages start empty
        for (int64_t t = blockIdx.x / 2; t < tiles && ok; t += step) {
            int64_t tn, tm;
            pair_tile(g, t, tn, tm);
            // past the last record the last one again: its results are not stored
            const int64_t rb = tn * 2 + rank < g.recs_n ? tn * 2 + rank : g.recs_n - 1;
            const int64_t ra0 = tm * 2, ra1 = ra0 + 1 < g.recs_m ? ra0 + 1 : ra0;
            int32_t yb = (int32_t)(rb * g.kt * kMxLines);
            int32_t y0 = (int32_t)(ra0 * g.kt * kMxLines), y1 = (int32_t)(ra1 * g.kt * kMxLines);
            for (int64_t kt = 0; kt < g.kt; ++kt) {
                ok = bar_wait(empty(s), phase);
                if (!ok) break;
                if (one) {
                    const uint32_t st = ring + s * kPairStage, bar = peer_addr(full(s), 0);
                    if (rank == 0) bar_expect(full(s), 2 * kPairStage);
                    tensor_load(st, &g.lanes, yb, bar);
                    tensor_load(st + kMxRecord, &g.codes, rank ? y1 : y0, bar);
                    tensor_load(st + kMxRecord + kMxCodes, &g.scales, y0 + 128, bar);
                    tensor_load(st + kMxRecord + kMxCodes + kMxScales, &g.scales, y1 + 128, bar);
                }
                __syncwarp();
                yb += kMxLines;
                y0 += kMxLines;
                y1 += kMxLines;
                if (++s == kPairStages) s = 0, phase ^= 1;
            }
        }
    } else if (warp == 6 && rank == 0) {                     // the scales
        const bool one = elect_one();
        const uint32_t sets = tmem + kPairScales;
        const int64_t total = pair_stages(g, blockIdx.x / 2, step);
        int s = 0, last = 0;                                 // the stage, and that of kSets before
        uint32_t phase = 0, last_phase = 0;
        for (int64_t it = 0; it < total; ++it) {
            // the products kSets stages before have read this set of columns
            ok = it < kSets ? bar_wait(full(s), phase)
                        : bar_wait_both(full(s), phase, empty(last), last_phase);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (one) {
                const uint32_t sb = sets + (uint32_t)(it % kSets) * 24, sa = sb + 8;
                const uint64_t db = scale_desc(ring + s * kPairStage + kMxCodes);
                const uint64_t da = db + ((kMxScales + kMxCodes) >> 4);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    copy_scales2(sb + 4 * h, db + h * (512 >> 4));
                    copy_scales2(sa + 8 * h, da + h * (512 >> 4));
                    copy_scales2(sa + 8 * h + 4, da + ((kMxScales + h * 512) >> 4));
                }
                commit2_first(scaled((int)(it % kSets)));
            }
            __syncwarp();
            if (++s == kPairStages) s = 0, phase ^= 1;
            if (it >= kSets && ++last == kPairStages) last = 0, last_phase ^= 1;
        }
    } else if (warp == 5 && rank == 0) {                     // the products
        const bool one = elect_one();
        constexpr uint32_t desc = (1u << 7) | (1u << 10) | ((256u >> 3) << 17) | (1u << 23) |
                                  (2u << 27);
        const uint32_t sets = tmem + kPairScales;
        int s = 0;
        uint32_t phase = 0, scaled_phase = 0;
        uint32_t i = 0, it = 0;                              // the tile's parity, the set
        // the record's columns past k are zeros: their products are left out
        const int last_steps = (int)((a.k - (g.kt - 1) * kMxCols + 63) / 64);
        for (int64_t t = blockIdx.x / 2; t < tiles && ok; t += step) {
            const uint32_t acc = tmem + (i & 1) * kPairAcc;
            // the tile before has left the columns that this one shares with it
            // (and so, read earlier by the same warps, the one before that all)
            if (t >= step) ok = bar_wait(drained, (i & 1) ^ 1);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            for (int64_t kt = 0; kt < g.kt; ++kt) {
                ok = bar_wait_both(full(s), phase, scaled((int)it), scaled_phase);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                if (one) {
                    const uint32_t sb = sets + it * 24, sa = sb + 8;
                    const uint64_t db = operand_desc(ring + s * kPairStage);
                    const uint64_t da = db + (kMxRecord >> 4);
                    const int steps = kt == g.kt - 1 ? last_steps : 4;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j >= steps) break;
                        const uint32_t id = (j & 1) * 2;
                        mma2(acc, db + j * 2, da + j * 2, desc | (id << 4) | (id << 29),
                             sb + 4 * (j >> 1), sa + 8 * (j >> 1), kt > 0 || j > 0);
                    }
                    commit2(empty(s));
                    if (kt == g.kt - 1) commit2(done((int)i));
                }
                __syncwarp();
                if (++s == kPairStages) s = 0, phase ^= 1;
                if (++it == kSets) it = 0, scaled_phase ^= 1;
            }
            i ^= 1;
        }
    } else if (warp < 4) {                                   // the results
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        uint32_t b = 0, done_phase = 0;
        for (int64_t t = blockIdx.x / 2; t < tiles; t += step) {
            int64_t tn, tm;
            pair_tile(g, t, tn, tm);
            ok = bar_wait(done((int)b), done_phase);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const int64_t l = (tn * 2 + rank) * kMxRows + warp * 32 + lane, c0 = tm * 256;
#pragma unroll 1
            for (int q = 0; q < 8; ++q) {
                // the shared columns first: the last of the lower accumulator,
                // the first of the upper one
                const int c = (b == 0 ? 7 - q : q) * 32;
                uint32_t r[32];
                load32(tmem + lanes + b * kPairAcc + c, r);
                if (q == kOverlap / 32 - 1) {
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) arrive_first(drained);
                }
                if constexpr (WIDE) {
                    if (l < a.m) put_row32<DT>(a, l, c0 + c, r);
                } else if (l < a.n) {
                    const int64_t left = a.m - (c0 + c);
                    float v[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
                    put_run<DT, 32>(a, (c0 + c) * a.stride + l, a.stride, v,
                                    left < 32 ? (int)left : 32);
                }
            }
            b ^= 1;
            if (b == 0) done_phase ^= 1;
        }
    }
    if (!ok) {
        if (lane == 0) atomicAdd(&g_mx4_timeouts, 1u);
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
    if (warp == 5) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(512u));
    }
}

// A quantised matrix as a tensor of 128-byte lines, copied `box` at a time.
cudaError_t record_map(CUtensorMap *map, const void *base, int64_t lines, int box)
{
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<Encode> encode{nullptr};
    Encode f = encode.load(std::memory_order_relaxed);
    if (!f) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                         cudaEnableDefault, &found);
        if (e != cudaSuccess) return e;
        if (!p || found != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
        f = reinterpret_cast<Encode>(p);
        encode.store(f, std::memory_order_relaxed);
    }
    const cuuint64_t dims[2] = {128, (cuuint64_t)lines}, strides[1] = {128};
    const cuuint32_t boxes[2] = {128, (cuuint32_t)box}, one[2] = {1, 1};
    const CUresult r = f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims,
                         strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The lines of both operands; whether the copies' 32-bit coordinates reach them.
bool pair_lines(const MxMatmulArgs &a, int64_t &la, int64_t &lb)
{
    const int64_t kt = (a.k + kMxCols - 1) / kMxCols * kMxLines;
    la = (a.m + kMxRows - 1) / kMxRows * kt;
    lb = (a.n + kMxRows - 1) / kMxRows * kt;
    return la <= 0x7fffffff && lb <= 0x7fffffff;
}

template <int DT, bool WIDE> cudaError_t pair_go(const MxMatmulArgs &a, int sms, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_shared(reinterpret_cast<const void *>(mx4_pair_kernel<DT, WIDE>),
                                 kSmemBlock, done);
    if (e != cudaSuccess) return e;
    MxPair g;
    int64_t lines_a = 0, lines_b = 0;
    pair_lines(a, lines_a, lines_b);
    const void *lanes = WIDE ? a.a : a.b, *cols = WIDE ? a.b : a.a;
    const int64_t lines_l = WIDE ? lines_a : lines_b, lines_c = WIDE ? lines_b : lines_a;
    e = record_map(&g.lanes, lanes, lines_l, kMxLines);
    if (e == cudaSuccess) e = record_map(&g.codes, cols, lines_c, kMxCodes / 128);
    if (e == cudaSuccess) e = record_map(&g.scales, cols, lines_c, kMxScales / 128);
    if (e != cudaSuccess) return e;
    g.kt = (a.k + kMxCols - 1) / kMxCols;
    g.recs_n = ((WIDE ? a.m : a.n) + kMxRows - 1) / kMxRows;
    g.recs_m = ((WIDE ? a.n : a.m) + kMxRows - 1) / kMxRows;
    g.tiles_n = (g.recs_n + 1) / 2;
    g.tiles_m = (g.recs_m + 1) / 2;
    const int64_t tiles = g.tiles_n * g.tiles_m;
    const int64_t pairs = tiles < sms / 2 ? tiles : sms / 2;
    return launch_dependent(mx4_pair_kernel<DT, WIDE>, dim3((unsigned)(2 * pairs)),
                            dim3(kPairThreads), kSmemBlock, s, a, g);
}

// NT < 128 serves m <= NT: a single tile of rows of A.
template <int DT, int NT>
cudaError_t mm_go(const MxMatmulArgs &a, int sms, cudaStream_t s)
{
    using Tl = Tile<NT>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_shared(reinterpret_cast<const void *>(mx4_matmul_kernel<DT, NT>),
                                 Tl::smem(Tl::kStages), done);
    if (e != cudaSuccess) return e;
    MxSplit sp;
    sp.kt = (a.k + kMxCols - 1) / kMxCols;
    sp.tiles_n = (a.n + kMxRows - 1) / kMxRows;
    const int64_t tiles = sp.tiles_n * ((a.m + NT - 1) / NT);
    // The split that leaves the fullest SM the fewest records, a join counting
    // as kJoin of them, as long as all blocks find a place at once.  (Measured:
    // 64 rows by 11008 x 4096 whole 7.2 us, in halves 8.1; one row by 4096 x 11008
    // in two 8.0, in four 7.0, in eight 6.7; by 4096 x 4096 in two 4.6, in four 3.8.)
    constexpr int kJoin = 2;
    auto stages = [&](int splits) {
        const int64_t most = (sp.kt + splits - 1) / splits;
        return most < 1 ? 1 : most < Tl::kStages ? (int)most : Tl::kStages;
    };
    sp.splits = 1;
    int64_t least = (tiles + sms - 1) / sms * sp.kt;
    for (int n = 2; n <= 8 && sp.kt >= 2 * n; n *= 2) {
        const int64_t per_sm = (tiles * n + sms - 1) / sms;
        if (per_sm > kSmemSm / (Tl::smem(stages(n)) + 1024)) break;
        const int64_t cost = per_sm * ((sp.kt + n - 1) / n) + kJoin;
        if (cost < least) least = cost, sp.splits = n;
    }
    sp.stages = stages(sp.splits);
    const int64_t blocks = tiles * sp.splits;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = Tl::smem(sp.stages);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)sp.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, mx4_matmul_kernel<DT, NT>, a, sp);
}

template <int DT> cudaError_t mm_pick(const MxMatmulArgs &a, int sms, cudaStream_t s)
{
    // Few rows, or no more tiles of 128 by 128 than SMs: the single blocks, whose
    // columns can be split (4096 x 4096 by 512 rows, 128 tiles: 7.5 us against the
    // pairs' 10.2).  Beyond that the pairs (768 rows, 192 tiles: 10.5 us against
    // 13.6).
    const int64_t tiles = ((a.n + 127) / 128) * ((a.m + 127) / 128);
    int64_t la, lb;
    if (a.k > 0 && a.m > 64 && tiles > sms && pair_lines(a, la, lb)) {
        const int es = DT == F32 ? 4 : 2;
        const bool wide = ((uintptr_t)a.out & 31) == 0 && a.stride * es % 32 == 0;
        return wide ? pair_go<DT, true>(a, sms, s) : pair_go<DT, false>(a, sms, s);
    }
    return a.m <= 16 ? mm_go<DT, 16>(a, sms, s)
           : a.m <= 32 ? mm_go<DT, 32>(a, sms, s)
           : a.m <= 64 ? mm_go<DT, 64>(a, sms, s) : mm_go<DT, 128>(a, sms, s);
}

}  // namespace

cudaError_t launch_mx4_matmul(int32_t dt, const MxMatmulArgs &a, int sms, cudaStream_t s)
{
    if (a.m <= 0 || a.n <= 0) return cudaSuccess;
    return dt == F32 ? mm_pick<F32>(a, sms, s) : dt == BF16 ? mm_pick<BF16>(a, sms, s)
                                                            : mm_pick<F16>(a, sms, s);
}

cudaError_t mx4_timeouts(unsigned int *count)
{
    // the copy alone would not wait for streams that do not synchronise with the
    // default one
    const cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return e;
    return cudaMemcpyFromSymbol(count, g_mx4_timeouts, sizeof(unsigned int));
}

}  // namespace zgb
