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
#include "zero_elems.cuh"
#include "zero_ops.h"

namespace zgb {
namespace {

constexpr long long kPolls = 1ll << 22;
__device__ unsigned int g_mx4_timeouts;

__device__ __forceinline__ uint32_t saddr(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity)
{
    for (long long i = 0; i < kPolls; ++i) {
        uint32_t done;
        asm volatile("{\n .reg .pred p;\n"
                     " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                     " selp.u32 %0, 1, 0, p;\n}"
                     : "=r"(done) : "r"(bar), "r"(parity) : "memory");
        if (done) return true;
    }
    return false;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// Shared-memory matrix descriptors: start address, stride between groups of
// 8 rows, the descriptor version and the swizzle, as PTX defines them.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr)     // 128-byte rows, swizzled
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ uint64_t scale_desc(uint32_t addr)       // 16-byte rows, as they lie
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}

// Instruction descriptor of kind mxf4 without the scale ids: both operands
// E2M1 and K-major, scales UE8M0, 128 lanes by NT columns.
constexpr uint32_t kDescBase = (1u << 7) | (1u << 10) | (1u << 23) | (1u << 27);

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

__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::
                     "r"(bar) : "memory");
}

__device__ __forceinline__ void load16(uint32_t tmem, float (&v)[16])
{
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32"
                 " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                   "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(tmem));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float load_peer(uint32_t addr, uint32_t rank)
{
    uint32_t p;
    float v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(p) : "memory");
    return v;
}

template <int NT> struct Tile {
    static constexpr int kRecs = (NT + 127) / 128;          // records of A side by side
    static constexpr int kACodes = NT * 128;                // their codes
    static constexpr int kStage = kMxRecord + kACodes + kRecs * kMxScales;
    // the accumulator, 8 columns of B's scales, 8 a record of A's
    static constexpr int kTmemUsed = NT + 8 + 8 * kRecs;
    static constexpr int kTmem = kTmemUsed <= 32 ? 32 : kTmemUsed <= 64 ? 64
                                 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
    // Shared memory holds at most 512 / kTmem blocks on an SM, so that no block
    // waits for tensor memory that another one holds.
    static constexpr int kStages = NT >= 256 ? 4 : NT >= 128 ? 3 : 4;
    static constexpr int kPart = NT * 128 * 4;              // a split's partial sums
    static constexpr int kSmem = (kStages * kStage > kPart ? kStages * kStage : kPart) + 1024;
    static_assert(kStage % 1024 == 0, "stages start on the swizzle's boundary");
    static_assert((232448 / kSmem) * kTmem <= 512, "tensor memory for every resident block");
};

constexpr int kMmThreads = 192;

struct MxSplit {
    int64_t kt, tiles_n;
    int32_t splits;
};

template <int DT>
__device__ __forceinline__ void put(const MxMatmulArgs &a, int64_t i, int64_t j, float v)
{
    const int64_t at = i * a.stride + j;
    v = __fmul_rn(v, a.alpha);
    if (a.accumulate) v = __fadd_rn(elems::load1<DT>(a.out, at), v);
    elems::store1<DT>(a.out, at, v);
}

template <int DT, int NT>
__global__ void __launch_bounds__(kMmThreads)
mx4_matmul_kernel(const __grid_constant__ MxMatmulArgs a, const __grid_constant__ MxSplit sp)
{
    using Tl = Tile<NT>;
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t bars[2 * Tl::kStages + 1];
    __shared__ uint32_t tmem_base, failed;
    unsigned char *ring = dyn + ((1024 - (saddr(dyn) & 1023)) & 1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = sp.splits > 1 ? cluster_rank() : 0;
    const int64_t tile = blockIdx.x / sp.splits;
    const int64_t tn = tile % sp.tiles_n, tm = tile / sp.tiles_n;
    const int64_t k0 = sp.kt * rank / sp.splits, k1 = sp.kt * (rank + 1) / sp.splits;
    const uint32_t done_bar = saddr(&bars[2 * Tl::kStages]);
    auto full = [&](int s) { return saddr(&bars[s]); };
    auto empty = [&](int s) { return saddr(&bars[Tl::kStages + s]); };

    if (warp == 4) {
        if (lane == 0) {
            for (int s = 0; s < Tl::kStages; ++s) {
                bar_init(full(s), 1);
                bar_init(empty(s), 1);
            }
            bar_init(done_bar, 1);
            failed = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
    } else if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         saddr(&tmem_base)), "r"((uint32_t)Tl::kTmem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_base;
    pdl_wait();
    pdl_launch_dependents();

    const int64_t arecs = (a.m + kMxRows - 1) / kMxRows;
    const int64_t arec0 = tm * Tl::kRecs;                    // NT < 128: a record's first rows
    const int nrec = Tl::kRecs == 2 && arec0 + 1 < arecs ? 2 : 1;

    if (warp == 4 && lane == 0) {                            // the copies
        const uint32_t bytes = kMxRecord + (NT < kMxRows ? Tl::kACodes : nrec * kMxCodes) +
                               nrec * kMxScales;
        for (int64_t kt = k0; kt < k1; ++kt) {
            const int it = (int)(kt - k0), s = it % Tl::kStages;
            if (it >= Tl::kStages && !bar_wait(empty(s), ((it / Tl::kStages) - 1) & 1)) {
                atomicAdd(&g_mx4_timeouts, 1u);
                failed = 1;
                break;
            }
            const uint32_t st = saddr(ring) + s * Tl::kStage;
            bar_expect(full(s), bytes);
            bulk_load(st, a.b + (tn * sp.kt + kt) * kMxRecord, kMxRecord, full(s));
            const uint32_t ac = st + kMxRecord, as = ac + Tl::kACodes;
            for (int r = 0; r < nrec; ++r) {
                const unsigned char *rec = a.a + ((arec0 + r) * sp.kt + kt) * kMxRecord;
                bulk_load(ac + r * kMxCodes, rec,
                          NT < kMxRows ? Tl::kACodes : kMxCodes, full(s));
                bulk_load(as + r * kMxScales, rec + kMxCodes, kMxScales, full(s));
            }
        }
    } else if (warp == 5 && lane == 0) {                     // the products
        const uint32_t sb = tmem + NT, sa = sb + 8;
        bool ok = true;
        for (int64_t kt = k0; kt < k1; ++kt) {
            const int it = (int)(kt - k0), s = it % Tl::kStages;
            if (!bar_wait(full(s), (it / Tl::kStages) & 1)) {
                ok = false;
                break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t st = saddr(ring) + s * Tl::kStage;
            const uint32_t ac = st + kMxRecord, as = ac + Tl::kACodes;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                copy_scales(sb + 4 * g, scale_desc(st + kMxCodes + g * 512));
#pragma unroll
                for (int r = 0; r < Tl::kRecs; ++r)
                    copy_scales(sa + 4 * (g * Tl::kRecs + r),
                                scale_desc(as + r * kMxScales + g * 512));
            }
            // the record's columns past k are zeros: their products are left out
            const int64_t left = a.k - kt * kMxCols;
            const int steps = left >= kMxCols ? 4 : (int)((left + 63) / 64);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j >= steps) break;
                const uint32_t id = (j & 1) * 2;             // which half of the scale words
                mma(tmem, operand_desc(st + j * 32), operand_desc(ac + j * 32),
                    kDescBase | ((uint32_t)(NT >> 3) << 17) | (id << 4) | (id << 29), sb + 4 * (j >> 1),
                    sa + 4 * Tl::kRecs * (j >> 1), it > 0 || j > 0);
            }
            commit(empty(s));
        }
        if (ok) {
            commit(done_bar);
        } else {
            atomicAdd(&g_mx4_timeouts, 1u);
            failed = 1;
        }
    }
    __syncwarp();

    bool ok = true;
    if (warp < 4) {
        ok = bar_wait(done_bar, 0);
        if (!ok && lane == 0) failed = 1;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    }
    const int64_t j = tn * kMxRows + warp * 32 + lane;       // this thread's column of the result
    const int64_t i0 = tm * NT;
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    if (sp.splits == 1) {
        if (warp < 4 && ok) {
#pragma unroll 1
            for (int c = 0; c < NT; c += 16) {
                if (i0 + c >= a.m) break;
                float v[16];
                load16(lanes + c, v);
                if (sp.kt == 0) {                            // an empty sum
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (i0 + c + e < a.m && j < a.n) put<DT>(a, i0 + c + e, j, v[e]);
            }
        }
    } else {
        // partial sums [column][lane] where the stages were: all copies have
        // landed and all products have read them
        float *part = reinterpret_cast<float *>(ring);
        if (warp < 4 && ok) {
#pragma unroll 1
            for (int c = 0; c < NT; c += 16) {
                if (i0 + c >= a.m) break;
                float v[16];
                load16(lanes + c, v);
#pragma unroll
                for (int e = 0; e < 16; ++e) part[(c + e) * 128 + warp * 32 + lane] = v[e];
            }
        }
        cluster_sync();
        if (warp < 4 && ok) {
            for (int c = (int)rank; c < NT; c += sp.splits) {
                if (i0 + c >= a.m) break;
                float v = 0.0f;
                for (int q = 0; q < sp.splits; ++q) {
                    const float u = load_peer(saddr(part + c * 128 + warp * 32 + lane), q);
                    v = q == 0 ? u : __fadd_rn(v, u);
                }
                if (j < a.n) put<DT>(a, i0 + c, j, v);
            }
        }
        cluster_sync();       // the peers have read this block's shared memory
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (failed && threadIdx.x == 0)       // copies still in flight land before the block ends
        for (int s = 0; s < Tl::kStages; ++s) bar_wait(full(s), 0), bar_wait(full(s), 1);
    __syncthreads();
    if (warp == 5)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"((uint32_t)Tl::kTmem));
}

// NT < 128 serves m <= NT: a single tile of rows of A.
template <int DT, int NT>
cudaError_t mm_go(const MxMatmulArgs &a, int sms, cudaStream_t s)
{
    using Tl = Tile<NT>;
    static int attr_device = -1;   // the attribute is per device
    int dev = 0;
    cudaGetDevice(&dev);
    if (attr_device != dev) {
        cudaError_t e = cudaFuncSetAttribute(mx4_matmul_kernel<DT, NT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Tl::kSmem);
        if (e != cudaSuccess) return e;
        attr_device = dev;
    }
    MxSplit sp;
    sp.kt = (a.k + kMxCols - 1) / kMxCols;
    sp.tiles_n = (a.n + kMxRows - 1) / kMxRows;
    const int64_t tiles = sp.tiles_n * ((a.m + NT - 1) / NT);
    // halve the columns while there are SMs without a tile and each
    // part keeps two records
    sp.splits = 1;
    while (sp.splits < 8 && tiles * sp.splits < sms && sp.kt >= 4 * sp.splits) sp.splits *= 2;
    const int64_t blocks = tiles * sp.splits;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = Tl::kSmem;
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
    return a.m <= 16 ? mm_go<DT, 16>(a, sms, s)
           : a.m <= 64 ? mm_go<DT, 64>(a, sms, s)
           : a.m <= 128 ? mm_go<DT, 128>(a, sms, s) : mm_go<DT, 256>(a, sms, s);
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
    return cudaMemcpyFromSymbol(count, g_mx4_timeouts, sizeof(unsigned int));
}

}  // namespace zgb
