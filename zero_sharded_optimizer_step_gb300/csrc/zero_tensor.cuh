// What the tensor-core products share: barriers in shared memory, the elected
// lane, matrix descriptors, tensor memory and clusters (tcgen05 and TMA as PTX
// defines them).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "zero_product_sizes.h"

namespace zgb {

constexpr long long kPolls = 1ll << 22;

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

__device__ __forceinline__ bool bar_poll(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n .reg .pred p;\n"
                 " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                 " selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}

// A wait by all lanes of a warp, which get one answer: were it each lane's own, some
// could give up in the poll in which others succeed, and the two would then wait for
// one another at the warp's next barrier or shuffle.  A phase that has ended stays so
// until this warp has gone on, so that every poll after that one is unanimous.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity)
{
    for (long long i = 0; i < kPolls; ++i)
        if (__all_sync(0xffffffffu, bar_poll(bar, parity))) return true;
    return false;
}

// A wait by a single thread.
__device__ __forceinline__ bool bar_wait_alone(uint32_t bar, uint32_t parity)
{
    for (long long i = 0; i < kPolls; ++i)
        if (bar_poll(bar, parity)) return true;
    return false;
}

// Both barriers' phases, by a warp; the two polls' latencies overlap.
__device__ __forceinline__ bool bar_wait_both(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1)
{
    for (long long i = 0; i < kPolls; ++i) {
        uint32_t done;
        asm volatile("{\n .reg .pred p, q;\n"
                     " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                     " mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n"
                     " and.pred p, p, q;\n selp.u32 %0, 1, 0, p;\n}"
                     : "=r"(done) : "r"(b0), "r"(p0), "r"(b1), "r"(p1) : "memory");
        if (__all_sync(0xffffffffu, done)) return true;
    }
    return false;
}

// One lane of a converged warp.  The warps that issue run whole, with a lane
// elected for the instructions themselves: their addresses are then
// uniform over the warp and need no copies to uniform registers, which would cost
// more than the products take.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(p));
    return p != 0;
}

// Shared-memory matrix descriptors: start address, stride between groups of
// 8 rows, the descriptor version and the swizzle, as PTX defines them.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr)     // 128-byte rows, swizzled
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::
                     "r"(bar) : "memory");
}

// 16 columns of tensor memory, the warp's 32 lanes.  (The .aligned instructions want
// the warp converged, which it need not be after a store that some of its lanes made.)
__device__ __forceinline__ void load16(uint32_t tmem, float (&v)[16])
{
    uint32_t r[16];
    __syncwarp();
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

// (The barrier's instructions want their warp converged.)
__device__ __forceinline__ void cluster_sync()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Its two halves, with other work between them.
__device__ __forceinline__ void cluster_arrive()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait()
{
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// All blocks have come here; nothing is said of what they wrote (no store is waited for).
__device__ __forceinline__ void cluster_meet()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank)
{
    uint32_t p;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(addr), "r"(rank));
    return p;
}

__device__ __forceinline__ float load_peer(uint32_t addr, uint32_t rank)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer_addr(addr, rank))
                 : "memory");
    return v;
}

__device__ __forceinline__ float4 load_peer4(uint32_t addr, uint32_t rank)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(peer_addr(addr, rank)) : "memory");
    return v;
}

// At the pair's first block.  The accumulator's order is kept by the tcgen05
// fences around it, so the arrival itself need not wait for earlier stores.
__device__ __forceinline__ void arrive_first(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(peer_addr(bar, 0))
                 : "memory");
}

__device__ __forceinline__ void commit2(uint32_t bar)             // at both blocks
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
                 ".multicast::cluster.b64 [%0], %1;" ::"r"(bar), "h"((uint16_t)3) : "memory");
}

// 32 columns, as load16.
__device__ __forceinline__ void load32(uint32_t tmem, uint32_t (&r)[32])
{
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32"
        " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(tmem));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

}  // namespace zgb
