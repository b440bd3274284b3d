// Dropout from a counter-based generator, the mask never stored.
//
// Element e is kept where word e % 4 of Philox4x32-10 (Salmon, Moraes, Dror
// and Shaw 2011, "Parallel random numbers: as easy as 1, 2, 3") under the key
// `seed` at the counter (e / 4, offset) is at least p * 2^32, and multiplied by
// 1 / (1 - p).  The gradient is the same map of dy, so the forward stores
// nothing for it: the same call with the same seed and offset makes the mask
// again.  One IEEE multiplication and, with a residual, one addition per
// element in fp32, rounded once to the type.
//
// What bounds it: four words cost 18 wide multiplications and 18 three-way
// exclusive ors (two of the 20 of either are the offset's alone), about 19
// instructions an element with the conversion and the comparison, so that 16-bit
// elements are bound by the integer pipes and fp32 ones by memory.  Measured for
// 2^26 elements: bf16 52 us (5.2 TB/s), with a residual 58 us (6.9 TB/s); fp32
// 77 us (6.9 TB/s), with a residual 113 us (7.1 TB/s).
#include "zero_elems.cuh"
#include "zero_ops.h"

namespace zgb {
namespace {

// The words at the counters c[0 .. N).  The chains go round by round together,
// so that a round's keys are fetched once for all of them.  LOW: counters below 2^32, and
// half of the first two rounds' products are those of the offset alone, made
// on the host (a.pre).
template <bool LOW, int N>
__device__ __forceinline__ void philox(const unsigned long long (&c)[N], const DropoutArgs &a,
                                       uint4 (&w)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (LOW) {
            const unsigned long long p0 = (unsigned long long)(uint32_t)c[i] * 0xD2511F53u;
            const unsigned long long p1 =
                (unsigned long long)((uint32_t)(p0 >> 32) ^ a.pre[0]) * 0xCD9E8D57u;
            w[i] = make_uint4((uint32_t)(p1 >> 32) ^ a.pre[1], (uint32_t)p1,
                              (uint32_t)p0 ^ a.pre[2], a.pre[3]);
        } else {
            w[i] = make_uint4((uint32_t)c[i], (uint32_t)(c[i] >> 32), a.off0, a.off1);
        }
    }
#pragma unroll
    for (int r = LOW ? 2 : 0; r < 10; ++r) {
        const uint32_t k0 = a.key0[r], k1 = a.key1[r];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const unsigned long long p0 = (unsigned long long)w[i].x * 0xD2511F53u;
            const unsigned long long p1 = (unsigned long long)w[i].z * 0xCD9E8D57u;
            w[i] = make_uint4((uint32_t)(p1 >> 32) ^ w[i].y ^ k0, (uint32_t)p1,
                              (uint32_t)(p0 >> 32) ^ w[i].w ^ k1, (uint32_t)p0);
        }
    }
}

__device__ __forceinline__ float drop(float x, uint32_t word, const DropoutArgs &a)
{
    return word >= a.threshold ? __fmul_rn(x, a.up) : 0.0f;
}

// VEC: kGroups groups of 8 elements a thread, on their boundaries, all loaded
// before the words are made.  Otherwise (an unaligned buffer, and the ragged
// end) 4 elements a thread, one by one.
constexpr int kGroups = 2;

template <int DT, bool RES, bool VEC, bool LOW>
__global__ void __launch_bounds__(kThreads)
dropout_kernel(const __grid_constant__ DropoutArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t groups = VEC ? a.n / 8 : 0;
    if (VEC) {
        const int64_t g0 = (int64_t)blockIdx.x * (kThreads * kGroups) + threadIdx.x;
        elems::Raw<DT> rx[kGroups], rr[kGroups];
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int64_t g = g0 + k * kThreads;
            if (g < groups) {
                rx[k].load(a.x, g * 8);
                if (RES) rr[k].load(a.residual, g * 8);
            }
        }
        unsigned long long c[2 * kGroups];
        uint4 w[2 * kGroups];
#pragma unroll
        for (int k = 0; k < 2 * kGroups; ++k)
            c[k] = a.first + 2 * (g0 + (k >> 1) * kThreads) + (k & 1);
        philox<LOW>(c, a, w);
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int64_t g = g0 + k * kThreads;
            if (g >= groups) break;
            const uint32_t u[8] = {w[2 * k].x,     w[2 * k].y,     w[2 * k].z,     w[2 * k].w,
                                   w[2 * k + 1].x, w[2 * k + 1].y, w[2 * k + 1].z, w[2 * k + 1].w};
            float x[8];
            rx[k].get(x);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = drop(x[i], u[i], a);
            if (RES) {
                float r[8];
                rr[k].get(r);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(x[i], r[i]);
            }
            rx[k].set(x);
            rx[k].store(a.out, g * 8);
        }
    }
    const int64_t T = (int64_t)gridDim.x * kThreads;
    for (int64_t e = groups * 8 + ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4; e < a.n;
         e += T * 4) {
        const unsigned long long c[1] = {a.first + e / 4};
        uint4 v[1];
        philox<LOW>(c, a, v);
        const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (e + i >= a.n) break;
            float y = drop(elems::load1<DT>(a.x, e + i), w[i], a);
            if (RES) y = __fadd_rn(y, elems::load1<DT>(a.residual, e + i));
            elems::store1<DT>(a.out, e + i, y);
        }
    }
}

// p = 1: nothing is kept (2^32 is no 32-bit threshold), and x is not read.
template <int DT>
__global__ void __launch_bounds__(kThreads)
dropout_all_kernel(const __grid_constant__ DropoutArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t T = (int64_t)gridDim.x * kThreads;
    for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < a.n; e += T)
        elems::store1<DT>(a.out, e, a.residual ? __fadd_rn(0.0f, elems::load1<DT>(a.residual, e))
                                               : 0.0f);
}

template <int DT, bool RES, bool VEC, bool LOW>
cudaError_t go(const DropoutArgs &a, cudaStream_t s)
{
    const int64_t per_block = (int64_t)kThreads * (VEC ? 8 * kGroups : 4);
    int64_t blocks = (a.n + per_block - 1) / per_block;
    if (VEC ? blocks > 0x7fffffff : blocks > (1 << 20)) {
        if (VEC) return cudaErrorInvalidValue;
        blocks = 1 << 20;       // element by element, the threads go around
    }
    return launch_dependent(dropout_kernel<DT, RES, VEC, LOW>, dim3((unsigned)blocks), dim3(kThreads),
                            0, s, a);
}

template <int DT> cudaError_t pick(const DropoutArgs &a, cudaStream_t s)
{
    if (a.all) {
        const int64_t blocks = (a.n + kThreads - 1) / kThreads;
        return launch_dependent(dropout_all_kernel<DT>,
                                dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)),
                                dim3(kThreads), 0, s, a);
    }
    const bool vec = (((uintptr_t)a.x | (uintptr_t)a.residual | (uintptr_t)a.out) &
                      (8 * elem_size(DT) - 1)) == 0;
    const bool low = a.first + (unsigned long long)a.n / 4 < 0xffffffffull;
    if (vec && low) return a.residual ? go<DT, true, true, true>(a, s) : go<DT, false, true, true>(a, s);
    if (vec) return a.residual ? go<DT, true, true, false>(a, s) : go<DT, false, true, false>(a, s);
    return a.residual ? go<DT, true, false, false>(a, s) : go<DT, false, false, false>(a, s);
}

}  // namespace

cudaError_t launch_dropout(int32_t dt, const DropoutArgs &a, cudaStream_t s)
{
    if (a.n <= 0) return cudaSuccess;
    return dt == F32 ? pick<F32>(a, s) : dt == BF16 ? pick<BF16>(a, s)
                                                         : pick<F16>(a, s);
}

}  // namespace zgb
