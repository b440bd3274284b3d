// Dropout from a counter-based generator, the mask never stored.
//
// Element e is kept where word e % 4 of Philox4x32-10 (Salmon, Moraes, Dror
// and Shaw 2011, "Parallel random numbers: as easy as 1, 2, 3") under the key
// `seed` at the counter (e / 4, offset) is at least p * 2^32, and multiplied by
// 1 / (1 - p).  The gradient is the same map of dy, so the forward stores
// nothing for it: the same call with the same seed and offset makes the mask
// again.  One IEEE multiplication and, with a residual, one addition per
// element in fp32, rounded once to the type.
#include "zero_elems.cuh"
#include "zero_ops.h"

namespace zgb {
namespace {

__device__ __forceinline__ uint4 philox(unsigned long long c, const DropoutArgs &a)
{
    uint32_t c0 = (uint32_t)c, c1 = (uint32_t)(c >> 32), c2 = a.off0, c3 = a.off1;
    uint32_t k0 = a.key0, k1 = a.key1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const unsigned long long p0 = (unsigned long long)c0 * 0xD2511F53u;
        const unsigned long long p1 = (unsigned long long)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ float drop(float x, uint32_t word, const DropoutArgs &a)
{
    return (unsigned long long)word >= a.threshold ? __fmul_rn(x, a.up) : 0.0f;
}

// VEC: 8 elements a thread on 16-byte boundaries.  Otherwise (an unaligned
// buffer, and the ragged end) 4 elements a thread, one by one.
template <int DT, bool RES, bool VEC>
__global__ void __launch_bounds__(kThreads)
dropout_kernel(const __grid_constant__ DropoutArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t T = (int64_t)gridDim.x * kThreads;
    const int64_t t0 = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t groups = VEC ? a.n / 8 : 0;
    for (int64_t g = t0; g < groups; g += T) {
        elems::Raw<DT, 8> rx, rr;
        rx.load(a.x, g * 8);
        if (RES) rr.load(a.residual, g * 8);
        const uint4 w0 = philox(a.first + 2 * g, a), w1 = philox(a.first + 2 * g + 1, a);
        const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
        float x[8];
        rx.get(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = drop(x[i], w[i], a);
        if (RES) {
            float r[8];
            rr.get(r);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(x[i], r[i]);
        }
        rx.set(x);
        rx.store(a.out, g * 8);
    }
    for (int64_t e = groups * 8 + t0 * 4; e < a.n; e += T * 4) {
        const uint4 v = philox(a.first + e / 4, a);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (e + i >= a.n) break;
            float y = drop(elems::load1<DT>(a.x, e + i), w[i], a);
            if (RES) y = __fadd_rn(y, elems::load1<DT>(a.residual, e + i));
            elems::store1<DT>(a.out, e + i, y);
        }
    }
}

template <int DT, bool RES, bool VEC>
cudaError_t go(const DropoutArgs &a, int sms, cudaStream_t s)
{
    const int per_sm = resident_blocks_per_sm(
        reinterpret_cast<const void *>(dropout_kernel<DT, RES, VEC>), kThreads);
    const int64_t per_block = (int64_t)kThreads * (VEC ? 8 : 4);
    int64_t blocks = (a.n + per_block - 1) / per_block;
    if (blocks > (int64_t)sms * per_sm) blocks = (int64_t)sms * per_sm;
    return launch_dependent(dropout_kernel<DT, RES, VEC>, dim3((unsigned)blocks), dim3(kThreads),
                            0, s, a);
}

template <int DT> cudaError_t pick(const DropoutArgs &a, int sms, cudaStream_t s)
{
    const bool vec = (((uintptr_t)a.x | (uintptr_t)a.residual | (uintptr_t)a.out) & 15) == 0;
    if (a.residual) return vec ? go<DT, true, true>(a, sms, s) : go<DT, true, false>(a, sms, s);
    return vec ? go<DT, false, true>(a, sms, s) : go<DT, false, false>(a, sms, s);
}

}  // namespace

cudaError_t launch_dropout(int32_t dt, const DropoutArgs &a, int sms, cudaStream_t s)
{
    if (a.n <= 0) return cudaSuccess;
    return dt == F32 ? pick<F32>(a, sms, s) : dt == BF16 ? pick<BF16>(a, sms, s)
                                                         : pick<F16>(a, sms, s);
}

}  // namespace zgb
