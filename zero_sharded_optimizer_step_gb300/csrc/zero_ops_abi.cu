// C ABI of the training operators: the embedding and its gradient, dropout,
// and the microscaled 4-bit quantisation and product.  Argument checks and
// the launches; the declarations and their contracts are in include/zero.h.
#include <atomic>
#include <cmath>

#include "../../include/zero.h"
#include "zero_ops.h"

namespace {

using zgb::report;

constexpr int64_t kMost = 0x7ffffffe;   // rows, columns, tokens

bool valid_dtype(int32_t d) { return d == ZERO_F32 || d == ZERO_BF16 || d == ZERO_F16; }

int launched(cudaError_t e, const char *what)
{
    if (e == cudaSuccess) return ZERO_OK;
    return report(ZERO_ECUDA, "%s: %s (%d)", what, cudaGetErrorString(e), (int)e);
}

// SMs of the current device (0 and a message when there is none).
int sm_count()
{
    static std::atomic<int> known[64];
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev < 64 && known[dev].load(std::memory_order_relaxed) > 0)
        return known[dev].load(std::memory_order_relaxed);
    int sms = 0;
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess || sms < 1) {
        report(ZERO_ECUDA, "reading the device's SM count: %s", cudaGetErrorString(e));
        return 0;
    }
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

bool aligned(const void *p, int64_t a) { return ((uintptr_t)p % (uintptr_t)a) == 0; }

// A matrix argument: pointer, type, extents and row stride (in elements).
int check_matrix(const char *name, const void *p, int32_t dt, int64_t rows, int64_t cols,
                 int64_t stride)
{
    if (!valid_dtype(dt)) return report(ZERO_EINVAL, "%s: unknown element type %d", name, dt);
    if (rows < 0 || cols < 0 || rows > kMost || cols > kMost)
        return report(ZERO_EINVAL, "%s: %lld by %lld is not a valid size", name, (long long)rows,
                      (long long)cols);
    if (stride < cols)
        return report(ZERO_EINVAL, "%s: row stride %lld is below the row length %lld", name,
                      (long long)stride, (long long)cols);
    if (rows > 0 && stride > (int64_t)(0x7fffffffffffffffll / 4) / rows)
        return report(ZERO_EINVAL, "%s: row stride %lld is too large", name, (long long)stride);
    if (rows > 0 && cols > 0 && !p) return report(ZERO_EINVAL, "%s must not be null", name);
    const int es = zgb::elem_size(dt);
    if (!aligned(p, es)) return report(ZERO_EALIGN, "%s is not aligned to %d bytes", name, es);
    return ZERO_OK;
}

int check_tokens(const void *tokens, int32_t token_bytes, int64_t n)
{
    if (token_bytes != 4 && token_bytes != 8)
        return report(ZERO_EINVAL, "token ids take 4 or 8 bytes, not %d", token_bytes);
    if (n < 0 || n > kMost) return report(ZERO_EINVAL, "%lld tokens", (long long)n);
    if (n > 0 && !tokens) return report(ZERO_EINVAL, "tokens must not be null");
    if (!aligned(tokens, token_bytes))
        return report(ZERO_EALIGN, "tokens are not aligned to %d bytes", token_bytes);
    return ZERO_OK;
}

int check_records(const char *name, const void *q, int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 0 || rows > kMost || cols > kMost)
        return report(ZERO_EINVAL, "%s: %lld by %lld is not a valid size", name, (long long)rows,
                      (long long)cols);
    if (rows > 0 && cols > 0 && !q) return report(ZERO_EINVAL, "%s must not be null", name);
    if (!aligned(q, 16)) return report(ZERO_EALIGN, "%s is not aligned to 16 bytes", name);
    return ZERO_OK;
}

}  // namespace

#define ZERO_TRY(call)                 \
    do {                               \
        const int rc_ = (call);        \
        if (rc_ != ZERO_OK) return rc_; \
    } while (0)

extern "C" {

int zero_embed(const void *table, int32_t dtype, int64_t rows, int64_t dim, int64_t table_stride,
               const void *tokens, int32_t token_bytes, int64_t n, int64_t pad, float scale,
               void *out, int64_t out_stride, uint64_t *bad, void *stream)
{
    ZERO_TRY(check_matrix("table", table, dtype, rows, dim, table_stride));
    ZERO_TRY(check_tokens(tokens, token_bytes, n));
    ZERO_TRY(check_matrix("out", out, dtype, n, dim, out_stride));
    if (!std::isfinite(scale)) return report(ZERO_EINVAL, "scale must be finite");
    if (!aligned(bad, 8)) return report(ZERO_EALIGN, "bad must be 8-byte aligned");
    if (n == 0 || dim == 0) return ZERO_OK;
    zgb::EmbedArgs a = {};
    a.tok = {tokens, token_bytes == 8, n, pad, rows};
    a.table = table;
    a.dim = dim;
    a.table_stride = table_stride;
    a.out_stride = out_stride;
    a.scale = scale;
    a.out = out;
    a.bad = reinterpret_cast<unsigned long long *>(bad);
    return launched(zgb::launch_embed(dtype, a, (cudaStream_t)stream), "the embedding lookup");
}

int64_t zero_embed_grad_workspace(int64_t rows, int64_t dim, int64_t n)
{
    if (rows < 0 || dim < 0 || n < 0 || rows > kMost || dim > kMost || n > kMost) return -1;
    zgb::EmbedGradArgs a = {};
    a.tok.n = n;
    a.tok.rows = rows;
    a.dim = dim;
    return zgb::embed_grad_layout(a, nullptr);
}

int zero_embed_grad(const void *dy, int32_t dy_dtype, int64_t dy_stride, const void *tokens,
                    int32_t token_bytes, int64_t n, int64_t pad, float scale, void *dtable,
                    int32_t grad_dtype, int64_t rows, int64_t dim, int64_t dtable_stride,
                    int32_t accumulate, void *workspace, int64_t workspace_bytes, void *stream)
{
    ZERO_TRY(check_tokens(tokens, token_bytes, n));
    ZERO_TRY(check_matrix("dy", dy, dy_dtype, n, dim, dy_stride));
    ZERO_TRY(check_matrix("dtable", dtable, grad_dtype, rows, dim, dtable_stride));
    if (!std::isfinite(scale)) return report(ZERO_EINVAL, "scale must be finite");
    if (rows == 0 || dim == 0 || (n == 0 && accumulate)) return ZERO_OK;
    zgb::EmbedGradArgs a = {};
    a.tok = {tokens, token_bytes == 8, n, pad, rows};
    a.dy = dy;
    a.dim = dim;
    a.dy_stride = dy_stride;
    a.grad_stride = dtable_stride;
    a.scale = scale;
    a.grad = dtable;
    a.accumulate = accumulate != 0;
    const int64_t need = zgb::embed_grad_layout(a, static_cast<char *>(workspace));
    if (!workspace || workspace_bytes < need)
        return report(ZERO_EINVAL, "the workspace has %lld bytes of the %lld needed",
                      (long long)(workspace ? workspace_bytes : 0), (long long)need);
    if (!aligned(workspace, 16))
        return report(ZERO_EALIGN, "the workspace is not aligned to 16 bytes");
    const int sms = sm_count();
    if (!sms) return ZERO_ECUDA;
    return launched(zgb::launch_embed_grad(dy_dtype, grad_dtype, a, sms, (cudaStream_t)stream),
                    "the embedding gradient");
}

int zero_dropout(const void *x, const void *residual, void *out, int32_t dtype, int64_t n,
                 double p, uint64_t seed, uint64_t offset, int64_t first, void *stream)
{
    if (!valid_dtype(dtype)) return report(ZERO_EINVAL, "unknown element type %d", dtype);
    if (n < 0 || n > (1ll << 42)) return report(ZERO_EINVAL, "%lld elements", (long long)n);
    if (!(p >= 0.0 && p <= 1.0)) return report(ZERO_EINVAL, "p must be in [0, 1]");
    if (first < 0 || first % 4)
        return report(ZERO_EINVAL, "the first element must be a multiple of 4, not %lld",
                      (long long)first);
    if (n > 0 && (!x || !out)) return report(ZERO_EINVAL, "x and out must not be null");
    const int es = zgb::elem_size(dtype);
    if (!aligned(x, es) || !aligned(residual, es) || !aligned(out, es))
        return report(ZERO_EALIGN, "x, residual and out must be aligned to %d bytes", es);
    if (n == 0) return ZERO_OK;
    zgb::DropoutArgs a = {};
    a.x = x;
    a.residual = residual;
    a.out = out;
    a.n = n;
    const double words = std::floor(p * 4294967296.0);
    a.all = words >= 4294967296.0;
    a.threshold = a.all ? 0 : (uint32_t)words;
    a.up = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.0f;
    for (uint32_t r = 0; r < 10; ++r) {
        a.key0[r] = (uint32_t)seed + r * 0x9E3779B9u;
        a.key1[r] = (uint32_t)(seed >> 32) + r * 0xBB67AE85u;
    }
    a.off0 = (uint32_t)offset;
    a.off1 = (uint32_t)(offset >> 32);
    a.first = (unsigned long long)first / 4;
    {   // round 1's product of off0, and round 2's of the word that it makes
        const uint64_t p1 = (uint64_t)a.off0 * 0xCD9E8D57u;
        const uint64_t p0 = (uint64_t)((uint32_t)(p1 >> 32) ^ a.key0[0]) * 0xD2511F53u;
        a.pre[0] = a.off1 ^ a.key1[0];
        a.pre[1] = (uint32_t)p1 ^ a.key0[1];
        a.pre[2] = (uint32_t)(p0 >> 32) ^ a.key1[1];
        a.pre[3] = (uint32_t)p0;
    }
    return launched(zgb::launch_dropout(dtype, a, (cudaStream_t)stream), "dropout");
}

int64_t zero_mx4_bytes(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 0 || rows > kMost || cols > kMost) return -1;
    return (rows + zgb::kMxRows - 1) / zgb::kMxRows * ((cols + zgb::kMxCols - 1) / zgb::kMxCols) *
           zgb::kMxRecord;
}

int zero_mx4_quantize(const void *x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride,
                      void *q, void *qt, void *stream)
{
    ZERO_TRY(check_matrix("x", x, dtype, rows, cols, stride));
    if (rows == 0 || cols == 0) return ZERO_OK;
    if (!q && !qt) return report(ZERO_EINVAL, "q and qt must not both be null");
    if (!aligned(q, 16) || !aligned(qt, 16))
        return report(ZERO_EALIGN, "q and qt must be aligned to 16 bytes");
    const int sms = sm_count();
    if (!sms) return ZERO_ECUDA;
    zgb::MxQuantArgs a = {x, rows, cols, stride, static_cast<unsigned char *>(q),
                          static_cast<unsigned char *>(qt)};
    return launched(zgb::launch_mx4_quantize(dtype, a, sms, (cudaStream_t)stream),
                    "the quantisation");
}

int zero_mx4_dequantize(const void *q, int64_t rows, int64_t cols, void *out, int32_t dtype,
                        int64_t stride, void *stream)
{
    ZERO_TRY(check_records("q", q, rows, cols));
    ZERO_TRY(check_matrix("out", out, dtype, rows, cols, stride));
    if (rows == 0 || cols == 0) return ZERO_OK;
    const int sms = sm_count();
    if (!sms) return ZERO_ECUDA;
    zgb::MxDequantArgs a = {static_cast<const unsigned char *>(q), rows, cols, stride, out};
    return launched(zgb::launch_mx4_dequantize(dtype, a, sms, (cudaStream_t)stream),
                    "the values");
}

int zero_mx4_matmul(const void *a, int64_t m, const void *b, int64_t n, int64_t k, float alpha,
                    int32_t accumulate, void *out, int32_t dtype, int64_t stride, void *stream)
{
    ZERO_TRY(check_records("a", a, m, k));
    ZERO_TRY(check_records("b", b, n, k));
    ZERO_TRY(check_matrix("out", out, dtype, m, n, stride));
    if (!std::isfinite(alpha)) return report(ZERO_EINVAL, "alpha must be finite");
    if (m == 0 || n == 0 || (k == 0 && accumulate)) return ZERO_OK;
    const int sms = sm_count();
    if (!sms) return ZERO_ECUDA;
    zgb::MxMatmulArgs g = {static_cast<const unsigned char *>(a),
                           static_cast<const unsigned char *>(b), m, n, k, alpha,
                           accumulate != 0, out, stride};
    return launched(zgb::launch_mx4_matmul(dtype, g, sms, (cudaStream_t)stream), "the product");
}

int zero_mx4_timeouts(uint32_t *count)
{
    if (!count) return report(ZERO_EINVAL, "null argument");
    unsigned int h = 0;
    cudaError_t e = zgb::mx4_timeouts(&h);
    if (e != cudaSuccess) return launched(e, "reading the product's timeout counter");
    *count = h;
    return h ? ZERO_ETIMEOUT : ZERO_OK;
}

}  // extern "C"
