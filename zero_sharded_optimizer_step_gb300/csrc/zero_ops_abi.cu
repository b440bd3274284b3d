// C ABI of the training operators: the embedding and its gradient, dropout,
// the microscaled 4-bit quantisation and product, the norm, 16-bit products and
// gated blocks, and rows kept in 8 bits.  Argument checks and
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

bool valid_16(int32_t d) { return d == ZERO_BF16 || d == ZERO_F16; }

bool valid_activation(int32_t a) { return a >= ZERO_ACT_NONE && a <= ZERO_ACT_SILU; }

int check_activation(int32_t a)
{
    return valid_activation(a) ? ZERO_OK : report(ZERO_EINVAL, "unknown activation %d", a);
}

bool size_ok(int64_t v) { return v >= 0 && v <= kMost; }

// A matrix that may be NULL.
int check_optional(const char *name, const void *p, int32_t dt, int64_t rows, int64_t cols,
                   int64_t stride)
{
    return p ? check_matrix(name, p, dt, rows, cols, stride) : ZERO_OK;
}

// A vector of `n` elements.
int check_vector(const char *name, const void *p, int32_t dt, int64_t n)
{
    return check_matrix(name, p, dt, 1, n, n);
}

int check_workspace(const void *workspace, int64_t bytes, int64_t need)
{
    if (need == 0) return ZERO_OK;
    if (!workspace || bytes < need)
        return report(ZERO_EINVAL, "the workspace has %lld bytes of the %lld needed",
                      (long long)(workspace ? bytes : 0), (long long)need);
    if (!aligned(workspace, 16))
        return report(ZERO_EALIGN, "the workspace is not aligned to 16 bytes");
    return ZERO_OK;
}

// What a call keeps or reads back: in the type, packed, or not at all.
int check_kept(const char *name, const void *kept, const void *q, int32_t dt, int64_t rows,
               int64_t cols, int64_t stride)
{
    if (kept && q) return report(ZERO_EINVAL, "%s is given in the type and in 8 bits", name);
    const int rc = check_optional(name, kept, dt, rows, cols, stride);
    return rc != ZERO_OK ? rc : q ? check_records(name, q, rows, cols) : ZERO_OK;
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

int64_t zero_pack8_bytes(int64_t rows, int64_t cols)
{
    if (!size_ok(rows) || !size_ok(cols)) return -1;
    return zgb::pack8_bytes(rows, cols);
}

int zero_pack8(const void *x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride, void *q,
               void *stream)
{
    ZERO_TRY(check_matrix("x", x, dtype, rows, cols, stride));
    ZERO_TRY(check_records("q", q, rows, cols));
    if (rows == 0 || cols == 0) return ZERO_OK;
    return launched(zgb::launch_pack8(dtype, x, rows, cols, stride,
                                      static_cast<unsigned char *>(q), (cudaStream_t)stream),
                    "the packing");
}

int zero_unpack8(const void *q, int64_t rows, int64_t cols, void *out, int32_t dtype,
                 int64_t stride, void *stream)
{
    ZERO_TRY(check_records("q", q, rows, cols));
    ZERO_TRY(check_matrix("out", out, dtype, rows, cols, stride));
    if (rows == 0 || cols == 0) return ZERO_OK;
    return launched(zgb::launch_unpack8(dtype, static_cast<const unsigned char *>(q), rows, cols,
                                        out, stride, (cudaStream_t)stream),
                    "the values");
}

int zero_rms_norm(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                  const void *weight, int32_t dtype, int64_t rows, int64_t dim, float eps,
                  void *sum, int64_t sum_stride, void *y, int64_t y_stride, void *q, float *rstd,
                  void *stream)
{
    ZERO_TRY(check_matrix("x", x, dtype, rows, dim, x_stride));
    ZERO_TRY(check_optional("residual", residual, dtype, rows, dim, residual_stride));
    ZERO_TRY(check_vector("weight", weight, dtype, dim));
    ZERO_TRY(check_optional("sum", sum, dtype, rows, dim, sum_stride));
    ZERO_TRY(check_optional("y", y, dtype, rows, dim, y_stride));
    if (!(eps >= 0.0f) || !std::isfinite(eps))
        return report(ZERO_EINVAL, "eps must be finite and not negative");
    if (!aligned(rstd, 4)) return report(ZERO_EALIGN, "rstd is not aligned to 4 bytes");
    if (q) ZERO_TRY(check_records("q", q, rows, dim));
    if (rows == 0 || dim == 0) return ZERO_OK;
    if (!y && !q) return report(ZERO_EINVAL, "y and q must not both be null");
    const int sms = sm_count();
    if (!sms) return ZERO_ECUDA;
    zgb::NormArgs a = {x, residual, weight, rows, dim, x_stride, residual_stride, eps, sum, y,
                       sum_stride, y_stride, static_cast<unsigned char *>(q), rstd};
    return launched(zgb::launch_norm(dtype, a, sms, (cudaStream_t)stream), "the norm");
}

int64_t zero_rms_norm_grad_workspace(int64_t rows, int64_t dim)
{
    if (!size_ok(rows) || !size_ok(dim)) return -1;
    return zgb::norm_grad_workspace(rows, dim);
}

int zero_rms_norm_grad(const void *dy, int64_t dy_stride, const void *dsum, int64_t dsum_stride,
                       const void *sum, int64_t sum_stride, const void *weight, const float *rstd,
                       int32_t dtype, int64_t rows, int64_t dim, void *dx, int64_t dx_stride,
                       void *dweight, int32_t grad_dtype, int32_t accumulate, void *workspace,
                       int64_t workspace_bytes, void *stream)
{
    ZERO_TRY(check_matrix("dy", dy, dtype, rows, dim, dy_stride));
    ZERO_TRY(check_optional("dsum", dsum, dtype, rows, dim, dsum_stride));
    ZERO_TRY(check_matrix("sum", sum, dtype, rows, dim, sum_stride));
    ZERO_TRY(check_vector("weight", weight, dtype, dim));
    ZERO_TRY(check_matrix("dx", dx, dtype, rows, dim, dx_stride));
    if (dweight) ZERO_TRY(check_vector("dweight", dweight, grad_dtype, dim));
    if (rows > 0 && dim > 0 && !rstd) return report(ZERO_EINVAL, "rstd must not be null");
    if (!aligned(rstd, 4)) return report(ZERO_EALIGN, "rstd is not aligned to 4 bytes");
    if (dim == 0 || (rows == 0 && (!dweight || accumulate))) return ZERO_OK;
    if (dweight)
        ZERO_TRY(check_workspace(workspace, workspace_bytes, zgb::norm_grad_workspace(rows, dim)));
    zgb::NormGradArgs a = {dy, dsum, sum, weight, rstd, rows, dim, dy_stride, dsum_stride,
                           sum_stride, dx, dweight, dx_stride, accumulate != 0};
    return launched(zgb::launch_norm_grad(dtype, grad_dtype, a, static_cast<float *>(workspace),
                                          (cudaStream_t)stream),
                    "the norm's gradient");
}

int64_t zero_matmul_workspace(const void *a, int32_t a_cols, int64_t a_stride, const void *b,
                              int32_t b_cols, int64_t b_stride, const void *a2, int64_t a2_stride,
                              const void *b2, int64_t b2_stride, int64_t m, int64_t n, int64_t k)
{
    if (!size_ok(m) || !size_ok(n) || !size_ok(k)) return -1;
    zgb::ProductArgs p = {};
    p.a = a, p.b = b, p.a2 = a2, p.b2 = b2;
    p.a_stride = a_stride, p.b_stride = b_stride, p.a2_stride = a2_stride, p.b2_stride = b2_stride;
    p.a_cols = a_cols != 0, p.b_cols = b_cols != 0;
    p.m = m, p.n = n, p.k = k;
    return zgb::product_workspace(p);
}

int zero_matmul(const void *a, int32_t a_cols, int64_t a_stride, const void *b, int32_t b_cols,
                int64_t b_stride, const void *a2, int64_t a2_stride, const void *b2,
                int64_t b2_stride, int32_t dtype, int64_t m, int64_t n, int64_t k,
                const void *bias, int32_t activation, const void *residual,
                int64_t residual_stride, void *kept, int64_t kept_stride, void *kept_q, void *out,
                int32_t out_dtype, int64_t out_stride, int32_t accumulate, void *workspace,
                int64_t workspace_bytes, void *stream)
{
    if (!valid_16(dtype)) return report(ZERO_EINVAL, "the operands are bf16 or fp16, not %d", dtype);
    if (out_dtype != dtype && out_dtype != ZERO_F32)
        return report(ZERO_EINVAL, "the result is of the operands' type or fp32, not %d", out_dtype);
    auto operand = [&](const char *name, const void *p, int64_t rows, int32_t cols, int64_t stride) {
        return cols ? check_matrix(name, p, dtype, k, rows, stride)
                    : check_matrix(name, p, dtype, rows, k, stride);
    };
    ZERO_TRY(operand("a", a, m, a_cols, a_stride));
    ZERO_TRY(operand("b", b, n, b_cols, b_stride));
    if (m > 0 && n > 0 && k > 0 && (a2 != nullptr) != (b2 != nullptr))   // empty ones have no place
        return report(ZERO_EINVAL, "a2 and b2 are given together");
    if (a2 && b2) {
        ZERO_TRY(operand("a2", a2, m, a_cols, a2_stride));
        ZERO_TRY(operand("b2", b2, n, b_cols, b2_stride));
    }
    if (bias) ZERO_TRY(check_vector("bias", bias, dtype, n));
    ZERO_TRY(check_activation(activation));
    ZERO_TRY(check_optional("residual", residual, out_dtype, m, n, residual_stride));
    if (residual && accumulate)
        return report(ZERO_EINVAL, "a residual and accumulate are not given together");
    ZERO_TRY(check_kept("kept", kept, kept_q, dtype, m, n, kept_stride));
    ZERO_TRY(check_matrix("out", out, out_dtype, m, n, out_stride));
    if (m == 0 || n == 0) return ZERO_OK;
    zgb::ProductArgs p = {};
    p.a = a, p.b = b, p.a2 = a2, p.b2 = b2;
    p.a_stride = a_stride, p.b_stride = b_stride, p.a2_stride = a2_stride, p.b2_stride = b2_stride;
    p.a_cols = a_cols != 0, p.b_cols = b_cols != 0;
    p.act = activation;
    p.m = m, p.n = n, p.k = k;
    p.bias = bias;
    p.residual = accumulate ? out : residual;
    p.residual_stride = accumulate ? out_stride : residual_stride;
    p.kept = kept, p.kept_stride = kept_stride, p.kept_q = static_cast<unsigned char *>(kept_q);
    p.out = out, p.stride = out_stride;
    ZERO_TRY(check_workspace(workspace, workspace_bytes, zgb::product_workspace(p)));
    const int sms = sm_count();
    if (!sms) return ZERO_ECUDA;
    return launched(zgb::launch_product(dtype, out_dtype, p, workspace, sms, (cudaStream_t)stream),
                    "the product");
}

int64_t zero_gated_workspace(const void *x, int64_t x_stride, const void *w_gate,
                             int64_t gate_stride, const void *w_up, int64_t up_stride, int64_t m,
                             int64_t n, int64_t k)
{
    return zero_matmul_workspace(x, 0, x_stride, w_gate, 0, gate_stride, nullptr, 0, w_up,
                                 up_stride, m, n, k);
}

int zero_gated(const void *x, int64_t x_stride, const void *w_gate, int64_t gate_stride,
               const void *w_up, int64_t up_stride, int32_t dtype, int64_t m, int64_t n, int64_t k,
               int32_t activation, void *gate, void *up, int64_t kept_stride, void *gate_q,
               void *up_q, void *h, int64_t h_stride, void *workspace, int64_t workspace_bytes,
               void *stream)
{
    if (!valid_16(dtype)) return report(ZERO_EINVAL, "the operands are bf16 or fp16, not %d", dtype);
    ZERO_TRY(check_matrix("x", x, dtype, m, k, x_stride));
    ZERO_TRY(check_matrix("w_gate", w_gate, dtype, n, k, gate_stride));
    ZERO_TRY(check_matrix("w_up", w_up, dtype, n, k, up_stride));
    ZERO_TRY(check_activation(activation));
    if ((gate != nullptr) != (up != nullptr) || (gate_q != nullptr) != (up_q != nullptr))
        return report(ZERO_EINVAL, "the gate and the other projection are kept together");
    ZERO_TRY(check_kept("gate", gate, gate_q, dtype, m, n, kept_stride));
    ZERO_TRY(check_kept("up", up, up_q, dtype, m, n, kept_stride));
    ZERO_TRY(check_matrix("h", h, dtype, m, n, h_stride));
    if (m == 0 || n == 0) return ZERO_OK;
    zgb::ProductArgs p = {};
    p.a = x, p.b = w_gate, p.b2 = w_up;
    p.a_stride = x_stride, p.b_stride = gate_stride, p.b2_stride = up_stride;
    p.gated = 1;
    p.act = activation;
    p.m = m, p.n = n, p.k = k;
    p.kept = gate, p.kept2 = up, p.kept_stride = kept_stride;
    p.kept_q = static_cast<unsigned char *>(gate_q);
    p.kept2_q = static_cast<unsigned char *>(up_q);
    p.out = h, p.stride = h_stride;
    ZERO_TRY(check_workspace(workspace, workspace_bytes, zgb::product_workspace(p)));
    const int sms = sm_count();
    if (!sms) return ZERO_ECUDA;
    return launched(zgb::launch_product(dtype, dtype, p, workspace, sms, (cudaStream_t)stream),
                    "the gated block");
}

int64_t zero_activation_grad_workspace(int64_t rows, int64_t cols)
{
    if (!size_ok(rows) || !size_ok(cols)) return -1;
    return zgb::activation_grad_workspace(rows, cols);
}

int zero_activation_grad(const void *dy, int64_t dy_stride, const void *kept, int64_t kept_stride,
                         const void *kept_q, int32_t activation, int32_t dtype, int64_t rows,
                         int64_t cols, void *dz, int64_t dz_stride, void *dbias,
                         int32_t bias_dtype, int32_t accumulate, void *workspace,
                         int64_t workspace_bytes, void *stream)
{
    ZERO_TRY(check_matrix("dy", dy, dtype, rows, cols, dy_stride));
    ZERO_TRY(check_activation(activation));
    ZERO_TRY(check_kept("kept", kept, kept_q, dtype, rows, cols, kept_stride));
    ZERO_TRY(check_optional("dz", dz, dtype, rows, cols, dz_stride));
    if (dbias) ZERO_TRY(check_vector("dbias", dbias, bias_dtype, cols));
    if (cols == 0) return ZERO_OK;
    if (!dz && !dbias) return report(ZERO_EINVAL, "dz and dbias must not both be null");
    if (rows > 0 && activation != ZERO_ACT_NONE && !kept && !kept_q)
        return report(ZERO_EINVAL, "kept and kept_q must not both be null");
    if (rows == 0 && (!dbias || accumulate)) return ZERO_OK;
    if (dbias)
        ZERO_TRY(check_workspace(workspace, workspace_bytes,
                                 zgb::activation_grad_workspace(rows, cols)));
    zgb::ActGradArgs a = {dy, kept, static_cast<unsigned char *>(const_cast<void *>(kept_q)),
                          rows, cols, dy_stride, kept_stride, activation, dz, dbias, dz_stride,
                          accumulate != 0};
    return launched(zgb::launch_activation_grad(dtype, bias_dtype, a,
                                                static_cast<float *>(workspace),
                                                (cudaStream_t)stream),
                    "the activation's gradient");
}

int zero_gated_grad(const void *dh, int64_t dh_stride, const void *gate, const void *up,
                    int64_t kept_stride, const void *gate_q, const void *up_q, int32_t activation,
                    int32_t dtype, int64_t rows, int64_t cols, void *dgate, void *dup,
                    int64_t grad_stride, void *h, int64_t h_stride, void *stream)
{
    ZERO_TRY(check_matrix("dh", dh, dtype, rows, cols, dh_stride));
    ZERO_TRY(check_activation(activation));
    if ((gate != nullptr) != (up != nullptr) || (gate_q != nullptr) != (up_q != nullptr))
        return report(ZERO_EINVAL, "the gate and the other projection are given together");
    ZERO_TRY(check_kept("gate", gate, gate_q, dtype, rows, cols, kept_stride));
    ZERO_TRY(check_kept("up", up, up_q, dtype, rows, cols, kept_stride));
    ZERO_TRY(check_matrix("dgate", dgate, dtype, rows, cols, grad_stride));
    ZERO_TRY(check_matrix("dup", dup, dtype, rows, cols, grad_stride));
    ZERO_TRY(check_optional("h", h, dtype, rows, cols, h_stride));
    if (rows == 0 || cols == 0) return ZERO_OK;
    if (!gate && !gate_q) return report(ZERO_EINVAL, "gate and gate_q must not both be null");
    auto bytes = [](const void *p) { return static_cast<unsigned char *>(const_cast<void *>(p)); };
    zgb::GatedGradArgs a = {dh, gate, up, bytes(gate_q), bytes(up_q), rows, cols, dh_stride,
                            kept_stride, activation, dgate, dup, h, grad_stride, h_stride};
    return launched(zgb::launch_gated_grad(dtype, a, (cudaStream_t)stream),
                    "the gated block's gradient");
}

int zero_matmul_timeouts(uint32_t *count)
{
    if (!count) return report(ZERO_EINVAL, "null argument");
    unsigned int h = 0;
    cudaError_t e = zgb::matmul_timeouts(&h);
    if (e != cudaSuccess) return launched(e, "reading the products' timeout counter");
    *count = h;
    return h ? ZERO_ETIMEOUT : ZERO_OK;
}

}  // extern "C"
