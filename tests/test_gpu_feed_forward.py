"""The norm, the 16-bit products, the gated block and the rows kept in 8 bits on
a GPU, against their definitions in 64 bits (tests/ff_ref.py)."""
import itertools

import pytest
import torch

import tests.ff_ref as F

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import zero_sharded_optimizer_step_gb300 as z
    CODE = {torch.float32: z.ZERO_F32, torch.bfloat16: z.ZERO_BF16, torch.float16: z.ZERO_F16}

DEV = "cuda"
ALL = [torch.float32, torch.bfloat16, torch.float16]
LOW = [torch.bfloat16, torch.float16]
U = 2.0 ** -24


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, sigma=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * sigma).to(dtype)


class Held:
    """rows x cols inside a larger buffer, at `offset` elements with `stride`
    between the rows, everything around it NaN (or the pattern that NaN bits
    are): untouched() says whether that is still so."""

    def __init__(self, rows, cols, stride, offset, dtype, fill=None):
        n = offset + max(rows, 1) * stride + 64
        self.buf = torch.full((n,), float("nan"), dtype=dtype, device=DEV)
        self.t = self.buf.as_strided((rows, cols), (stride, 1), offset)
        if fill is not None:
            self.t.copy_(fill)
        self.mask = torch.ones(n, dtype=torch.bool, device=DEV)
        self.mask.as_strided((rows, cols), (stride, 1), offset).fill_(False)

    def untouched(self):
        return bool(torch.isnan(self.buf[self.mask]).all())


def held(x, stride=None, offset=0):
    rows, cols = x.shape
    return Held(rows, cols, stride or cols, offset, x.dtype, x)


def space(rows, cols, dtype, stride=None, offset=0):
    return Held(rows, cols, stride or max(cols, 1), offset, dtype)


def packed(rows, cols):
    """Room for 8-bit rows, and a guard behind them."""
    n = z.zero_pack8_bytes(rows, cols)
    return torch.full((n + 64,), 0xA5, dtype=torch.uint8, device=DEV)


def unpack(q, rows, cols, dtype=torch.float32):
    out = torch.empty(rows, cols, dtype=dtype, device=DEV)
    z.zero_unpack8(q, rows, cols, out, CODE[dtype], cols)
    return out


def parts(q, rows, cols):
    """(codes past the columns, scales, guard)."""
    pitch = -(-cols // 32) * 32
    n = rows * pitch
    codes = q[:n].view(rows, pitch)
    return codes[:, cols:], q[n:n + n // 32].view(rows, pitch // 32), q[n + n // 32:]


# ------------------------------------------------------------------ 8-bit rows

@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,cols,stride,offset", [
    (1, 1, 1, 0), (3, 31, 31, 0), (5, 32, 32, 0), (2, 33, 40, 3), (9, 256, 256, 0),
    (7, 257, 259, 1), (300, 1600, 1600, 0), (33, 4099, 4100, 5), (1, 20000, 20000, 0)])
def test_pack8(dtype, rows, cols, stride, offset):
    g = gen(rows * cols)
    x = held(randn(g, rows, cols, dtype=dtype) * torch.where(
        torch.rand(cols, generator=g, device=DEV) < 0.1, 40.0, 1.0).to(dtype), stride, offset)
    q = packed(rows, cols)
    z.zero_pack8(x.t, CODE[dtype], rows, cols, stride, q)
    want, scales = F.pack(x.t.double())
    tail, got_scales, guard = parts(q, rows, cols)
    assert torch.equal(got_scales, scales) and not tail.any() and bool((guard == 0xA5).all())
    for out_dtype in ALL:
        out = space(rows, cols, out_dtype, stride, offset)
        z.zero_unpack8(q, rows, cols, out.t, CODE[out_dtype], stride)
        assert torch.equal(out.t, F.rounded(want, out_dtype)) and out.untouched()


@pytest.mark.parametrize("dtype", ALL)
def test_pack8_extremes(dtype):
    """Every tie of e4m3 at every power of two of the type, both signs, zeros,
    the largest and smallest values, infinities and NaN."""
    f = torch.finfo(dtype)
    grid = torch.cat([1 + torch.arange(16, device=DEV).double() / 16,
                      torch.tensor([448.0, 449, 224, 225, 0.001, 2 ** -9, 2 ** -10,
                                    1.5 * 2 ** -10], device=DEV).double()])
    lines = [torch.cat([grid, -grid[:8]]) * 2.0 ** e for e in range(-160, 128, 5)]
    x = torch.stack(lines).clamp(-f.max, f.max).to(dtype)
    more = torch.zeros(6, 32, dtype=dtype, device=DEV)
    more[1], more[2] = f.max, f.smallest_normal / 2
    more[3, 7], more[4, 31], more[5, 0] = float("inf"), float("nan"), float("-inf")
    x = torch.cat([x, more])
    q = packed(*x.shape)
    z.zero_pack8(x, CODE[dtype], *x.shape, 32, q)
    want, scales = F.pack(x.double())
    _, got, _ = parts(q, *x.shape)
    assert torch.equal(got, scales)
    for out_dtype in ALL:
        v = unpack(q, *x.shape, out_dtype)
        w = F.rounded(want, out_dtype)
        assert torch.equal(torch.isnan(v), torch.isnan(w))
        assert torch.equal(v.nan_to_num(), w.nan_to_num())


# -------------------------------------------------------------------- the norm

def norm(x, residual, w, eps, sum=None, y=None, q=None, rstd=None):
    rows, dim = x.t.shape

    def p(h):
        return (h.t, h.t.stride(0)) if h is not None else (None, 0)

    z.zero_rms_norm(*p(x), *p(residual), w, CODE[x.t.dtype], rows, dim, eps, *p(sum), *p(y), q,
                    rstd)


def norm_want(x, residual, w, eps):
    """sum, rstd, y in 64 bits, and y's error in fp32: the squares' sum of dim
    additions is off by (dim + 2) U at most, relatively, which the root halves; half a dozen
    more roundings follow."""
    s = x.double()
    if residual is not None:
        s = (s + residual.double()).to(x.dtype).double()
    dim = x.shape[1]
    rstd = ((s * s).sum(1, keepdim=True) / dim + eps) ** -0.5
    y = s * rstd * w.double()
    return s, rstd, y, (0.5 * (dim + 2) + 8) * U * y.abs()


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,dim", [(1, 1), (1, 64), (3, 255), (48, 768), (5, 1600), (2500, 200),
                                      (2500, 257), (2600, 1001), (2432, 1024), (2433, 2056),
                                      (2440, 4096), (17, 8192), (3, 8200), (9, 12289)])
@pytest.mark.parametrize("stride,offset", [(0, 0), (8, 8), (3, 1)])
def test_norm(dtype, rows, dim, stride, offset):
    g = gen(rows + dim)
    stride += dim
    x = held(randn(g, rows, dim, dtype=dtype, sigma=3), stride, offset)
    r = held(randn(g, rows, dim, dtype=dtype), stride, offset)
    w = randn(g, dim, dtype=dtype)
    for residual in (None, r):
        s, rstd, y, err = norm_want(x.t, residual and residual.t, w, 1e-5)
        gs, gy = space(rows, dim, dtype, stride, offset), space(rows, dim, dtype, stride, offset)
        q = packed(rows, dim)
        gr = torch.empty(rows, device=DEV)
        norm(x, residual, w, 1e-5, gs, gy, q, gr)
        assert torch.equal(gs.t.double(), s) and gs.untouched() and gy.untouched()
        F.within(gr[:, None], rstd, (0.5 * (dim + 2) + 6) * U * rstd, torch.float32)
        F.within(gy.t, y, err)
        # packed from fp32: a step of the element's own, or of a scale that is next to a border
        top = F.pack(y)[0].abs().reshape(rows, -1)
        v = unpack(q, rows, dim).double()
        block = torch.nn.functional.pad(y.abs(), (0, -dim % 32)).reshape(rows, -1, 32).amax(
            2, keepdim=True).expand(-1, -1, 32).reshape(rows, -1)[:, :dim]
        # half a step is 2^-4 of the value, or 2^-10 of a scale of at most max / 224
        assert bool(((v - y).abs() <= (2.0 ** -4 * y.abs()).maximum(2.0 ** -10 * block / 224)
                     * 1.001 + 2.0 ** -137).all()), top.shape
        _, _, guard = parts(q, rows, dim)
        assert bool((guard == 0xA5).all())
        # each output alone gives the same bits
        gy2, q2 = space(rows, dim, dtype, stride, offset), packed(rows, dim)
        norm(x, residual, w, 1e-5, None, gy2)
        norm(x, residual, w, 1e-5, None, None, q2)
        assert torch.equal(gy2.t, gy.t) and torch.equal(q2, q)


@pytest.mark.parametrize("dim", [100, 768, 4096, 9000])
@pytest.mark.parametrize("into", ["x", "residual"])
def test_norm_in_place(dim, into):
    g = gen(dim)
    x, r = (held(randn(g, 50, dim, dtype=torch.bfloat16)) for _ in range(2))
    w = randn(g, dim, dtype=torch.bfloat16)
    s, y = space(50, dim, torch.bfloat16), space(50, dim, torch.bfloat16)
    norm(x, r, w, 1e-6, s, y)
    y2 = space(50, dim, torch.bfloat16)
    norm(x, r, w, 1e-6, x if into == "x" else r, y2)
    assert torch.equal((x if into == "x" else r).t, s.t) and torch.equal(y2.t, y.t)


def test_norm_of_zeros_infinities_and_nan():
    x = torch.zeros(4, 512, device=DEV)
    x[1, 3], x[2, 5] = float("inf"), float("nan")
    x[3] = 2.0
    y, w = space(4, 512, torch.float32), torch.ones(512, device=DEV)
    q = packed(4, 512)
    norm(held(x), None, w, 1e-5, None, y, q)
    assert not y.t[0].any() and torch.isnan(y.t[2]).all()
    assert torch.isnan(y.t[1, 3]) and not y.t[1, 4:].any()
    assert float((y.t[3] - 1).abs().max()) < 1e-5
    v = unpack(q, 4, 512)
    assert torch.isnan(v[1, :32]).all() and not v[1, 32:].any() and torch.isnan(v[2]).all()


def norm_grad(dy, ds, s, w, rstd, dx, dw=None, accumulate=False):
    rows, dim = dy.t.shape
    need = z.zero_rms_norm_grad_workspace(rows, dim)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    z.zero_rms_norm_grad(dy.t, dy.t.stride(0), ds.t if ds else None, ds.t.stride(0) if ds else 0,
                         s.t, s.t.stride(0), w, rstd, CODE[dy.t.dtype], rows, dim, dx.t,
                         dx.t.stride(0), dw, CODE[dw.dtype] if dw is not None else 0, accumulate,
                         ws, need)
    assert bool((ws[need:] == 0xA5).all())


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,dim", [(1, 1), (2, 64), (700, 200), (9, 255), (5000, 257),
                                      (100, 1024), (70, 1600), (700, 4096), (3, 4099), (17, 8192),
                                      (300, 8200), (5, 12289)])
@pytest.mark.parametrize("stride,offset", [(0, 0), (3, 1)])
def test_norm_gradient(dtype, rows, dim, stride, offset):
    g = gen(rows + dim)
    stride += dim
    s = held(randn(g, rows, dim, dtype=dtype, sigma=2), stride, offset)
    dy = held(randn(g, rows, dim, dtype=dtype), stride, offset)
    ds = held(randn(g, rows, dim, dtype=dtype), stride, offset)
    w = randn(g, dim, dtype=dtype)
    rstd64 = ((s.t.double() ** 2).mean(1, keepdim=True) + 1e-5) ** -0.5
    rstd = rstd64[:, 0].float()
    n, wdy = s.t.double() * rstd[:, None].double(), dy.t.double() * w.double()
    share = (wdy * n).sum(1, keepdim=True) / dim
    dw = (dy.t.double() * n).sum(0)
    # dim (rows) additions and a few roundings of what is added
    dw_err = (rows + 4) * U * (dy.t.double() * n).abs().sum(0)
    share_err = (dim + 6) * U * (wdy * n).abs().sum(1, keepdim=True) / dim
    r = rstd[:, None].double()
    for extra in (None, ds):
        dx = r * (wdy - n * share) + (extra.t.double() if extra else 0.0)
        err = r * n.abs() * share_err + 6 * U * (
            r * (wdy.abs() + (n * share).abs()) + (extra.t.double().abs() if extra else 0.0))
        got = space(rows, dim, dtype, stride, offset)
        gw = torch.full((dim,), float("nan"), dtype=dtype, device=DEV)
        norm_grad(dy, extra, s, w, rstd, got, gw)
        F.within(got.t, dx, err)
        F.within(gw, dw, dw_err)
        assert got.untouched()
        # without the weight's, and the weight's added to fp32: the same dx
        got2 = space(rows, dim, dtype, stride, offset)
        norm_grad(dy, extra, s, w, rstd, got2)
        acc = torch.full((dim,), 3.0, device=DEV)
        norm_grad(dy, extra, s, w, rstd, got2, acc, True)
        assert torch.equal(got2.t, got.t)
        F.within(acc, dw + 3.0, dw_err + U * (dw_err + dw.abs() + 3.0))


def test_norm_gradient_against_differences():
    g = gen(1)
    rows, dim = 4, 40
    x, w = randn(g, rows, dim), randn(g, dim)
    v = randn(g, rows, dim).double()

    def loss(x, w):
        return float((norm_want(x, None, w, 1e-3)[2] * v).sum())

    rstd = torch.empty(rows, device=DEV)
    y = space(rows, dim, torch.float32)
    norm(held(x), None, w, 1e-3, None, y, None, rstd)
    dx, dw = space(rows, dim, torch.float32), torch.empty(dim, device=DEV)
    norm_grad(held(v.float()), None, held(x), w, rstd, dx, dw)
    h = 1e-4

    def nudged(t, i, by):
        t = t.double().clone()
        t.view(-1)[i] += by
        return t

    for i in (0, 41, 159):
        d = (loss(nudged(x, i, h), w.double()) - loss(nudged(x, i, -h), w.double())) / (2 * h)
        # the difference's own error is of the order of h^2 (1e-8) and v is rounded
        assert abs(d - float(dx.t.reshape(-1)[i])) < 1e-4 * max(1.0, abs(d))
    for i in (0, 39):
        d = (loss(x.double(), nudged(w, i, h)) - loss(x.double(), nudged(w, i, -h))) / (2 * h)
        assert abs(d - float(dw[i])) < 1e-4 * max(1.0, abs(d))


def test_norm_gradient_without_rows():
    w = torch.ones(8, device=DEV)
    dw = torch.full((8,), 5.0, device=DEV)
    e = space(0, 8, torch.float32)
    rstd = torch.empty(0, device=DEV)
    norm_grad(e, None, e, w, rstd, e, dw, True)
    assert bool((dw == 5).all())
    norm_grad(e, None, e, w, rstd, e, dw)
    assert not dw.any()


# ---------------------------------------------------------------- the products

def product(a, a_cols, b, b_cols, out, a2=None, b2=None, bias=None, act=F.NONE, residual=None,
            kept=None, kept_q=None, accumulate=False):
    (m, k) = reversed(a.t.shape) if a_cols else a.t.shape
    n = b.t.shape[1] if b_cols else b.t.shape[0]
    dtype = a.t.dtype

    def p(h):
        return (h.t, max(h.t.stride(0), h.t.shape[1])) if h is not None else (None, 0)

    pa, pb = p(a), p(b)
    need = z.zero_matmul_workspace(pa[0], a_cols, pa[1], pb[0], b_cols, pb[1], *p(a2), *p(b2), m,
                                   n, k)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    z.zero_matmul(pa[0], a_cols, pa[1], pb[0], b_cols, pb[1], *p(a2), *p(b2), CODE[dtype], m, n,
                  k, bias, act, *p(residual), *p(kept), kept_q, out.t, CODE[out.t.dtype],
                  max(out.t.stride(0), n), accumulate, ws, need)
    assert bool((ws[need:] == 0xA5).all())
    return need


def as_lies(x, cols, pad=0, offset=0):
    t = x.t().contiguous() if cols else x
    return held(t, t.shape[1] + pad, offset)


SIZES = [(1, 1, 1), (1, 128, 64), (1, 300, 1000), (2, 130, 72), (7, 40, 33), (16, 256, 512),
         (17, 200, 100), (64, 1000, 520), (65, 129, 40), (100, 256, 64), (128, 384, 200),
         (200, 40, 300), (333, 520, 130)]
BIG = [(1500, 2000, 200), (1537, 1601, 65), (257, 10000, 96), (4000, 640, 328), (2560, 1040, 16)]


@pytest.mark.parametrize("dtype", LOW)
@pytest.mark.parametrize("a_cols,b_cols", list(itertools.product([False, True], repeat=2)))
@pytest.mark.parametrize("m,n,k", SIZES + BIG)
def test_product(dtype, a_cols, b_cols, m, n, k):
    g = gen(m * n + k)
    a, b = randn(g, m, k, dtype=dtype), randn(g, n, k, dtype=dtype)
    want, err = F.product(a.double(), b.double())
    out = space(m, n, dtype)
    product(as_lies(a, a_cols), a_cols, as_lies(b, b_cols), b_cols, out)
    F.within(out.t, want, err)
    assert out.untouched()
    wide = space(m, n, torch.float32, n + 3, 1)
    need = product(as_lies(a, a_cols, 3, 1), a_cols, as_lies(b, b_cols, 5, 3), b_cols, wide)
    assert need > 0 or (m <= 4 and not a_cols and not b_cols)     # few rows need no copy
    F.within(wide.t, want, err)
    assert wide.untouched()
    assert z.zero_matmul_timeouts() == 0


@pytest.mark.parametrize("a_cols,b_cols", [(False, False), (False, True), (True, True)])
@pytest.mark.parametrize("m,n,k", [(5, 100, 70), (130, 260, 72), (1500, 2100, 100)])
def test_product_of_two_pairs(a_cols, b_cols, m, n, k):
    g = gen(m)
    a, a2 = (randn(g, m, k, dtype=torch.bfloat16) for _ in range(2))
    b, b2 = (randn(g, n, k, dtype=torch.bfloat16) for _ in range(2))
    want, err = F.product(torch.cat([a, a2], 1).double(), torch.cat([b, b2], 1).double())
    for pad in (0, 1):
        out = space(m, n, torch.bfloat16)
        product(as_lies(a, a_cols, pad), a_cols, as_lies(b, b_cols), b_cols, out,
                as_lies(a2, a_cols), as_lies(b2, b_cols, pad))
        F.within(out.t, want, err)


@pytest.mark.parametrize("dtype", LOW)
@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("m,n,k,pad,offset", [
    (3, 100, 64, 0, 0), (77, 257, 40, 1, 1), (128, 256, 72, 0, 0), (1500, 2016, 72, 0, 0),
    (1500, 2010, 72, 6, 16), (1400, 2100, 64, 1, 1)])
def test_product_with_everything(dtype, act, m, n, k, pad, offset):
    """Bias, activation, residual and both ways of keeping, whole rows and
    rows off the boundaries."""
    g = gen(m + n + act)
    a, b = randn(g, m, k, dtype=dtype), randn(g, n, k, dtype=dtype, sigma=k ** -0.5 * 3)
    bias, r = randn(g, n, dtype=dtype), randn(g, m, n, dtype=dtype)
    zz, err = F.product(a.double(), b.double())
    zz = zz + bias.double()
    err = err + U * (zz.abs() + err)
    y = F.activation(zz, act)[0]
    yerr = F.value_error(zz, err, act)
    out, kept = (space(m, n, dtype, n + pad, offset) for _ in range(2))
    res = held(r, n + pad, offset)
    product(held(a), False, held(b), False, out, bias=bias, act=act, residual=res, kept=kept)
    F.within(kept.t, zz, err)
    F.within(out.t, y + r.double(), yerr + U * (y + r.double()).abs() + U * yerr)
    assert out.untouched() and kept.untouched()
    q = packed(m, n)
    out2 = space(m, n, dtype, n + pad, offset)
    product(held(a), False, held(b), False, out2, bias=bias, act=act, residual=res, kept_q=q)
    assert torch.equal(out2.t, out.t)
    # within half a step of the value, or of the block's smallest numbers
    v = unpack(q, m, n).double()
    block = torch.nn.functional.pad(zz.abs(), (0, -n % 32)).reshape(m, -1, 32).amax(
        2, keepdim=True).expand(-1, -1, 32).reshape(m, -1)[:, :n]
    step = (2.0 ** -4 * zz.abs()).maximum(2.0 ** -10 * block / 224)
    assert bool(((v - zz).abs() <= step * 1.001 + 1.1 * err).all())
    tail, _, guard = parts(q, m, n)
    assert not tail.any() and bool((guard == 0xA5).all())
    # into the residual itself, and as accumulation
    again = held(r, n + pad, offset)
    product(held(a), False, held(b), False, again, bias=bias, act=act, residual=again)
    assert torch.equal(again.t, out.t)
    again = held(r, n + pad, offset)
    product(held(a), False, held(b), False, again, bias=bias, act=act, accumulate=True)
    assert torch.equal(again.t, out.t)


@pytest.mark.parametrize("m,n", [(3, 40), (128, 256), (1500, 2016)])
def test_product_accumulates_in_fp32(m, n):
    g = gen(n)
    k = 200
    a, b = randn(g, m, k, dtype=torch.bfloat16), randn(g, n, k, dtype=torch.bfloat16)
    start = randn(g, m, n)
    want, err = F.product(a.double(), b.double())
    out = held(start)
    product(as_lies(a, True), True, as_lies(b, True), True, out, accumulate=True)
    want = want + start.double()
    F.within(out.t, want, err + U * want.abs())


@pytest.mark.parametrize("m,n", [(3, 100), (1500, 2016)])
def test_product_of_nothing(m, n):
    """k = 0: the activation of the bias."""
    bias, r = randn(gen(1), n, dtype=torch.bfloat16), randn(gen(2), m, n, dtype=torch.bfloat16)
    out = space(m, n, torch.bfloat16)
    a, b = space(m, 0, torch.bfloat16, 8), space(n, 0, torch.bfloat16, 8)
    product(a, False, b, False, out, bias=bias, act=F.SILU, residual=held(r))
    y = F.activation(bias.double(), F.SILU)[0]
    F.within(out.t, y + r.double(), F.value_error(bias.double(), 0 * y, F.SILU)
             + U * (y + r.double()).abs())


@pytest.mark.parametrize("m,n,k", [(2, 100, 64), (70, 130, 200), (1500, 2016, 72)])
def test_product_of_infinities_and_nan(m, n, k):
    """They reach their own row or column alone."""
    g = gen(3)
    a, b = randn(g, m, k, dtype=torch.bfloat16), randn(g, n, k, dtype=torch.bfloat16)
    a[1, 5], b[7, 2] = float("inf"), float("nan")
    out = space(m, n, torch.bfloat16)
    product(held(a), False, held(b), False, out)
    rows = torch.isfinite(out.t)
    assert not rows[1].any() and not rows[:, 7].any()
    rows[1], rows[:, 7] = True, True
    assert bool(rows.all())
    want = a.double() @ b.double().t()
    assert torch.equal(torch.isnan(out.t), torch.isnan(want))


def test_product_is_the_same_on_every_run():
    g = gen(8)
    for m, n, k in [(1, 6400, 1600), (40, 500, 3000), (130, 260, 2000), (2000, 3000, 500)]:
        a, b = held(randn(g, m, k, dtype=torch.float16)), held(randn(g, n, k, dtype=torch.float16))
        first = space(m, n, torch.float32)
        product(a, False, b, False, first)
        for _ in range(3):
            again = space(m, n, torch.float32)
            product(a, False, b, False, again)
            assert torch.equal(again.t, first.t)


# ------------------------------------------------------------- the gated block

def gated(x, wg, wu, h, act, gate=None, up=None, gate_q=None, up_q=None):
    m, k = x.t.shape
    n = wg.t.shape[0]

    def p(t):
        return t.t, max(t.t.stride(0), t.t.shape[1])

    need = z.zero_gated_workspace(*p(x), *p(wg), *p(wu), m, n, k)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    z.zero_gated(*p(x), *p(wg), *p(wu), CODE[x.t.dtype], m, n, k, act, gate.t if gate else None,
                 up.t if up else None, gate.t.stride(0) if gate else 0, gate_q, up_q, *p(h), ws,
                 need)
    assert bool((ws[need:] == 0xA5).all())


@pytest.mark.parametrize("dtype", LOW)
@pytest.mark.parametrize("act", [F.SILU, F.GELU_TANH, F.NONE])
@pytest.mark.parametrize("m,n,k,pad,offset", [
    (1, 1, 1, 0, 0), (1, 300, 1000, 0, 0), (5, 33, 40, 3, 1), (17, 128, 128, 0, 0),
    (77, 260, 72, 0, 0), (130, 384, 64, 0, 0), (1500, 2016, 72, 0, 0), (1500, 2000, 40, 0, 0),
    (1401, 2001, 33, 1, 1), (2600, 1000, 200, 0, 0)])
def test_gated(dtype, act, m, n, k, pad, offset):
    g = gen(m + n + act)
    x = randn(g, m, k, dtype=dtype)
    wg, wu = (randn(g, n, k, dtype=dtype, sigma=k ** -0.5) for _ in range(2))
    gate, gerr = F.product(x.double(), wg.double())
    up, uerr = F.product(x.double(), wu.double())
    f, ferr = F.activation(gate, act)[0], F.value_error(gate, gerr, act)
    want = f * up
    err = ferr * up.abs() + f.abs() * uerr + ferr * uerr + 2 * U * want.abs()
    h, kg, ku = (space(m, n, dtype, n + pad, offset) for _ in range(3))
    gated(held(x, k + pad, offset), held(wg, k + pad, offset), held(wu), h, act, kg, ku)
    F.within(h.t, want, err)
    F.within(kg.t, gate, gerr)
    F.within(ku.t, up, uerr)
    assert h.untouched() and kg.untouched() and ku.untouched()
    qg, qu = packed(m, n), packed(m, n)
    h2 = space(m, n, dtype, n + pad, offset)
    gated(held(x, k + pad, offset), held(wg, k + pad, offset), held(wu), h2, act, None, None, qg,
          qu)
    assert torch.equal(h2.t, h.t)
    for q, v, e in ((qg, gate, gerr), (qu, up, uerr)):
        block = torch.nn.functional.pad(v.abs(), (0, -n % 32)).reshape(m, -1, 32).amax(
            2, keepdim=True).expand(-1, -1, 32).reshape(m, -1)[:, :n]
        step = (2.0 ** -4 * v.abs()).maximum(2.0 ** -10 * block / 224)
        assert bool(((unpack(q, m, n).double() - v).abs() <= step * 1.001 + 1.1 * e).all())
        tail, _, guard = parts(q, m, n)
        assert not tail.any() and bool((guard == 0xA5).all())
    assert z.zero_matmul_timeouts() == 0


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("rows,cols,stride,offset", [(1, 1, 1, 0), (5, 33, 34, 1), (70, 256, 256, 0),
                                                     (33, 1601, 1608, 8), (300, 520, 523, 3)])
@pytest.mark.parametrize("keep8", [False, True])
def test_gated_gradient(dtype, act, rows, cols, stride, offset, keep8):
    g = gen(rows + act)
    dh, gate, up = (held(randn(g, rows, cols, dtype=dtype, sigma=2), stride, offset)
                    for _ in range(3))
    qs = [None, None]
    gv, uv = gate.t.double(), up.t.double()
    if keep8:
        qs = [packed(rows, cols) for _ in range(2)]
        for q, t in zip(qs, (gate, up)):
            z.zero_pack8(t.t, CODE[dtype], rows, cols, stride, q)
        gv, uv = (unpack(q, rows, cols, dtype).double() for q in qs)
    dg, du, h = (space(rows, cols, dtype, stride, offset) for _ in range(3))
    z.zero_gated_grad(dh.t, stride, None if keep8 else gate.t, None if keep8 else up.t, stride,
                      qs[0], qs[1], act, CODE[dtype], rows, cols, dg.t, du.t, stride, h.t, stride)
    f, slope = F.activation(gv, act)
    ferr, serr = F.value_error(gv, 0 * gv, act), F.slope_error(gv, act)
    d = dh.t.double()
    F.within(dg.t, d * uv * slope, (d * uv).abs() * (serr + 3 * U * slope.abs()))
    F.within(du.t, d * f, d.abs() * (ferr + 2 * U * f.abs()))
    F.within(h.t, f * uv, uv.abs() * (ferr + 2 * U * f.abs()))
    assert dg.untouched() and du.untouched() and h.untouched()


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("rows,cols,stride,offset", [
    (1, 1, 1, 0), (5, 33, 34, 1), (70, 256, 256, 0), (2000, 264, 264, 0), (300, 1601, 1604, 2)])
@pytest.mark.parametrize("keep8", [False, True])
def test_activation_gradient(dtype, act, rows, cols, stride, offset, keep8):
    g = gen(rows + act)
    dy, kept = (held(randn(g, rows, cols, dtype=dtype, sigma=2), stride, offset) for _ in range(2))
    v, q = kept.t.double(), None
    if keep8:
        q = packed(rows, cols)
        z.zero_pack8(kept.t, CODE[dtype], rows, cols, stride, q)
        v = unpack(q, rows, cols, dtype).double()
    slope, serr = F.activation(v, act)[1], F.slope_error(v, act)
    d = dy.t.double()
    want, err = d * slope, d.abs() * (serr + 2 * U * slope.abs())
    db = want.sum(0)
    db_err = err.sum(0) + (rows + 1) * U * (want.abs() + err).sum(0)
    need = z.zero_activation_grad_workspace(rows, cols)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device=DEV)

    def call(dz, bias, accumulate=False):
        z.zero_activation_grad(dy.t, stride, None if keep8 else kept.t, stride, q, act, CODE[dtype],
                               rows, cols, dz.t if dz else None, stride, bias,
                               CODE[bias.dtype] if bias is not None else 0, accumulate, ws, need)
        assert bool((ws[need:] == 0xA5).all())

    dz = space(rows, cols, dtype, stride, offset)
    bias = torch.full((cols,), float("nan"), dtype=dtype, device=DEV)
    call(dz, bias)
    F.within(dz.t, want, err)
    F.within(bias, db, db_err)
    assert dz.untouched()
    acc = torch.full((cols,), 2.0, device=DEV)
    call(None, acc, True)
    F.within(acc, db + 2.0, db_err + U * (db.abs() + db_err + 2.0))
    dz2 = space(rows, cols, dtype, stride, offset)
    call(dz2, None)
    assert torch.equal(dz2.t, dz.t)
    z.zero_activation_grad(dy.t, stride, None if keep8 else kept.t, stride, q, act, CODE[dtype],
                           rows, cols, dy.t, stride, None, 0, False)
    assert torch.equal(dy.t, dz.t) and dy.untouched()


@pytest.mark.parametrize("act", range(1, 5))
def test_activation_slopes_against_differences_and_far_out(act):
    v = torch.tensor([-200.0, -30.0, -8.0, -3.0, -1.0, -0.3, 0.3, 1.0, 3.0, 8.0, 30.0, 200.0],
                     device=DEV)
    one, dz = torch.ones_like(v), torch.empty_like(v)
    z.zero_activation_grad(one, 12, v, 12, None, act, z.ZERO_F32, 1, 12, dz, 12, None, 0, False)
    h = 1e-5
    d = (F.activation(v.double() + h, act)[0] - F.activation(v.double() - h, act)[0]) / (2 * h)
    # the difference: h^2 / 6 times a third derivative below 4, and 1e-16 |y| / h
    assert float((dz.double() - d).abs().max()) < 1e-9 + 4e-9 + 64 * F.ULP
    far = torch.tensor([-3e38, -1e20, 1e20, 3e38], device=DEV)
    dz = torch.empty_like(far)
    z.zero_activation_grad(torch.ones_like(far), 4, far, 4, None, act, z.ZERO_F32, 1, 4, dz, 4,
                           None, 0, False)
    assert dz.tolist() == [0.0, 0.0, 1.0, 1.0]
