"""The training operators on the GPU against their definitions in 64 bits
(tests/ops_ref.py).

The bounds, with u the unit roundoff of the output's type and 2^-24 that of
fp32:
  embed       one fp32 product, one rounding: (u + 2^-24) |y|
  embed_grad  a sum of c terms in any order loses at most c * 2^-24 of the sum
              of their magnitudes, then one product, one addition, one rounding
  dropout     1 / (1 - p) rounded to fp32, one product, one addition, one
              rounding
  quantise    codes and scales equal
  product     k exact products summed in fp32: the tensor cores may cut off
              instead of rounding, so k * 2^-23 of the sum of magnitudes
each with the loss of rounding among subnormal numbers (TINY)."""
import numpy as np
import pytest
import torch

import zero_sharded_optimizer_step_gb300 as z
from tests import ops_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda"
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
CODE = {torch.float32: z.ZERO_F32, torch.bfloat16: z.ZERO_BF16, torch.float16: z.ZERO_F16}
E24 = 2.0 ** -24


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, sigma=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * sigma).to(dtype)


def rows_of(g, rows, cols, stride, dtype, offset=0, sigma=1.0):
    """A [rows, cols] view with that row stride, `offset` elements into its
    buffer."""
    buf = randn(g, rows * stride + offset + 8, dtype=dtype, sigma=sigma)
    return buf[offset:offset + rows * stride].view(rows, stride)[:, :cols]


# ----------------------------------------------------------------- embedding

def embed(table, tokens, scale, pad=-1, out=None, bad=None):
    n, dim = tokens.numel(), table.shape[1]
    if out is None:
        out = torch.empty(n, dim, dtype=table.dtype, device=DEV)
    z.zero_embed(table, CODE[table.dtype], table.shape[0], dim, table.stride(0), tokens,
                 tokens.element_size(), n, pad, scale, out, out.stride(0), bad)
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,rows,dim,stride,offset,tt", [
    (1, 1, 1, 1, 0, torch.int64), (1, 50, 4096, 4096, 0, torch.int32),
    (33, 1000, 768, 768, 0, torch.int64), (300, 77, 257, 260, 3, torch.int32),
    (2000, 300, 130, 130, 2, torch.int64), (70, 5000, 1601, 1601, 0, torch.int64),
    (5, 9, 8, 64, 8, torch.int32), (1500, 100, 1025, 1032, 0, torch.int32)])
def test_embed(dtype, n, rows, dim, stride, offset, tt):
    g = gen(n + dim)
    table = rows_of(g, rows, dim, stride, dtype, offset)
    tokens = torch.randint(0, rows, (n,), generator=g, device=DEV).to(tt)
    pad = int(tokens[0]) if n > 30 else -1
    bad = torch.full((1,), 5, dtype=torch.int64, device=DEV)
    outside = 0
    if n > 30:
        tokens[7], tokens[9], tokens[11] = rows, -3, 2 ** 31 - 1
        outside = 3
    got = R.host(embed(table, tokens, 22.627, pad, bad=bad))
    t = tokens.cpu().numpy().astype(np.int64)
    live = (t != pad) & (t >= 0) & (t < rows)
    want = R.host(table)[np.where(live, t, 0)] * float(np.float32(22.627)) * live[:, None]
    R.within(got, want, (R.ROUND[dtype] + E24) * np.abs(want) + R.TINY[dtype])
    assert (got[~live] == 0).all() and int(bad) == 5 + outside


def test_embed_into_a_strided_output_leaves_the_gaps():
    g = gen(1)
    table = randn(g, 40, 24, dtype=torch.bfloat16)
    tokens = torch.randint(0, 40, (50,), generator=g, device=DEV)
    buf = torch.full((50, 31), 7.0, dtype=torch.bfloat16, device=DEV)
    embed(table, tokens, 1.0, out=buf[:, :24])
    assert torch.equal(buf[:, :24], table[tokens]) and bool((buf[:, 24:] == 7).all())


def test_embed_keeps_infinities_and_nans():
    table = torch.tensor([[1.0, float("inf")], [float("nan"), -2.0]], device=DEV)
    got = embed(table, torch.tensor([1, 0, 7, 1], device=DEV), 2.0)
    want = np.array([[np.nan, -4.0], [2.0, np.inf], [0.0, 0.0], [np.nan, -4.0]])
    R.within(R.host(got), want, 0.0)


def test_embed_beyond_32_bit_offsets():
    """A table of more than 2^31 elements, read at its end."""
    rows, dim = 1_100_000, 2048
    table = torch.zeros(rows, dim, dtype=torch.bfloat16, device=DEV)
    table[-2:] = randn(gen(3), 2, dim, dtype=torch.bfloat16)
    got = embed(table, torch.tensor([rows - 1, 0, rows - 2], device=DEV), 1.0)
    assert torch.equal(got[0], table[-1]) and torch.equal(got[2], table[-2])
    assert not got[1].any()


def embed_grad(dy, tokens, rows, scale=1.0, pad=-1, grad=None, accumulate=False,
               dtype=torch.float32):
    n, dim = dy.shape
    if grad is None:
        grad = torch.full((rows, dim), 77.0, dtype=dtype, device=DEV)
    need = z.zero_embed_grad_workspace(rows, dim, n)
    ws = torch.full((need,), 0xEE, dtype=torch.uint8, device=DEV)
    z.zero_embed_grad(dy, CODE[dy.dtype], dy.stride(0), tokens, tokens.element_size(), n, pad,
                      scale, grad, CODE[grad.dtype], rows, dim, grad.stride(0), accumulate, ws,
                      need)
    return grad


def check_embed_grad(dy, tokens, rows, scale, pad, got, old=None):
    t = tokens.cpu().numpy().astype(np.int64)
    live = (t != pad) & (t >= 0) & (t < rows)
    y = R.host(dy)[live]
    dim = dy.shape[1]
    total, mag = np.zeros((rows, dim)), np.zeros((rows, dim))
    count = np.bincount(t[live], minlength=rows)
    np.add.at(total, t[live], y)
    np.add.at(mag, t[live], np.abs(y))
    s = float(np.float32(scale))
    want, bound = total * s, (count[:, None] + 2) * E24 * mag * s * 1.01
    if old is not None:
        want = want + old
        bound = bound + E24 * (np.abs(want) + np.abs(old))
    u = R.ROUND[got.dtype]
    R.within(R.host(got), want, (1 + u) * bound + (u + E24) * np.abs(want) + R.TINY[got.dtype])
    return count


@pytest.mark.parametrize("ydt,gdt", [(a, b) for a in DTYPES for b in DTYPES])
@pytest.mark.parametrize("n,rows,dim", [(1, 3, 1), (700, 90, 770), (9000, 70_000, 33)])
def test_embed_grad_types(ydt, gdt, n, rows, dim):
    g = gen(n)
    dy = randn(g, n, dim, dtype=ydt)
    tokens = torch.randint(0, rows, (n,), generator=g, device=DEV)
    got = embed_grad(dy, tokens, rows, 1.5, dtype=gdt)
    count = check_embed_grad(dy, tokens, rows, 1.5, -1, got)
    assert not got[torch.from_numpy(count == 0).to(DEV)].any()


@pytest.mark.parametrize("n", [0, 1, 7, 8, 9, 31, 32, 33, 1023, 1025, 8191, 8192, 8193, 8200,
                               12289, 100_001])
@pytest.mark.parametrize("kind", ["zipf", "one", "two", "each"])
def test_embed_grad_lengths_and_runs(n, kind):
    """Runs of one id of every length, up to all tokens; a padding token; ids
    outside the table."""
    rows, dim = 257, 20
    g = gen(n + 5)
    if kind == "zipf":
        t = (torch.exp(torch.rand(n, generator=g, device=DEV) * 5.5).long() * 37) % rows
    elif kind == "one":
        t = torch.full((n,), 200, device=DEV)
    elif kind == "two":
        t = torch.where(torch.rand(n, generator=g, device=DEV) < 0.5, 0, rows - 1)
    else:
        t = torch.arange(n, device=DEV) % rows
    if n > 20:
        t[3], t[5], t[n // 2] = rows, -1, 10 ** 12
    dy = randn(g, n, dim, dtype=torch.bfloat16)
    got = embed_grad(dy, t, rows, 1.0, pad=100)
    check_embed_grad(dy, t, rows, 1.0, 100, got)


@pytest.mark.parametrize("n", [511, 512, 513, 2047, 2048, 2049, 4097])
@pytest.mark.parametrize("rows,dim", [(300, 8), (524_287, 24), (524_288, 33), (900, 1111)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_path_boundaries(n, rows, dim, accumulate):
    """Lengths and table sizes at which another way of sorting takes over."""
    g = gen(n + rows)
    t = (torch.exp(torch.rand(n, generator=g, device=DEV) * 6).long() * 7919) % rows
    t[::9] = torch.randint(0, rows, (len(t[::9]),), generator=g, device=DEV)
    t[1], t[n - 2] = -7, rows
    dy = randn(g, n, dim, dtype=torch.float16)
    grad = randn(g, rows, dim) if accumulate else None
    old = R.host(grad) if accumulate else None
    got = embed_grad(dy, t, rows, 0.25, grad=grad, accumulate=accumulate)
    check_embed_grad(dy, t, rows, 0.25, -1, got, old)


@pytest.mark.parametrize("rows", [1, 255, 256, 65_535, 65_536, 16_777_217])
@pytest.mark.parametrize("n", [100, 10_000])
def test_embed_grad_digit_counts(rows, n):
    """Row counts around the sort's digit boundaries (1 to 4 passes)."""
    g = gen(rows % 1000)
    t = torch.randint(max(0, rows - 2000), rows, (n,), generator=g, device=DEV)
    t[::7] = torch.randint(0, rows, (len(t[::7]),), generator=g, device=DEV)
    dy = randn(g, n, 4)
    got = embed_grad(dy, t, rows)
    check_embed_grad(dy, t, rows, 1.0, -1, got)


@pytest.mark.parametrize("n", [50, 9001])
@pytest.mark.parametrize("gdt", DTYPES)
def test_embed_grad_accumulates_into_named_rows_only(n, gdt):
    rows, dim = 3000, 100
    g = gen(n)
    buf = randn(g, rows, 113, dtype=gdt)
    grad = buf[:, 5:105]
    before = buf.clone()
    t = torch.randint(0, rows // 2, (n,), generator=g, device=DEV).int()
    dy = rows_of(g, n, dim, 101, torch.float16, 1)
    embed_grad(dy, t, rows, 0.5, grad=grad, accumulate=True)
    check_embed_grad(dy, t, rows, 0.5, -1, grad, R.host(before[:, 5:105]))
    touched = torch.zeros(rows, dtype=torch.bool, device=DEV)
    touched[t.long()] = True
    assert torch.equal(buf[~touched], before[~touched])
    assert torch.equal(buf[:, :5], before[:, :5]) and torch.equal(buf[:, 105:], before[:, 105:])


@pytest.mark.parametrize("n", [6000, 60_000])
def test_embed_grad_is_the_same_on_every_run(n):
    g = gen(n)
    t = (torch.exp(torch.rand(n, generator=g, device=DEV) * 9).long() * 31) % 5000
    dy = randn(g, n, 300, dtype=torch.bfloat16)
    first = embed_grad(dy, t, 5000)
    for _ in range(5):
        assert torch.equal(embed_grad(dy, t, 5000), first)


@pytest.mark.parametrize("n", [40, 8500])
def test_embed_grad_with_nothing_but_padding(n):
    t = torch.full((n,), 3, device=DEV)
    dy = torch.full((n, 16), float("nan"), device=DEV)
    assert not embed_grad(dy, t, 50, pad=3).any()
    keep = torch.full((50, 16), 2.0, device=DEV)
    assert bool((embed_grad(dy, t, 50, pad=3, grad=keep, accumulate=True) == 2.0).all())


def test_embed_grad_against_differences():
    """L = sum(w * embed(table)) is linear in the table: its central difference
    is the gradient, exactly where every sum is of small whole numbers."""
    g = gen(9)
    rows, dim, n = 30, 5, 200
    table = torch.randint(-8, 9, (rows, dim), generator=g, device=DEV).float()
    w = torch.randint(-8, 9, (n, dim), generator=g, device=DEV).float()
    t = torch.randint(0, rows, (n,), generator=g, device=DEV)
    got = embed_grad(w, t, rows, 2.0, pad=4)

    def loss(tb):
        return float((w * embed(tb, t, 2.0, pad=4)).double().sum())

    for r, c in [(0, 0), (4, 2), (17, 4), (29, 1)]:
        up, down = table.clone(), table.clone()
        up[r, c] += 1
        down[r, c] -= 1
        assert (loss(up) - loss(down)) / 2 == float(got[r, c])


# ------------------------------------------------------------------- dropout

def dropout(x, p, seed, offset, residual=None, first=0, out=None):
    out = torch.empty_like(x) if out is None else out
    z.zero_dropout(x, residual, out, CODE[x.dtype], x.numel(), p, seed, offset, first)
    return out


def check_dropout(x, p, seed, offset, residual, first, got):
    n = x.numel()
    kept = R.keep(n, p, seed, offset, first)
    up = 1.0 / (1.0 - p) if p < 1 else 0.0
    with np.errstate(invalid="ignore"):
        y = np.where(kept, R.host(x) * up, 0.0)
    want = y + (R.host(residual) if residual is not None else 0.0)
    u = R.ROUND[x.dtype]
    bound = (1 + u) * (2 * E24 * np.abs(y) + E24 * np.abs(want)) * 1.01 + u * np.abs(want)
    R.within(R.host(got), want, np.nan_to_num(bound) + R.TINY[x.dtype])
    return kept


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [0, 1, 3, 4, 5, 8, 9, 1000, 4097, 1_000_003])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
@pytest.mark.parametrize("with_residual", [False, True])
def test_dropout(dtype, n, p, with_residual):
    g = gen(n)
    x = randn(g, n, dtype=dtype)
    r = randn(g, n, dtype=dtype) if with_residual else None
    seed, offset = 0xFEDCBA9876543210, 0x1234567890ABCDEF
    got = dropout(x, p, seed, offset, r)
    kept = check_dropout(x, p, seed, offset, r, 0, got)
    if n > 100_000:      # within 6 standard deviations of n (1 - p)
        assert abs(kept.sum() - n * (1 - p)) <= 6 * np.sqrt(n * p * (1 - p))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ox,orr,oo", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (3, 5, 7), (8, 8, 8)])
def test_dropout_of_unaligned_buffers(dtype, ox, orr, oo):
    g, n = gen(3), 5003
    x, r, o = (randn(g, n + 8, dtype=dtype)[k:k + n] for k in (ox, orr, oo))
    check_dropout(x, 0.3, 5, 6, r, 0, dropout(x, 0.3, 5, 6, r, out=o))


def test_dropout_in_place_and_in_pieces():
    g, n = gen(4), 100_000
    x, r = randn(g, n, dtype=torch.bfloat16), randn(g, n, dtype=torch.bfloat16)
    whole = dropout(x, 0.25, 1, 2, r)
    pieces = torch.empty_like(x)
    for lo, hi in [(0, 4), (4, 1000), (1000, 50_004), (50_004, n)]:
        dropout(x[lo:hi], 0.25, 1, 2, r[lo:hi], first=lo, out=pieces[lo:hi])
    assert torch.equal(pieces, whole)
    a, b = x.clone(), r.clone()
    assert torch.equal(dropout(a, 0.25, 1, 2, r, out=a), whole)
    assert torch.equal(dropout(x, 0.25, 1, 2, b, out=b), whole)


@pytest.mark.parametrize("first", [2 ** 32 * 4 - 16, 2 ** 40, 2 ** 62])
def test_dropout_counters_past_32_bits(first):
    x = torch.ones(64, device=DEV)
    check_dropout(x, 0.5, 77, 3, None, first, dropout(x, 0.5, 77, 3, first=first))


def test_dropout_drops_infinities_and_nans():
    x = torch.full((4000,), float("nan"), device=DEV)
    x[::2] = float("inf")
    got = dropout(x, 0.5, 9, 9)
    kept = torch.from_numpy(R.keep(4000, 0.5, 9, 9)).to(DEV)
    assert not got[~kept].any() and not torch.isfinite(got[kept]).any()


def test_dropout_gradient_is_the_same_map():
    """Against the formula and, with p = 1/2 and whole numbers (so that every
    value is exact), against central differences."""
    g, n = gen(6), 600
    x = torch.randint(-50, 51, (n,), generator=g, device=DEV).float()
    dy = torch.randint(-50, 51, (n,), generator=g, device=DEV).float()
    dx = dropout(dy, 0.5, 11, 12)
    kept = torch.from_numpy(R.keep(n, 0.5, 11, 12)).to(DEV)
    assert torch.equal(dx, dy * kept * 2)
    for e in (0, 5, 300, 599):
        up, down = x.clone(), x.clone()
        up[e] += 1
        down[e] -= 1
        d = [(dropout(v, 0.5, 11, 12) * dy).double().sum() for v in (up, down)]
        assert float(d[0] - d[1]) / 2 == float(dx[e])


# -------------------------------------------------------------- 4-bit numbers

def room(rows, cols, fill=0xFF):
    """A buffer for a quantised matrix, filled with NaN scales."""
    return torch.full((z.zero_mx4_bytes(rows, cols),), fill, dtype=torch.uint8, device=DEV)


def quantize(x, q=True, qt=False):
    rows, cols = x.shape
    a = room(rows, cols) if q else None
    b = room(cols, rows) if qt else None
    z.zero_mx4_quantize(x, CODE[x.dtype], rows, cols, x.stride(0), a, b)
    return a, b


def check_records(q, x64):
    """Codes and scales equal, zeros in the columns that fill the records."""
    rows, cols = x64.shape
    codes, scales = R.unpack(q.cpu().numpy(), rows, cols)
    want, wscales = R.quantize(x64)
    nb = wscales.shape[1]
    assert np.array_equal(scales[:, :nb], wscales) and not scales[:, nb:].any()
    fine = np.repeat(wscales != 255, 32, 1)[:, :cols]      # a NaN block's codes mean nothing
    assert np.array_equal(np.where(fine, codes[:, :cols], 0), np.where(fine, want, 0))
    assert not codes[:, 32 * nb:].any()
    assert not (codes[:, cols:32 * nb] & 7).any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,stride,offset", [
    (1, 1, 1, 0), (1, 4096, 4096, 0), (3, 33, 33, 0), (128, 256, 256, 0), (129, 257, 260, 1),
    (300, 514, 514, 2), (77, 1600, 1608, 8), (257, 40, 40, 0)])
@pytest.mark.parametrize("which", ["rows", "columns", "both"])
def test_quantize(dtype, rows, cols, stride, offset, which):
    g = gen(rows + cols)
    x = rows_of(g, rows, cols, stride, dtype, offset)
    x[:, ::5] *= 0.01
    q, qt = quantize(x, which != "columns", which != "rows")
    if q is not None:
        check_records(q, R.host(x))
    if qt is not None:
        check_records(qt, R.host(x).T)


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_extremes(dtype):
    """Every tie and power of two of the type's range, zeros of both signs,
    subnormals, the largest finite value, infinities and NaN."""
    f = torch.finfo(dtype)
    ties = torch.tensor([.25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.9],
                        device=DEV)
    lines = []
    for e in range(-150, 128, 3):
        lines.append(torch.cat([ties, -ties]).double() * 2.0 ** e)
    x = torch.stack(lines).clamp(-f.max, f.max).to(dtype)
    x = torch.cat([x, torch.zeros(1, 32, device=DEV, dtype=dtype),
                   -torch.zeros(1, 32, device=DEV, dtype=dtype),
                   torch.full((1, 32), f.max, device=DEV, dtype=dtype),
                   torch.full((1, 32), f.smallest_normal / 4, device=DEV, dtype=dtype),
                   torch.ones(3, 32, device=DEV, dtype=dtype)])
    x[-3, 4], x[-2, 31], x[-1, 0] = float("inf"), float("nan"), float("-inf")
    q, qt = quantize(x, True, True)
    check_records(q, R.host(x))
    check_records(qt, R.host(x).T)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,stride,offset", [(1, 1, 1, 0), (200, 300, 303, 1),
                                                     (130, 512, 512, 0), (5, 1030, 1032, 2)])
def test_dequantize(dtype, rows, cols, stride, offset):
    g = gen(rows)
    x = randn(g, rows, cols)
    q, _ = quantize(x)
    out = rows_of(g, rows, cols, stride, dtype, offset)
    base = out.as_strided((rows * stride,), (1,), offset)
    gaps = base.clone().view(rows, stride)[:, cols:]
    z.zero_mx4_dequantize(q, rows, cols, out, CODE[dtype], stride)
    want = R.values(*R.quantize(R.host(x)))
    R.within(R.host(out), want, R.ROUND[dtype] * np.abs(want) + R.TINY[dtype])
    assert torch.equal(base.view(rows, stride)[:, cols:], gaps)


def test_dequantize_gives_nan_for_a_nan_block():
    x = torch.ones(2, 64, device=DEV)
    x[1, 40] = float("inf")
    q, _ = quantize(x)
    out = torch.empty(2, 64, device=DEV)
    z.zero_mx4_dequantize(q, 2, 64, out, z.ZERO_F32, 64)
    assert torch.isnan(out[1, 32:]).all() and bool((out[:, :32] == 1).all())
    assert bool((out[0] == 1).all())


# ----------------------------------------------------------------- the product

def matmul(a, m, b, n, k, out, alpha=1.0, accumulate=False):
    z.zero_mx4_matmul(a, m, b, n, k, alpha, accumulate, out, CODE[out.dtype], out.stride(0))
    return out


def check_product(av, bv, alpha, got, old=None):
    """av [m, k] and bv [n, k]: the quantised operands' values (float64)."""
    want = av @ bv.T * alpha
    mag = np.abs(av) @ np.abs(bv).T * abs(alpha)
    k = av.shape[1]
    bound = (k + 2) * 2.0 ** -23 * mag
    if old is not None:
        want = want + old
        bound = bound + E24 * np.abs(old)
    u = R.ROUND[got.dtype]
    R.within(R.host(got), want, (1 + u) * bound + (u + E24) * np.abs(want) + R.TINY[got.dtype])


def operands(seed, m, n, k):
    g = gen(seed)
    x, w = randn(g, m, k), randn(g, n, k)
    (a, _), (b, _) = quantize(x), quantize(w)
    return a, b, R.values(*R.quantize(R.host(x))), R.values(*R.quantize(R.host(w)))


SIZES = [(1, 1, 1), (1, 127, 64), (2, 129, 257), (16, 128, 256), (17, 300, 1600), (33, 1000, 96),
         (64, 128, 5000), (65, 200, 2048), (100, 64, 31), (128, 384, 1024), (129, 130, 300),
         (255, 257, 512), (256, 128, 65), (257, 640, 1000), (513, 129, 4096), (1000, 1000, 999),
         (1, 11008, 4096), (700, 4100, 260)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_matmul(m, n, k, dtype):
    a, b, av, bv = operands(m + n + k, m, n, k)
    buf = torch.full((m, n + 3), 9.0, dtype=dtype, device=DEV)
    got = matmul(a, m, b, n, k, buf[:, :n])
    check_product(av, bv, 1.0, got)
    assert bool((buf[:, n:] == 9.0).all())
    assert z.zero_mx4_timeouts() == 0


@pytest.mark.parametrize("m,n,k", [(3, 200, 700), (40, 300, 3000), (300, 500, 800)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_matmul_adds_to_its_output(m, n, k, dtype):
    a, b, av, bv = operands(7, m, n, k)
    out = randn(gen(1), m, n, dtype=dtype, sigma=30.0)
    old = R.host(out)
    matmul(a, m, b, n, k, out, alpha=-0.75, accumulate=True)
    check_product(av, bv, -0.75, out, old)


def test_matmul_of_nothing():
    a, b = room(300, 0), room(200, 0)
    out = torch.full((300, 200), 4.0, device=DEV)
    matmul(a, 300, b, 200, 0, out, accumulate=True)
    assert bool((out == 4.0).all())
    matmul(a, 300, b, 200, 0, out)
    assert not out.any()
    matmul(None, 0, b, 200, 0, out[:0])
    matmul(a, 300, None, 0, 0, out[:, :0])


@pytest.mark.parametrize("m", [5, 60, 300])
def test_matmul_keeps_nan_to_its_row_and_column(m):
    n, k = 260, 600
    g = gen(2)
    x, w = randn(g, m, k), randn(g, n, k)
    x[3, 500], w[200, 10] = float("inf"), float("nan")
    (a, _), (b, _) = quantize(x), quantize(w)
    got = matmul(a, m, b, n, k, torch.empty(m, n, device=DEV))
    want = torch.zeros(m, n, dtype=torch.bool, device=DEV)
    want[3], want[:, 200] = True, True
    assert torch.equal(torch.isnan(got), want)


def test_matmul_wide_scales():
    """Blocks whose scales lie far apart: exact where one block stands out."""
    m, n, k = 20, 140, 512
    g = gen(8)
    x = torch.zeros(m, k, device=DEV)
    w = torch.zeros(n, k, device=DEV)
    for blk in range(k // 32):
        x[:, blk * 32] = 2.0 ** (blk - 40)
        w[blk % n, blk * 32] = 1.5 * 2.0 ** (30 - 3 * blk)
    (a, _), (b, _) = quantize(x), quantize(w)
    got = matmul(a, m, b, n, k, torch.empty(m, n, device=DEV))
    want = R.host(x) @ R.host(w).T
    R.within(R.host(got), want, 0.0)


def test_linear_layer_gradients():
    """dx and dW of y = Q(x) Q(W)^T by the three products, against the
    formulas on the values that the quantisation gives."""
    g = gen(5)
    m, n, k = 150, 300, 200
    x, w = randn(g, m, k, dtype=torch.bfloat16), randn(g, n, k, dtype=torch.bfloat16)
    dy = randn(g, m, n, dtype=torch.bfloat16)
    (xq, xt), (wq, wt), (dq, dt) = (quantize(v, True, True) for v in (x, w, dy))
    y = matmul(xq, m, wq, n, k, torch.empty(m, n, device=DEV))
    dx = matmul(dq, m, wt, k, n, torch.empty(m, k, device=DEV))
    dw = matmul(dt, n, xt, k, m, torch.empty(n, k, device=DEV))
    val = [R.values(*R.quantize(v)) for v in (R.host(x), R.host(w), R.host(dy))]
    valt = [R.values(*R.quantize(v.T)) for v in (R.host(x), R.host(w), R.host(dy))]
    check_product(val[0], val[1], 1.0, y)
    check_product(val[2], valt[1], 1.0, dx)
    check_product(valt[2], valt[0], 1.0, dw)


def test_linear_layer_gradients_against_differences():
    """Operands that 4 bits hold exactly: y is then linear in each of them, and
    the central differences of L = sum(dy * y) are whole multiples of 1/4 that
    every sum here holds exactly."""
    g = gen(10)
    m, n, k = 40, 70, 50
    grid = torch.tensor([-2, -1.5, -1, -.5, .5, 1, 1.5, 2], device=DEV)

    def draw(*shape):
        t = grid[torch.randint(0, 8, shape, generator=g, device=DEV)]
        return t

    x, w, dy = draw(m, k), draw(n, k), draw(m, n)
    # 4 in every block makes its scale 1 whichever element changes
    x[:, 0], x[:, 32], w[:, 0], w[:, 32] = 4, 4, 4, 4
    x[0], x[32], w[0], w[32], w[64], dy[0], dy[32] = 4, 4, 4, 4, 4, 4, 4
    dy[:, 0], dy[:, 32], dy[:, 64] = 4, 4, 4
    (_, xt), (_, wt), (dq, dt) = (quantize(v, True, True) for v in (x, w, dy))
    dx = matmul(dq, m, wt, k, n, torch.empty(m, k, device=DEV))
    dw = matmul(dt, n, xt, k, m, torch.empty(n, k, device=DEV))

    def loss(xx, ww):
        y = matmul(quantize(xx)[0], m, quantize(ww)[0], n, k, torch.empty(m, n, device=DEV))
        return float((y.double() * dy).sum())

    for i, c in [(1, 1), (20, 40), (39, 49)]:
        up, down = x.clone(), x.clone()
        up[i, c], down[i, c] = 1.5, 0.5
        assert loss(up, w) - loss(down, w) == float(dx[i, c])
        up, down = w.clone(), w.clone()
        up[i + 5, c], down[i + 5, c] = 1.5, 0.5
        assert loss(x, up) - loss(x, down) == float(dw[i + 5, c])


# ------------------------------------------------- more than 2^31 (2^32) elements

def test_embed_grad_of_a_long_list():
    """dy of more than 2^31 elements: rows that one token each names hold that
    token's row, the last of them among them; one frequent row, of whole numbers,
    the exact sum."""
    n, dim, rows = 1_100_000, 2048, 3000
    dy = torch.ones(n, dim, dtype=torch.bfloat16, device=DEV)
    t = torch.full((n,), 7, dtype=torch.int32, device=DEV)
    single = torch.tensor([0, 1, 65_536, n // 2, n - 2, n - 1], device=DEV)
    t[single] = torch.arange(100, 106, device=DEV, dtype=torch.int32)
    dy[single] = randn(gen(1), 6, dim, dtype=torch.bfloat16)
    got = embed_grad(dy, t, rows)
    assert torch.equal(got[100:106], dy[single].float())
    assert bool((got[7] == n - 6).all())               # below 2^24: exact in any order
    got[7], got[100:106] = 0, 0
    assert not got.any()


def test_embed_grad_into_a_large_table():
    rows, dim = 1_100_000, 2048
    grad = torch.zeros(rows, dim, dtype=torch.bfloat16, device=DEV)
    t = torch.tensor([rows - 1, 5, rows - 2, 5], device=DEV)
    dy = torch.ones(4, dim, dtype=torch.bfloat16, device=DEV)
    embed_grad(dy, t, rows, grad=grad, accumulate=True)
    assert bool((grad[-2:] == 1).all()) and bool((grad[5] == 2).all())
    assert not grad[6:-2].any()
    grad.fill_(3)
    embed_grad(dy, t, rows, grad=grad)
    assert bool((grad[-2:] == 1).all()) and bool((grad[5] == 2).all())
    assert not grad[6:-2].any() and not grad[:5].any()


def test_dropout_of_more_than_2_to_32_elements():
    n = 2 ** 32 + 24
    x = torch.ones(n, dtype=torch.float16, device=DEV)
    dropout(x, 0.5, 3, 4, out=x)
    for lo in (0, 2 ** 31 - 8, 2 ** 32 - 8, n - 24):
        m = min(64, n - lo)
        kept = R.keep(m, 0.5, 3, 4, lo)
        assert np.array_equal(R.host(x[lo:lo + m]), kept * 2.0)


def test_quantize_of_more_than_2_to_31_elements():
    rows, cols = 70_000, 32_768
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[-300:, -600:] = randn(gen(2), 300, 600, dtype=torch.bfloat16)
    q, qt = quantize(x, True, True)
    out = torch.empty_like(x)
    z.zero_mx4_dequantize(q, rows, cols, out, z.ZERO_BF16, cols)
    part = R.host(x[-304:, -608:])                      # whole blocks of 32 columns
    assert np.array_equal(R.host(out[-304:, -608:]), R.values(*R.quantize(part)))
    assert not out[:-300].any()
    back = torch.empty(cols, rows, dtype=torch.bfloat16, device=DEV)
    z.zero_mx4_dequantize(qt, cols, rows, back, z.ZERO_BF16, rows)
    part = R.host(x[69_664:, -608:]).T                  # 69,664 is a multiple of 32
    assert np.array_equal(R.host(back[-608:, 69_664:]), R.values(*R.quantize(part)))
    assert not back[:-600].any()


@pytest.mark.parametrize("n,stride", [(46_400, 46_400), (46_401, 46_401)])
def test_matmul_into_more_than_2_to_31_elements(n, stride):
    m, k = 46_500, 64
    g = gen(3)
    x, w = randn(g, m, k), randn(g, n, k)
    (a, _), (b, _) = quantize(x), quantize(w)
    out = torch.full((m, stride), 5.0, dtype=torch.bfloat16, device=DEV)
    matmul(a, m, b, n, k, out)
    av, bv = R.values(*R.quantize(R.host(x))), R.values(*R.quantize(R.host(w)))
    for rows in (slice(0, 3), slice(m // 2, m // 2 + 3), slice(m - 3, m)):
        check_product(av[rows], bv, 1.0, out[rows])


# ------------------------------------------------------------ streams, graphs

def _all_operators(state):
    """Every operator once, on the current stream, into state's buffers."""
    s = state
    st = torch.cuda.current_stream()
    n, dim, rows, cols = s["n"], s["dim"], s["rows"], s["cols"]
    bf = z.ZERO_BF16
    z.zero_embed(s["table"], bf, rows, dim, dim, s["tokens"], 8, n, -1, 2.0, s["e"], dim, None, st)
    z.zero_dropout(s["e"], None, s["d"], bf, n * dim, 0.25, 3, 4, 0, st)
    z.zero_mx4_quantize(s["d"], bf, n, dim, dim, s["q"], s["qt"], st)
    z.zero_mx4_quantize(s["w"], bf, cols, dim, dim, s["wq"], None, st)
    z.zero_mx4_matmul(s["q"], n, s["wq"], cols, dim, 1.0, False, s["y"], bf, cols, st)
    z.zero_mx4_dequantize(s["q"], n, dim, s["v"], bf, dim, st)
    z.zero_embed_grad(s["v"], bf, dim, s["tokens"], 8, n, -1, 2.0, s["g"], bf, rows, dim, dim,
                      False, s["ws"], s["ws"].numel(), st)


def _operator_state(n):
    g = gen(n)
    dim, rows, cols = 136, 500, 333
    e = dict(dtype=torch.bfloat16, device=DEV)
    return dict(n=n, dim=dim, rows=rows, cols=cols, table=randn(g, rows, dim, dtype=e["dtype"]),
                tokens=torch.randint(0, rows, (n,), generator=g, device=DEV),
                w=randn(g, cols, dim, dtype=e["dtype"]), e=torch.empty(n, dim, **e),
                d=torch.empty(n, dim, **e), q=room(n, dim), qt=room(dim, n), wq=room(cols, dim),
                y=torch.empty(n, cols, **e), v=torch.empty(n, dim, **e),
                g=torch.empty(rows, dim, **e),
                ws=torch.empty(z.zero_embed_grad_workspace(rows, dim, n), dtype=torch.uint8,
                               device=DEV))


@pytest.mark.parametrize("n", [5, 400, 9000])
def test_operators_on_another_stream_and_in_a_graph(n):
    s = _operator_state(n)
    _all_operators(s)
    torch.cuda.synchronize()
    outs = ("e", "d", "y", "v", "g")
    want = {k: s[k].clone() for k in outs}
    side = torch.cuda.Stream()
    for k in outs:
        s[k].fill_(3.0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _all_operators(s)
        _all_operators(s)
    side.synchronize()
    for k in outs:
        assert torch.equal(s[k], want[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _all_operators(s)
    for k in outs:
        s[k].fill_(3.0)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for k in outs:
        assert torch.equal(s[k], want[k]), k
