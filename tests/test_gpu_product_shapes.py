"""16-bit products and gated blocks at the sizes where their kernels change course:
sums split over blocks, tiles in parts and narrower ones, one row, more than 2^31
elements, and calls whose first time is inside a captured graph."""
import pytest
import torch

import tests.ff_ref as F
from tests.test_gpu_feed_forward import (DEV, U, as_lies, gated, gen, held, packed, parts,
                                         product, randn, space, unpack)

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import zero_sharded_optimizer_step_gb300 as z

BF = torch.bfloat16


def eight_bits(q, m, n, v, err):
    """q holds v, known to err, to half a step of its own or of the block's smallest."""
    block = torch.nn.functional.pad(v.abs(), (0, -n % 32)).reshape(m, -1, 32).amax(
        2, keepdim=True).expand(-1, -1, 32).reshape(m, -1)[:, :n]
    step = (2.0 ** -4 * v.abs()).maximum(2.0 ** -10 * block / 224)
    assert bool(((unpack(q, m, n).double() - v).abs() <= step * 1.001 + 1.1 * err).all())
    tail, _, guard = parts(q, m, n)
    assert not tail.any() and bool((guard == 0xA5).all())


# one row; split sums of few, of some rows; whole blocks of several tiles of rows
SPLITS = [(1, 300, 1500), (2, 300, 1500), (9, 129, 2100), (16, 1000, 4000), (40, 300, 1500),
          (64, 130, 5000), (65, 260, 2000), (130, 260, 2000), (300, 515, 1111), (140, 1000, 900)]


@pytest.mark.parametrize("m,n,k", SPLITS)
@pytest.mark.parametrize("pad,offset", [(0, 0), (16, 16), (1, 1)])
def test_split_sums_with_everything(m, n, k, pad, offset):
    g = gen(m + n)
    a, b = randn(g, m, k, dtype=BF), randn(g, n, k, dtype=BF, sigma=k ** -0.5 * 2)
    bias, r = randn(g, n, dtype=BF), randn(g, m, n, dtype=BF)
    zz, err = F.product(a.double(), b.double())
    zz = zz + bias.double()
    err = err + U * (zz.abs() + err)
    y, yerr = F.activation(zz, F.GELU)[0], F.value_error(zz, err, F.GELU)
    want = y + r.double()
    for dtype in (BF, torch.float32):
        out, kept = space(m, n, dtype, n + pad, offset), space(m, n, BF, n + pad, offset)
        res = held(r.to(dtype), n + pad, offset)
        product(held(a), False, held(b), False, out, bias=bias, act=F.GELU, residual=res,
                kept=kept)
        F.within(out.t, want, yerr + U * (want.abs() + yerr))
        F.within(kept.t, zz, err)
        assert out.untouched() and kept.untouched()
        q, again = packed(m, n), space(m, n, dtype, n + pad, offset)
        product(held(a), False, held(b), False, again, bias=bias, act=F.GELU, residual=res,
                kept_q=q)
        assert torch.equal(again.t, out.t)
        eight_bits(q, m, n, zz, err)
        product(held(a), False, held(b), False, res, bias=bias, act=F.GELU, accumulate=True)
        assert torch.equal(res.t, out.t)
    assert z.zero_matmul_timeouts() == 0


@pytest.mark.parametrize("m,n,k", SPLITS)
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 1)])
def test_split_gated(m, n, k, pad, offset):
    g = gen(m + k)
    x = randn(g, m, k, dtype=BF)
    wg, wu = (randn(g, n, k, dtype=BF, sigma=k ** -0.5) for _ in range(2))
    gate, gerr = F.product(x.double(), wg.double())
    up, uerr = F.product(x.double(), wu.double())
    f, ferr = F.activation(gate, F.SILU)[0], F.value_error(gate, gerr, F.SILU)
    want = f * up
    err = ferr * up.abs() + f.abs() * uerr + ferr * uerr + 2 * U * want.abs()
    h, kg, ku = (space(m, n, BF, n + pad, offset) for _ in range(3))
    gated(held(x, k + pad, offset), held(wg), held(wu, k + pad, offset), h, F.SILU, kg, ku)
    F.within(h.t, want, err)
    F.within(kg.t, gate, gerr)
    F.within(ku.t, up, uerr)
    assert h.untouched() and kg.untouched() and ku.untouched()
    qg, qu, again = packed(m, n), packed(m, n), space(m, n, BF, n + pad, offset)
    gated(held(x), held(wg), held(wu), again, F.SILU, None, None, qg, qu)
    F.within(again.t, want, err)
    eight_bits(qg, m, n, gate, gerr)
    eight_bits(qu, m, n, up, uerr)


@pytest.mark.parametrize("a_cols,b_cols", [(False, False), (False, True), (True, True)])
@pytest.mark.parametrize("m,n,k", [
    (2560, 2048, 72),        # 80 tiles of 256 x 256: the last four in quarters
    (2560, 2008, 40),        # the same, the last tile of a row narrower
    (2816, 2048, 24),        # 88: the last twelve in quarters
    (4096, 1800, 136),       # 16 x 8: the last 52 whole
    (6400, 1600, 32),        # 25 x 7 of 256, narrower tiles
    (6400, 1601, 40), (5000, 1100, 72)])
def test_tiles_in_parts(a_cols, b_cols, m, n, k):
    g = gen(m + n)
    a, b = randn(g, m, k, dtype=torch.float16), randn(g, n, k, dtype=torch.float16)
    want, err = F.product(a.double(), b.double())
    for pad in (0, 3):
        out = space(m, n, torch.float16, n + pad)
        product(as_lies(a, a_cols), a_cols, as_lies(b, b_cols), b_cols, out)
        F.within(out.t, want, err)
        assert out.untouched()


# tiles of 192, 160, 176 and 240 rows of A, split over blocks, and what splits too little
# once the rows of the result need a place to be turned in
WIDE = [(384, 4096, 2112), (300, 4000, 2112), (333, 1600, 6400), (230, 6397, 1800)]


@pytest.mark.parametrize("m,n,k", WIDE)
@pytest.mark.parametrize("pad,offset", [(0, 0), (16, 16), (1, 1)])
def test_wide_tiles_with_everything(m, n, k, pad, offset):
    test_split_sums_with_everything(m, n, k, pad, offset)


@pytest.mark.parametrize("m,n,k", [(384, 4096, 1090), (333, 1600, 3208)])
def test_wide_tiles_of_two_pairs(m, n, k):
    g = gen(m)
    a, a2 = (randn(g, m, k, dtype=BF) for _ in range(2))
    b, b2 = (randn(g, n, k, dtype=BF) for _ in range(2))
    want, err = F.product(torch.cat([a, a2], 1).double(), torch.cat([b, b2], 1).double())
    for b_cols in (False, True):
        for pad in (0, 1):
            out = space(m, n, BF)
            product(as_lies(a, False, pad), False, as_lies(b, b_cols), b_cols, out,
                    as_lies(a2, False), as_lies(b2, b_cols, pad))
            F.within(out.t, want, err)
            assert out.untouched()


@pytest.mark.parametrize("m,n,k", [(2, 9801, 72), (77, 9900, 136), (128, 16001, 72),
                                   (300, 4096, 200), (130, 6000, 500)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (16, 16), (1, 1)])
def test_gated_in_one_tile_a_sm(m, n, k, pad, offset):
    test_split_gated(m, n, k, pad, offset)


@pytest.mark.parametrize("m,n,k", [(2560, 1024, 72), (2560, 1000, 40), (6400, 800, 32),
                                   (6400, 801, 40), (5000, 600, 72)])
def test_gated_tiles_in_parts(m, n, k):
    g = gen(m + n)
    x = randn(g, m, k, dtype=BF)
    wg, wu = (randn(g, n, k, dtype=BF, sigma=k ** -0.5) for _ in range(2))
    gate, gerr = F.product(x.double(), wg.double())
    up, uerr = F.product(x.double(), wu.double())
    f, ferr = F.activation(gate, F.SILU)[0], F.value_error(gate, gerr, F.SILU)
    want = f * up
    err = ferr * up.abs() + f.abs() * uerr + ferr * uerr + 2 * U * want.abs()
    qg, qu, h = packed(m, n), packed(m, n), space(m, n, BF)
    gated(held(x), held(wg), held(wu), h, F.SILU, None, None, qg, qu)
    F.within(h.t, want, err)
    assert h.untouched()
    eight_bits(qg, m, n, gate, gerr)
    eight_bits(qu, m, n, up, uerr)


def captured(call):
    """call() in a captured graph, replayed once."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    graph.replay()
    torch.cuda.synchronize()


@pytest.mark.parametrize("m,n,k", [(1, 640, 704), (24, 384, 3008), (144, 400, 2112),
                                   (200, 72, 136), (2570, 2056, 56)])
def test_a_shape_that_is_first_met_in_a_captured_graph(m, n, k):
    """Nothing that a first call sets up disturbs the capture."""
    g = gen(k)
    a, b = held(randn(g, m, k, dtype=BF)), held(randn(g, n, k, dtype=BF))
    out = space(m, n, BF)
    captured(lambda: z.zero_matmul(a.t, False, k, b.t, False, k, None, 0, None, 0, z.ZERO_BF16, m,
                                   n, k, None, 0, None, 0, None, 0, None, out.t, z.ZERO_BF16, n,
                                   False))
    F.within(out.t, *F.product(a.t.double(), b.t.double()))


def test_results_of_more_than_2_to_31_elements():
    """Rows far beyond 32-bit offsets, in every kernel that writes such a matrix."""
    m, n, k = 70_000, 32_768, 64
    g = gen(1)
    a, b = randn(g, m, k, dtype=BF), randn(g, n, k, dtype=BF, sigma=k ** -0.5)
    rows = torch.cat([torch.arange(4, device=DEV), torch.arange(65_530, 65_540, device=DEV),
                      torch.arange(m - 4, m, device=DEV)])
    zz, err = F.product(a[rows].double(), b.double())
    out = torch.empty(m, n, dtype=BF, device=DEV)
    q = torch.empty(z.zero_pack8_bytes(m, n), dtype=torch.uint8, device=DEV)
    z.zero_matmul(a, False, k, b, False, k, None, 0, None, 0, z.ZERO_BF16, m, n, k, None, 0, None,
                  0, None, 0, q, out, z.ZERO_BF16, n, False)
    F.within(out[rows], zz, err)
    v = torch.empty(m, n, dtype=BF, device=DEV)
    z.zero_unpack8(q, m, n, v, z.ZERO_BF16, n)
    assert float((v[rows].double() - zz).abs().max()) <= 2.0 ** -4 * float(zz.abs().max()) * 1.01
    del q
    # its gradient through an activation, with the bias's, and through the norm
    dz, db = torch.empty_like(out), torch.empty(n, device=DEV)
    need = z.zero_activation_grad_workspace(m, n)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    z.zero_activation_grad(v, n, out, n, None, F.RELU, z.ZERO_BF16, m, n, dz, n, db, z.ZERO_F32,
                           False, ws, need)
    want = torch.where(out[rows] > 0, v[rows], 0.0)
    assert torch.equal(dz[rows], want)
    w = randn(g, n, dtype=BF)
    rstd = torch.empty(m, device=DEV)
    z.zero_rms_norm(out, n, None, 0, w, z.ZERO_BF16, m, n, 1e-5, None, 0, dz, n, None, rstd)
    s = out[rows].double()
    r = ((s * s).mean(1, keepdim=True) + 1e-5) ** -0.5
    F.within(dz[rows], s * r * w.double(), (0.5 * n + 9) * U * (s * r * w.double()).abs())
    # a strided view far into a buffer: rows 2^16 elements apart
    wide = out.view(-1)[: 40_000 * 57_344].view(40_000, 57_344)
    part = wide[:, :96]
    b2 = randn(g, 200, 96, dtype=BF)
    o2 = torch.empty(40_000, 200, dtype=BF, device=DEV)
    z.zero_matmul(part, False, 57_344, b2, False, 96, None, 0, None, 0, z.ZERO_BF16, 40_000, 200,
                  96, None, 0, None, 0, None, 0, None, o2, z.ZERO_BF16, 200, False)
    last = torch.arange(39_990, 40_000, device=DEV)
    F.within(o2[last], *F.product(part[last].double(), b2.double()))

