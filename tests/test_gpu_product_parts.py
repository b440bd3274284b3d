"""Large products whose last, unfilled turn of tiles goes in halves or quarters, so that
all pairs of SMs share it: every layout and everything beside the result, ragged last
tiles and parts with nothing left among them."""
import pytest
import torch

import tests.ff_ref as F
from tests.product_sizes import pair_shape
from tests.test_gpu_feed_forward import (DEV, U, as_lies, gated, gen, held, packed, product,
                                         randn, space)
from tests.test_gpu_product_shapes import eight_bits

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import zero_sharded_optimizer_step_gb300 as z

BF = torch.bfloat16

# (rows, columns, half a tile's width, parts, whether a part of the last tile in a row
# has no columns left), at 152 SMs
PLAIN = [(9984, 2560, 128, 4, False), (9984, 2501, 128, 4, False), (9216, 2696, 128, 4, True),
         (4352, 4968, 128, 2, True), (13056, 328, 96, 2, False), (13056, 1128, 64, 4, False),
         (11264, 1352, 64, 2, False)]
GATED = [(2304, 4352, 128, 4, False), (13056, 712, 128, 4, True), (13056, 711, 128, 4, True),
         (2304, 4608, 128, 2, False), (9984, 488, 64, 2, False), (11776, 392, 64, 2, True)]


def in_parts(m, n, gated):
    """The division is the one that the test is for: this device's."""
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    shape = pair_shape(m, n, sms, gated)
    assert shape["cut"] > 1 and shape["whole"] < shape["tiles_m"] * shape["tiles_n"]


@pytest.mark.parametrize("a_cols,b_cols", [(False, False), (False, True), (True, True),
                                           (True, False)])
@pytest.mark.parametrize("m,n,half,cut,empty", PLAIN)
def test_tiles_in_parts_in_every_layout(a_cols, b_cols, m, n, half, cut, empty):
    in_parts(m, n, False)
    k = 72
    g = gen(m + n)
    a, b = randn(g, m, k, dtype=torch.float16), randn(g, n, k, dtype=torch.float16)
    want, err = F.product(a.double(), b.double())
    for pad in (0, 3):
        out = space(m, n, torch.float16, n + pad)
        product(as_lies(a, a_cols), a_cols, as_lies(b, b_cols), b_cols, out)
        F.within(out.t, want, err)
        assert out.untouched()


@pytest.mark.parametrize("m,n,half,cut,empty", PLAIN)
@pytest.mark.parametrize("pad,offset", [(0, 0), (16, 16), (1, 1)])
def test_tiles_in_parts_with_everything(m, n, half, cut, empty, pad, offset):
    in_parts(m, n, False)
    k = 136
    g = gen(m + n)
    a, b = randn(g, m, k, dtype=BF), randn(g, n, k, dtype=BF, sigma=k ** -0.5 * 2)
    bias, r = randn(g, n, dtype=BF), randn(g, m, n, dtype=BF)
    zz, err = F.product(a.double(), b.double())
    zz = zz + bias.double()
    err = err + U * (zz.abs() + err)
    y, yerr = F.activation(zz, F.GELU_TANH)[0], F.value_error(zz, err, F.GELU_TANH)
    want = y + r.double()
    for dtype in (BF, torch.float32):
        out, kept = space(m, n, dtype, n + pad, offset), space(m, n, BF, n + pad, offset)
        res = held(r.to(dtype), n + pad, offset)
        product(held(a), False, held(b), False, out, bias=bias, act=F.GELU_TANH, residual=res,
                kept=kept)
        F.within(out.t, want, yerr + U * (want.abs() + yerr))
        F.within(kept.t, zz, err)
        assert out.untouched() and kept.untouched()
        q = packed(m, n)
        product(held(a), False, held(b), False, res, bias=bias, act=F.GELU_TANH, kept_q=q,
                accumulate=True)
        assert torch.equal(res.t, out.t)
        eight_bits(q, m, n, zz, err)
    assert z.zero_matmul_timeouts() == 0


@pytest.mark.parametrize("m,n,half,cut,empty", GATED)
@pytest.mark.parametrize("pad,offset", [(0, 0), (16, 16), (1, 1)])
def test_gated_tiles_in_parts_with_everything(m, n, half, cut, empty, pad, offset):
    in_parts(m, n, True)
    k = 136
    g = gen(m + n)
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
    assert torch.equal(again.t, h.t)
    eight_bits(qg, m, n, gate, gerr)
    eight_bits(qu, m, n, up, uerr)
    assert z.zero_matmul_timeouts() == 0


@pytest.mark.parametrize("m,n", [(9216, 2696), (13056, 328)])
def test_tiles_in_parts_of_two_pairs(m, n):
    in_parts(m, n, False)
    k = 100
    g = gen(m)
    a, a2 = (randn(g, m, k, dtype=BF) for _ in range(2))
    b, b2 = (randn(g, n, k, dtype=BF) for _ in range(2))
    want, err = F.product(torch.cat([a, a2], 1).double(), torch.cat([b, b2], 1).double())
    out = space(m, n, BF)
    product(as_lies(a, False), False, as_lies(b, True), True, out, as_lies(a2, False),
            as_lies(b2, True))
    F.within(out.t, want, err)
    assert out.untouched()
