"""As many rows as there can be: what is counted in rows, and every row's place."""
import pytest
import torch

import tests.ff_ref as F

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import zero_sharded_optimizer_step_gb300 as z

DEV, BF = "cuda", torch.bfloat16
MOST = 2 ** 31 - 2


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def column(seed):
    g = torch.Generator(DEV).manual_seed(seed)
    x = torch.empty(MOST, 1, dtype=BF, device=DEV)
    return x.normal_(generator=g)


def some():
    return torch.cat([torch.arange(300, device=DEV),
                      torch.randint(0, MOST, (3000,), device=DEV,
                                    generator=torch.Generator(DEV).manual_seed(0)),
                      torch.arange(MOST - 300, MOST, device=DEV)])


def test_the_norm_and_its_gradient():
    x, w, at = column(1), torch.full((1,), 1.5, dtype=BF, device=DEV), some()
    y, rstd = torch.empty_like(x), torch.empty(MOST, device=DEV)
    z.zero_rms_norm(x, 1, None, 0, w, z.ZERO_BF16, MOST, 1, 1e-2, None, 0, y, 1, None, rstd)
    s = x[at].double()
    r = (s * s + 1e-2) ** -0.5
    F.within(y[at], s * r * 1.5, 10 * 2.0 ** -24 * (s * r * 1.5).abs())
    assert float((rstd[at].double() - r[:, 0]).abs().max()) < 1e-5
    dx, dw = torch.empty_like(x), torch.empty(1, device=DEV)
    need = z.zero_rms_norm_grad_workspace(MOST, 1)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    z.zero_rms_norm_grad(y, 1, None, 0, x, 1, w, rstd, z.ZERO_BF16, MOST, 1, dx, 1, dw,
                         z.ZERO_F32, False, ws, need)
    n, dy = s * rstd[at, None].double(), y[at].double()
    want = rstd[at, None].double() * (1.5 * dy - n * (1.5 * dy * n))
    # the terms cancel: an fp32 rounding or two of either
    F.within(dx[at], want, 8 * 2.0 ** -24 * (rstd[at, None].double() * 1.5 * dy).abs())


def test_gradients_through_activations():
    dy, kept, at = column(2), column(3), some()
    dz, db = torch.empty_like(dy), torch.empty(1, device=DEV)
    need = z.zero_activation_grad_workspace(MOST, 1)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    z.zero_activation_grad(dy, 1, kept, 1, None, F.RELU, z.ZERO_BF16, MOST, 1, dz, 1, db,
                           z.ZERO_F32, False, ws, need)
    assert torch.equal(dz[at], torch.where(kept[at] > 0, dy[at], 0.0))
    dg, du = dz, torch.empty_like(dy)
    z.zero_gated_grad(dy, 1, kept, dy, 1, None, None, F.RELU, z.ZERO_BF16, MOST, 1, dg, du, 1)
    assert torch.equal(du[at], dy[at] * kept[at].clamp(min=0))
    assert torch.equal(dg[at], torch.where(kept[at] > 0, dy[at] * dy[at], 0.0))


def test_rows_in_8_bits():
    x, at = column(4), some()
    q = torch.empty(z.zero_pack8_bytes(MOST, 1), dtype=torch.uint8, device=DEV)
    z.zero_pack8(x, z.ZERO_BF16, MOST, 1, 1, q)
    v = torch.empty_like(x)
    z.zero_unpack8(q, MOST, 1, v, z.ZERO_BF16, 1)
    assert torch.equal(v[at].double(), F.pack(x[at].double())[0])


@pytest.mark.parametrize("m,n", [(MOST, 1), (2, MOST), (1, MOST)])
def test_products(m, n):
    g = torch.Generator(DEV).manual_seed(5)

    def whole(rows):
        return torch.empty(rows, 8, dtype=torch.int8, device=DEV).random_(
            -4, 5, generator=g).to(BF)

    a, b = whole(m), whole(n)
    out = z.matmul(a, b)
    at = some()
    i, j = (at, slice(None)) if m == MOST else (slice(None), at)
    assert torch.equal(out[i, j].double(), (a[i].double() @ b[j].double().t()))
    assert z.zero_matmul_timeouts() == 0
