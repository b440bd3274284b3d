"""The training operators as torch functions (layers.py): values and gradients
against plain torch on the same quantised operands, refusals, and the token
model that runs them together under ZeroAdam."""
import numpy as np
import pytest
import torch

import zero_sharded_optimizer_step_gb300 as z
from tests import ops_ref as R

pytestmark = pytest.mark.gpu


def quantised(x):
    """The values of x quantised along its rows, float64 on the GPU."""
    return torch.from_numpy(R.values(*R.quantize(R.host(x)))).cuda()


def test_embed_and_its_gradient():
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randn(60, 40, generator=g, device="cuda", requires_grad=True)
    tokens = torch.randint(0, 60, (7, 9), generator=g, device="cuda").int()
    bad = torch.zeros(1, dtype=torch.int64, device="cuda")
    tokens[0, 0] = 99
    y = z.embed(table, tokens, scale=2.0, pad=5, bad=bad)
    live = ((tokens != 5) & (tokens < 60))[..., None]
    want = torch.where(live, table.detach()[tokens.clamp(max=59)] * 2.0, 0.0)
    assert y.shape == (7, 9, 40) and torch.equal(y, want) and int(bad) == 1
    w = torch.randn(7, 9, 40, generator=g, device="cuda")
    (y * w).sum().backward()
    ref = torch.zeros(60, 40, dtype=torch.float64, device="cuda")
    ref.index_add_(0, tokens.clamp(max=59).reshape(-1).long(),
                   (w * live).double().reshape(-1, 40) * 2.0)
    # at most 63 terms of magnitude up to 2 * max|w| in fp32
    assert float((table.grad.double() - ref).abs().max()) <= 65 * 2.0 ** -24 * 63 * 2 * float(
        w.abs().max())
    # a transposed gradient (no consecutive rows) is the same gradient
    first = table.grad.clone()
    table.grad = None
    z.embed(table, tokens, scale=2.0, pad=5).backward(
        w.permute(2, 0, 1).contiguous().permute(1, 2, 0))
    assert torch.equal(table.grad, first)


def test_dropout_and_its_gradient():
    x = torch.randn(30, 50, device="cuda", requires_grad=True)
    r = torch.randn(30, 50, device="cuda", requires_grad=True)
    y = z.dropout(x, 0.25, 7, 8, residual=r)
    kept = torch.from_numpy(R.keep(1500, 0.25, 7, 8)).cuda().view(30, 50)
    up = float(np.float32(1 / 0.75))
    assert torch.equal(y, torch.where(kept, x * up, 0.0) + r)
    w = torch.randn(30, 50, device="cuda")
    y.backward(w)
    assert torch.equal(x.grad, torch.where(kept, w * up, 0.0)) and torch.equal(r.grad, w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_linear_and_its_gradients(dtype):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(3, 20, 72, generator=g, device="cuda").to(dtype).requires_grad_()
    weight = torch.randn(100, 72, generator=g, device="cuda").to(dtype).requires_grad_()
    dy = torch.randn(3, 20, 100, generator=g, device="cuda").to(dtype)
    layer = z.Mx4Linear(weight)
    y = layer(x)
    y.backward(dy)
    x2, dy2 = x.detach().reshape(60, 72), dy.reshape(60, 100)
    u = R.ROUND[dtype]

    def check(got, a, b):
        want = a @ b.T
        bound = (a.shape[1] + 2) * 2.0 ** -23 * (a.abs() @ b.abs().T)
        off = (got.double().reshape(want.shape) - want).abs()
        assert bool((off <= (1 + u) * bound + (u + 2.0 ** -24) * want.abs()
                     + R.TINY[dtype]).all())

    check(y.detach(), quantised(x2), quantised(weight))
    check(x.grad, quantised(dy2), quantised(weight.detach().T))
    check(weight.grad, quantised(dy2.T), quantised(x2.T))
    # the same gradient written where a rank's gradient lies, and added to it
    buf = torch.zeros(100 * 72 + 6, dtype=dtype, device="cuda")
    view = buf[3:3 + 7200].view(100, 72)
    layer.weight_grad(x2, dy2, view)
    assert torch.equal(view, weight.grad) and not buf[:3].any() and not buf[-3:].any()
    # the weight's change is seen after refresh(), not before
    with torch.no_grad():
        before = layer(x)
        weight.mul_(2.0)
        assert torch.equal(layer(x), before)
        layer.refresh()
        assert not torch.equal(layer(x), before)


def test_backward_uses_the_weight_of_its_forward():
    weight = torch.randn(64, 64, device="cuda", requires_grad=True)
    layer = z.Mx4Linear(weight)
    x = torch.randn(8, 64, device="cuda", requires_grad=True)
    dy = torch.randn(8, 64, device="cuda")
    layer(x).backward(dy)
    want = x.grad.clone()
    x.grad = None
    y = layer(x)
    with torch.no_grad():
        weight.neg_()
    layer.refresh()
    y.backward(dy)
    assert torch.equal(x.grad, want)


def test_refusals():
    t = torch.zeros(4, 8, device="cuda")
    tok = torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (lambda: z.embed(t.cpu(), tok), lambda: z.embed(t.double(), tok),
                lambda: z.embed(t[0], tok), lambda: z.embed(t, tok.float()),
                lambda: z.embed(t, tok.cpu()), lambda: z.embed(t.t(), tok),
                lambda: z.embed_grad(t, tok, t), lambda: z.embed_grad(t[:3, :4], tok, t),
                lambda: z.dropout(t, 1.5, 0, 0), lambda: z.dropout(t.int(), 0.5, 0, 0),
                lambda: z.dropout(t, 0.5, 0, 0, residual=t[:2]),
                lambda: z.dropout(t, 0.5, 0, 0, residual=t.half()),
                lambda: z.Mx4Linear(t)(t[:, :4]), lambda: z.mx4_quantize(t.t()),
                lambda: z.mx4_matmul(z.mx4_quantize(t)[0], z.mx4_quantize(t)[1]),
                lambda: z.mx4_matmul(*[z.mx4_quantize(t)[0]] * 2, out=t),
                lambda: z.mx4_matmul(*[z.mx4_quantize(t)[0]] * 2, accumulate=True)):
        with pytest.raises(ValueError):
            bad()


def test_token_model_trains():
    """The loss of a fixed token map falls from about log(500) = 6.2 to well
    below 1 (dropout and 4-bit operands left in); the same run twice gives the
    same losses, bit for bit."""
    from workloads import token_model
    losses = token_model.train(steps=150)
    assert 5.5 < losses[0] < 8.0, losses[0]
    assert np.mean(losses[-10:]) < 1.0, losses[-10:]
    assert token_model.train(steps=5) == losses[:5]
    assert z.zero_mx4_timeouts() == 0
