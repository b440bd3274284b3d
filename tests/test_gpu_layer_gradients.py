"""Gradients of the torch functions in the layouts that torch hands them in, and
derivatives of derivatives."""
import pytest
import torch

import zero_sharded_optimizer_step_gb300 as z

pytestmark = pytest.mark.gpu

DEV = "cuda"


def randn(*shape, seed=0, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def gradient(fn, inputs, dy):
    """The inputs' gradients for the output's gradient dy."""
    return torch.autograd.grad(fn(*inputs), inputs, dy)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", [1, 24, 33])
@pytest.mark.parametrize("n", [1, 5, 700])
def test_a_gradient_that_is_the_same_for_all_rows(dtype, n, dim):
    """sum(0) hands its gradient on with a row stride of 0, sum() with both: the
    gradients are those of the same values written out."""
    table = randn(90, dim, dtype=dtype).requires_grad_()
    tokens = torch.arange(n, device=DEV) * 7 % 90
    weight = randn(20, dim, seed=1, dtype=dtype).requires_grad_()
    layer = z.Mx4Linear(weight)
    x = randn(n, dim, seed=2, dtype=dtype).requires_grad_()
    for fn, inputs, width in [(lambda t: z.embed(t, tokens, scale=2.0), (table,), dim),
                              (lambda v, w: layer(v), (x, weight), 20)]:
        v = randn(width, seed=3, dtype=dtype)
        want = gradient(fn, inputs, v.expand(n, width).contiguous())
        for got in (gradient(lambda *a: fn(*a).sum(0), inputs, v),
                    gradient(fn, inputs, v.expand(n, width)),
                    gradient(lambda *a: fn(*a)[None].sum(1), inputs, v[None])):
            assert all(torch.equal(g, w) for g, w in zip(got, want))
        one = torch.ones((), dtype=dtype, device=DEV)
        want = gradient(fn, inputs, one.expand(n, width).contiguous())
        got = gradient(lambda *a: fn(*a).sum(), inputs, one)
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_a_gradient_whose_rows_overlap():
    """Rows that share elements, as a sliding window's gradient may."""
    table = randn(30, 8).requires_grad_()
    tokens = torch.arange(12, device=DEV)
    dy = randn(41, seed=4).as_strided((12, 8), (3, 1))
    want = gradient(lambda t: z.embed(t, tokens), (table,), dy.contiguous())
    assert torch.equal(gradient(lambda t: z.embed(t, tokens), (table,), dy)[0], want[0])
