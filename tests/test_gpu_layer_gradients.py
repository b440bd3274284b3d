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


@pytest.mark.parametrize("with_residual", [False, True])
def test_dropout_can_be_differentiated_twice(with_residual):
    """L = sum of (m x^2 + r)^2, m = 0 or 1 / (1 - p): dL/dx = 4 m x (m x^2 + r),
    and the sum of that has the derivative 12 m^2 x^2 + 4 m r.  p = 1/2 and small
    whole numbers: every value is exact."""
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randint(-5, 6, (300,), generator=g, device=DEV).float().requires_grad_()
    r = torch.randint(-5, 6, (300,), generator=g, device=DEV).float()
    if not with_residual:
        r.zero_()
    m = z.dropout(torch.ones(300, device=DEV), 0.5, 3, 4)
    assert set(m.tolist()) == {0.0, 2.0}
    y = z.dropout(x * x, 0.5, 3, 4, residual=r if with_residual else None)
    first, = torch.autograd.grad((y * y).sum(), x, create_graph=True)
    xd = x.detach()
    assert torch.equal(first.detach(), 4 * m * xd * (m * xd * xd + r))
    second, = torch.autograd.grad(first.sum(), x)
    assert torch.equal(second, 12 * m * m * xd * xd + 4 * m * r)


def test_dropout_against_differences_of_its_gradient():
    """L = sum of (m x^2)^2 has the gradient 4 m^2 x^3, whose central difference at
    step 1 is its slope plus 4 m^2.  Whole numbers below 2^24 throughout."""
    x = (torch.arange(64, device=DEV) % 9 + 1).float().requires_grad_()
    w = torch.arange(1, 65, device=DEV).float()

    def gradient_of(v, **kw):
        y = z.dropout(v * v, 0.5, 7, 8)
        return torch.autograd.grad((y * y).sum(), v, **kw)[0]

    second, = torch.autograd.grad((gradient_of(x, create_graph=True) * w).sum(), x)
    m = z.dropout(torch.ones(64, device=DEV), 0.5, 7, 8)
    assert 0 < int((m == 2).sum()) < 64
    for e in range(0, 64, 5):
        up, down = (x.detach().clone().requires_grad_() for _ in range(2))
        with torch.no_grad():
            up[e] += 1
            down[e] -= 1
        slope = float((gradient_of(up)[e] - gradient_of(down)[e]) * w[e]) / 2
        assert slope - 4 * float(m[e]) ** 2 * float(w[e]) == float(second[e])


def test_the_lookup_can_be_differentiated_twice():
    """L = sum of y^4 / 4 over y = s table[tok]: with c the times that a row is
    named, dL/dtable = c s^4 table^3 and the derivative of its sum with weights w
    is 3 w c s^4 table^2.  Whole numbers; a padding token; an id outside."""
    g = torch.Generator(device=DEV).manual_seed(3)
    table = torch.randint(-3, 4, (20, 9), generator=g, device=DEV).float().requires_grad_()
    w = torch.randint(-3, 4, (20, 9), generator=g, device=DEV).float()
    tokens = torch.randint(0, 20, (6, 11), generator=g, device=DEV)
    tokens[0, 0], tokens[3, 4] = 33, -2
    count = torch.bincount(tokens.reshape(-1).clamp(0, 33), minlength=34)[:20].float()
    count[0] -= 1                                   # -2, which was counted as 0
    count[5] = 0
    y = z.embed(table, tokens, scale=2.0, pad=5)
    first, = torch.autograd.grad((y * y * y * y).sum() / 4, table, create_graph=True)
    t = table.detach()
    assert torch.equal(first.detach(), count[:, None] * 16 * t ** 3)
    second, = torch.autograd.grad((first * w).sum(), table, create_graph=True)
    assert torch.equal(second.detach(), 3 * w * count[:, None] * 16 * t ** 2)
    third, = torch.autograd.grad(second.sum(), table)
    assert torch.equal(third, 6 * w * count[:, None] * 16 * t)


def linear(seed=0):
    weight = randn(16, 8, seed=seed).requires_grad_()
    return z.Mx4Linear(weight), randn(12, 8, seed=2).requires_grad_(), weight


@pytest.mark.parametrize("by", ["inputs", "backward"])
@pytest.mark.parametrize("curved", [True, False])
@pytest.mark.parametrize("of,wrt", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_the_linear_layer_says_that_it_cannot(of, wrt, curved, by):
    """dx depends on the weight and dW on x even for a loss that is linear in y.
    The gradients themselves are there, and differentiating them raises also
    where other paths lead to the same input (cubes of both, here)."""
    layer, x, weight = linear()
    leaves = x, weight

    def loss():
        y = layer(x * 1.0)                          # x as an intermediate result
        return (y * y if curved else y).sum()

    plain = torch.autograd.grad(loss(), leaves)
    total = loss() + sum((v ** 3).sum() for v in leaves)
    first = torch.autograd.grad(total, leaves, create_graph=True)
    for f, p, v in zip(first, plain, leaves):
        want = p + 3 * v.detach() ** 2
        assert torch.allclose(f.detach(), want, rtol=1e-6, atol=1e-6)
    last = (first[of] ** 2).sum() + (leaves[wrt] ** 3).sum()
    with pytest.raises(RuntimeError, match="differentiated once"):
        if by == "inputs":
            torch.autograd.grad(last, leaves[wrt])
        else:
            last.backward()


def test_a_linear_layer_whose_result_goes_unused():
    """Only one of two results takes part in the loss."""
    layer, x, weight = linear()
    outer = z.Mx4Linear(randn(4, 16, seed=3).requires_grad_())
    y = layer(x)
    outer(y)
    y.sum().backward()
    assert x.grad is not None and weight.grad is not None and outer.weight.grad is None
