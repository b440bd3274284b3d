"""A norm whose weight alone is trained: the sum that it returns has no gradient, as torch's
own x + residual has none."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import zero_sharded_optimizer_step_gb300 as z

DEV, BF = "cuda", torch.bfloat16


def three(x_grad, r_grad, w_grad):
    g = torch.Generator(DEV).manual_seed(3)
    x, r = (torch.randn(24, 72, device=DEV, generator=g).to(BF) for _ in range(2))
    w = torch.randn(72, device=DEV, generator=g).to(BF)
    return x.requires_grad_(x_grad), r.requires_grad_(r_grad), w.requires_grad_(w_grad)


@pytest.mark.parametrize("packed", [False, True])
def test_the_sum_of_frozen_inputs_asks_for_no_gradient(packed):
    x, r, w = three(False, False, True)
    y, h = z.rms_norm(x, w, residual=r, packed=packed)[:2]
    assert y.requires_grad and not h.requires_grad and h.grad_fn is None
    assert torch.equal(h, x + r)
    # what follows takes both, and the weight's gradient is the norm's alone
    (y.float().square().sum() + (h.float() * 3).sum()).backward()
    w2 = w.detach().float().requires_grad_()
    s = (x + r).float()
    n = s * (s.square().mean(1, keepdim=True) + 1e-5).rsqrt()
    (n * w2).square().sum().backward()
    assert float((w.grad.float() - w2.grad).norm()) < 2 ** -7 * float(w2.grad.norm())


@pytest.mark.parametrize("grads", [(True, False, True), (False, True, True), (True, True, False),
                                   (False, True, False)])
def test_the_sum_of_others_does(grads):
    x, r, w = three(*grads)
    y, h = z.rms_norm(x, w, residual=r)
    assert h.requires_grad
    h.float().sum().backward()
    for t, g in ((x, grads[0]), (r, grads[1])):
        assert (t.grad is not None) == g
        if g:
            assert bool((t.grad == 1).all())


def test_it_can_be_captured():
    x, r, w = three(False, False, True)

    def step():
        w.grad = None
        y, h = z.rms_norm(x, w, residual=r)
        (y * h).sum().backward()
        return w.grad

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step().clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
