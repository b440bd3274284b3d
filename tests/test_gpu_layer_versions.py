"""A tensor that a call writes and that a backward pass still needs: refused, as after
torch's own operations in place."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import zero_sharded_optimizer_step_gb300 as z

DEV, BF = "cuda", torch.bfloat16


def randn(*shape):
    return torch.randn(*shape, device=DEV, dtype=BF)


def writers(x):
    """The calls that write x, [16, 64]."""
    ids = torch.arange(16, device=DEV)
    (a, _), (b, _) = z.mx4_quantize(randn(16, 32)), z.mx4_quantize(randn(64, 32))
    return {"matmul": lambda: z.matmul(randn(16, 32), randn(64, 32), out=x),
            "matmul_accumulate": lambda: z.matmul(randn(16, 32), randn(64, 32), out=x,
                                                  accumulate=True),
            "kept": lambda: z.matmul(randn(16, 32), randn(64, 32), kept=x),
            "mx4_matmul": lambda: z.mx4_matmul(a, b, out=x),
            "embed_grad": lambda: z.embed_grad(randn(16, 64), ids, x)}


NAMES = ["matmul", "matmul_accumulate", "kept", "mx4_matmul", "embed_grad"]


@pytest.mark.parametrize("name", NAMES)
def test_what_a_backward_pass_needs_is_not_overwritten_in_silence(name):
    x, w = randn(16, 64), randn(24, 64).requires_grad_()
    y = z.linear(x, w)
    before = x._version
    writers(x)[name]()
    assert x._version > before
    with pytest.raises(RuntimeError, match="in-?place"):
        y.sum().backward()


@pytest.mark.parametrize("name", NAMES)
def test_what_none_needs_may_be_written(name):
    x, w = randn(16, 64), randn(24, 64).requires_grad_()
    x0 = x.clone()
    y = z.linear(x, w)
    other = randn(16, 64)
    writers(other)[name]()
    y.sum().backward()
    want = torch.ones(24, 16, device=DEV) @ x0.float()
    assert torch.allclose(w.grad.float(), want, rtol=2 ** -7, atol=1e-3)
    with torch.inference_mode():
        writers(randn(16, 64))[name]()


def test_a_gradient_buffer_takes_sum_after_sum():
    """The rank's own use: a weight's gradient accumulated beside the graph."""
    x, w = randn(16, 64), randn(24, 64).requires_grad_()
    grad = torch.zeros(24, 64, device=DEV)
    for _ in range(2):
        z.linear(x, w).sum().backward()
        z.matmul(torch.ones(16, 24, device=DEV, dtype=BF), x, True, True, out=grad,
                 accumulate=True)
    want = 2 * torch.ones(24, 16, device=DEV) @ x.float()
    assert torch.allclose(grad, want, rtol=1e-5, atol=1e-4)
