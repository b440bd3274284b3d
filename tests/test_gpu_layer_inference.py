"""The 4-bit layer where no backward pass can follow."""
import pytest
import torch

import zero_sharded_optimizer_step_gb300 as z
from zero_sharded_optimizer_step_gb300 import layers

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [1, 70])
@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
def test_nothing_is_quantised_for_a_backward_pass_that_cannot_come(m, off, monkeypatch):
    weight = torch.randn(100, 640, device="cuda").requires_grad_()
    layer = z.Mx4Linear(weight)
    x = torch.randn(m, 640, device="cuda")
    both = []
    real = layers.z.zero_mx4_quantize

    def quantize(*args, **kw):
        both.append(args[6] is not None)
        return real(*args, **kw)

    monkeypatch.setattr(layers.z, "zero_mx4_quantize", quantize)
    with off():
        y = layer(x)
    assert both == [False] and not y.requires_grad
    # with gradients on: the weight's needs the transpose, and y is the same
    both.clear()
    w = layer(x)
    assert both == [True] and w.requires_grad and torch.equal(w.detach(), y)
    # a frozen weight needs none
    both.clear()
    weight.requires_grad_(False)
    xg = x.clone().requires_grad_()
    v = layer(xg)
    assert both == [False] and v.requires_grad and torch.equal(v.detach(), y)
    v.sum().backward()
    assert xg.grad is not None and weight.grad is None
