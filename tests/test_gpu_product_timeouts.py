"""The count of products that gave up: that reading it waits for the products,
and that the token model looks at it."""
import pytest
import torch

import zero_sharded_optimizer_step_gb300 as z

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_the_count_is_read_after_the_work_of_every_stream():
    """Streams that do not synchronise with the default one included: work that
    is still to come when the count is asked for has ended when it is there."""
    assert z.zero_mx4_timeouts() == 0
    (a, _), (b, _) = (z.mx4_quantize(torch.randn(64, 512, device=DEV)) for _ in range(2))
    z.mx4_matmul(a, b, torch.float32)              # what a first call sets up
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    done = torch.cuda.Event()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)             # some 50 ms
        out = z.mx4_matmul(a, b, torch.float32)
        done.record()
    assert not done.query()
    assert z.zero_mx4_timeouts() == 0
    assert done.query()
    assert torch.isfinite(out).all()


def test_the_token_model_stops_when_a_product_gave_up(monkeypatch):
    from workloads import token_model
    monkeypatch.setattr(token_model.z, "zero_mx4_timeouts", lambda: 3, raising=False)
    with pytest.raises(RuntimeError, match="3"):
        token_model.train(steps=1)
