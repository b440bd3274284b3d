"""The embedding gradient between other work of its stream: its lists, its
inputs and its output are written right before it and right after it."""
import pytest
import torch

import zero_sharded_optimizer_step_gb300 as z

pytestmark = pytest.mark.gpu

DEV = "cuda"


def tokens_of(n, rows, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(0, rows, (n,), generator=g, device=DEV)


def whole_rows(n, dim, seed):
    """Small whole numbers: every sum is exact, in any order."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-8, 9, (n, dim), generator=g, device=DEV).float()


def formula(t, dy, rows):
    out = torch.zeros(rows, dy.shape[1], dtype=torch.float64, device=DEV)
    return out.index_add_(0, t, dy.double()).float()


def call(dy, t, rows, grad, ws, accumulate=False):
    n, dim = dy.shape
    z.zero_embed_grad(dy, z.ZERO_F32, dim, t, 8, n, -1, 1.0, grad, z.ZERO_F32, rows, dim, dim,
                      accumulate, ws, ws.numel())


@pytest.mark.parametrize("n,rows", [(2049, 300), (4096, 70_000), (4097, 50_257), (8192, 50_257)])
def test_lists_sorted_by_a_cluster_back_to_back(n, rows):
    """Forty calls without a pause, each with a list of its own, so that a call's
    cluster starts beside the tail of the call before."""
    dim = 16
    lists = [tokens_of(n, rows, k) for k in range(8)]
    dy = whole_rows(n, dim, 9)
    want = [formula(t, dy, rows) for t in lists]
    ws = torch.empty(z.zero_embed_grad_workspace(rows, dim, n), dtype=torch.uint8, device=DEV)
    got = [torch.full((rows, dim), 7.0, device=DEV) for _ in range(40)]
    torch.cuda.synchronize()
    for k in range(40):
        call(dy, lists[k % 8], rows, got[k], ws)
    for k in range(40):
        assert torch.equal(got[k], want[k % 8]), k
