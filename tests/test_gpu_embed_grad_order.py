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


@pytest.mark.parametrize("n", [1, 2, 31, 255, 257, 512])
@pytest.mark.parametrize("rows,dim,gap,offset", [
    (1, 8, 0, 0), (7, 24, 0, 0), (300, 33, 0, 0), (300, 33, 4, 1), (20_000, 16, 8, 0),
    (1_000_003, 8, 0, 0), (5_300_000, 1, 0, 0), (50_257, 768, 0, 0)])
def test_few_tokens_right_after_their_inputs_are_written(n, rows, dim, gap, offset):
    """The list, dy and the gradient's old contents come from the kernels right in
    front; the rows that no token names are zero and those that one names hold
    their sum, for tables with fewer rows than blocks, of several thousand rows
    a block, and with gaps between the rows."""
    stride = dim + gap
    where = tokens_of(n, rows, n)
    where[n // 2], where[-1] = rows - 1, 0
    values = whole_rows(n, dim, n + 1)
    want = formula(where, values, rows)
    buf = torch.empty(rows * stride + offset, device=DEV)
    grad = buf[offset:].view(rows, stride)[:, :dim]
    ws = torch.empty(z.zero_embed_grad_workspace(rows, dim, n), dtype=torch.uint8, device=DEV)
    t, dy = torch.empty_like(where), torch.empty_like(values)
    for _ in range(3):
        t.fill_(0)
        dy.fill_(5.0)
        buf.fill_(9.0)
        t.copy_(where)
        dy.copy_(values)
        z.zero_embed_grad(dy, z.ZERO_F32, dim, t, 8, n, -1, 1.0, grad, z.ZERO_F32, rows, dim,
                          stride, False, ws, ws.numel())
        t.fill_(-3)                    # what comes after must not be seen
        dy.fill_(float("nan"))
        assert torch.equal(grad, want)
        assert bool((buf[:offset] == 9).all())
        if gap:
            assert bool((buf[offset:].view(rows, stride)[:, dim:] == 9).all())


def test_no_tokens_leave_zeros():
    grad = torch.full((5000, 40), 3.0, device=DEV)
    ws = torch.empty(z.zero_embed_grad_workspace(5000, 40, 0), dtype=torch.uint8, device=DEV)
    call(torch.empty(0, 40, device=DEV), None, 5000, grad, ws)
    assert not grad.any()
