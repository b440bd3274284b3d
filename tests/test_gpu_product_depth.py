"""16-bit products as deep as columns go: the stages of a block are counted in millions,
its waits last a large part of a second, and columns lie beyond 32-bit offsets."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import zero_sharded_optimizer_step_gb300 as z

DEV, BF = "cuda", torch.bfloat16


def sparse(rows, k, cols, at, seed):
    """Small whole numbers in the columns `at`, zeros elsewhere: (as it lies, those columns)."""
    g = torch.Generator(DEV).manual_seed(seed)
    v = torch.randint(-4, 5, (rows, at.numel()), device=DEV, generator=g).to(BF)
    x = torch.zeros((k, rows) if cols else (rows, k), dtype=BF, device=DEV)
    if cols:
        x[at] = v.t()
    else:
        x[:, at] = v
    return x, v.double()


@pytest.mark.parametrize("m,n,cols,k", [
    (2, 3, False, 2 ** 31 - 8),          # few rows, split over eight blocks
    (1, 2, False, 2 ** 31 - 8),          # a dot product
    (72, 8, False, 2 ** 28 + 24),        # some rows
    (8, 8, True, 2 ** 30 + 40)])         # a weight's gradient over a billion rows
def test_the_deepest_products(m, n, cols, k):
    at = torch.cat([torch.tensor([0, 1, k // 2, k - 65, k - 64, k - 2, k - 1], device=DEV),
                    torch.randint(0, k, (500,), device=DEV,
                                  generator=torch.Generator(DEV).manual_seed(k))]).unique()
    (a, av), (b, bv) = sparse(m, k, cols, at, 1), sparse(n, k, cols, at, 2)
    out = z.matmul(a, b, cols, cols, out=torch.full((m, n), 7.0, device=DEV))
    assert torch.equal(out.double(), av @ bv.t())            # whole numbers: every sum is exact
    assert z.zero_matmul_timeouts() == 0
