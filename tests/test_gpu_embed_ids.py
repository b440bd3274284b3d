"""The lookup's ids that name no row: tables without rows, ids outside the table
and what is counted of them."""
import pytest
import torch

import zero_sharded_optimizer_step_gb300 as z

pytestmark = pytest.mark.gpu

DEV = "cuda"
CODE = {torch.float32: z.ZERO_F32, torch.bfloat16: z.ZERO_BF16, torch.float16: z.ZERO_F16}


@pytest.mark.parametrize("dtype", list(CODE))
@pytest.mark.parametrize("dim,stride", [(7, 7), (7, 64), (1, 1000), (33, 40), (64, 64), (64, 96),
                                        (1025, 5000)])
@pytest.mark.parametrize("null", [True, False])
def test_a_table_without_rows(dtype, dim, stride, null):
    """Every id lies outside it: rows of zeros, all counted, nothing read."""
    n = 50
    table = None if null else torch.full((stride + 8,), 5.0, dtype=dtype, device=DEV)
    tokens = torch.arange(-3, n - 3, device=DEV)
    out = torch.full((n, dim), 7.0, dtype=dtype, device=DEV)
    bad = torch.zeros(1, dtype=torch.int64, device=DEV)
    z.zero_embed(table, CODE[dtype], 0, dim, stride, tokens, 8, n, 4, 2.0, out, dim, bad)
    assert not out.any() and int(bad) == n - 1          # id 4 is the padding token
