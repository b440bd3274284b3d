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


@pytest.mark.parametrize("tt", [torch.int32, torch.int64])
@pytest.mark.parametrize("pad,counted", [(-1, 4), (2, 4), (-7, 3), (100, 3)])
def test_what_is_counted_as_outside(tt, pad, counted):
    """Without a padding token (-1) an id of -1 is one outside the table like any
    other; a padding token outside the table is none."""
    table = torch.ones(10, 16, device=DEV)
    tokens = torch.tensor([0, -1, 2, 100, -7, 9, 10], device=DEV).to(tt)
    out = torch.full((7, 16), 7.0, device=DEV)
    bad = torch.zeros(1, dtype=torch.int64, device=DEV)
    z.zero_embed(table, z.ZERO_F32, 10, 16, 16, tokens, tokens.element_size(), 7, pad, 1.0, out,
                 16, bad)
    assert int(bad) == counted
    live = [0, 5] + ([2] if pad != 2 else [])
    want = torch.zeros(7, 16, device=DEV)
    want[live] = 1.0
    assert torch.equal(out, want)
