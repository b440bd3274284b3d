"""Codes past the columns are zero in everything that packs rows, whatever the rows hold."""
import pytest
import torch

import tests.ff_ref as F
from tests.test_gpu_feed_forward import DEV, gen, held, norm, packed, parts, product, randn, space

pytestmark = pytest.mark.gpu

ALL = [torch.float32, torch.bfloat16, torch.float16]


def rows_of(dim, dtype):
    """Rows of numbers, of zeros, with an infinity, with a NaN."""
    x = randn(gen(dim), 6, dim, dtype=dtype)
    x[1] = 0
    x[2, dim // 2], x[3, dim - 1], x[4, 0] = float("inf"), float("nan"), float("-inf")
    return x


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("dim,stride", [(8, 8), (72, 72), (33, 40), (200, 200), (777, 777),
                                        (1608, 1608), (4100, 4100), (8200, 8200), (9001, 9001)])
def test_the_norm_of_rows_without_a_finite_root(dtype, dim, stride):
    """eps = 0: a row of zeros has the root 1 / 0, and one with a NaN has none."""
    x = rows_of(dim, dtype)
    q, y = packed(6, dim), space(6, dim, dtype, stride)
    norm(held(x, stride), None, torch.ones(dim, dtype=dtype, device=DEV), 0.0, None, y, q)
    tail, scales, guard = parts(q, 6, dim)
    assert not tail.any() and bool((guard == 0xA5).all())
    assert torch.isnan(y.t[1]).all() and torch.isnan(y.t[3]).all()
    assert bool((scales[1] == 255).all()) and bool((scales[3] == 255).all())


@pytest.mark.parametrize("m,n,k", [(6, 33, 40), (1, 33, 64), (6, 72, 40), (130, 200, 72)])
@pytest.mark.parametrize("pad", [0, 1])
def test_a_products_kept_sums(m, n, k, pad):
    a, b = randn(gen(m), m, k, dtype=torch.bfloat16), randn(gen(n), n, k, dtype=torch.bfloat16)
    a[0, 0], b[n - 1, 1] = float("nan"), float("inf")
    q, out = packed(m, n), space(m, n, torch.bfloat16, n + pad)
    product(held(a), False, held(b), False, out, act=F.SILU, kept_q=q)
    tail, scales, guard = parts(q, m, n)
    assert not tail.any() and bool((guard == 0xA5).all())
    assert bool((scales[0] == 255).all())
