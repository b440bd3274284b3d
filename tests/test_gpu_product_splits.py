"""16-bit products whose split comes next to a limit."""
import pytest
import torch

import tests.ff_ref as F
from tests.test_gpu_feed_forward import gen, held, product, randn, space

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("m,n,k", [(170, 2000, 1600), (170, 2500, 6400), (176, 2300, 896)])
@pytest.mark.parametrize("pad", [0, 1])
def test_a_split_that_would_pass_a_blocks_shared_memory(m, n, k, pad):
    """Tiles of 176 rows in seven parts, the result's rows turned: 232,288 bytes of the
    231,424 that a block may have.  Another split is taken."""
    g = gen(m + n)
    a, b = randn(g, m, k, dtype=BF), randn(g, n, k, dtype=BF, sigma=k ** -0.5)
    want, err = F.product(a.double(), b.double())
    for dtype in (BF, torch.float32):
        out = space(m, n, dtype, n + pad)
        product(held(a), False, held(b), False, out)
        F.within(out.t, want, err)
        assert out.untouched()
