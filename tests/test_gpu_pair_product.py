"""The product where two SMs share a tile (more than one tile of 128 by 128 an
SM): several tiles a pair, more records of k than the ring has stages, ragged
ends of all three sizes, every type, both alignments of the result, alpha and
accumulation, and NaN.  The bounds are those of test_gpu_operators.py."""
import functools

import numpy as np
import pytest
import torch

import zero_sharded_optimizer_step_gb300 as z
from tests import ops_ref as R
from tests.test_gpu_operators import CODE, DTYPES, E24, gen, matmul, quantize, randn

pytestmark = pytest.mark.gpu

DEV = "cuda"
#: (m, n, k): 160 tiles of 256 x 256 on 76 pairs, eight records of k, both bands
#: of the sweep; 256 tiles, 3.4 a pair, with a last tile of one record either
#: way; few tiles, 17 records of k; more rows than columns; one row of tiles
SIZES = [(2560, 4088, 1900), (3900, 3850, 300), (300, 8200, 4130), (9001, 500, 70),
         (100, 20_011, 513)]


@functools.lru_cache(maxsize=None)
def problem(m, n, k):
    """The quantised operands, their product and the sum of its terms' magnitudes
    (float64, on the host)."""
    g = gen(m + n + k)
    x, w = randn(g, m, k), randn(g, n, k)
    (a, _), (b, _) = quantize(x), quantize(w)
    av, bv = R.values(*R.quantize(R.host(x))), R.values(*R.quantize(R.host(w)))
    return a, b, av @ bv.T, np.abs(av) @ np.abs(bv).T


def result(m, n, stride, dtype, offset, fill):
    """A result of m rows with a row in front and one behind, and its buffer; the
    result starts `offset` elements into a row of the buffer's."""
    buf = torch.full(((m + 2) * stride + 64,), fill, dtype=dtype, device=DEV)
    first = stride + offset
    return buf[first:first + m * stride].view(m, stride)[:, :n], buf, first


def check(size, dtype, stride, offset, alpha, accumulate):
    m, n, k = size
    a, b, want, mag = problem(m, n, k)
    out, buf, first = result(m, n, stride, dtype, offset, 9.0)
    old = None
    if accumulate:
        out.copy_(randn(gen(1), m, n, dtype=dtype, sigma=30.0))
        old = R.host(out)
    matmul(a, m, b, n, k, out, alpha=alpha, accumulate=accumulate)
    want, bound = want * alpha, (k + 2) * 2.0 ** -23 * mag * abs(alpha)
    if old is not None:
        want = want + old
        bound = bound + E24 * np.abs(old)
    u = R.ROUND[dtype]
    R.within(R.host(out), want, (1 + u) * bound + (u + E24) * np.abs(want) + R.TINY[dtype])
    assert bool((buf[:first] == 9).all()) and bool((buf[first + m * stride:] == 9).all())
    assert bool((buf[first:first + m * stride].view(m, stride)[:, n:] == 9).all())
    assert z.zero_mx4_timeouts() == 0


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("accumulate", [False, True])
def test_rows_on_32_byte_boundaries(size, dtype, accumulate):
    stride = (size[1] + 15) // 16 * 16 + 16
    check(size, dtype, stride, 0, -0.75 if accumulate else 1.0, accumulate)


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("accumulate", [False, True])
def test_rows_off_them(size, dtype, accumulate):
    check(size, dtype, size[1] + 3, 0, 1.0 if accumulate else 0.5, accumulate)


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_result_that_starts_off_a_boundary(dtype):
    """Row strides of whole boundaries, the first row beside one."""
    check(SIZES[0], dtype, 4096, 3, 1.0, True)


@pytest.mark.parametrize("gap", [16, 3])
@pytest.mark.parametrize("accumulate", [False, True])
def test_nan_stays_in_its_row_and_column(gap, accumulate):
    m, n, k = SIZES[0]
    n = n // 16 * 16
    g = gen(2)
    x, w = randn(g, m, k), randn(g, n, k)
    rows, cols = [0, 700, m - 1], [5, 2049, n - 1]
    x[rows, k - 1], w[cols, 40] = float("inf"), float("nan")
    (a, _), (b, _) = quantize(x), quantize(w)
    out, _, _ = result(m, n, n + gap, torch.bfloat16, 0, 1.0)
    matmul(a, m, b, n, k, out, accumulate=accumulate)
    want = torch.zeros(m, n, dtype=torch.bool, device=DEV)
    want[rows], want[:, cols] = True, True
    assert torch.equal(torch.isnan(out), want)


def test_the_same_bits_on_every_run():
    m, n, k = SIZES[1]
    a, b, _, _ = problem(m, n, k)
    first = matmul(a, m, b, n, k, torch.empty(m, n, device=DEV))
    for _ in range(20):
        assert torch.equal(matmul(a, m, b, n, k, torch.empty(m, n, device=DEV)), first)
