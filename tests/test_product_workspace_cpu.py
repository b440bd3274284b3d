"""When a 16-bit product needs its workspace: exactly."""
import itertools

import pytest

from tests.test_feed_forward_cpu import A, B, C, z  # noqa: F401  (a fixture)


def lies(rows, k, cols, pad):
    """(row stride, rows, columns) of an operand as it lies."""
    r, c = (k, rows) if cols else (rows, k)
    return c + pad, r, c


def room(r, c):
    return (r * ((c + 7) // 8 * 8) * 2 + 127) // 128 * 128


@pytest.mark.parametrize("a_cols,b_cols", list(itertools.product([False, True], repeat=2)))
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 16, 65, 300])
def test_operands_off_their_boundaries(z, m, a_cols, b_cols):  # noqa: F811
    """A single row of A against rows of B is read as it lies; everything else is copied."""
    n, k = 40, 72
    (sa, ra, ca), (sb, rb, cb) = lies(m, k, a_cols, 3), lies(n, k, b_cols, 5)
    for off in (0, 2, 6, 14):
        need = z.zero_matmul_workspace(A + off, a_cols, sa, B + off, b_cols, sb, None, 0, None, 0,
                                       m, n, k)
        one = m == 1 and not a_cols and not b_cols
        assert (need == 0) == one
        if not one:             # (a matrix of one row has no stride to be off by)
            want = (room(ra, ca) if off or (ra > 1 and sa % 8) else 0) + (
                room(rb, cb) if off or sb % 8 else 0)
            assert need == want
    for one_off in (True, False):
        need = z.zero_matmul_workspace(A + 2 * one_off, a_cols, (ca + 7) // 8 * 8,
                                       B + 2 * (not one_off), b_cols, (cb + 7) // 8 * 8, None, 0,
                                       None, 0, m, n, k)
        assert need == (0 if m == 1 and not a_cols and not b_cols
                        else room(ra, ca) if one_off else room(rb, cb))


@pytest.mark.parametrize("m", [1, 2, 64, 300])
def test_operands_on_them(z, m):  # noqa: F811
    for a_cols, b_cols in itertools.product([False, True], repeat=2):
        sa, sb = (304 if a_cols else 72), (40 if b_cols else 72)
        assert z.zero_matmul_workspace(A, a_cols, sa, B, b_cols, sb, None, 0, None, 0, m, 40,
                                       72) == 0
        assert z.zero_matmul_workspace(A, a_cols, sa, B, b_cols, sb, C, sa, B, sb, m, 40, 72) == 0


@pytest.mark.parametrize("m", [1, 2, 64, 300])
def test_a_gated_block(z, m):  # noqa: F811
    need = z.zero_gated_workspace(A + 2, 73, B, 73, C, 72, m, 40, 72)
    assert need == (0 if m == 1 else room(m, 72) + room(40, 72))
