"""Attention where the first rows of a sequence see nothing: rows before its first token, what a block of
such rows may write, and windows longer than any sequence."""
import numpy as np
import pytest

import block_ref as ref
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (8, 2, 128), (8, 1, 64), (6, 2, 64)])
@pytest.mark.parametrize("n,L", [(300, 100), (200, 10), (64, 30), (129, 128), (257, 1), (200, 72), (400, 272)])
def test_blocks_of_empty_rows_leave_the_next_block_alone(n, L, Hq, Hkv, D):
    """The first row that sees a token stands anywhere inside a block of 128 rows. Enough sequences
    that blocks start in any order, several times: every run gives the same, right, rows."""
    c = Case([(L, n)] * 3 + [(L + 40, n)], Hq, Hkv, D, 16).gpu()
    first = c.run()
    got = ref.bf16_bits_to_f64(first).reshape(c.T, Hq, D)
    want, bound = c.reference()
    assert (np.abs(got - want) <= bound).all()
    assert (got[:n - L] == 0).all() and (np.abs(got[n - L:n]).max((1, 2)) > 0).all()
    for _ in range(5):
        assert np.array_equal(c.run(), first)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 100, 2 ** 30])
def test_windows_beyond_every_length(window):
    """As no window at all, where rows stand before the first token too."""
    for seqs in ([(0, 3), (2, 9), (10, 200), (0, 150), (300, 1)], [(2, 3), (0, 1), (50, 4)]):
        c = Case(seqs, 8, 2, 64, 16).gpu()
        whole = c.run()
        assert np.array_equal(c.run(window), whole)
        c.check(window)
