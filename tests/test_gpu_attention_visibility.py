"""Attention where the first rows of a sequence see nothing: rows before its first token, and what a
block of such rows may write."""
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
