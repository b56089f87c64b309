"""Cuts after pages before the window were given back, as a server makes them that takes back rejected drafts."""
import numpy as np
import pytest

import pages_ref
from test_gpu_kv_pages import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P,window,sinks,most", [(16, 1, 0, 5), (16, 40, 5, 7), (32, 33, 32, 40), (16, 16, 17, 1), (64, 300, 0, 90)])
def test_a_window_larger_by_the_cut_keeps_what_the_next_query_sees(P, window, sinks, most):
    """Sequences go back by up to `most` tokens from the longest that they were released at: a release with that many tokens
    more gives back none that will be seen."""
    rng = np.random.default_rng([P, window])
    p = Pool(200, 3, 40, P)
    longest = np.zeros(3, dtype=np.int64)
    for _ in range(40):
        p.extend(rng.integers(1, most + 2, 3) * (p.cpu.length + most + 1 < 40 * P))
        p.release(None, window + most, sinks)
        longest = np.maximum(longest, p.cpu.length)
        p.release(np.maximum(p.cpu.length - rng.integers(0, most + 1, 3), np.maximum(longest - most, 0)))
        table = p.gpu.page_table.cpu().numpy()
        for s, L in enumerate(p.cpu.length):
            pos = np.arange(L)
            seen = pos[(pos > L - window) | (pos < sinks)]  # by a query at position L, itself aside
            assert (table[s, seen // P] >= 0).all()


def test_a_cut_behind_the_window_is_flagged():
    p = Pool(20, 2, 10, 16)
    p.extend([40, 40])
    p.release(None, 16, 0)                 # page 0 goes: the next query sees tokens 25 on
    p.release([10, 39])
    assert (p.cpu.table[:, 0] == -1).all()
    _, status = p.extend([1, 1])           # the one that would go on inside page 0 gets nothing
    assert status == pages_ref.BAD_SLOT and list(p.cpu.length) == [10, 40]
