"""Sliding windows over caches whose pages before the window were given back: what lies before the first
token that a sequence's rows see is not used, and its page table entries are not looked at."""
import numpy as np
import pytest

import block_ref as ref
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


def give_back(c, window, how):
    """Page table entries and codes before the window as a scheduler may leave them."""
    spare = np.setdiff1d(np.arange(c.codes["k"].shape[0]), c.table)         # nan codes, nan scales
    for s, (L, n) in enumerate(c.seqs):
        first = max(0, L - n - window + 1)                                  # first token that a row sees
        for i in range(first // c.P):
            c.table[s, i] = {"missing": -1, "past the end": 1 << 30, "stale": spare[i % len(spare)]}[how]
        page, tokens = c.table[s, first // c.P], first % c.P
        if L > first and tokens:
            for kind in "kv":
                c.codes[kind][page, :, :tokens] = 0x7F


def check(c, window, how):
    want, bound = c.reference(window)
    give_back(c, window, how)
    c.gpu()
    for _ in range(2):
        got = ref.bf16_bits_to_f64(c.run(window)).reshape(c.T, c.Hq, c.D)   # (and no status bit)
        assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("how", ["missing", "past the end", "stale"])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_pages_before_the_window(D, P, how):
    for window in (1, 50, 333):
        check(Case([(400, 1), (400, 200), (90, 90), (777, 3), (1500, 130)], 12, 3, D, P), window, how)
        check(Case([(400, 1), (777, 3), (1500, 4), (64, 1)], 12, 3, D, P), window, how)


@pytest.mark.parametrize("how", ["missing", "stale"])
def test_pages_before_the_window_of_many_sequences(how):
    check(Case([(int(L), 1) for L in np.random.default_rng(3).integers(1, 700, 130)], 8, 2, 64, 16), 75, how)


@pytest.mark.parametrize("how", ["missing", "stale"])
def test_pages_before_the_window_of_cut_sequences(how):
    check(Case([(9000, 1)], 8, 1, 128, 16), 4001, how)
    check(Case([(4100, 64)], 32, 4, 128, 16), 2001, how)
    check(Case([(1030, 17), (6000, 33), (40, 40)], 8, 2, 128, 16), 1801, how)


def test_pages_before_the_window_of_blocks_of_256_rows():
    check(Case([(450, 150)] * 6, 64, 32, 64, 16), 70, "stale")
