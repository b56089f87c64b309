"""Attention over pages whose scales differ by more than f16 holds: a row's result goes by the tokens that
it sees and by their weights, not by the largest page that the kernel reads beside them."""
import numpy as np
import pytest

import block_ref as ref
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu

LOG2E = 1 / np.log(2)


def reference(c, window=0):
    """The output in 64 bits and the bound on a bf16 result's error, by the tokens that a row sees.
    A weight is rounded to f16: 2^-11 of itself, or 2^-25 of the row's largest weight times page scale (and
    there times a code). Its exponent, a fp32 sum of D products plus the logarithms of weight and scale, is
    off by 16 units of the last place of their magnitudes. The output is rounded to bf16."""
    T, Hq, D, P = c.T, c.Hq, c.D, c.P
    G = Hq // c.Hkv
    q = ref.bf16_bits_to_f64(c.q_bits).reshape(T, Hq, D)
    out, bound = np.zeros_like(q), np.zeros_like(q)
    at = 0
    for s, (L, n) in enumerate(c.seqs):
        pages = np.asarray(c.table[s][:-(-L // P)], dtype=np.int64)
        for h in range(c.Hkv if n and L else 0):
            codes = {x: ref.E4M3[c.codes[x][pages, h]].reshape(-1, D)[:L] for x in "kv"}
            sc = {x: np.repeat(c.scales[x][pages, h].astype(np.float64), P)[:L] for x in "kv"}
            k, v = (codes[x] * sc[x][:, None] for x in "kv")
            lv = np.log2(sc["v"])
            for i in range(n):
                pos = L - n + i
                lo = max(0, pos - window + 1) if window else 0
                see = slice(lo, pos + 1)
                if pos < lo:
                    continue
                for g in range(G):
                    x = q[at + i, h * G + g]
                    t = k[see] @ x * c.scale
                    mag = np.abs(k[see]) @ np.abs(x) * abs(c.scale)
                    top = t.max()
                    p = np.exp(t - top)
                    l = p.sum()
                    o = p @ v[see] / l
                    rel = 2.0 ** -11 + 2.0 ** -21 + 16 * ref.U32 * (mag + np.abs(t) + abs(top) + 2 * np.abs(lv[see]).max())
                    b = ((p * rel) @ np.abs(v[see]) + np.abs(o) * (p * rel).sum()) / l
                    b = b + 2.0 ** -25 * (p * sc["v"][see]).max() * np.abs(codes["v"][see]).sum(0) / l
                    out[at + i, h * G + g] = o
                    bound[at + i, h * G + g] = b + ref.half_ulp_bf16(np.abs(o) + b)
        at += n
    return out, bound


def check(c, window=0):
    want, bound = reference(c, window)
    got = ref.bf16_bits_to_f64(c.gpu().run(window)).reshape(want.shape)
    worst = (np.abs(got - want) / np.maximum(bound, 1e-300)).max()
    print(f"worst error / bound {worst:.3f}")
    assert worst <= 1


# every way through the kernels: one row, a few rows, many sequences, blocks of 128 and 256 rows, units that are cut
SHAPES = {"one row": ([(300, 1)], 4, 1), "few rows": ([(300, 4), (90, 2)], 8, 2),
          "many": ([(200, 1)] * 60, 8, 4), "prompt": ([(300, 150)], 4, 2), "prompts": ([(150, 150)] * 5, 64, 32),
          "cut": ([(1700, 40)], 16, 2), "long": ([(3000, 1)], 8, 1)}


def shape(name, D, P):
    seqs, Hq, Hkv = SHAPES[name]
    return Case(seqs, Hq, Hkv, D, P, seed=3, spread=1)


@pytest.mark.parametrize("up", [20, 40])
@pytest.mark.parametrize("kind", ["k", "v"])
@pytest.mark.parametrize("name", ["few rows", "prompt", "prompts", "cut"])
def test_a_large_page_that_earlier_rows_do_not_see(name, kind, up):
    """The last page's scale is 2^up times the others'."""
    c = shape(name, 64, 16)
    for s, (L, n) in enumerate(c.seqs):
        if n > 1:
            c.scales[kind][c.table[s, (L - 1) // 16]] *= np.float32(2.0 ** up)
            if kind == "k":     # small scores all the same: its rows are compared too
                c.codes["k"][c.table[s, (L - 1) // 16]] = 0
    check(c)


@pytest.mark.parametrize("kind", ["k", "v"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", ["one row", "few rows", "many", "prompt", "long"])
def test_a_large_page_before_the_window(name, D, kind):
    c = shape(name, D, 16)
    for s, (L, n) in enumerate(c.seqs):
        first = max(0, L - n - 40)                       # (window 41: the first token that a row sees)
        if first >= 16:
            c.scales[kind][c.table[s, first // 16 - 1]] *= np.float32(2.0 ** 30)
    check(c, 41)


@pytest.mark.parametrize("page", [0, 4, -1])
@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("D,P", [(64, 16), (128, 32), (128, 64)])
def test_a_large_page_of_negligible_weight(name, D, P, page):
    """V of one page is 2^25 times the others', and its tokens' weights e^-60: below 2^-60."""
    c = shape(name, D, P)
    q = np.abs(ref.bf16_bits_to_f64(c.q_bits)) + 0.5
    from workloads import gen
    c.q_bits = gen.f32_to_bf16_bits(q.astype(np.float32))
    for s, (L, n) in enumerate(c.seqs):
        p = c.table[s, page % (-(-L // P))]
        if L <= P or (page == -1 and n > 1):             # (rows that see that page alone are another matter)
            p = c.table[s, 0]
        c.scales["v"][p] *= np.float32(2.0 ** 25)
        c.codes["k"][p] = 0xB8 + 0x30                    # -64 everywhere
        c.scales["k"][p] = np.float32(2.0 ** -1)
    c.scale = 0.06
    check(c)


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("D,P", [(64, 16), (128, 16), (128, 64)])
def test_pages_of_alternating_size(name, D, P):
    """Neighbouring pages 2^18 apart in V, and 2^9 in K, of like weights."""
    c = shape(name, D, P)
    for s, (L, _) in enumerate(c.seqs):
        for i in range(-(-L // P)):
            c.scales["v"][c.table[s, i]] *= np.float32(2.0 ** (18 if i % 2 else 0))
            c.scales["k"][c.table[s, i]] *= np.float32(2.0 ** (-9 if i % 3 else 0))
    check(c)


@pytest.mark.parametrize("big", [0, 30, 60])
@pytest.mark.parametrize("name", list(SHAPES))
def test_pages_of_zeros_keep_their_weight(name, big):
    """Zeros have the smallest scale there is, 2^-100, and their tokens count in the sum of the weights as
    others do, whatever the size of the values beside them."""
    c = shape(name, 64, 16)
    for s, (L, _) in enumerate(c.seqs):
        for i in range(-(-L // 16)):
            p = c.table[s, i]
            if i % 3 == 1:
                c.codes["v"][p] = 0
                c.scales["v"][p] = np.float32(2.0 ** -100)
            else:
                c.scales["v"][p] *= np.float32(2.0 ** big)
    check(c)


@pytest.mark.parametrize("name", list(SHAPES))
def test_scales_that_are_no_powers_of_two(name):
    """The cache's own append writes powers of two; any positive scales are read."""
    c = shape(name, 128, 32)
    rng = np.random.default_rng(5)
    for kind in "kv":
        c.scales[kind] *= rng.uniform(0.3, 3.0, c.scales[kind].shape).astype(np.float32)
    check(c)


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("n", [3, 150])
def test_a_scale_that_is_not_finite_reaches_the_rows_that_see_it(n, P, value):
    """The K scale of a sequence's last page: nan for the rows that see a token of it, nothing for others."""
    L = 400
    c = Case([(L, n), (200, n)], 8, 2, 64, P)
    want, bound = reference(c)
    last = (L - 1) // P
    c.scales["k"][c.table[0, last], 1] = value
    got = ref.bf16_bits_to_f64(c.gpu().run()).reshape(want.shape)
    hit = np.zeros(want.shape[:2], dtype=bool)
    hit[:n, 4:] = (np.arange(L - n, L) >= last * P)[:, None]
    assert np.isnan(got[hit]).all() and hit.any()
    assert (np.abs(got - want) <= bound)[~hit].all()


@pytest.mark.parametrize("zeros_first", [False, True])
@pytest.mark.parametrize("big", [0, 30, 60, 110])
@pytest.mark.parametrize("name", list(SHAPES))
def test_long_stretches_of_zeros(name, big, zeros_first):
    """Zeros over many pages in a row, so that a warp, a piece or a block meets nothing else for a while, beside values
    as large as bf16 holds."""
    c = shape(name, 64, 16)
    for s, (L, _) in enumerate(c.seqs):
        pages = -(-L // 16)
        for i in range(pages):
            p = c.table[s, i]
            if (i < pages // 2) == zeros_first:
                c.codes["v"][p] = 0
                c.scales["v"][p] = np.float32(2.0 ** -100)
            else:
                c.scales["v"][p] *= np.float32(2.0 ** big)
    check(c)


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("P", [16, 64])
def test_values_at_both_ends_of_the_range(name, P):
    """Pages of 2^-90, 1 and 2^110 times the usual values, of like weights."""
    c = shape(name, 128, P)
    for s, (L, _) in enumerate(c.seqs):
        for i in range(-(-L // P)):
            c.scales["v"][c.table[s, i]] *= np.float32(2.0 ** (-90, 0, 110)[i * 7 // 3 % 3])
    check(c)


@pytest.mark.parametrize("name", ["few rows", "prompt", "many"])
def test_a_missing_page_beside_huge_values(name):
    """Its tokens count as unseen, whatever the others' scales."""
    import int4_grouped_expert_gb300 as st
    c = shape(name, 64, 16)
    for kind in "v":
        c.scales[kind] *= np.float32(2.0 ** 100)
    c.codes["k"][c.table[0, 3]] = 0xFE                   # (as good as unseen: the largest key, against every query)
    from workloads import gen
    c.q_bits = gen.f32_to_bf16_bits((np.abs(ref.bf16_bits_to_f64(c.q_bits)) + 0.5).astype(np.float32))
    c.scales["k"][c.table[0, 3]] = np.float32(2.0 ** 4)
    want, bound = reference(c)
    c.table[0, 3] = -1
    got = ref.bf16_bits_to_f64(c.gpu().run(expect_status=st.STRATA_DEV_BAD_SLOT)).reshape(want.shape)
    assert (np.abs(got - want) <= bound).all()
