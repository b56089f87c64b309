"""Attention over the paged 8-bit cache against the 64-bit softmax (block_ref.attention states the
bound)."""
import numpy as np
import pytest

import block_ref as ref
from helpers import bf16_tensor, bf16_to_np_bits
from workloads import gen

pytestmark = pytest.mark.gpu


class Case:
    """Sequences [(tokens in the cache, query rows)] over shuffled pages. Pages that no sequence owns,
    and slots past a sequence's length, hold nan codes and (whole pages) nan scales; table entries
    past the last page are out of range."""

    def __init__(self, seqs, Hq, Hkv, D, P, seed=0, spread=2, q_scale=1.5, n_spare=2, extra_cols=3):
        rng = np.random.default_rng([seed, Hq, Hkv, D, P, len(seqs)])
        self.seqs, self.Hq, self.Hkv, self.D, self.P = seqs, Hq, Hkv, D, P
        need = [-(-L // P) for L, _ in seqs]
        n_pages = sum(need) + n_spare
        order = rng.permutation(n_pages)
        cols = max(need + [0]) + extra_cols
        self.table = np.full((len(seqs), cols), -123456, dtype=np.int32)
        self.table[:, cols // 2 + 1:] = 1 << 30
        codes = {k: np.full((n_pages, Hkv, P, D), 0x7F, dtype=np.uint8) for k in "kv"}
        scales = {k: np.full((n_pages, Hkv), np.nan, dtype=np.float32) for k in "kv"}
        at = 0
        for s, (L, _) in enumerate(seqs):
            for i in range(need[s]):
                p = order[at]
                at += 1
                self.table[s, i] = p
                n = min(P, L - i * P)
                for kind in "kv":
                    c = rng.integers(0, 256, (Hkv, n, D), dtype=np.uint8)
                    c[(c & 0x7F) == 0x7F] = 0x35                           # no nan among the tokens
                    big = (c & 0x7F) > 0x68                                # |code| > 64: few of them
                    c[big & (rng.random(c.shape) < 0.8)] ^= 0x30
                    codes[kind][p, :, :n] = c
                    scales[kind][p] = np.exp2(rng.integers(-5 - spread, -4 + spread, Hkv)).astype(np.float32)
        self.codes, self.scales = codes, scales
        self.T = sum(n for _, n in seqs)
        self.q_bits = gen.f32_to_bf16_bits(
            rng.standard_normal((self.T, Hq * D), dtype=np.float32) * np.float32(q_scale))
        self.scale = 0.25 / np.sqrt(D)

    def gpu(self):
        import torch
        import int4_grouped_expert_gb300 as st
        t = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.cache = st.PagedKVCache(self.codes["k"].shape[0], self.Hkv, self.D, self.P, t(self.codes["k"]),
                                     t(self.codes["v"]), t(self.scales["k"]), t(self.scales["v"]))
        start = np.cumsum([0] + [n for _, n in self.seqs]).astype(np.int32)
        self.q = bf16_tensor(self.q_bits)
        max_q, max_kv = max(n for _, n in self.seqs), max(L for L, _ in self.seqs)
        self.batch = st.kv_batch(t(start), t(np.array([L for L, _ in self.seqs], dtype=np.int32)), t(self.table),
                                 self.T, max_q, max_kv)
        return self

    def run(self, window=0, flags=0, ws=None, expect_status=0, q_stride=None, q=None):
        import torch
        import int4_grouped_expert_gb300 as st
        out = torch.full((self.T + 1, self.Hq * self.D), -7.0, dtype=torch.bfloat16, device="cuda")
        need = st.strata_attention_workspace_size(self.cache.struct(), self.batch, self.Hq)
        if ws is None:
            ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
        st.check(st.strata_attention_forward(self.cache.struct(), self.batch, self.q if q is None else q, self.Hq,
                                             self.scale, out, ws, ws.numel(), window=window, flags=flags,
                                             q_stride=q_stride), "strata_attention_forward")
        torch.cuda.synchronize()
        rc, bits = st.strata_workspace_status(ws)
        assert bits == expect_status, hex(bits)
        assert (out[self.T] == -7).all()
        return bf16_to_np_bits(out[:self.T])

    def reference(self, window=0):
        c = ref.Cache(self.codes["k"], self.codes["v"], self.scales["k"], self.scales["v"])
        q = ref.bf16_bits_to_f64(self.q_bits).reshape(self.T, self.Hq, self.D)
        return ref.attention(q, c, self.table, self.seqs, self.P, self.scale, window)

    def check(self, window=0, **kw):
        got = ref.bf16_bits_to_f64(self.run(window, **kw)).reshape(self.T, self.Hq, self.D)
        want, bound = self.reference(window)
        assert np.isfinite(want).all()
        worst = (np.abs(got - want) / np.maximum(bound, 1e-300)).max() if got.size else 0.0
        print(f"worst error / bound {worst:.3f}")
        assert (np.abs(got - want) <= bound).all()


HEADS = [(1, 1), (8, 8), (8, 1), (4, 1), (7, 1), (6, 2), (16, 1), (40, 2), (64, 4)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_single_tokens(Hq, Hkv, D):
    Case([(L, 1) for L in (1, 2, 15, 16, 17, 63, 64, 65, 300, 777)], Hq, Hkv, D, 64).gpu().check()


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_page_sizes(P, D):
    Case([(1000, 1), (P, 1), (P + 1, 2), (3 * P - 1, 5)], 8, 2, D, P).gpu().check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [2, 3, 8, 31, 32, 33, 127, 128, 129, 300])
def test_rows_per_sequence(n, D):
    Case([(n, n), (n + 70, n), (500 + n, n)], 8, 2, D, 32).gpu().check()


@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_prompt_pieces_with_every_head_ratio(Hq, Hkv):
    Case([(150, 150), (210, 61)], Hq, Hkv, 128, 64).gpu().check()
    Case([(150, 150), (210, 61)], Hq, Hkv, 64, 16).gpu().check()


@pytest.mark.parametrize("window", [1, 2, 16, 50, 333, 100000])
@pytest.mark.parametrize("D", [64, 128])
def test_windows(window, D):
    Case([(1, 1), (400, 1), (400, 200), (90, 90), (777, 3)], 12, 3, D, 16).gpu().check(window)


def test_mixed_lengths_and_empty_sequences():
    seqs = [(0, 0), (5, 0), (700, 1), (40, 40), (0, 0), (2000, 300), (1, 1), (129, 128), (0, 0)]
    Case(seqs, 8, 2, 128, 64).gpu().check()
    Case(seqs, 6, 2, 64, 16).gpu().check(100)


@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_nothing_are_zero(D):
    """No tokens in the cache, and more rows than tokens: the first rows stand before the first token."""
    c = Case([(0, 3), (2, 9), (10, 200), (0, 150), (300, 1)], 8, 2, D, 16).gpu()
    got = ref.bf16_bits_to_f64(c.run()).reshape(c.T, 8, D)
    want, bound = c.reference()
    assert (np.abs(got - want) <= bound).all()
    assert (got[:3] == 0).all() and (got[3:10] == 0).all() and (got[12:202] == 0).all()


@pytest.mark.parametrize("seqs", [[(9000, 1)], [(9000, 1), (3, 1), (2500, 1)], [(5000, 40)], [(6000, 200)]])
@pytest.mark.parametrize("D", [64, 128])
def test_long_caches_are_split_and_joined(seqs, D):
    Case(seqs, 8, 1, D, 128).gpu().check()
    Case(seqs, 8, 1, D, 16).gpu().check(window=4000)


def test_scales_far_apart():
    """Pages whose K or V scales differ by up to 2^20, and a page of zeros with the smallest scale."""
    c = Case([(600, 1), (600, 150)], 4, 2, 128, 32, spread=10, q_scale=0.05)
    for kind in "kv":
        p = c.table[0, 1]
        c.codes[kind][p] = 0
        c.scales[kind][p] = np.float32(2.0 ** -100)
    c.gpu().check()


@pytest.mark.parametrize("exponent", [-60, -12, 20, 60])
def test_queries_of_any_size(exponent):
    c = Case([(200, 1), (200, 140)], 8, 2, 64, 32)
    c.q_bits = gen.f32_to_bf16_bits(ref.bf16_bits_to_f64(c.q_bits).astype(np.float32) * np.float32(2.0 ** exponent))
    c.scale *= 2.0 ** -exponent
    c.gpu().check()


def test_a_sharp_softmax():
    """One score far above the others: the output is that token's value."""
    Case([(500, 1), (500, 130)], 8, 2, 128, 64, q_scale=30).gpu().check()


def test_negative_scale_and_zero_scale():
    for scale in (-0.05, 0.0):
        c = Case([(300, 1), (140, 140)], 4, 2, 64, 32).gpu()
        c.scale = scale
        c.check()


@pytest.mark.parametrize("n", [3, 150])
def test_nan_reaches_exactly_the_rows_that_see_it(n):
    """A token with nan keys and zero values, as the append marks one that was not finite."""
    L, at = 400, 399 - n // 2
    c = Case([(L, n), (L, n)], 8, 2, 64, 16)
    page = c.table[0, at // 16]
    c.codes["k"][page, 1, at % 16] = 0x7F
    c.codes["v"][page, 1, at % 16] = 0
    got = ref.bf16_bits_to_f64(c.gpu().run()).reshape(c.T, 8, 64)
    hit = np.zeros((c.T, 8), dtype=bool)
    hit[:n][np.arange(L - n, L) >= at, 4:] = True
    assert np.isnan(got[hit]).all()
    c.codes["k"][page, 1, at % 16] = 0
    want, bound = c.reference()
    assert (np.abs(got - want) <= bound)[~hit].all()


def test_bad_descriptions_are_flagged_and_cut():
    import torch
    import int4_grouped_expert_gb300 as st
    c = Case([(300, 1), (200, 20)], 4, 2, 64, 16).gpu()
    c.check()
    whole = c.run()
    # a page that does not exist: its tokens count as unseen
    for bad in (-1, c.codes["k"].shape[0], 1 << 30):
        t = torch.from_numpy(c.table).cuda()
        t[0, 3] = bad
        b = st.kv_batch(c.batch.tensors[0], c.batch.tensors[1], t, c.T, 20, 300)
        keep, c.batch = c.batch, b
        got = ref.bf16_bits_to_f64(c.run(expect_status=st.STRATA_DEV_BAD_SLOT))
        c.batch = keep
        seen = np.r_[0:48, 64:300]
        q = ref.bf16_bits_to_f64(c.q_bits)[0].reshape(4, 64)
        for h in range(4):
            k, v = [(ref.E4M3[c.codes[n][c.table[0, :19], h // 2]] *
                     c.scales[n][c.table[0, :19], h // 2].astype(np.float64)[:, None, None]).reshape(-1, 64)[seen]
                    for n in "kv"]
            w = np.exp(k @ q[h] * c.scale)
            o = w @ v / w.sum()
            assert np.abs(got[0].reshape(4, 64)[h] - o).max() < 2e-2 * np.abs(v).max()
    # row ranges and lengths outside the limits: nothing outside q and out is touched
    for start, lens in (([0, 5, 1 << 30], [300, 200]), ([-4, 1, 21], [300, 200]), ([0, 30, 21], [300, 200]),
                        ([0, 1, 21], [-5, 200]), ([0, 1, 21], [1 << 30, 200])):
        t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        keep, c.batch = c.batch, st.kv_batch(t(start), t(lens), c.batch.tensors[2], c.T, 20, 300)
        c.run(expect_status=st.STRATA_DEV_BAD_SLOT)
        c.batch = keep
    assert np.array_equal(c.run(), whole)


@pytest.mark.parametrize("seqs", [[(9000, 1), (100, 1)], [(3000, 90)], [(700, 1), (300, 130)]])
def test_a_kept_workspace_gives_the_same_bits(seqs):
    import torch
    import int4_grouped_expert_gb300 as st
    c = Case(seqs, 8, 2, 128, 64).gpu()
    first = c.run()
    need = st.strata_attention_workspace_size(c.cache.struct(), c.batch, 8)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for _ in range(20):
        assert np.array_equal(c.run(flags=st.STRATA_WS_REUSE, ws=ws), first)


def test_strided_queries_and_another_stream():
    import torch
    import int4_grouped_expert_gb300 as st
    c = Case([(300, 1), (200, 33)], 8, 2, 64, 32).gpu()
    want = c.run()
    wide = torch.full((c.T, 8 * 64 + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :512] = c.q
    assert np.array_equal(c.run(q=wide, q_stride=536), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert np.array_equal(c.run(), want)


def test_limits_above_the_lengths():
    """max_q, max_kv and T may be larger than what the call holds, as in a captured graph."""
    import torch
    import int4_grouped_expert_gb300 as st
    c = Case([(300, 1), (77, 1)], 8, 2, 128, 64, extra_cols=200).gpu()
    t = c.batch.tensors
    for max_q, max_kv in ((1, 9000), (5, 300), (64, 13000)):
        keep, c.batch = c.batch, st.kv_batch(*t, c.T, max_q, max_kv)
        c.check()
        c.batch = keep


def test_a_cache_of_more_than_4_gb():
    """Pages whose codes lie past 2^32 bytes from the start of the cache (and element counts past 2^31)."""
    import torch
    import int4_grouped_expert_gb300 as st
    Hkv, D, P = 8, 128, 128
    n_pages = (9 << 30) // (2 * Hkv * D * P)                              # 4.5 GB each of K and V
    small = Case([(500, 1), (200, 40)], 16, Hkv, D, P).gpu()
    want = small.run()
    big = st.PagedKVCache(n_pages, Hkv, D, P)
    n = small.codes["k"].shape[0]
    shift = n_pages - n
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        dst, src = getattr(big, name), getattr(small.cache, name)
        dst.view(torch.uint8 if "codes" in name else dst.dtype)[shift:] = src
    table = small.batch.tensors[2]
    table = torch.where((table >= 0) & (table < n), table + shift, table)
    small.cache = big
    small.batch = st.kv_batch(small.batch.tensors[0], small.batch.tensors[1], table, small.T, 40, 500)
    assert np.array_equal(small.run(), want)
    # and an append up there, read back
    k = torch.randn(2, Hkv * D, device="cuda").bfloat16()
    slots = torch.tensor([(n_pages - 1) * P, (n_pages - 1) * P + 1], dtype=torch.int32, device="cuda")
    st.check(st.strata_kv_append(big.struct(), k, k, 2, slots), "append")
    got = big.k_codes[-1, :, :2].float() * big.k_scales[-1][:, None, None]
    x = k.view(2, Hkv, D).transpose(0, 1).float()
    assert ((got - x).abs() <= x.abs() / 16 + big.k_scales[-1][:, None, None] * 2.0 ** -10).all()


def many(n, seed, longest, rows=1):
    """Lengths of n sequences: some empty, some without queries, a few long ones."""
    rng = np.random.default_rng(seed)
    seqs = [(int(L), int(q)) for L, q in zip(rng.integers(1, 260, n), rng.integers(1, rows + 1, n))]
    for i in range(0, n, 7):
        seqs[i] = (seqs[i][0], 0) if i % 2 else (0, 1)
    for i, L in enumerate((longest, longest // 2 + 1, 32, 33, 31)):
        seqs[(i * 17 + 3) % n] = (L, 1)
    return seqs


@pytest.mark.parametrize("window", [0, 75])
@pytest.mark.parametrize("n,Hq,Hkv,D,rows", [(60, 16, 4, 128, 1), (60, 64, 4, 128, 1), (300, 2, 1, 64, 1),
                                             (1100, 1, 1, 64, 1), (58, 32, 8, 64, 4), (77, 6, 3, 128, 3)])
def test_many_sequences(n, Hq, Hkv, D, rows, window):
    """More pairs of sequence and head than blocks that run at once: warps go from pair to pair, and
    the long sequences are cut over many of them."""
    Case(many(n, 5, 6000, rows), Hq, Hkv, D, 32).gpu().check(window)


def test_many_equal_sequences():
    Case([(96, 1)] * 64, 32, 8, 128, 32).gpu().check()
    Case([(1, 1)] * 230, 2, 1, 64, 16).gpu().check()


@pytest.mark.parametrize("n", [2, 9, 20, 33, 57])
def test_pairs_that_do_not_fill_the_blocks_evenly(n):
    Case([(1500, 1)] * n, 8, 4, 64, 64).gpu().check()


def test_many_sequences_beside_prompts():
    Case(many(130, 6, 2000) + [(700, 300), (90, 90)], 8, 2, 128, 64).gpu().check()


def test_many_sequences_with_a_kept_workspace_give_the_same_bits():
    import torch
    import int4_grouped_expert_gb300 as st
    c = Case(many(90, 7, 9000), 12, 3, 128, 64).gpu()
    first = c.run()
    ws = torch.zeros(st.strata_attention_workspace_size(c.cache.struct(), c.batch, c.Hq), dtype=torch.uint8,
                     device="cuda")
    c.run(ws=ws)
    for _ in range(4):
        assert (c.run(ws=ws, flags=st.STRATA_WS_REUSE) == first).all()


def test_many_sequences_with_pages_that_do_not_exist():
    """A page number out of range is flagged and its tokens count as unseen, whatever warp meets it."""
    import int4_grouped_expert_gb300 as st
    c = Case([(200, 1)] * 120, 4, 2, 64, 32)
    want, bound = c.reference()
    c.table[50, 2] = -5
    c.gpu()
    got = ref.bf16_bits_to_f64(c.run(expect_status=st.STRATA_DEV_BAD_SLOT)).reshape(c.T, c.Hq, c.D)
    others = np.arange(c.T) != 50
    assert (np.abs(got - want) <= bound)[others].all()
    assert np.isfinite(got[50]).all()


def test_a_kept_workspace_serves_batches_of_other_shapes():
    """What one call leaves in the workspace is clean for the next, whatever its lengths, heads and rows."""
    import torch
    import int4_grouped_expert_gb300 as st
    cases = [Case([(20000, 1)], 8, 2, 128, 64), Case(many(90, 7, 5000), 12, 3, 128, 64),
             Case([(3000, 1)] * 40, 16, 2, 64, 32), Case([(2000, 300), (900, 1)], 8, 2, 128, 64),
             Case([(5000, 2)] * 3, 64, 4, 64, 16), Case([(6000, 70)], 8, 1, 128, 64)]
    cases = [c.gpu() for c in cases]
    first = [c.run() for c in cases]
    size = max(st.strata_attention_workspace_size(c.cache.struct(), c.batch, c.Hq) for c in cases)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for i in (0, 1, 2, 3, 4, 5, 1, 0, 3, 2, 5, 4, 1, 5, 0):
        assert (cases[i].run(ws=ws, flags=st.STRATA_WS_REUSE) == first[i]).all(), i


@pytest.mark.parametrize("seqs,Hq,Hkv,D,window", [
    ([(4100, 64)], 32, 4, 128, 0),                       # few units: pieces of each
    ([(4100, 64)], 32, 4, 128, 2000),
    ([(2600, 300)], 8, 8, 64, 0),
    ([(1030, 17), (6000, 33), (40, 40)], 8, 2, 128, 0),  # units too short for as many pieces as others
    ([(1030, 17), (6000, 33), (40, 40)], 8, 2, 128, 1800),
    ([(3000, 300), (9, 9), (2222, 1)], 28, 4, 64, 0),
    ([(1560, 620)], 64, 32, 64, 0),                      # 160 units: the last ones are cut
    ([(1600, 450)], 64, 2, 64, 0),
])
def test_units_cut_along_the_tokens(seqs, Hq, Hkv, D, window):
    Case(seqs, Hq, Hkv, D, 64).gpu().check(window)


def test_one_long_prompt_among_many_single_rows():
    """Blocks by the longest sequence would mostly be empty: they find their units in the lengths."""
    Case([(500, 400)] + [(300, 1)] * 40, 8, 2, 64, 32).gpu().check()


def test_nan_in_one_piece_of_a_cut_unit():
    c = Case([(4100, 40)], 16, 2, 128, 64)
    c.codes["v"][c.table[0, 20], 1, 5, :] = 0x7F
    c.codes["k"][c.table[0, 40], 0, 7, :] = 0x7F
    c.gpu()
    got = ref.bf16_bits_to_f64(c.run()).reshape(c.T, 16, 128)
    assert np.isnan(got).all()          # every row sees both tokens: a head's K, the other's V


@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("seqs,Hq,Hkv,D", [
    ([(150, 150)] * 6, 64, 32, 64),                 # 300 rows a head: a block of 256 and one of 44
    ([(300, 200), (129, 129), (70, 1), (256, 256)], 40, 40, 128),
    ([(190, 64)] * 3, 96, 24, 128),                 # exactly 256 rows
])
def test_blocks_of_two_row_tiles(seqs, Hq, Hkv, D, window):
    """Enough units of 128 rows to fill the GPU: a block takes 256."""
    Case(seqs, Hq, Hkv, D, 32).gpu().check(window)
