"""Attention with a window and first tokens that stay visible, against a 64-bit softmax over the tokens that a row sees.
What lies between the first tokens and the window holds nan, and the table's entries for pages wholly there
are not pages."""
import numpy as np
import pytest

import block_ref as ref
from helpers import bf16_to_np_bits
from test_gpu_attention import HEADS, Case

pytestmark = pytest.mark.gpu


def reference(c, window, sinks):
    """Output and the bound on a bf16 result's error. A weight is rounded to f16: 2^-11 of itself, or 2^-25 of the row's
    largest weight times page scale (and there times a code). Its exponent, a fp32 sum of D products plus the
    logarithms of weight and scale, is off by 16 units of the last place of their magnitudes. The output is rounded
    to bf16."""
    T, Hq, D, P, G = c.T, c.Hq, c.D, c.P, c.Hq // c.Hkv
    q = ref.bf16_bits_to_f64(c.q_bits).reshape(T, Hq, D)
    out, bound = np.zeros_like(q), np.zeros_like(q)
    at = 0
    for s, (L, n) in enumerate(c.seqs):
        first = max(0, L - n - window + 1)
        tok = np.r_[0:min(first, sinks, L), first:L].astype(np.int64)
        pos = L - n + np.arange(n)
        far = pos[:, None] - tok[None]
        sees = (far >= 0) & ((far < window) | (tok[None] < sinks))
        page, off = c.table[s][tok // P], tok % P
        for h in range(c.Hkv if n and len(tok) else 0):
            heads = slice(h * G, (h + 1) * G)
            sc = {x: c.scales[x][page, h].astype(np.float64)[:, None] for x in "kv"}
            k, vc = (ref.E4M3[c.codes[x][page, h, off]] for x in "kv")
            k, v = k * sc["k"], vc * sc["v"]
            x = q[at:at + n, heads]
            t = np.where(sees[:, None], np.einsum("ngd,ld->ngl", x, k) * c.scale, -np.inf)
            mag = np.einsum("ngd,ld->ngl", np.abs(x), np.abs(k)) * abs(c.scale)
            top = t.max(-1, keepdims=True)
            top = np.where(np.isfinite(top), top, 0.0)
            p = np.exp(t - top)
            l = p.sum(-1, keepdims=True)
            l = np.where(l == 0, 1.0, l)
            o = np.einsum("ngl,ld->ngd", p, v) / l
            lv = np.where(sees, np.abs(np.log2(sc["v"][:, 0]))[None], 0).max(-1)[:, None, None]
            rel = 2.0 ** -11 + 2.0 ** -21 + 16 * ref.U32 * (mag + np.abs(np.where(sees[:, None], t, 0)) + np.abs(top) + 2 * lv)
            pr = p * rel
            b = (np.einsum("ngl,ld->ngd", pr, np.abs(v)) + np.abs(o) * pr.sum(-1, keepdims=True)) / l
            most = (p * sc["v"][:, 0]).max(-1, keepdims=True)
            b = b + 2.0 ** -25 * most * np.einsum("nl,ld->nd", sees.astype(float), np.abs(vc))[:, None] / l
            out[at:at + n, heads] = o
            bound[at:at + n, heads] = b + ref.half_ulp_bf16(np.abs(o) + b)
        at += n
    return out, bound


def empty_the_gap(c, window, sinks, how=-1):
    """Between the first tokens and the window of each sequence's first row: no pages, and nan in the pages that are."""
    for s, (L, n) in enumerate(c.seqs):
        first = min(max(0, L - n - window + 1), L)
        for e in range(-(-L // c.P)):
            lo, hi = max(e * c.P, sinks), min((e + 1) * c.P, first)  # unseen tokens of the page
            if lo >= hi:
                continue
            if hi - lo == c.P:
                c.table[s, e] = how
                continue
            for kind in "kv":
                c.codes[kind][c.table[s, e], :, lo - e * c.P:hi - e * c.P] = 0x7F


class SinkCase(Case):
    def run(self, window, sinks, flags=0, ws=None, expect_status=0, out=None):
        import torch
        import int4_grouped_expert_gb300 as st
        out = torch.full((self.T + 1, self.Hq * self.D), -7.0, dtype=torch.bfloat16, device="cuda")
        need = st.strata_attention_workspace_size(self.cache.struct(), self.batch, self.Hq)
        if ws is None:
            ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
        st.check(st.strata_attention_sinks_forward(self.cache.struct(), self.batch, self.q, self.Hq, self.scale, out, ws,
                                                   ws.numel(), window=window, n_sinks=sinks, flags=flags),
                 "strata_attention_sinks_forward")
        torch.cuda.synchronize()
        assert st.strata_workspace_status(ws)[1] == expect_status
        assert (out[self.T] == -7).all()
        return bf16_to_np_bits(out[:self.T])

    def check(self, window, sinks, how=-1):
        empty_the_gap(self, window, sinks, how)
        got = ref.bf16_bits_to_f64(self.gpu().run(window, sinks)).reshape(self.T, self.Hq, self.D)
        want, bound = reference(self, window, sinks)
        assert np.isfinite(want).all()
        worst = (np.abs(got - want) / np.maximum(bound, 1e-300)).max()
        print(f"worst error / bound {worst:.3f}")
        assert worst <= 1


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_single_tokens(Hq, Hkv, D):
    SinkCase([(L, 1) for L in (1, 2, 15, 16, 17, 63, 64, 65, 300, 777)], Hq, Hkv, D, 64).check(50, 4)


@pytest.mark.parametrize("window", [1, 2, 16, 50, 333])
@pytest.mark.parametrize("sinks", [1, 4, 16, 31, 32, 33, 63, 64, 65, 200, 2 ** 31 - 1])
def test_windows_and_first_tokens(window, sinks):
    """One row, a few rows and prompts, first tokens that end in a step, at its end and past the window."""
    SinkCase([(1, 1), (400, 1), (400, 200), (90, 90), (777, 3)], 12, 3, 64, 16).check(window, sinks)
    SinkCase([(400, 1), (777, 3), (33, 1)], 12, 3, 128, 16, seed=1).check(window, sinks)
    SinkCase([(700, 100), (300, 300)], 8, 2, 128, 64, seed=2).check(window, sinks, how=1 << 30)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_page_sizes(P, D):
    SinkCase([(1000, 1), (P, 1), (P + 1, 2), (3 * P - 1, 5), (900, 70)], 8, 2, D, P).check(2 * P - 3, P // 2 + 1)
    SinkCase([(1000, 1), (P, 1), (P + 1, 2), (3 * P - 1, 2)], 8, 2, D, P).check(P, P)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [2, 3, 8, 31, 33, 127, 128, 129, 300])
def test_rows_per_sequence(n, D):
    SinkCase([(n, n), (n + 70, n), (500 + n, n)], 8, 2, D, 32).check(100, 7)


@pytest.mark.parametrize("D", [64, 128])
def test_many_sequences(D):
    """More pairs of sequence and head than blocks: a warp walks through several, some of them cut."""
    lens = np.random.default_rng(5).integers(1, 900, 130)
    SinkCase([(int(L), 1) for L in lens], 8, 2, D, 16).check(75, 40)
    SinkCase([(int(L), 1) for L in lens], 8, 4, D, 64).check(300, 3)
    SinkCase([(5000, 1)] + [(int(L), 1) for L in lens], 8, 2, D, 16).check(2500, 100)


@pytest.mark.parametrize("seqs,window,sinks", [
    ([(9000, 1)], 4001, 5), ([(9000, 1), (3, 1), (2500, 1)], 1000, 700), ([(5000, 40)], 2000, 300),
    ([(9000, 33)], 3000, 64), ([(1030, 17), (6000, 33), (40, 40)], 1801, 130), ([(20000, 2)], 9000, 9000)])
@pytest.mark.parametrize("P", [16, 128])
def test_long_caches_are_split_and_joined(seqs, window, sinks, P):
    SinkCase(seqs, 8, 1, 128, P).check(window, sinks)
    SinkCase(seqs, 32, 2, 64, P).check(window, sinks)


def test_blocks_of_256_rows():
    SinkCase([(450, 150)] * 6, 64, 32, 64, 16).check(70, 30)
    SinkCase([(1200, 300)] * 3, 32, 8, 128, 64).check(400, 130)


def test_mixed_lengths_and_empty_sequences():
    seqs = [(0, 0), (5, 0), (700, 1), (40, 40), (0, 0), (2000, 300), (1, 1), (129, 128), (0, 0)]
    SinkCase(seqs, 8, 2, 128, 64).check(90, 10)
    SinkCase(seqs, 6, 2, 64, 16).check(100, 20)


@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_nothing_are_zero(D):
    c = SinkCase([(0, 3), (2, 9), (10, 200), (0, 150), (300, 1)], 8, 2, D, 16).gpu()
    got = ref.bf16_bits_to_f64(c.run(20, 5)).reshape(c.T, 8, D)
    want, bound = reference(c, 20, 5)
    assert (np.abs(got - want) <= bound).all()
    assert (got[:3] == 0).all() and (got[3:10] == 0).all() and (got[12:202] == 0).all()


@pytest.mark.parametrize("seqs", [[(300, 1), (90, 2)], [(200, 1)] * 60, [(500, 150)], [(3000, 60)]])
def test_without_a_gap_it_is_the_plain_call(seqs):
    """No first tokens, no window, or a window that reaches them for every row: the same bits as strata_attention_forward."""
    c = SinkCase(seqs, 8, 4, 64, 16).gpu()
    most = max(L for L, _ in seqs)
    assert np.array_equal(c.run(70, 0), Case.run(c, window=70))
    assert np.array_equal(c.run(0, 9), Case.run(c))
    assert np.array_equal(c.run(most - 9, 9), Case.run(c))


@pytest.mark.parametrize("up", [-90, -30, 20, 40])
@pytest.mark.parametrize("kind", ["k", "v"])
@pytest.mark.parametrize("seqs", [[(300, 1), (90, 2)], [(250, 1)] * 60, [(500, 150)], [(3000, 60)]])
def test_first_tokens_of_another_size(seqs, kind, up):
    """The first page's scale is 2^up times the others': rows that give it no weight lose nothing, the others follow it."""
    c = SinkCase(seqs, 8, 4, 64, 16, spread=1, seed=7)
    for s in range(len(seqs)):
        c.scales[kind][c.table[s, 0]] *= np.float32(2.0 ** up)
        if kind == "k" and up > 0:  # (scores stay within reach)
            c.codes["k"][c.table[s, 0]] = 0x08 | (c.codes["k"][c.table[s, 0]] & 0x80)
    if kind == "k" and up > 0:
        c.scale *= 2.0 ** -up
    c.check(60, 6)


@pytest.mark.parametrize("n", [1, 150])
def test_nan_in_a_first_token_reaches_every_row(n):
    L = 400
    c = SinkCase([(L, n), (L, n)], 8, 2, 64, 16)
    c.codes["k"][c.table[0, 0], 1, 2] = 0x7F
    c.codes["v"][c.table[0, 0], 1, 2] = 0
    hit = np.zeros((c.T, 8), dtype=bool)
    hit[:n, 4:] = True
    seen = ref.bf16_bits_to_f64(c.gpu().run(40, 3)).reshape(c.T, 8, 64)
    assert np.isnan(seen[hit]).all() and np.isfinite(seen[~hit]).all()
    unseen = ref.bf16_bits_to_f64(c.run(40, 2))
    assert np.isfinite(unseen).all()


@pytest.mark.parametrize("seqs", [[(300, 1), (200, 20)], [(500, 150)], [(200, 1)] * 130])
def test_pages_that_do_not_exist(seqs):
    """Among the first tokens one is flagged and its tokens count as unseen; between them and the window none is."""
    import int4_grouped_expert_gb300 as st
    c = SinkCase(seqs, 4, 2, 64, 16)
    empty_the_gap(c, 50, 40)
    good = c.gpu().run(50, 40)
    assert np.array_equal(good, c.run(50, 40))
    c.table[0, 1] = c.codes["k"].shape[0]
    got = ref.bf16_bits_to_f64(c.gpu().run(50, 40, expect_status=st.STRATA_DEV_BAD_SLOT)).reshape(c.T, 4, 64)
    assert np.array_equal(bf16_rows(got[seqs[0][1]:]), bf16_rows(ref.bf16_bits_to_f64(good).reshape(c.T, 4, 64)[seqs[0][1]:]))
    L, n = seqs[0]
    for i in (0, n - 1):
        pos = L - n + i
        tok = np.array([j for j in range(pos + 1) if (j > pos - 50 or j < 40) and j // 16 != 1])
        q = ref.bf16_bits_to_f64(c.q_bits)[i].reshape(4, 64)
        for h in range(4):
            page = c.table[0][tok // 16]
            k, v = (ref.E4M3[c.codes[x][page, h // 2, tok % 16]] *
                    c.scales[x][page, h // 2].astype(np.float64)[:, None] for x in "kv")
            w = np.exp(k @ q[h] * c.scale)
            assert np.abs(got[i, h] - w @ v / w.sum()).max() < 2e-2 * np.abs(v).max()


def bf16_rows(a):
    return a.astype(np.float32)


@pytest.mark.parametrize("seqs", [[(9000, 1), (100, 1)], [(3000, 90)], [(700, 1), (300, 130)], [(200, 1)] * 130])
def test_a_workspace_goes_between_the_calls(seqs):
    """The same bits every time, with and without first tokens in turn, on one kept workspace."""
    import torch
    import int4_grouped_expert_gb300 as st
    c = SinkCase(seqs, 8, 2, 128, 64).gpu()
    need = st.strata_attention_workspace_size(c.cache.struct(), c.batch, 8)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    plain, sink = Case.run(c, window=150), c.run(150, 70)
    for _ in range(8):
        assert np.array_equal(c.run(150, 70, flags=st.STRATA_WS_REUSE, ws=ws), sink)
        assert np.array_equal(Case.run(c, window=150, flags=st.STRATA_WS_REUSE, ws=ws), plain)


def test_replayed_with_other_lengths():
    """A captured call follows the lengths and the table that stand there when it runs."""
    import torch
    import int4_grouped_expert_gb300 as st
    a, b = ([(900, 1), (40, 1), (300, 1)], [(77, 1), (901, 1), (2, 1)])
    big = SinkCase(a, 8, 2, 128, 16).gpu()
    start, length, table = big.batch.tensors
    batch = st.kv_batch(start, length, table, 3, 1, 901)
    out = torch.empty(3, 8 * 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(st.strata_attention_workspace_size(big.cache.struct(), batch, 8), dtype=torch.uint8, device="cuda")

    def call():
        st.check(st.strata_attention_sinks_forward(big.cache.struct(), batch, big.q, 8, big.scale, out, ws, ws.numel(),
                                                   window=100, n_sinks=5, flags=st.STRATA_WS_REUSE), "attention")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.synchronize()
    for lens in ([900, 40, 300], [500, 1, 16], [0, 39, 299]):
        big.seqs = [(n, 1) for n in lens]
        length.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = ref.bf16_bits_to_f64(bf16_to_np_bits(out)).reshape(3, 8, 128)
        want, bound = reference(big, 100, 5)
        assert (np.abs(got - want) <= bound).all()
