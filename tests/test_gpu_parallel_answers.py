"""The page calls, the append with norms and the attention with first tokens in a run, as the example uses them: several
answers share a prompt's pages, are extended through a captured graph, forked again, and end."""
import os
import sys

import numpy as np
import pytest

import block_ref as ref
import pages_ref
from helpers import bf16_to_np_bits
from test_gpu_attention_sinks import reference

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

N_PAGES, N_SEQ, E, P, WINDOW, SINKS = 150, 7, 24, 16, 50, 5


def f64(t):
    return ref.bf16_bits_to_f64(bf16_to_np_bits(t.contiguous()))


class View:
    """What test_gpu_attention_sinks.reference asks of a case, of a server's state."""

    def __init__(self, server, q, seqs, table):
        k, c = server.block, server.cache
        self.T, self.Hq, self.Hkv, self.D, self.P, self.scale = len(q), k.Hq, k.Hkv, k.D, P, k.scale
        self.q_bits, self.seqs, self.table = q, seqs, table
        self.codes = {x: t.view(torch_uint8()).cpu().numpy() for x, t in (("k", c.k_codes), ("v", c.v_codes))}
        self.scales = {x: t.cpu().numpy() for x, t in (("k", c.k_scales), ("v", c.v_scales))}


def torch_uint8():
    import torch
    return torch.uint8


class Twin:
    """The tables on host lists, and every sequence's keys and values in 64 bits."""

    def __init__(self, server):
        self.server = server
        self.pages = pages_ref.Pages(N_PAGES, N_SEQ, E, P)
        shape = (0, server.block.Hkv, server.block.D)
        self.k, self.v = [np.zeros(shape)] * N_SEQ, [np.zeros(shape)] * N_SEQ

    def same_tables(self):
        p = self.server.pages
        np.testing.assert_array_equal(p.kv_len.cpu().numpy(), self.pages.length)
        np.testing.assert_array_equal(p.refs.cpu().numpy(), self.pages.refs)
        np.testing.assert_array_equal(p.page_table.cpu().numpy(), self.pages.table)
        self.pages.check()

    def fork(self, parent):
        self.server.fork(parent)
        assert self.pages.fork(parent) == 0
        for s, of in enumerate(parent):
            if of >= 0:
                self.k[s], self.v[s] = self.k[of], self.v[of]
        self.same_tables()

    def end(self, sequences):
        self.server.end(sequences)
        self.pages.release([0 if s in sequences else -1 for s in range(N_SEQ)])
        for s in sequences:
            self.k[s], self.v[s] = self.k[s][:0], self.v[s][:0]
        self.same_tables()

    def run(self, rows, x, new):
        s, k = self.server, self.server.block
        out = rows.run(x, new).clone()
        s.check(rows)
        slots, positions, q_start, copies, status = self.pages.extend(new, rows.T)
        assert status == 0
        n = int(q_start[-1])
        for got, want in ((rows.slots, slots), (rows.positions, positions), (rows.q_start, q_start)):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        # keys and values of the new tokens, from what the projection gave (q in the buffer is finished already)
        Hq, Hkv, D = k.Hq, k.Hkv, k.D
        qkv = f64(rows.b["qkv"])[:n]
        kk = qkv[:, Hq * D:(Hq + Hkv) * D].reshape(n, Hkv, D)
        kk = kk / np.sqrt((kk * kk).mean(-1, keepdims=True) + s.norm.eps) * s.norm.k_weight.cpu().numpy().astype(np.float64)
        rope = k.rope.cpu().numpy().astype(np.float64)[positions[:n]]
        kk, _ = ref.rotate(kk, rope[:, :k.rot // 2], rope[:, k.rot // 2:], k.rot, False)
        vv = qkv[:, (Hq + Hkv) * D:].reshape(n, Hkv, D)
        for i in range(N_SEQ):
            at = slice(q_start[i], q_start[i + 1])
            self.k[i], self.v[i] = np.concatenate([self.k[i], kk[at]]), np.concatenate([self.v[i], vv[at]])
        # the attention, over the pages as they lay there before pages were given back
        seqs = [(int(self.pages.length[i]), int(new[i])) for i in range(N_SEQ)]
        view = View(s, bf16_to_np_bits(rows.b["qkv"][:n, :Hq * D].contiguous()), seqs, self.pages.table.copy())
        want, bound = reference(view, WINDOW, SINKS)
        assert (np.abs(f64(rows.b["att"])[:n].reshape(n, Hq, D) - want) <= bound).all()
        self.same_values(view, new)
        self.pages.release(None, WINDOW, SINKS)
        self.same_tables()
        return out

    def same_values(self, view, new):
        """Each sequence's pages hold its own keys and values. A code is rounded once, by half a step (2^-4 of its value, or
        half of the smallest step, 2^-10 of the scale), and once more each time its page's scale grows: at most 7 times
        here, as scales differ by less than 2^7."""
        for i in range(N_SEQ):
            L = int(self.pages.length[i])
            first = max(0, L - int(new[i]) - WINDOW + 1)
            tok = np.r_[0:min(first, SINKS), first:L]
            if not len(tok):
                continue
            page, off = view.table[i][tok // P], tok % P
            for x, mine in (("k", self.k[i]), ("v", self.v[i])):
                scale = view.scales[x][page].astype(np.float64)[:, :, None]
                held = ref.E4M3[view.codes[x][page, :, off]] * scale
                want = mine[tok]
                step = np.maximum(2.0 ** -4 * np.abs(want) * 1.01, 2.0 ** -10 * scale)
                assert (np.abs(held - want) <= 7 * step).all(), (i, x)
                assert np.linalg.norm(held - want) <= 0.05 * np.linalg.norm(want), (i, x)


def test_answers_that_share_a_prompt():
    import torch
    import decoder_block
    import parallel_answers as ex
    torch.manual_seed(5)
    block = decoder_block.random_block(H=512, I=256, E=8, k=2, Hq=8, Hkv=2, D=64, seed=3)
    server = ex.Server(block, WINDOW, SINKS, N_PAGES, N_SEQ, E, P, seed=1)
    twin = Twin(server)
    rand = lambda n: torch.randn(n, 512, device="cuda").bfloat16()  # noqa: E731
    prompts, tokens = ex.Rows(server, 150, 140), ex.Rows(server, N_SEQ, 1, capture=True)
    twin.run(prompts, rand(150), [87, 0, 0, 0, 0, 0, 63])   # two prompts, one of a whole number of pages but for one token
    twin.fork([-1, 0, 0, 0, 6, -1, -1])
    same = rand(1).expand(5, -1)
    out = twin.run(tokens, same, [1, 1, 1, 1, 0, 0, 1])     # the same token for all answers of the first prompt
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[3]) and not torch.equal(out[0], out[4])
    for step in range(40):
        if step == 12:
            twin.end([2, 6])
        if step == 15:
            twin.fork([-1, -1, 1, -1, -1, 1, 4])            # answers of an answer
        if step == 30:
            twin.end([0])
        live = [s for s in range(N_SEQ) if twin.pages.length[s] > 0 and (step + s) % 5]
        twin.run(tokens, rand(len(live)), [int(s in live) for s in range(N_SEQ)])
    twin.run(prompts, rand(100), [30, 0, 20, 0, 50, 0, 0])  # pieces of new prompts, and of answers that are rather long
    twin.end(list(range(N_SEQ)))
    assert not server.pages.refs.any()


def test_the_example_runs(capsys):
    import parallel_answers as ex
    ex.main()
    assert "8 answers of 200 tokens" in capsys.readouterr().out
