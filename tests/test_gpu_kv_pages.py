"""The page calls against host lists (pages_ref), entry by entry; copies byte by byte."""
import numpy as np
import pytest

import pages_ref

pytestmark = pytest.mark.gpu


class Pool:
    """Page tables on the GPU and their host twin, changed by the same calls."""

    def __init__(self, n_pages, n_seq, max_pages, P, apart=0):
        import torch
        import int4_grouped_expert_gb300 as st
        self.st, self.torch = st, torch
        self.cpu = pages_ref.Pages(n_pages, n_seq, max_pages, P)
        wide = torch.full((n_seq, max_pages + apart), -1, dtype=torch.int32, device="cuda")
        self.wide, self.max_pages = wide, max_pages
        wide[:, max_pages:] = -77
        self.gpu = st.PageTable(n_pages, n_seq, max_pages, P, page_table=wide[:, :max_pages])
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def i32(self, a):
        return self.torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    def settle(self, expect):
        self.torch.cuda.synchronize()
        assert self.st.strata_read_status(self.status)[1] == expect
        p, c = self.gpu, self.cpu
        np.testing.assert_array_equal(p.kv_len.cpu().numpy(), c.length)
        np.testing.assert_array_equal(p.refs.cpu().numpy(), c.refs)
        np.testing.assert_array_equal(p.page_table.cpu().numpy(), c.table)
        assert (self.wide[:, self.max_pages:] == -77).all()

    def extend(self, new, T_max=None):
        st, torch = self.st, self.torch
        T = int(max(0, np.sum(new))) if T_max is None else T_max
        out = {k: torch.full((n + 2,), -9, dtype=torch.int32, device="cuda")
               for k, n in (("slots", T), ("positions", T), ("q_start", len(new) + 1), ("copies", 2 * len(new)), ("n", 1))}
        slots, positions, q_start, copies, status = self.cpu.extend(new, T)
        st.check(st.strata_kv_pages_extend(self.gpu.struct(), self.i32(new), T, out["slots"], out["positions"],
                                           out["q_start"], out["copies"], out["n"], self.status), "extend")
        self.settle(status)
        got = {k: v.cpu().numpy() for k, v in out.items()}
        want = {"slots": slots, "positions": positions, "q_start": q_start, "n": [len(copies)],
                "copies": np.array(copies, dtype=np.int64).reshape(-1)}
        for k, w in want.items():
            np.testing.assert_array_equal(got[k][:len(w)], w, err_msg=k)
            assert (got[k][len(w):] == -9).all(), k
        return copies, status

    def fork(self, parent):
        status = self.cpu.fork(parent)
        self.st.check(self.st.strata_kv_pages_fork(self.gpu.struct(), self.i32(parent), self.status), "fork")
        self.settle(status)

    def release(self, keep=None, window=0, sinks=0):
        self.cpu.release(keep, window, sinks)
        self.st.check(self.st.strata_kv_pages_release(self.gpu.struct(), None if keep is None else self.i32(keep), window,
                                                      sinks, self.status), "release")
        self.settle(0)

    def compact(self, n_pages, more=0):
        st, torch = self.st, self.torch
        to = Pool(n_pages, self.cpu.n_seq, self.max_pages + more, self.cpu.P, apart=more)
        to.gpu.kv_len.fill_(55)  # (written whole, whatever was there)
        to.gpu.refs.fill_(66)
        to.gpu.page_table.fill_(44)
        copies = torch.full((n_pages + 1, 2), -9, dtype=torch.int32, device="cuda")
        n = torch.full((1,), -9, dtype=torch.int32, device="cuda")
        need = st.strata_kv_pages_compact_workspace_size(self.gpu.struct())
        ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
        to.cpu, want, status = self.cpu.compact(n_pages, self.max_pages + more)
        st.check(st.strata_kv_pages_compact(self.gpu.struct(), to.gpu.struct(), copies, n, ws, need, to.status), "compact")
        to.settle(status)
        self.settle(0)
        assert n.item() == len(want)
        np.testing.assert_array_equal(copies[:len(want)].cpu().numpy(), np.array(want).reshape(-1, 2))
        assert (copies[len(want):] == -9).all()
        return to


@pytest.mark.parametrize("n_seq,n_pages,max_pages,P", [
    (1, 9, 9, 16), (5, 33, 20, 16), (7, 300, 50, 128), (300, 5001, 40, 32), (1100, 9000, 7, 64), (9000, 70003, 5, 16)])
def test_sequences_come_and_go(n_seq, n_pages, max_pages, P):
    """Rounds of every call with what a server does to its sequences; pages and rows run out now and then."""
    rng = np.random.default_rng([n_seq, n_pages, P])
    p = Pool(n_pages, n_seq, max_pages, P, apart=n_seq % 4)
    for step in range(12):
        room = max_pages * P - p.cpu.length
        want = rng.integers(0, 3, n_seq) if step % 3 else (rng.random(n_seq) < 0.5) * rng.integers(0, 2 * P + 2, n_seq)
        new = np.minimum(want, room)
        T = int(new.sum())
        p.extend(new, [T, T + 37, max(0, T - 2), T][step % 4])
        empty, held = np.nonzero(p.cpu.length == 0)[0], np.nonzero(p.cpu.length)[0]
        parent = np.full(n_seq, -1)
        if len(held):
            parent[empty[:len(empty) // 2]] = rng.choice(held, len(empty) // 2)
        p.fork(parent)
        keep = np.where(rng.random(n_seq) < 0.3, rng.integers(0, max_pages * P, n_seq), -1)
        keep[rng.random(n_seq) < 0.15] = 0
        p.release(keep if step % 2 else None, window=[0, P + 3, 1, 2 * P][step % 4] if step > 5 else 0, sinks=step)
        p.cpu.check()
        if step % 4 == 3:
            live = int((p.cpu.refs > 0).sum())
            p.compact(live + 3)
            p.compact(live, more=2)
            if live:
                p.compact(live - 1)


def test_many_answers_of_one_prompt():
    p = Pool(400, 40, 30, 16)
    p.extend([333] + [0] * 39)
    p.fork([-1] + [0] * 39)
    copies, _ = p.extend([1] * 40)  # all of them write: the shared page is left by everybody
    assert len(copies) == 40 and p.cpu.refs[copies[0][0]] == 0
    copies, _ = p.extend([1] * 40)
    assert not copies
    p.release([0] * 40)
    assert not p.cpu.refs.any()


def test_a_cut_inside_a_shared_page():
    p = Pool(50, 3, 10, 16)
    p.extend([64, 0, 0])
    p.fork([-1, 0, 0])
    p.release([-1, 40, -1])
    copies, _ = p.extend([0, 1, 1])
    assert copies == [(2, 4)]
    p.release([40, 40, 40])
    copies, _ = p.extend([3, 3, 30])  # (sequence 0 and 2 still share; sequence 1 has its own)
    assert len(copies) == 2


def test_a_long_prompt_beside_single_tokens():
    p = Pool(9000, 6, 8200, 16)
    p.extend([3, 130000, 1, 0, 17, 900])
    p.fork([-1, -1, -1, 1, -1, -1])
    p.extend([1, 1, 1, 1000, 1, 0])
    p.release([-1, -1, -1, 70000, 0, -1], window=5000, sinks=100)


def test_windows_give_pages_back_step_by_step():
    for P, window, sinks in ((16, 1, 0), (16, 40, 5), (32, 33, 32), (16, 16, 17), (64, 300, 0)):
        p = Pool(200, 3, 40, P)
        for step in range(60):
            p.extend([[1, 0, 7], [P, 3, 0], [0, 1, 1]][step % 3])
            p.release(None, window, sinks)


def test_more_pages_than_are_free():
    p = Pool(20, 4, 20, 16)
    p.extend([100, 0, 30, 0])
    _, status = p.extend([12, 170, 1, 0])  # 0 fits its page, 1 needs 11 pages and 11 are free
    assert status == 0
    _, status = p.extend([0, 6, 1, 1])     # 1 fits its page, 2 as well, and 3 finds none
    assert status == pages_ref.NO_PAGES
    _, status = p.extend([1, 0, 1, 0])     # 0 finds none: 2 does not get its row either
    assert status == pages_ref.NO_PAGES
    _, status = p.extend([0, 0, 2, 0], T_max=1)
    assert status == pages_ref.NO_PAGES
    _, status = p.extend([0, 0, 1, 0], T_max=0)
    assert status == pages_ref.NO_PAGES
    _, status = p.extend([0, 0, 0, 0], T_max=0)
    assert status == 0


def test_counts_that_make_no_sense():
    p = Pool(50, 5, 4, 16)
    _, status = p.extend([-1, 65, 64, 1 << 30, 2], T_max=70)
    assert status == pages_ref.BAD_SLOT and list(p.cpu.length) == [0, 0, 64, 0, 2]
    _, status = p.extend([1, 1, 1, 1, -(1 << 31)], T_max=9)
    assert status == pages_ref.BAD_SLOT


def test_forks_that_make_no_sense():
    p = Pool(50, 6, 4, 16)
    p.extend([20, 5, 0, 0, 0, 0])
    # onto one that holds tokens, of itself, of one that does not exist, of one that is being forked itself
    p.fork([1, -1, 2, 6, 1, 4])
    assert list(p.cpu.length) == [20, 5, 0, 0, 5, 0]
    p.fork([-1, -1, 3, -5, -1, 1 << 30])  # (of an empty one: nothing; negative: none)


@pytest.mark.parametrize("what", ["no page", "past the end", "uncounted"])
def test_tables_that_make_no_sense(what):
    """An unfinished page that is none: the sequence gets nothing, the others theirs."""
    p = Pool(50, 3, 4, 16)
    p.extend([20, 20, 5])
    if what == "uncounted":
        page = p.cpu.table[1, 1]
        p.cpu.refs[page] = 0
        p.gpu.refs[int(page)] = 0
        # (it counts as free, and nobody is given it: the first free pages come before it)
        p.cpu.table[1, 1] = p.gpu.page_table[1, 1] = 49
    else:
        p.cpu.table[1, 1] = {"no page": -1, "past the end": 50}[what]
        p.gpu.page_table[1, 1] = int(p.cpu.table[1, 1])
    _, status = p.extend([1, 1, 1])
    assert status == pages_ref.BAD_SLOT and list(p.cpu.length) == [21, 20, 6]


def test_arrays_that_make_no_sense_touch_nothing_else():
    """Lengths, entries and counts out of range: flagged, and no access leaves the arrays (guards on both sides)."""
    import torch
    import int4_grouped_expert_gb300 as st
    i32 = dict(dtype=torch.int32, device="cuda")
    for length in (-5, 1 << 30, -(1 << 31), (1 << 31) - 1):
        for entry in (-(1 << 31), 50, (1 << 31) - 1):
            mem = torch.full((400,), -3, **i32)
            table, n, refs = mem[64:76].view(3, 4), mem[128:131], mem[192:242]
            table.fill_(entry), refs.fill_(1), refs[:10].zero_(), n.copy_(torch.tensor([length, 0, 20]))
            p = st.PageTable(50, 3, 4, 16, table, n, refs)
            status, out = torch.zeros(1, **i32), torch.zeros(64, **i32)
            def flagged():  # noqa: E306
                bits = st.strata_read_status(status)[1]
                assert (mem[:64] == -3).all() and (mem[76:128] == -3).all() and (mem[131:192] == -3).all()
                assert (mem[242:] == -3).all()
                return bits == pages_ref.BAD_SLOT
            to = st.PageTable(60, 3, 4, 16)
            ws = torch.zeros(st.strata_kv_pages_compact_workspace_size(p.struct()), dtype=torch.uint8, device="cuda")
            st.check(st.strata_kv_pages_compact(p.struct(), to.struct(), torch.zeros(60, 2, **i32), out, ws, ws.numel(),
                                                status), "compact")
            assert flagged() and (to.page_table == -1).all()
            st.check(st.strata_kv_pages_extend(p.struct(), torch.ones(3, **i32), 3, out, out[8:], out[16:], out[32:],
                                               out[48:], status), "extend")
            assert flagged()
            n[1] = 0
            st.check(st.strata_kv_pages_fork(p.struct(), torch.tensor([-1, 0, -1], **i32), status), "fork")
            flagged()
            st.check(st.strata_kv_pages_release(p.struct(), torch.zeros(3, **i32), 7, 3, status), "release")
            flagged()


CACHES = [(1, 64, 16, 1), (8, 128, 64, 3), (3, 64, 32, 2), (256, 128, 16, 2), (5, 128, 128, 1), (2, 64, 16, 100)]


@pytest.mark.parametrize("Hkv,D,P,layers", CACHES)
def test_copies(Hkv, D, P, layers):
    import torch
    import int4_grouped_expert_gb300 as st
    rng = np.random.default_rng([Hkv, D, layers])
    N, M = 21, 34

    def caches(n):
        return [st.PagedKVCache(n, Hkv, D, P, *(torch.randint(0, 256, (n, Hkv, P, D), dtype=torch.uint8, device="cuda")
                                                for _ in "kv"), *(torch.rand(n, Hkv, device="cuda") for _ in "kv"))
                for _ in range(layers)]

    names = ("k_codes", "v_codes", "k_scales", "v_scales")
    bits = lambda c: [getattr(c, n).view(torch.uint8).cpu().numpy().copy() for n in names]  # noqa: E731
    src, dst = caches(N), caches(M)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = [(-1, 3), (4, -1), (N, 1), (2, M), (1 << 30, 1 << 30)]
    pairs = list(zip(rng.integers(0, N, 12), rng.permutation(np.arange(5, M))[:12]))  # (a page may be copied twice)
    for listed, count, flag in ((pairs, None, 0), (pairs[:7], 7, 0), (pairs, 3, 0), (pairs, 0, 0),
                                (pairs[:4] + bad[:2] + pairs[4:], None, 0), (bad + pairs, len(pairs) + 5, 0x10),
                                (pairs[:5], 9, 0x10), (pairs[:5], -1, 0x10)):
        n = len(listed) if count is None else min(max(count, 0), len(listed))
        before = [bits(c) for c in dst]
        dev = torch.tensor(np.array(listed), dtype=torch.int32, device="cuda")
        cnt = None if count is None else torch.tensor([count], dtype=torch.int32, device="cuda")
        st.check(st.strata_kv_copy_pages(st.cache_array(src), st.cache_array(dst), dev, cnt, len(listed), status), "copy")
        assert st.strata_read_status(status)[1] == flag
        for c, d, was in zip(src, dst, before):
            for got, want, x in zip(bits(d), was, bits(c)):
                for a, b in listed[:n]:
                    if 0 <= a < N and 0 <= b < M:
                        want.reshape(M, -1)[b] = x.reshape(N, -1)[a]
                assert np.array_equal(got, want)
        for d in dst:
            d.k_codes.random_(0, 256)
    # within one cache, and one descriptor instead of an array
    before = bits(src[0])
    st.check(st.strata_kv_copy_pages(src[0].struct(), src[0].struct(),
                                     torch.tensor([[3, 7], [3, 8], [0, 20]], dtype=torch.int32, device="cuda"), None, 3,
                                     status), "copy")
    for got, want in zip(bits(src[0]), before):
        for a, b in ((3, 7), (3, 8), (0, 20)):
            want.reshape(N, -1)[b] = want.reshape(N, -1)[a]
        assert np.array_equal(got, want)


def test_copies_past_4_gb():
    """Pages whose codes lie past 2^32 bytes from the start of the cache."""
    import torch
    import int4_grouped_expert_gb300 as st
    n = 36000  # pages of 128 KB
    c = st.PagedKVCache(n, 8, 128, 128)
    c.k_codes.view(torch.uint8).view(n, -1)[[5, n - 1]] = torch.randint(0, 256, (2, 131072), dtype=torch.uint8, device="cuda")
    c.v_codes.view(torch.uint8).view(n, -1)[[5, n - 1]] = torch.randint(0, 256, (2, 131072), dtype=torch.uint8, device="cuda")
    c.k_scales.fill_(1.0), c.v_scales.fill_(2.0)
    pairs = torch.tensor([[5, n - 2], [n - 1, 6]], dtype=torch.int32, device="cuda")
    st.check(st.strata_kv_copy_pages(c.struct(), c.struct(), pairs, None, 2), "copy")
    for a, b in ((5, n - 2), (n - 1, 6)):
        for x in (c.k_codes, c.v_codes):
            assert torch.equal(x.view(torch.uint8)[a], x.view(torch.uint8)[b])


def test_replayed_on_a_stream():
    """Captured calls follow the arrays as they are at each replay: a round of a server without the host."""
    import torch
    import int4_grouped_expert_gb300 as st
    n_seq, P = 6, 16
    p = Pool(300, n_seq, 40, P)
    i32 = dict(dtype=torch.int32, device="cuda")
    new, parent, keep = (torch.full((n_seq,), v, **i32) for v in (0, -1, -1))
    slots, positions, q_start = torch.zeros(32, **i32), torch.zeros(32, **i32), torch.zeros(n_seq + 1, **i32)
    copies, n = torch.zeros(n_seq, 2, **i32), torch.zeros(1, **i32)

    def calls():
        s = p.gpu.struct()
        st.check(st.strata_kv_pages_release(s, keep, 50, 3, p.status), "release")
        st.check(st.strata_kv_pages_fork(s, parent, p.status), "fork")
        st.check(st.strata_kv_pages_extend(s, new, 32, slots, positions, q_start, copies, n, p.status), "extend")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            calls()
    torch.cuda.synchronize()
    rng = np.random.default_rng(1)
    for step in range(25):
        k = np.where(rng.random(n_seq) < 0.1, 0, -1)
        gone = (p.cpu.length == 0) | (k == 0)
        par = np.where(gone & (step > 3) & ~gone[0] & (np.arange(n_seq) > 0), 0, -1)
        add = rng.integers(0, 6, n_seq)
        for dst, src in ((keep, k), (parent, par), (new, add)):
            dst.copy_(torch.from_numpy(src.astype(np.int32)))
        graph.replay()
        p.cpu.release(k, 50, 3)
        status = p.cpu.fork(par)
        s, pos, start, pairs, more = p.cpu.extend(add, 32)
        p.settle(status | more)
        for got, want in ((slots, s), (positions, pos), (q_start, start), (n, [len(pairs)])):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        np.testing.assert_array_equal(copies[:len(pairs)].cpu().numpy(), np.array(pairs).reshape(-1, 2))
