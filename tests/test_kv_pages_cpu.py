"""Argument checks of the page calls, on the host before any CUDA call; the tensors behind a page table; and the host
lists that the GPU tests compare with."""
import numpy as np
import pytest
import torch

import pages_ref
from test_block_abi_cpu import A, CACHE_REFUSALS, cache, st  # noqa: F401


def pages(st, **kw):  # noqa: F811
    d = dict(n_seq=4, page_size=64, n_pages=100, max_pages=20, table_stride=22, page_table=A, kv_len=A, refs=A)
    d.update(kw)
    return st.strata_kv_pages(**d)


REFUSALS = [(dict(page_size=48), 3), (dict(page_size=0), 3), (dict(page_size=256), 3), (dict(n_seq=-1), 2),
            (dict(n_seq=65536), 2), (dict(n_pages=-1), 2), (dict(n_pages=1 << 25), 2), (dict(max_pages=-1), 2),
            (dict(max_pages=1 << 25, table_stride=1 << 25), 2), (dict(table_stride=19), 2), (dict(page_table=None), 1), (dict(kv_len=None), 1), (dict(refs=None), 1),
            (dict(page_table=A + 2), 1), (dict(kv_len=A + 1), 1), (dict(refs=A + 4), 1)]


@pytest.mark.parametrize("kw,expect", REFUSALS)
def test_descriptor_refusals(st, kw, expect):  # noqa: F811
    p = pages(st, **kw)
    assert st.strata_kv_pages_extend(p, A, 8, A, A, A, A, A) == expect
    assert st.strata_kv_pages_fork(p, A) == expect
    assert st.strata_kv_pages_release(p, A) == expect
    big = pages(st, n_pages=200, page_table=2 * A, kv_len=2 * A, refs=2 * A)
    assert st.strata_kv_pages_compact(p, big, A, A, A, 1 << 30) == expect
    assert st.strata_kv_pages_compact(big, p, A, A, A, 1 << 30) == expect
    assert st.strata_kv_pages_compact_workspace_size(p) == 0


def test_call_refusals(st):  # noqa: F811
    p = pages(st)
    f = st.strata_kv_pages_extend
    assert f(p, A, -1, A, A, A, A, A) == 2
    assert f(p, A, (1 << 22) + 1, A, A, A, A, A) == 2
    for at in range(6):  # each array missing, then unaligned
        for bad in (None, A + 2):
            args = [A] * 6
            args[at] = bad
            assert f(p, args[0], 8, *args[1:]) == 1
    assert f(p, A, 8, A, A, A, A, A, dev_status=A + 2) == 1
    assert st.strata_kv_pages_fork(p, None) == 1
    assert st.strata_kv_pages_fork(p, A + 2) == 1
    assert st.strata_kv_pages_fork(p, A, dev_status=A + 1) == 1
    assert st.strata_kv_pages_fork(pages(st, n_seq=0), None) == 0
    r = st.strata_kv_pages_release
    assert r(p, A + 2) == 1
    assert r(p, A, window=-1) == 1
    assert r(p, A, window=4, n_sinks=-1) == 1
    assert r(p, A, dev_status=A + 2) == 1
    assert r(p) == 0                                              # nothing to give back
    assert r(pages(st, n_seq=0), None, window=5) == 0


def test_compact_refusals(st):  # noqa: F811
    src, other = pages(st), dict(page_table=2 * A, kv_len=2 * A, refs=2 * A)
    need = st.strata_kv_pages_compact_workspace_size(src)
    assert need >= 256 + 400 and need % 256 == 0
    f = st.strata_kv_pages_compact
    ok = (A, A, A, need)
    assert f(src, pages(st, **other, n_seq=5), *ok) == 2
    assert f(src, pages(st, **other, page_size=32), *ok) == 2
    assert f(src, pages(st, **other, max_pages=19), *ok) == 2
    for name in other:  # an array that serves both
        assert f(src, pages(st, **{**other, name: A}), *ok) == 1
    dst = pages(st, **other)
    assert f(src, dst, None, A, A, need) == 1
    assert f(src, dst, A, None, A, need) == 1
    assert f(src, dst, A, A + 2, A, need) == 1
    assert f(src, dst, A, A, None, need) == 4
    assert f(src, dst, A, A, A + 64, need) == 4
    assert f(src, dst, A, A, A, need - 1) == 4


@pytest.mark.parametrize("kw,expect", CACHE_REFUSALS)
def test_copies_refuse_caches(st, kw, expect):  # noqa: F811
    good, bad = cache(st), cache(st, **kw)
    f = st.strata_kv_copy_pages
    assert f(bad, good, A, A, 5) == expect
    assert f(good, bad, A, A, 5) == expect


def test_copy_refusals(st):  # noqa: F811
    c = cache(st)
    arr = lambda *x: (st.strata_kv_cache * len(x))(*x)  # noqa: E731
    f = st.strata_kv_copy_pages
    for kw in (dict(n_kv_heads=4), dict(head_dim=64), dict(page_size=32)):
        assert f(c, cache(st, **kw), A, A, 5) == 2
        assert f(arr(c, cache(st, **kw)), arr(c, c), A, A, 5) == 2
    assert f(arr(c, cache(st, n_pages=99)), arr(c, c), A, A, 5) == 2
    assert f(arr(c, c), arr(cache(st, n_pages=99), c), A, A, 5) == 2
    assert f(c, c, A, A, -1) == 2
    assert f(c, c, A, A, 1 << 30) == 2
    assert f(c, c, None, A, 5) == 1
    assert f(c, c, A + 2, A, 5) == 1
    assert f(c, c, A, A + 2, 5) == 1
    assert f(c, c, A, A, 5, dev_status=A + 2) == 1
    assert f(arr(*[c] * 1025), arr(*[c] * 1025), A, A, 5) == 2
    assert f(c, c, None, None, 0) == 0                            # nothing to do
    assert f(arr(), arr(), None, None, 5) == 0
    with pytest.raises(ValueError):
        f(arr(c, c), arr(c), A, A, 5)


def test_tables_that_are_taken_and_refused():
    import int4_grouped_expert_gb300 as st
    i32 = dict(dtype=torch.int32)
    p = st.PageTable(10, 3, 4, 16, device="cpu")
    assert (p.page_table == -1).all() and p.page_table.shape == (3, 4)
    assert not p.kv_len.any() and not p.refs.any() and p.struct().table_stride == 4
    wide = torch.zeros(3, 9, **i32)[:, :4]
    table, length, refs = torch.zeros(3, 4, **i32), torch.zeros(3, **i32), torch.zeros(10, **i32)
    assert st.PageTable(10, 3, 4, 16, wide, length, refs).struct().table_stride == 9
    assert st.PageTable(10, 0, 4, 16, device="cpu").struct().n_seq == 0
    assert st.PageTable(10, 3, 4, 16, table, length, refs).batch(torch.zeros(4, **i32), 5, 2, 60).T == 5
    for t, n, r, error in ((table.long(), length, refs, TypeError), (table[:2], length, refs, ValueError),
                           (torch.zeros(4, 3, **i32).t(), length, refs, ValueError), (table, length[:2], refs, ValueError),
                           (table[:1].expand(3, 4), length, refs, ValueError), (table, length.long(), refs, TypeError),
                           (table, length, torch.zeros(20, **i32)[::2], ValueError),
                           (table, length, refs.float(), TypeError)):
        with pytest.raises(error):
            st.PageTable(10, 3, 4, 16, t, n, r)


def test_host_lists():
    """Two sequences share pages, part, and give them back."""
    p = pages_ref.Pages(8, 3, 4, 16)
    slots, pos, start, copies, status = p.extend([20, 0, 0], 24)
    assert status == 0 and not copies and list(p.table[0]) == [0, 1, -1, -1] and list(start) == [0, 20, 20, 20]
    assert list(slots[:20]) == list(range(20)) and list(pos[:20]) == list(range(20)) and (slots[20:] == -1).all()
    assert p.fork([-1, 0, 0]) == 0 and list(p.refs) == [3, 3, 0, 0, 0, 0, 0, 0]
    *_, copies, status = p.extend([0, 1, 14], 15)
    assert copies == [(1, 2), (1, 3)] and list(p.table[2]) == [0, 3, 4, -1] and list(p.refs) == [3, 1, 1, 1, 1, 0, 0, 0]
    p.check()
    p.release([-1, 0, 30])
    assert list(p.refs) == [2, 1, 0, 1, 0, 0, 0, 0]
    to, copies, _ = p.compact(5, 4)
    assert copies == [(0, 0), (1, 1), (3, 2)] and list(to.table[2]) == [0, 2, -1, -1]
    to.check()
    assert np.array_equal(to.refs, [2, 1, 1, 0, 0])
