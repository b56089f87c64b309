"""Argument checks of the projection, cache-append and attention calls: all on the host, before any
CUDA call, so they run without a GPU."""
import pytest

A = 1 << 12  # an aligned fake address: the checks fail before anything is read


@pytest.fixture(scope="module")
def st():
    from int4_grouped_expert_gb300 import build
    build.build()
    import int4_grouped_expert_gb300 as mod
    mod.lib()
    return mod


def lin(st, **kw):
    d = dict(N=512, K=1024, group_size=128, bits=4, codes=A, scales=A, bias=None)
    d.update(kw)
    return st.strata_linear(**d)


@pytest.mark.parametrize("kw,expect", [
    (dict(group_size=32), 3), (dict(bits=3), 3), (dict(N=0), 2), (dict(N=(1 << 20) + 1), 2),
    (dict(K=1000), 2), (dict(K=1 << 17), 2), (dict(K=192), 2), (dict(codes=None), 1),
    (dict(codes=A + 8), 1), (dict(scales=None), 1), (dict(scales=A + 1), 1), (dict(bias=A + 2), 1)])
def test_linear_descriptor_refusals(st, kw, expect):
    assert st.strata_linear_forward(lin(st, **kw), A, 4, 2 * A, A, 1 << 30) == expect
    assert st.strata_linear_workspace_size(lin(st, **kw), 4) == 0


def test_linear_call_refusals(st):
    L = lin(st)
    need = st.strata_linear_workspace_size(L, 4)
    assert need > 0 and need % 256 == 0
    assert st.strata_linear_workspace_size(L, -1) == 0
    ok = dict(workspace=A, ws_bytes=1 << 40)
    f = st.strata_linear_forward
    assert f(L, A, -1, 2 * A, **ok) == 2
    assert f(L, A, (1 << 22) + 1, 2 * A, **ok) == 2
    assert f(L, None, 4, 2 * A, **ok) == 1
    assert f(L, A + 8, 4, 2 * A, **ok) == 1                       # x misaligned
    assert f(L, A, 4, 2 * A, x_stride=1023, **ok) == 1            # shorter than a row
    assert f(L, A, 4, 2 * A, x_stride=1028, **ok) == 1            # rows lose their alignment
    assert f(L, A, 4, None, **ok) == 1
    assert f(L, A, 4, 2 * A + 1, **ok) == 1
    assert f(L, A, 4, 2 * A, out_stride=511, **ok) == 1
    assert f(L, A, 4, A, **ok) == 1                               # out is x
    assert f(L, A, 4, 2 * A, residual=3 * A, residual_stride=8, **ok) == 1
    assert f(L, A, 4, 2 * A, residual=2 * A, residual_stride=600, **ok) == 1  # in place, other rows
    assert f(L, A, 4, 2 * A, None, need) == 4
    assert f(L, A, 4, 2 * A, A + 16, need) == 4
    assert f(L, A, 4, 2 * A, A, need - 1) == 4
    assert f(L, A, 0, 2 * A, None, 0) == 0                        # nothing to do


def cache(st, **kw):
    d = dict(n_kv_heads=8, head_dim=128, page_size=64, n_pages=100, k_codes=A, v_codes=A, k_scales=A,
             v_scales=A)
    d.update(kw)
    return st.strata_kv_cache(**d)


CACHE_REFUSALS = [(dict(head_dim=96), 3), (dict(head_dim=256), 3), (dict(page_size=8), 3),
                  (dict(page_size=48), 3), (dict(page_size=256), 3), (dict(n_kv_heads=0), 3),
                  (dict(n_kv_heads=257), 3), (dict(n_pages=-1), 2), (dict(n_pages=1 << 26), 2),
                  (dict(k_codes=None), 1), (dict(v_codes=A + 8), 1), (dict(k_scales=A + 2), 1),
                  (dict(v_scales=None), 1)]


@pytest.mark.parametrize("kw,expect", CACHE_REFUSALS)
def test_cache_refusals(st, kw, expect):
    C = cache(st, **kw)
    assert st.strata_kv_append(C, A, A, 4, A) == expect
    b = st.strata_kv_batch(n_seq=1, max_q=1, T=1, max_kv=64, q_start=A, kv_len=A, page_table=A, table_stride=4)
    assert st.strata_attention_workspace_size(C, b, 8) == 0
    assert st.strata_attention_forward(C, b, A, 8, 0.1, 2 * A, A, 1 << 30) == expect


def test_append_refusals(st):
    C = cache(st)
    f = st.strata_kv_append
    q = dict(q=A, n_heads=32, q_out=2 * A)
    rope = dict(positions=A, rope=A, n_pos=100, rot_dim=128)
    assert f(C, A, A, -1, A) == 2
    assert f(C, A, A, (1 << 22) + 1, A) == 2
    assert f(C, None, A, 4, A) == 1
    assert f(C, A, None, 4, A) == 1
    assert f(C, A, A, 4, None) == 1
    assert f(C, A, A, 4, A + 2) == 1
    assert f(C, A + 2, A, 4, A) == 1
    assert f(C, A, A, 4, A, k_stride=1000) == 1                   # shorter than a row
    assert f(C, A, A, 4, A, v_stride=1028) == 1                   # not a multiple of 8
    assert f(C, A, A, 4, A, flags=2) == 1
    assert f(C, A, A, 4, A, dev_status=A + 2) == 1
    assert f(C, A, A, 4, A, q=A, n_heads=32) == 1                 # q without q_out
    assert f(C, A, A, 4, A, q_out=A, n_heads=32) == 1
    assert f(C, A, A, 4, A, **{**q, "n_heads": 0}) == 3
    assert f(C, A, A, 4, A, **{**q, "n_heads": 1025}) == 3
    assert f(C, A, A, 4, A, q=A, n_heads=32, q_out=A, q_stride=8192) == 1  # in place, other rows
    assert f(C, A, A, 4, A, **{**rope, "rot_dim": 24}) == 2
    assert f(C, A, A, 4, A, **{**rope, "rot_dim": 144}) == 2
    assert f(C, A, A, 4, A, **{**rope, "rot_dim": -16}) == 2
    assert f(C, A, A, 4, A, **{**rope, "positions": None}) == 1
    assert f(C, A, A, 4, A, **{**rope, "rope": None}) == 1
    assert f(C, A, A, 4, A, **{**rope, "rope": A + 4}) == 1
    assert f(C, A, A, 4, A, **{**rope, "n_pos": 0}) == 1
    assert f(C, A, A, 0, None) == 0                               # nothing to do


def batch(st, **kw):
    d = dict(n_seq=3, max_q=5, T=9, max_kv=500, q_start=A, kv_len=A, page_table=A, table_stride=8)
    d.update(kw)
    return st.strata_kv_batch(**d)


@pytest.mark.parametrize("kw,expect", [
    (dict(n_seq=-1), 2), (dict(n_seq=65536), 2), (dict(T=-1), 2), (dict(T=(1 << 22) + 1), 2),
    (dict(max_q=0), 2), (dict(max_q=-1), 2), (dict(max_kv=-1), 2), (dict(max_kv=513), 2),
    (dict(table_stride=-1), 2), (dict(q_start=None), 1), (dict(kv_len=None), 1),
    (dict(page_table=None), 1), (dict(q_start=A + 2), 1), (dict(kv_len=A + 1), 1)])
def test_batch_refusals(st, kw, expect):
    C, b = cache(st), batch(st, **kw)
    assert st.strata_attention_workspace_size(C, b, 32) == 0
    assert st.strata_attention_forward(C, b, A, 32, 0.1, 2 * A, A, 1 << 30) == expect


def test_attention_refusals(st):
    C, b = cache(st), batch(st)
    need = st.strata_attention_workspace_size(C, b, 32)
    assert need > 0 and need % 256 == 0
    ok = dict(workspace=A, ws_bytes=1 << 40)
    f = st.strata_attention_forward
    for heads in (0, 12, 1032):
        assert f(C, b, A, heads, 0.1, 2 * A, **ok) == 3
    assert f(C, b, A, 32, float("nan"), 2 * A, **ok) == 1
    assert f(C, b, A, 32, float("inf"), 2 * A, **ok) == 1
    assert f(C, b, A, 32, 0.1, 2 * A, window=-1, **ok) == 1
    assert f(C, b, A, 32, 0.1, 2 * A, flags=1, **ok) == 1
    assert f(C, b, None, 32, 0.1, 2 * A, **ok) == 1
    assert f(C, b, A + 8, 32, 0.1, 2 * A, **ok) == 1
    assert f(C, b, A, 32, 0.1, 2 * A + 4, **ok) == 1
    assert f(C, b, A, 32, 0.1, A, **ok) == 1                      # out is q
    assert f(C, b, A, 32, 0.1, 2 * A, q_stride=4095, **ok) == 1
    assert f(C, b, A, 32, 0.1, 2 * A, out_stride=4100, **ok) == 1
    assert f(C, b, A, 32, 0.1, 2 * A, None, need) == 4
    assert f(C, b, A, 32, 0.1, 2 * A, A + 128, need) == 4
    assert f(C, b, A, 32, 0.1, 2 * A, A, need - 1) == 4
    assert f(C, batch(st, n_seq=0), A, 32, 0.1, 2 * A, None, 0) == 0
    assert f(C, batch(st, T=0), A, 32, 0.1, 2 * A, None, 0) == 0
