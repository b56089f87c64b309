"""Argument checks of the append with norms, on the host before any CUDA call, and of the tensors behind its weights."""
import pytest
import torch

from test_block_abi_cpu import A, cache, st  # noqa: F401


def norm(st, **kw):  # noqa: F811
    d = dict(q_weight=A, q_head_stride=0, k_weight=A, k_head_stride=128, eps=1e-6)
    d.update(kw)
    return st.strata_qk_norm(**d)


@pytest.mark.parametrize("kw", [
    dict(eps=0.0), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e-31),
    dict(q_weight=A + 4), dict(k_weight=A + 8), dict(q_head_stride=64), dict(k_head_stride=130),
    dict(k_head_stride=-128)])
def test_norm_refusals(st, kw):  # noqa: F811
    f = st.strata_kv_append_normed
    for T in (4, 0):
        assert f(cache(st), norm(st, **kw), A, A, T, A) == 1


def test_call_refusals(st):  # noqa: F811
    C, N = cache(st), norm(st)
    f = st.strata_kv_append_normed
    assert st.lib().strata_kv_append_normed(C, None, A, 4096, 32, A, 1024, A, 1024, 4, A, None, None, 0, 0, 0, A, 4096,
                                            None, None) == 1
    q = dict(q=A, n_heads=32, q_out=2 * A)
    rope = dict(positions=A, rope=A, n_pos=100, rot_dim=128)
    assert f(cache(st, head_dim=96), N, A, A, 4, A) == 3
    assert f(C, N, A, A, -1, A) == 2
    assert f(C, N, None, A, 4, A) == 1
    assert f(C, N, A, A, 4, None) == 1
    assert f(C, N, A, A, 4, A, k_stride=1000) == 1
    assert f(C, N, A, A, 4, A, flags=2) == 1
    assert f(C, N, A, A, 4, A, q=A, n_heads=32) == 1
    assert f(C, N, A, A, 4, A, **{**q, "n_heads": 0}) == 3
    assert f(C, N, A, A, 4, A, **{**rope, "rot_dim": 24}) == 2
    assert f(C, N, A, A, 4, A, **{**rope, "rope": None}) == 1
    assert f(C, N, A, A, 0, None) == 0                            # nothing to do
    assert f(C, norm(st, q_weight=None, k_weight=None, q_head_stride=3), A, A, 0, None) == 0  # (no weights: no strides)


def test_weights_that_are_taken_and_refused():
    import int4_grouped_expert_gb300 as st
    one, heads = torch.ones(64), torch.ones(4, 64)
    n = st.QKNorm(one, heads, 64, eps=1e-5).struct()
    assert (n.q_head_stride, n.k_head_stride, n.k_weight) == (0, 64, heads.data_ptr())
    assert st.QKNorm(None, heads[:1], 64).struct().k_head_stride == 0
    assert st.QKNorm(None, None, 64).struct().q_weight is None
    for w, error in ((one.half(), TypeError), (one.double(), TypeError), (torch.ones(65), ValueError),
                     (torch.ones(2, 2, 64), ValueError), (torch.ones(64, 4).t(), ValueError),
                     (torch.ones(4, 128)[:, ::2], ValueError)):
        with pytest.raises(error):
            st.QKNorm(w, None, 64)
        with pytest.raises(error):
            st.QKNorm(None, w, 64)


def test_fewer_rows_of_weights_than_heads(st):  # noqa: F811
    C = cache(st, head_dim=64, n_kv_heads=4)
    f = st.strata_kv_append_normed
    for q, k in ((torch.ones(7, 64), None), (torch.ones(8, 64), torch.ones(3, 64))):
        with pytest.raises(ValueError):
            f(C, st.QKNorm(q, k, 64).struct(), A, A, 4, A, q=A, n_heads=8, q_out=2 * A)
    assert f(C, st.QKNorm(torch.ones(8, 64), torch.ones(4, 64), 64).struct(), A, A, 0, A, q=A, n_heads=8, q_out=2 * A) == 0
    assert f(C, st.QKNorm(torch.ones(7, 64), torch.ones(5, 64), 64).struct(), A, A, 0, A) == 0
