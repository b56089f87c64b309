"""What the weights behind the norms of queries and keys have to be beside dtype and layout: rows that exist, as wide as the
cache's heads, and alive as long as the descriptor."""
import pytest
import torch

from test_block_abi_cpu import A, cache, st  # noqa: F401


@pytest.mark.parametrize("w", [torch.ones(0, 64), torch.ones(0)])
def test_weights_without_rows_are_refused(w):
    """(Their address is null, which to the library means no norm.)"""
    import int4_grouped_expert_gb300 as st  # noqa: F811
    for q, k in ((w, None), (None, w), (torch.ones(64), w)):
        with pytest.raises(ValueError):
            st.QKNorm(q, k, w.shape[-1])


@pytest.mark.parametrize("dim,other", [(64, 128), (128, 64)])
def test_weights_of_another_width_than_the_heads(st, dim, other):  # noqa: F811
    C = cache(st, head_dim=other, n_kv_heads=4)
    f = st.strata_kv_append_normed
    for q, k in ((torch.ones(dim), None), (None, torch.ones(dim)), (torch.ones(8, dim), torch.ones(4, dim))):
        n = st.QKNorm(q, k, dim).struct()
        with pytest.raises(ValueError):
            f(C, n, A, A, 4, A, q=A, n_heads=8, q_out=2 * A)
        assert f(cache(st, head_dim=dim, n_kv_heads=4), n, A, A, 0, A, q=A, n_heads=8, q_out=2 * A) == 0
    assert f(C, st.QKNorm(None, None, dim).struct(), A, A, 0, A) == 0  # (no weights: no width)
