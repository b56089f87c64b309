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
