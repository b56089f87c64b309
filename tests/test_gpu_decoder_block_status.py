"""The example's decoder block keeps what its calls report: the projections and the MoE layer clear their status
words at every call."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("call,workspace", [("strata_linear_forward", 4), ("strata_moe_forward", 4)])
def test_a_status_of_one_step_survives_the_next(monkeypatch, call, workspace):
    """A call whose workspace says that a wait gave up (written by the test, after the call), then a step
    without a fault."""
    import torch
    import int4_grouped_expert_gb300 as st
    import decoder_block as ex
    block = ex.random_block()
    cache = st.PagedKVCache(8, block.Hkv, block.D, 32)
    pages = ex.Pages(8, 32, 2, 128)
    batch, slots, positions = ex.prompt_batch(pages, [3, 40])
    b = block.buffers(cache, batch)
    x = torch.randn(batch.T, block.H, device="cuda").bfloat16()
    args = (x, cache, batch, slots, positions, b)
    block.forward(*args)
    block.check(b)
    real = getattr(st, call)

    def faulty(*a, **kw):
        rc = real(*a, **kw)
        a[workspace][:4].view(torch.int32).fill_(st.STRATA_DEV_TIMEOUT)
        return rc

    monkeypatch.setattr(st, call, faulty)
    block.forward(*args)
    monkeypatch.undo()
    block.forward(*args)
    with pytest.raises(st.StrataError):
        block.check(b)
    block.forward(*args)
    block.check(b)
