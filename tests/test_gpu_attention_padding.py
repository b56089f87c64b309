"""Row buffers larger than the rows of a batch: rows of no sequence are neither read nor written, also where the
sizes are those of sequences of equal length."""
import numpy as np
import pytest

import block_ref as ref
from helpers import bf16_tensor
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,max_q", [
    ([(300, 1), (90, 0), (17, 1)], 1),                    # T of 3 single tokens, 2 of them there
    ([(300, 4), (90, 2), (64, 1)], 4),
    ([(300, 20), (200, 3), (50, 0)], 20),                 # some rows few, some many
    ([(700, 300), (200, 17), (300, 150)], 300),
    ([(4100, 64), (900, 1)], 64),                         # cut along the tokens
    ([(200, 1)] * 100 + [(300, 0)] * 20, 1)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T_more", [0, 5])
def test_rows_of_no_sequence(seqs, max_q, D, T_more):
    import torch
    import int4_grouped_expert_gb300 as st
    c = Case(seqs, 8, 2, D, 32).gpu()
    want, bound = c.reference()
    T = len(seqs) * max_q + T_more
    q = np.full((T, 8 * D), 0x7FC0, dtype=np.uint16)      # nan in the rows of no sequence
    q[:c.T] = c.q_bits
    out = torch.full((T, 8 * D), -7.0, dtype=torch.bfloat16, device="cuda")
    batch = st.kv_batch(*c.batch.tensors, T, max_q, max(L for L, _ in seqs))
    n = st.strata_attention_workspace_size(c.cache.struct(), batch, 8)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    st.check(st.strata_attention_forward(c.cache.struct(), batch, bf16_tensor(q), 8, c.scale, out, ws, n), "attention")
    torch.cuda.synchronize()
    assert st.strata_workspace_status(ws) == (0, 0)
    got = out[:c.T].float().cpu().numpy().astype(np.float64).reshape(want.shape)
    assert (np.abs(got - want) <= bound).all()
    assert (out[c.T:] == -7).all()
