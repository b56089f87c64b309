"""Weights quantized on another stream than the one that makes them."""
import pytest

pytestmark = pytest.mark.gpu


def test_quantizing_on_another_stream_waits_for_the_weights():
    import torch
    import int4_grouped_expert_gb300 as st
    torch.manual_seed(0)
    w = torch.randn(2048, 2048, device="cuda")
    want = st.QuantLinear.from_fp16(w, bits=4)
    big = torch.randn(8192, 8192, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        late = torch.zeros_like(w)
        for _ in range(4):
            big = big @ big * 1e-3                 # the current stream is busy for a while,
        late.copy_(w)                              # then makes the weights
        got = st.QuantLinear.from_fp16(late, bits=4, stream=handle)
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
