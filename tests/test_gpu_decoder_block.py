"""The example's decoder block: every call against its 64-bit definition on the inputs it got on the GPU, for
a batch of prompts, for pieces of prompts beside single tokens, and for steps through a captured graph."""
import os
import sys

import numpy as np
import pytest

import block_ref as ref
import oracle
from helpers import bf16_to_np_bits, compare_output

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

P, N_PAGES = 32, 30


def f64(t):
    return ref.bf16_bits_to_f64(bf16_to_np_bits(t.contiguous()))


class Twin:
    """Checks one forward call of the block, given what its buffers hold afterwards."""

    def __init__(self, block, cache):
        self.block, self.cache = block, cache
        codes = np.full((N_PAGES, block.Hkv, P, block.D), 0x7F, dtype=np.uint8)
        scales = np.full((N_PAGES, block.Hkv), np.nan, dtype=np.float32)
        self.cpu = ref.Cache(codes, codes, scales, scales)
        self.w_moe = {e: tuple((c[e].cpu().numpy(), s[e].cpu().numpy()) for c, s in (
            (block.moe.gate_codes, block.moe.gate_scales), (block.moe.up_codes, block.moe.up_scales),
            (block.moe.down_codes, block.moe.down_scales))) for e in range(block.moe.E)}

    def linear(self, lin, x, out, residual=None):
        want, bound = ref.linear(x, lin.codes.cpu().numpy().view(np.uint8), lin.scales.cpu().numpy(), lin.bits, 128,
                                 residual=residual, rounded_weights=len(x) > 64)
        assert (np.abs(out - want) <= bound).all()

    def check(self, x, batch_new, pages, slots, positions, b):
        k = self.block
        T, D, Hq, Hkv = len(x), k.D, k.Hq, k.Hkv
        qkv = f64(b["qkv"])
        # q in the buffer is rotated already: k and v show the projection, then q after the rotation
        w = np.s_[Hq * D:]
        full, bound = ref.linear(x, k.qkv.codes.cpu().numpy().view(np.uint8), k.qkv.scales.cpu().numpy(), 8, 128,
                                 rounded_weights=T > 64)
        assert (np.abs(qkv[:, w] - full[:, w]) <= bound[:, w]).all()
        rope = k.rope.cpu().numpy().astype(np.float64)
        h = k.rot // 2
        cos, sin = rope[positions, :h], rope[positions, h:]
        q, qm = ref.rotate(full[:, :Hq * D].reshape(T, Hq, D), cos, sin, k.rot, False)
        qb = bound[:, :Hq * D].reshape(T, Hq, D)
        # the projection's own error turns with it: at most the sum of the pair's two bounds
        pair = qb + np.concatenate([qb[..., h:], qb[..., :h]], -1)
        got_q = qkv[:, :Hq * D].reshape(T, Hq, D)
        lim = pair + 3 * ref.U32 * qm
        assert (np.abs(got_q - q) <= lim + ref.half_ulp_bf16(np.abs(q) + lim)).all()
        kk = qkv[:, Hq * D:(Hq + Hkv) * D].reshape(T, Hkv, D)
        vv = qkv[:, (Hq + Hkv) * D:].reshape(T, Hkv, D)
        kr, km = ref.rotate(kk, cos, sin, k.rot, False)
        want = ref.append(self.cpu, kr, vv, 3 * ref.U32 * km, slots, P)
        for kind, codes, scales in (("k", self.cache.k_codes, self.cache.k_scales),
                                    ("v", self.cache.v_codes, self.cache.v_scales)):
            import torch
            c = ref.E4M3[codes.view(torch.uint8).cpu().numpy()]
            s = scales.cpu().numpy().astype(np.float64)
            used = np.unique(pages.table[pages.table >= 0])
            np.testing.assert_array_equal(s[used], self.cpu.scales[kind][used])
            val, (wv, allow) = c * s[:, :, None, None], want[kind]
            at = np.asarray(slots)
            assert (np.abs(val - wv) <= allow)[at // P, :, at % P].all()
            self.cpu.codes[kind], self.cpu.scales[kind] = c, s
        seqs = [(int(L), int(n)) for L, n in zip(pages.length, batch_new)]
        att, bound = ref.attention(got_q, self.cpu, pages.table, seqs, P, k.scale)
        got = f64(b["att"]).reshape(T, Hq, D)
        assert (np.abs(got - att) <= bound).all()
        self.linear(k.o, got.reshape(T, -1), f64(b["mid"]), residual=x)
        m = k.moe
        r = oracle.moe_forward(bf16_to_np_bits(b["mid"]), m.w_router.cpu().numpy(), None, m.k,
                               lambda e: self.w_moe[e], m.E, 0, residual=True)
        compare_output(bf16_to_np_bits(b["out"]), r["out"], scale_max_abs=True)


def test_prompts_pieces_and_a_captured_step():
    import torch
    import int4_grouped_expert_gb300 as st
    import decoder_block as ex
    block = ex.random_block()
    cache = st.PagedKVCache(N_PAGES, block.Hkv, block.D, P)
    cache.k_codes.view(torch.uint8).fill_(0x7F)
    cache.v_codes.view(torch.uint8).fill_(0x7F)
    pages = ex.Pages(N_PAGES, P, 3, 320)
    twin = Twin(block, cache)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for new in ([37, 1, 140], [1, 60, 1], [33, 1, 1]):
        batch, slots, positions = ex.prompt_batch(pages, new)
        b = block.buffers(cache, batch)
        x = torch.randn(batch.T, block.H, device="cuda", generator=gen).bfloat16()
        block.forward(x, cache, batch, slots, positions, b)
        torch.cuda.synchronize()
        assert st.strata_read_status(b["status"]) == (0, 0)
        assert st.strata_workspace_status(b["ws_att"]) == (0, 0)
        twin.check(f64(x), new, pages, slots.cpu().numpy(), positions.cpu().numpy(), b)
    graph = ex.DecodeGraph(block, cache, pages, 3, 320)
    for _ in range(4):
        x = torch.randn(3, block.H, device="cuda", generator=gen).bfloat16()
        graph.step(x, pages)
        torch.cuda.synchronize()
        assert st.strata_read_status(graph.b["status"]) == (0, 0)
        assert st.strata_workspace_status(graph.b["ws_att"]) == (0, 0)
        twin.check(f64(x), [1, 1, 1], pages, graph.slots.cpu().numpy(), graph.positions.cpu().numpy(), graph.b)
