"""One decoder block on the library's calls: quantized q/k/v projection, rotation and cache append, attention
over the paged 8-bit cache, quantized output projection with residual, routed MoE layer with residual.

    python examples/decoder_block.py

runs three prompts of different lengths in one batch, then single tokens through a CUDA graph that was
captured once (lengths, slots and positions are device arrays that the host rewrites before each
replay), and prints the time of a step. The q/k/v projection has 8-bit weights and the output projection
4-bit ones, as "Strata" MoE tuning notes (lpnh.cn/news/2730718, §2.1) keep them; weights are random and
no normalisation is applied (none is named there).
"""
from __future__ import annotations

import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402
import torch  # noqa: E402

import int4_grouped_expert_gb300 as st  # noqa: E402


class Pages:
    """Host-side page tables: hands out cache pages and lists the slots of new tokens."""

    def __init__(self, n_pages: int, page_size: int, n_seq: int, max_len: int):
        self.free = list(range(n_pages - 1, -1, -1))
        self.P = page_size
        self.table = np.full((n_seq, -(-max_len // page_size)), -1, dtype=np.int32)
        self.length = np.zeros(n_seq, dtype=np.int32)

    def extend(self, new):
        """Makes room for new[s] tokens of each sequence: (slots, positions) of the rows, in order."""
        slots, positions = [], []
        for s, n in enumerate(new):
            for pos in range(self.length[s], self.length[s] + n):
                if pos % self.P == 0:
                    self.table[s, pos // self.P] = self.free.pop()
                slots.append(self.table[s, pos // self.P] * self.P + pos % self.P)
                positions.append(pos)
            self.length[s] += n
        return np.array(slots, dtype=np.int32), np.array(positions, dtype=np.int32)


class DecoderBlock:
    def __init__(self, H, Hq, Hkv, D, moe: "st.MoELayer", wqkv, wo, max_pos=4096, rot_dim=None):
        """wqkv [(Hq + 2 Hkv) D, H] and wo [H, Hq D]: fp16; moe: a layer of hidden size H."""
        self.H, self.Hq, self.Hkv, self.D = H, Hq, Hkv, D
        self.qkv = st.QuantLinear.from_fp16(wqkv, bits=8)
        self.o = st.QuantLinear.from_fp16(wo, bits=4)
        self.moe = moe
        moe.flags |= st.STRATA_ADD_RESIDUAL
        self.rot = D if rot_dim is None else rot_dim
        self.rope = st.rope_table(max_pos, self.rot)
        self.scale = 1.0 / math.sqrt(D)

    def buffers(self, cache, batch):
        """Activations and workspaces of a batch of up to batch.T rows, allocated once."""
        T = batch.T
        bf = dict(dtype=torch.bfloat16, device="cuda")
        b = {"qkv": torch.empty(T, (self.Hq + 2 * self.Hkv) * self.D, **bf),
             "att": torch.empty(T, self.Hq * self.D, **bf), "mid": torch.empty(T, self.H, **bf),
             "out": torch.empty(T, self.H, **bf), "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
        sizes = {"ws_qkv": self.qkv.workspace_size(T), "ws_o": self.o.workspace_size(T),
                 "ws_att": st.strata_attention_workspace_size(cache.struct(), batch, self.Hq),
                 "ws_moe": self.moe.workspace_size(T)}
        for name, n in sizes.items():
            b[name] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        b["words"] = [b[name][:4].view(torch.int32) for name in ("ws_qkv", "ws_o", "ws_moe")]
        return b

    def forward(self, x, cache, batch, slots, positions, b):
        """x [T, H] bf16 -> b["out"]. Every call is asynchronous on torch's current stream."""
        T, D = batch.T, self.D
        q, k = self.Hq * D, (self.Hq + self.Hkv) * D
        qkv, wide = b["qkv"], b["qkv"].stride(0)
        st.check(st.strata_linear_forward(self.qkv.struct(), x, T, qkv, b["ws_qkv"], b["ws_qkv"].numel()), "q/k/v")
        # q turns in place, k and v go to the cache
        st.check(st.strata_kv_append(cache.struct(), qkv[:, q:], qkv[:, k:], T, slots, positions, self.rope,
                                     self.rope.shape[0], self.rot, q=qkv, n_heads=self.Hq, q_out=qkv, k_stride=wide,
                                     v_stride=wide, q_stride=wide, q_out_stride=wide, dev_status=b["status"]), "append")
        st.check(st.strata_attention_forward(cache.struct(), batch, qkv, self.Hq, self.scale, b["att"], b["ws_att"],
                                             b["ws_att"].numel(), flags=st.STRATA_WS_REUSE, q_stride=wide), "attention")
        st.check(st.strata_linear_forward(self.o.struct(), b["att"], T, b["mid"], b["ws_o"], b["ws_o"].numel(),
                                          residual=x), "output projection")
        st.check(st.strata_moe_forward(self.moe.struct(), b["mid"], T, b["out"], b["ws_moe"], b["ws_moe"].numel()),
                 "MoE layer")
        # projections and the MoE layer clear their status words at every call: what they found is kept here
        for word in b["words"]:
            b["status"] |= word
        return b["out"]

    @staticmethod
    def check(b):
        """Raises if a call since the last check reported a fault. Waits for the current stream."""
        for name, (rc, bits) in (("attention", st.strata_workspace_status(b["ws_att"])),
                                 ("append, projections, MoE layer", st.strata_read_status(b["status"]))):
            if rc != 0:
                raise st.StrataError(rc, f"{name}: device status 0x{bits:x}")


def random_block(H=1024, I=512, E=16, k=2, Hq=8, Hkv=2, D=128, seed=0):
    g = torch.Generator().manual_seed(seed)
    moe = st.MoELayer(H, I, E, k, shared=0)
    moe.set_router(torch.randn(E, H, generator=g) * 0.02)
    for e in range(E):
        moe.load_expert_fp16(e, *((torch.randn(s, generator=g) * 0.02).half() for s in ((I, H), (I, H), (H, I))))
    wqkv = (torch.randn((Hq + 2 * Hkv) * D, H, generator=g) * 0.03).half()
    wo = (torch.randn(H, Hq * D, generator=g) * 0.03).half()
    return DecoderBlock(H, Hq, Hkv, D, moe, wqkv, wo)


def to_gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def prompt_batch(pages: Pages, new):
    """Descriptor, slots and positions of a batch that adds new[s] tokens to each sequence."""
    slots, positions = pages.extend(new)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    batch = st.kv_batch(to_gpu(start), to_gpu(pages.length), to_gpu(pages.table), T=int(start[-1]),
                        max_q=int(max(new)), max_kv=int(pages.length.max()))
    return batch, to_gpu(slots), to_gpu(positions)


class DecodeGraph:
    """One captured step of a token per sequence; lengths up to max_kv."""

    def __init__(self, block, cache, pages: Pages, n_seq, max_kv):
        dev = dict(dtype=torch.int32, device="cuda")
        self.start = torch.arange(n_seq + 1, **dev)
        self.length, self.slots = torch.zeros(n_seq, **dev), torch.full((n_seq,), -1, **dev)
        self.positions, self.table = torch.zeros(n_seq, **dev), to_gpu(pages.table)
        self.batch = st.kv_batch(self.start, self.length, self.table, T=n_seq, max_q=1, max_kv=max_kv)
        self.b = block.buffers(cache, self.batch)
        self.x = torch.zeros(n_seq, block.H, dtype=torch.bfloat16, device="cuda")
        args = (self.x, cache, self.batch, self.slots, self.positions, self.b)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):   # once outside the capture (slots of -1: nothing is stored)
            block.forward(*args)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            block.forward(*args)

    def step(self, x, pages: Pages):
        slots, positions = pages.extend([1] * len(pages.length))
        for dst, src in ((self.slots, slots), (self.positions, positions), (self.length, pages.length),
                         (self.table, pages.table)):
            dst.copy_(torch.from_numpy(src))
        self.x.copy_(x)
        self.graph.replay()
        return self.b["out"]


def main():
    block = random_block()
    prompts, steps, P = [37, 300, 129], 20, 64
    max_len = max(prompts) + steps + 1
    pages = Pages(40, P, len(prompts), max_len)
    cache = st.PagedKVCache(40, block.Hkv, block.D, P)
    batch, slots, positions = prompt_batch(pages, prompts)
    b = block.buffers(cache, batch)
    x = torch.randn(batch.T, block.H, device="cuda").bfloat16()
    out = block.forward(x, cache, batch, slots, positions, b)
    block.check(b)
    last = np.cumsum(prompts) - 1
    graph = DecodeGraph(block, cache, pages, len(prompts), max_len)
    tok = out[to_gpu(last)]

    def next_input(row):  # (a model would sample here: the output row stands in for the next input)
        return torch.nn.functional.normalize(row.float(), dim=1).mul(math.sqrt(block.H)).bfloat16()

    tok = graph.step(next_input(tok), pages)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(steps):
        tok = graph.step(next_input(tok), pages)
    end.record()
    torch.cuda.synchronize()
    block.check(graph.b)
    assert torch.isfinite(tok.float()).all()
    print(f"{sum(prompts)} prompt tokens, then {steps} steps of {len(prompts)} tokens: "
          f"{begin.elapsed_time(end) / steps * 1e3:.0f} us a step (host work between replays included)")


if __name__ == "__main__":
    main()
