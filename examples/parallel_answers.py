"""Several answers to one prompt from shared pages, without the host in a step: normalised queries and keys, a window with
first tokens that stay visible, and page tables that live on the device.

    python examples/parallel_answers.py

A prompt goes through the decoder block of decoder_block.py once; its sequence is forked, so that all answers share its
pages; then a captured graph takes a token of every answer per replay: room for the tokens (an answer that would write
into a shared page gets one of its own), page copies, projection, append with norms, attention, output projection, MoE
layer, and the pages that fall between the first tokens and the window are given back. The host says which sequences go
on, and nothing else. Weights are random.
"""
from __future__ import annotations

import torch

from decoder_block import DecoderBlock, ROOT, random_block  # noqa: F401  (ROOT: the package is found)

import int4_grouped_expert_gb300 as st


class Server:
    """A decoder block, its cache, and who holds which pages."""

    def __init__(self, block: DecoderBlock, window, n_sinks, n_pages, n_seq, max_pages, page_size, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.block, self.window, self.n_sinks = block, window, n_sinks
        self.norm = st.QKNorm(*((1 + 0.2 * torch.randn(block.D, generator=g)).cuda() for _ in "qk"), block.D)
        self.pages = st.PageTable(n_pages, n_seq, max_pages, page_size)
        self.cache = st.PagedKVCache(n_pages, block.Hkv, block.D, page_size)
        self.layers = st.cache_array([self.cache])
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def fork(self, parent):
        """Sequence s goes on from where parent[s] is (-1: stays as it is)."""
        st.check(st.strata_kv_pages_fork(self.pages.struct(), torch.tensor(parent, dtype=torch.int32, device="cuda"),
                                         self.status), "fork")

    def end(self, sequences):
        keep = torch.full((self.pages.n_seq,), -1, dtype=torch.int32)
        keep[list(sequences)] = 0
        st.check(st.strata_kv_pages_release(self.pages.struct(), keep.cuda(), dev_status=self.status), "release")

    def check(self, rows: "Rows"):
        """Raises if a call since the last check reported a fault. Waits for the current stream."""
        DecoderBlock.check(rows.b)
        rc, bits = st.strata_read_status(self.status)
        if rc != 0:
            raise st.StrataError(rc, f"pages: device status 0x{bits:x}")


class Rows:
    """Calls for up to T new tokens at a time, at most max_q of one sequence; captured once if asked for."""

    def __init__(self, server: Server, T, max_q, capture=False):
        self.server, self.T = server, T
        p, ints = server.pages, dict(dtype=torch.int32, device="cuda")
        self.new, self.q_start = torch.zeros(p.n_seq, **ints), torch.zeros(p.n_seq + 1, **ints)
        self.slots, self.positions = torch.zeros(T, **ints), torch.zeros(T, **ints)
        self.copies, self.n_copies = torch.zeros(p.n_seq, 2, **ints), torch.zeros(1, **ints)
        self.x = torch.zeros(T, server.block.H, dtype=torch.bfloat16, device="cuda")
        self.batch = p.batch(self.q_start, T, max_q, p.max_pages * p.page_size)
        self.b = server.block.buffers(server.cache, self.batch)
        self.graph = None
        if capture:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):  # once outside the capture (no new token: nothing changes)
                self.calls()
            torch.cuda.current_stream().wait_stream(side)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.calls()

    def calls(self):
        s, b, T = self.server, self.b, self.T
        k, p = s.block, s.pages.struct()
        at_k, at_v, qkv = k.Hq * k.D, (k.Hq + k.Hkv) * k.D, b["qkv"]
        wide = qkv.stride(0)
        st.check(st.strata_kv_pages_extend(p, self.new, T, self.slots, self.positions, self.q_start, self.copies,
                                           self.n_copies, s.status), "extend")
        st.check(st.strata_kv_copy_pages(s.layers, s.layers, self.copies, self.n_copies, s.pages.n_seq, s.status), "copy")
        st.check(st.strata_linear_forward(k.qkv.struct(), self.x, T, qkv, b["ws_qkv"], b["ws_qkv"].numel()), "q/k/v")
        st.check(st.strata_kv_append_normed(
            s.cache.struct(), s.norm.struct(), qkv[:, at_k:], qkv[:, at_v:], T, self.slots, self.positions, k.rope,
            k.rope.shape[0], k.rot, q=qkv, n_heads=k.Hq, q_out=qkv, k_stride=wide, v_stride=wide, q_stride=wide,
            q_out_stride=wide, dev_status=s.status), "append")
        st.check(st.strata_attention_sinks_forward(
            s.cache.struct(), self.batch, qkv, k.Hq, k.scale, b["att"], b["ws_att"], b["ws_att"].numel(),
            window=s.window, n_sinks=s.n_sinks, flags=st.STRATA_WS_REUSE, q_stride=wide), "attention")
        st.check(st.strata_linear_forward(k.o.struct(), b["att"], T, b["mid"], b["ws_o"], b["ws_o"].numel(),
                                          residual=self.x), "output projection")
        st.check(st.strata_moe_forward(k.moe.struct(), b["mid"], T, b["out"], b["ws_moe"], b["ws_moe"].numel()), "MoE layer")
        st.check(st.strata_kv_pages_release(p, None, s.window, s.n_sinks, s.status), "release")
        for word in b["words"]:
            b["status"] |= word

    def run(self, x, new):
        """new[s] more tokens of each sequence, whose rows x holds one sequence after another; their outputs."""
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.x[:x.shape[0]].copy_(x)
        if self.graph is None:
            self.calls()
        else:
            self.graph.replay()
        return self.b["out"][:x.shape[0]]


def next_inputs(out):  # (a model would sample here: rows with a little noise stand in for the next inputs)
    y = torch.nn.functional.normalize(out.float(), dim=1) * out.shape[1] ** 0.5
    return (y + 0.3 * torch.randn_like(y)).bfloat16()


def main():
    answers, prompt, steps, P = 8, 300, 200, 32
    server = Server(random_block(), window=128, n_sinks=4, n_pages=120, n_seq=answers, max_pages=20, page_size=P)
    first = Rows(server, prompt, prompt)
    out = first.run(torch.randn(prompt, server.block.H, device="cuda").bfloat16(), [prompt] + [0] * (answers - 1))
    server.check(first)
    server.fork([-1] + [0] * (answers - 1))
    tokens = Rows(server, answers, 1, capture=True)
    x = next_inputs(out[-1:].expand(answers, -1))
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(steps):
        x = next_inputs(tokens.run(x, [1] * answers))
    end.record()
    torch.cuda.synchronize()
    server.check(tokens)
    assert torch.isfinite(x.float()).all()
    used = int((server.pages.refs > 0).sum())
    server.end(range(answers))
    assert not server.pages.refs.any()
    print(f"{answers} answers of {steps} tokens to a prompt of {prompt}: {begin.elapsed_time(end) / steps * 1e3:.0f} us a "
          f"step (host work between replays included), {used} pages in use at the end")


if __name__ == "__main__":
    main()
