"""Calls of different sizes from two host threads at once: every launch is taken, whatever shared memory the other's needs."""
import threading

import pytest

pytestmark = pytest.mark.gpu


def refused(sizes, make, calls):
    """How many calls of each thread failed. make(size) gives a call on the thread's own stream and tensors."""
    import torch
    count = [None] * len(sizes)

    def work(i):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            call = make(sizes[i])
            n = sum(call(side) != 0 for _ in range(calls))
            side.synchronize()
            count[i] = n

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return count


def test_grouping_of_rows():
    import torch
    import int4_grouped_expert_gb300 as st
    T, k = 30, 8

    def make(E):
        i32 = dict(dtype=torch.int32, device="cuda")
        ids, ws = torch.randint(0, E, (T, k), **i32), torch.zeros(st.GROUP_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
        out = [torch.zeros(n, **i32) for n in (E, E + 1, T * k, T * k)]
        return lambda side: st.strata_group_rows(ids, T, k, E, *out, ws, ws.numel(), stream=side)

    assert refused((700, 1024), make, 30000) == [0, 0]


def test_layers_of_few_tokens():
    import torch
    import int4_grouped_expert_gb300 as st
    T = 64  # (T * k rows: 800 experts take 54 KB, 1024 69 KB)

    def make(E):
        L = st.MoELayer(128, 128, E, 8, 0)
        x = torch.randn(T, 128, device="cuda").bfloat16()
        out, s = torch.empty_like(x), L.struct()
        ws = torch.zeros(L.workspace_size(T), dtype=torch.uint8, device="cuda")
        call = lambda side: st.strata_moe_forward(s, x, T, out, ws, ws.numel(), stream=side)  # noqa: E731
        call.holds = L
        return call

    assert refused((800, 1024), make, 10000) == [0, 0]
