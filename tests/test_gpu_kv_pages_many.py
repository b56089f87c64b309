"""The page calls with as many sequences as they take, and room made from two threads at once."""
import threading

import numpy as np
import pytest

from test_gpu_kv_pages import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_seq", [24576, 24577, 30000, 65535])
def test_many_sequences(n_seq):
    rng = np.random.default_rng(n_seq)
    p = Pool(2 * n_seq + 50, n_seq, 3, 16, apart=1)
    p.extend(rng.integers(0, 20, n_seq))
    held, empty = np.nonzero(p.cpu.length)[0], np.nonzero(p.cpu.length == 0)[0]
    parent = np.full(n_seq, -1)
    parent[empty] = rng.choice(held, len(empty))
    p.fork(parent)
    p.extend(np.minimum(rng.integers(0, 9, n_seq), 48 - p.cpu.length))
    p.extend((p.cpu.length < 48) * 1, T_max=n_seq // 2)
    p.release(np.where(rng.random(n_seq) < 0.3, rng.integers(0, 30, n_seq), -1), window=20, sinks=3)
    p.cpu.check()
    p.compact(int((p.cpu.refs > 0).sum()))


def test_two_threads_make_room_for_different_numbers_of_sequences():
    """Every call is taken: what one thread's launch needs of shared memory does not go by the other's."""
    import torch
    import int4_grouped_expert_gb300 as st
    sizes, refused = (25000, 65535), [None, None]
    i32 = dict(dtype=torch.int32, device="cuda")

    def work(i):
        n = sizes[i]
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            p, new = st.PageTable(n, n, 1, 16), torch.zeros(n, **i32)
            out = [torch.zeros(k, **i32) for k in (8, 8, n + 1, 2 * n, 1)]
            n = sum(st.strata_kv_pages_extend(p.struct(), new, 8, *out, stream=side) != 0 for _ in range(3000))
            side.synchronize()
            refused[i] = n

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert refused == [0, 0]
