"""A descriptor keeps the tensors alive whose addresses it holds, also where the object that made it is gone."""
import gc
import weakref

import torch


def alive(make, *shapes):
    """make(*tensors) gives the descriptor; shapes: (dtype, size ...) of each tensor."""
    tensors = [torch.zeros(size, dtype=dtype) for dtype, *size in shapes]
    refs = [weakref.ref(t) for t in tensors]
    kept = make(*tensors)
    del tensors
    gc.collect()
    return kept is not None and all(r() is not None for r in refs)


U8, F16, F32, I32 = torch.uint8, torch.float16, torch.float32, torch.int32
CACHE = [(U8, 3, 2, 16, 64), (U8, 3, 2, 16, 64), (F32, 3, 2), (F32, 3, 2)]


def test_norms():
    import int4_grouped_expert_gb300 as st
    assert alive(lambda q, k: st.QKNorm(q, k, 64).struct(), (F32, 64), (F32, 4, 64))


def test_page_tables():
    import int4_grouped_expert_gb300 as st
    assert alive(lambda t, n, r: st.PageTable(10, 3, 4, 16, t, n, r).struct(), (I32, 3, 4), (I32, 3), (I32, 10))


def test_batches():
    import int4_grouped_expert_gb300 as st
    assert alive(lambda s, n, t: st.kv_batch(s, n, t, T=3, max_q=2, max_kv=9), (I32, 4), (I32, 3), (I32, 3, 4))


def test_caches():
    import int4_grouped_expert_gb300 as st
    assert alive(lambda *t: st.PagedKVCache(3, 2, 64, 16, *t).struct(), *CACHE)


def test_arrays_of_caches():
    import int4_grouped_expert_gb300 as st
    assert alive(lambda *t: st.cache_array([st.PagedKVCache(3, 2, 64, 16, *t)]), *CACHE)


def test_projections():
    import int4_grouped_expert_gb300 as st
    assert alive(lambda c, s, b: st.QuantLinear(c, s, 6, 256, bias=b).struct(), (U8, 6, 128), (F16, 6, 2), (F32, 6))
