"""What the tensors behind the projection, cache and batch descriptors have to be: the library sees addresses
only, so the binding refuses other element types and layouts. No GPU is needed."""
import pytest
import torch

import int4_grouped_expert_gb300 as st


def i32(*a):
    return torch.tensor(a, dtype=torch.int32)


TABLE = torch.zeros(2, 6, dtype=torch.int32)


def test_batches_that_are_taken():
    b = st.kv_batch(i32(0, 1, 3), i32(5, 9), TABLE, T=3, max_q=2, max_kv=9)
    assert b.n_seq == 2 and b.table_stride == 6 and b.q_start == b.tensors[0].data_ptr()
    wide = torch.zeros(4, 50, dtype=torch.int32)
    assert st.kv_batch(i32(0, 1, 3, 7), i32(5, 9), wide[:, 10:20], T=3, max_q=2, max_kv=9).table_stride == 50
    assert st.kv_batch(i32(0, 1), i32(5), torch.zeros(1, 1, dtype=torch.int32), T=1, max_q=1, max_kv=5).n_seq == 1
    assert st.kv_batch(i32(0), i32(), torch.zeros(0, 4, dtype=torch.int32), T=0, max_q=0, max_kv=0).n_seq == 0


@pytest.mark.parametrize("start,length,table,error", [
    (torch.cumsum(i32(0, 1, 2), 0), i32(5, 9), TABLE, TypeError),          # (int64)
    (i32(0, 1, 3), i32(5, 9).long(), TABLE, TypeError),
    (i32(0, 1, 3), i32(5, 9), TABLE.long(), TypeError),
    (i32(0, 1), i32(5, 9), TABLE, ValueError),                             # a start is missing
    (i32(0, 9, 1, 9, 3, 9)[::2], i32(5, 9), TABLE, ValueError),
    (i32(0, 1, 3), i32(5, 0, 9, 0)[::2], TABLE, ValueError),
    (i32(0, 1, 3), i32(5, 9), torch.zeros(6, 2, dtype=torch.int32).t(), ValueError),
    (i32(0, 1, 3), i32(5, 9), TABLE[:1], ValueError)])
def test_batches_that_are_refused(start, length, table, error):
    with pytest.raises(error):
        st.kv_batch(start, length, table, T=3, max_q=2, max_kv=9)


def test_projections():
    N, K = 6, 256
    u8, f16 = torch.uint8, torch.float16
    st.QuantLinear(torch.zeros(N, K // 2, dtype=u8), torch.zeros(N, 2, dtype=f16), N, K)
    st.QuantLinear(torch.zeros(N, K, dtype=torch.int8), torch.zeros(N, 4, dtype=f16), N, K, 8, 64, torch.zeros(N))
    st.QuantLinear(1 << 12, 1 << 12, N, K)                                 # addresses
    st.QuantLinear(torch.zeros(N, K // 2, dtype=u8), torch.zeros(N, 2, dtype=f16), N, K, 0, 0)  # (the defaults)
    for codes, scales, bias, error in (
            (torch.zeros(N, K // 2, dtype=torch.int16), torch.zeros(N, 2, dtype=f16), None, TypeError),
            (torch.zeros(N, K, dtype=u8), torch.zeros(N, 2, dtype=f16), None, ValueError),
            (torch.zeros(K // 2, N, dtype=u8).t(), torch.zeros(N, 2, dtype=f16), None, ValueError),
            (torch.zeros(N, K // 2, dtype=u8), torch.zeros(N, 2), None, TypeError),
            (torch.zeros(N, K // 2, dtype=u8), torch.zeros(2, N, dtype=f16).t(), None, ValueError),
            (torch.zeros(N, K // 2, dtype=u8), torch.zeros(N, 2, dtype=f16), torch.zeros(N).double(), TypeError)):
        with pytest.raises(error):
            st.QuantLinear(codes, scales, N, K, bias=bias)


def test_caches():
    shape = (3, 2, 16, 64)
    codes, scales = torch.zeros(shape, dtype=torch.uint8), torch.zeros(3, 2)
    st.PagedKVCache(3, 2, 64, 16, codes, codes.view(torch.float8_e4m3fn), scales, scales, device="cpu")
    for c, s, error in ((codes.half(), scales, TypeError), (codes[:2], scales, ValueError),
                        (codes.transpose(1, 2), scales, ValueError), (codes, scales.half(), TypeError),
                        (codes, torch.zeros(2, 3).t(), ValueError)):
        with pytest.raises(error):
            st.PagedKVCache(3, 2, 64, 16, c, codes, s, scales, device="cpu")
        with pytest.raises(error):
            st.PagedKVCache(3, 2, 64, 16, codes, c, scales, s, device="cpu")
