"""The cache append with norms where a block takes 16, 8 or 4 heads of a row at a time, and where a thread goes on to more
heads than the five that it has on their way at the start. (On 152 SMs 16 heads up to 1216 rows of 128-wide
heads, 8 up to 2432; twice as many rows of 64-wide heads.)"""
import numpy as np
import pytest

from test_gpu_kv_append import slots_of
from test_gpu_kv_append_normed import NormRun

pytestmark = pytest.mark.gpu


def rows_of(r, T, P):
    """T rows of three sequences, which end inside pages. The cache's last page is left."""
    n = [T // 2 + 1, T // 3, T - T // 2 - 1 - T // 3]
    order, at, parts = r.rng.permutation(r.shape[0] - 1), 0, []
    for i in n:
        pages = -(-i // P)
        parts.append(slots_of(order[at:at + pages], 0, i, P))
        at += pages
    return np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts]) % r.n_pos


@pytest.mark.parametrize("D,T", [(128, 1216), (128, 1217), (128, 1500), (128, 2432), (128, 2433), (128, 3001),
                                 (64, 2432), (64, 2433), (64, 2600), (64, 4864), (64, 4865), (64, 5003)])
@pytest.mark.parametrize("Hq,per_head", [(28, False), (50, True)])
def test_prompts(D, T, Hq, per_head):
    P = 64
    r = NormRun(-(-T // P) + 4, 2, D, P, seed=T)
    r.append(*rows_of(r, T, P), Hq=Hq, per_head=per_head, in_place=T % 2, neighbours=T % 3 == 0, pad=8)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq", [80, 81, 96, 97, 160, 200])
def test_more_heads_than_are_on_their_way(D, Hq):
    """Few rows, 16 heads at a time: from the 81st head on a thread's copies take places that it has read."""
    r = NormRun(8, 2, D, 16)
    r.append(*rows_of(r, 45, 16), Hq=Hq, per_head=True)
    r.append(*slots_of([7], 0, 1, 16), Hq=Hq, in_place=True)


@pytest.mark.parametrize("T", [1300, 2500])
def test_many_heads_of_prompts(T):
    r = NormRun(-(-T // 128) + 4, 1, 128, 128, seed=T)
    r.append(*rows_of(r, T, 128), Hq=66, rot=64, in_place=True)
