"""The cache append with rows that are skipped inside a page: a position out of range between good
rows leaves a hole, and the page keeps one scale for what was stored around it."""
import numpy as np
import pytest

import block_ref as ref
from helpers import bf16_tensor
from workloads import gen

pytestmark = pytest.mark.gpu

Hkv, N_POS = 2, 500


def bf16(a):
    return gen.f32_to_bf16_bits(np.asarray(a, dtype=np.float32))


class Cache:
    def __init__(self, n_pages, P, D, seed):
        import torch
        import int4_grouped_expert_gb300 as st
        self.P, self.D, self.rng = P, D, np.random.default_rng(seed)
        shape = (n_pages, Hkv, P, D)
        c = np.full(shape, 0x7F, dtype=np.uint8)
        s = np.full(shape[:2], np.nan, dtype=np.float32)
        t = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        self.gpu = st.PagedKVCache(n_pages, Hkv, D, P, t(c), t(c), t(s), t(s))
        ang = self.rng.uniform(0, 2 * np.pi, (N_POS, D // 2))
        self.table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
        self.stored = {}                     # slot -> (k, v, k error) in 64 bits
        self.scales = {}                     # page -> {"k": [Hkv], "v": [Hkv]}

    def bits(self):
        return [t.cpu().numpy().tobytes() for t in (self.gpu.k_codes, self.gpu.v_codes, self.gpu.k_scales,
                                                    self.gpu.v_scales)]

    def append(self, slots, bad, size=1.0):
        """Rows with good positions but for those in `bad`; checks every stored slot of the cache."""
        import torch
        import int4_grouped_expert_gb300 as st
        T, D, P, h = len(slots), self.D, self.P, self.D // 2
        k, v = (bf16(self.rng.standard_normal((T, Hkv, D)) * size) for _ in "kv")
        for i in bad:
            k[i] = bf16(1e30)                # would give the page another scale
            v[i] = bf16(1e30)
        pos = self.rng.integers(0, N_POS, T).astype(np.int32)
        for n, i in enumerate(bad):
            pos[i] = (-1, N_POS, 1 << 30, -(1 << 31))[n % 4]
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        st.check(st.strata_kv_append(self.gpu.struct(), bf16_tensor(k.reshape(T, -1)), bf16_tensor(v.reshape(T, -1)), T,
                                     t(np.asarray(slots, dtype=np.int32)), t(pos), t(self.table), N_POS, D,
                                     dev_status=status), "append")
        torch.cuda.synchronize()
        assert st.strata_read_status(status)[1] == (st.STRATA_DEV_BAD_SLOT if bad else 0)
        good = np.array([i for i in range(T) if i not in set(bad)], dtype=int)
        at = np.where(np.isin(np.arange(T), good), pos, 0)
        kr, km = ref.rotate(ref.bf16_bits_to_f64(k), self.table[at, :h].astype(float), self.table[at, h:].astype(float),
                            D, False)
        vr = ref.bf16_bits_to_f64(v)
        slots = np.asarray(slots)
        for p in np.unique(slots[good] // P):
            rows = good[slots[good] // P == p]
            first = slots[slots // P == p].min() % P
            old = self.scales.get(p, {}) if first else {}
            if not first:
                self.stored = {s: x for s, x in self.stored.items() if s // P != p}
            now = {}
            for kind, x in (("k", kr), ("v", vr)):
                now[kind] = np.array([ref.append_scale(np.abs(x[rows, n]).max()) for n in range(Hkv)])
                if old:
                    now[kind] = np.maximum(now[kind], old[kind])
            self.scales[p] = now
            for i in rows:
                self.stored[slots[i]] = (kr[i], vr[i], 3 * ref.U32 * km[i])
        self.check()

    def check(self):
        import torch
        P = self.P
        codes = {n: ref.E4M3[getattr(self.gpu, n + "_codes").view(torch.uint8).cpu().numpy()] for n in "kv"}
        scales = {n: getattr(self.gpu, n + "_scales").cpu().numpy().astype(np.float64) for n in "kv"}
        for p in range(scales["k"].shape[0]):
            for n in "kv":
                want = self.scales[p][n] if p in self.scales else np.full(Hkv, np.nan)
                np.testing.assert_array_equal(scales[n][p], want)
        for s, (k, v, err) in self.stored.items():
            p, o = divmod(s, P)
            for n, x, e in (("k", k, err), ("v", v, 0.0)):
                now = self.scales[p][n][:, None]
                # each rounding to a code is off by half a step at most: one when it was stored, one for
                # every time the page's scale grew since (three here, each at a larger scale: their sum is
                # below twice the last)
                allow = 2 * 0.5 * ref.e4m3_step(x / now) * now + e
                assert (np.abs(codes[n][p, :, o] * now - x) <= allow).all(), (s, n)
        return codes


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_a_hole_inside_a_page(P, D):
    """On a fresh page and on one with older tokens, growing scales, holes first, last and between."""
    c = Cache(4, P, D, P + D)
    page = lambda p, a, b: list(range(p * P + a, p * P + b))  # noqa: E731
    c.append(page(1, 0, 7), [3])
    c.append(page(1, 7, 10), [1], size=30.0)
    c.append(page(1, 10, 13), [0], size=1e3)
    c.append(page(1, 13, 16), [2], size=1.0)
    c.append(page(2, 0, 9), [0, 1, 4, 8])                    # the page begins with holes
    c.append(page(2, 9, 12), [0, 2], size=100.0)
    c.append(page(3, 0, P), [P // 2, P // 2 + 1, P - 1])     # a whole page
    codes = c.check()
    assert np.isnan(codes["k"][3, :, P // 2]).all() and np.isnan(codes["v"][3, :, P - 1]).all()


def test_a_run_of_holes_changes_nothing():
    c = Cache(3, 16, 64, 1)
    c.append(list(range(16, 24)), [])
    before = c.bits()
    c.append([24, 25, 32, 33, 34], [0, 1, 2, 3, 4])
    assert c.bits() == before
    c.append([26, 27], [], size=50.0)


@pytest.mark.parametrize("P,D", [(16, 64), (32, 128), (128, 64), (128, 128)])
def test_holes_in_prompts(P, D):
    """Long calls: a block starts the runs of many rows, and pages end inside its share."""
    n_pages = 60
    c = Cache(n_pages, P, D, 7)
    order = c.rng.permutation(n_pages)[:min(n_pages, 2400 // P)]
    slots = (order[:, None] * P + np.arange(P)).reshape(-1)
    c.append(slots[:-5], sorted(c.rng.choice(len(slots) - 5, 150, replace=False).tolist()))
    c.append(slots[-5:], [1, 3], size=20.0)


def test_several_sequences_with_holes_give_the_same_bits():
    """Single tokens and short pieces, each page one writer: the same codes every time."""
    first = None
    for _ in range(10):
        c = Cache(40, 16, 64, 11)
        c.append([p * 16 + o for p in range(40) for o in range(6)], [5, 9, 14, 60, 61, 62, 100, 150])
        c.append([p * 16 + o for p in range(40) for o in range(6, 9)], [1, 4, 7, 90], size=40.0)
        first = first or c.bits()
        assert c.bits() == first
