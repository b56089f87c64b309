"""The cache append against 64-bit rotation and e4m3 rounding (block_ref.append)."""
import numpy as np
import pytest

import block_ref as ref
from helpers import bf16_tensor, bf16_to_np_bits
from workloads import gen

pytestmark = pytest.mark.gpu

GARBAGE_CODE = 0x7F       # nan: what a page holds before its first token
GARBAGE_SCALE = np.float32(np.nan)


def bf16(a):
    return gen.f32_to_bf16_bits(np.asarray(a, dtype=np.float32))


class Run:
    """One cache on the GPU and its 64-bit twin, appended to by the same calls."""

    def __init__(self, n_pages, Hkv, D, P, n_pos=5000, seed=0):
        import torch
        import int4_grouped_expert_gb300 as st
        self.rng = np.random.default_rng(seed)
        self.shape = (n_pages, Hkv, P, D)
        self.P, self.D, self.Hkv = P, D, Hkv
        codes = np.full(self.shape, GARBAGE_CODE, dtype=np.uint8)
        scales = np.full(self.shape[:2], GARBAGE_SCALE, dtype=np.float32)
        self.cpu = ref.Cache(codes, codes, scales, scales)
        t = torch.from_numpy
        self.gpu = st.PagedKVCache(n_pages, Hkv, D, P, t(codes).cuda(), t(codes.copy()).cuda(),
                                   t(scales).cuda(), t(scales.copy()).cuda())
        self.rope = self.rng.uniform(0, 2 * np.pi, (n_pos, D // 2))
        self.n_pos = n_pos

    def append(self, slots, positions, Hq=4, rot=None, neighbours=False, k=None, v=None, in_place=False,
               expect_status=0, pad=0, flaws=()):
        import torch
        import int4_grouped_expert_gb300 as st
        T, D, Hkv = len(slots), self.D, self.Hkv
        rot = D if rot is None else rot
        rng = self.rng
        q = rng.standard_normal((T, Hq, D))
        k = rng.standard_normal((T, Hkv, D)) if k is None else k
        v = rng.standard_normal((T, Hkv, D)) if v is None else v
        wide = np.zeros((T, (Hq + 2 * Hkv) * D + pad), dtype=np.uint16)
        qb, kb, vb = bf16(q), bf16(k), bf16(v)
        for which, i, val in flaws:
            {"k": kb, "v": vb}[which][i] = val
        a, b, c = Hq * D, (Hq + Hkv) * D, (Hq + 2 * Hkv) * D
        wide[:, :a], wide[:, a:b], wide[:, b:c] = qb.reshape(T, -1), kb.reshape(T, -1), vb.reshape(T, -1)
        x = bf16_tensor(wide)
        h = max(rot // 2, 1)
        cs = np.concatenate([np.cos(self.rope[:, :h]), np.sin(self.rope[:, :h])], 1).astype(np.float32)
        q_out = x[:, :a] if in_place else torch.full((T, Hq * D), -7.0, dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        g = lambda z: torch.from_numpy(np.ascontiguousarray(z, dtype=np.int32)).cuda()  # noqa: E731
        ds, dp, dr = g(slots), g(positions), torch.from_numpy(cs).cuda()
        before = x.clone()
        st.check(st.strata_kv_append(
            self.gpu.struct(), x[:, a:b], x[:, b:c], T, ds, dp if rot else None, dr if rot else None,
            self.n_pos, rot, q=x, n_heads=Hq, q_out=q_out, k_stride=x.stride(0), v_stride=x.stride(0),
            q_stride=x.stride(0), q_out_stride=q_out.stride(0),
            flags=st.STRATA_ROPE_NEIGHBOURS if neighbours else 0, dev_status=status), "strata_kv_append")
        torch.cuda.synchronize()
        rc, bits = st.strata_read_status(status)
        assert bits == expect_status, hex(bits)
        assert torch.equal(x[:, a:].view(torch.int16), before[:, a:].view(torch.int16))  # only q is written
        # the same in 64 bits, on the rows that are neither padding nor out of range
        slots, positions = np.asarray(slots), np.asarray(positions)
        n_slots = self.shape[0] * self.P
        good = (slots >= 0) & (slots < n_slots) & ((rot == 0) | ((positions >= 0) & (positions < self.n_pos)))
        at = np.where(good & (rot > 0), positions, 0)
        cos, sin = cs[at, :h].astype(np.float64), cs[at, h:].astype(np.float64)
        f64 = ref.bf16_bits_to_f64
        with np.errstate(invalid="ignore"):
            qr, qm = ref.rotate(f64(qb), cos, sin, rot, neighbours) if rot else (f64(qb), 0 * f64(qb))
            kr, km = ref.rotate(f64(kb), cos, sin, rot, neighbours) if rot else (f64(kb), 0 * f64(kb))
            got = f64(bf16_to_np_bits(q_out.contiguous())).reshape(T, Hq, D)
            err = 3 * ref.U32 * qm                       # two products and a sum in fp32
            assert (np.abs(got - qr) <= err + ref.half_ulp_bf16(np.abs(qr) + err))[good].all()
            if not in_place:
                assert (got[~good] == -7).all()          # skipped rows are not written
            want = ref.append(self.cpu, kr, f64(vb), 3 * ref.U32 * km, np.where(good, slots, -1), self.P)
        self.compare(want)

    def compare(self, want=None):
        for kind, codes, scales in (("k", self.gpu.k_codes, self.gpu.k_scales),
                                    ("v", self.gpu.v_codes, self.gpu.v_scales)):
            c = ref.E4M3[codes.cpu().numpy()]
            s = scales.cpu().numpy().astype(np.float64)
            np.testing.assert_array_equal(s, self.cpu.scales[kind])
            val = c * s[:, :, None, None]
            w, allow = want[kind]
            nan = np.isnan(w)
            assert np.array_equal(np.isnan(val), nan), kind
            assert (np.abs(val - w) <= allow)[~nan].all(), kind
            # go on from the GPU's codes: a value in 2^20 may have rounded the other way
            self.cpu.codes[kind] = c


def slots_of(pages, old, new, P):
    pos = np.arange(old, old + new)
    return np.asarray(pages)[pos // P] * P + pos % P, pos


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_sequences_grow(P, D):
    """Three sequences: prompts of odd lengths, pieces, then single tokens, each page order shuffled."""
    r = Run(40, 3, D, P)
    order = r.rng.permutation(40)
    pages = [order[:12], order[12:24], order[24:36]]
    length = [0, 0, 0]
    for step in ([37, 5, 1], [P, 3, P + 1], [1, 1, 1], [1, 0, 1], [2, P - 1, 0], [1, 1, 1]):
        parts = [slots_of(pages[s], length[s], n, P) for s, n in enumerate(step)]
        r.append(np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts]))
        length = [a + b for a, b in zip(length, step)]


@pytest.mark.parametrize("rot", [0, 16, 48, 64, 128])
@pytest.mark.parametrize("neighbours", [False, True])
def test_rotations(rot, neighbours):
    r = Run(8, 2, 128, 32)
    s, p = slots_of(np.arange(8), 0, 100, 32)
    r.append(s, p * 37 % 5000, rot=rot, neighbours=neighbours, Hq=6)
    r.append(*slots_of(np.arange(8), 100, 1, 32), rot=rot, neighbours=neighbours, Hq=6, in_place=True)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 1), (28, 4), (5, 5), (64, 8)])
def test_head_counts_and_strides(Hq, Hkv):
    r = Run(6, Hkv, 64, 16)
    r.append(*slots_of([4, 0, 5], 0, 45, 16), Hq=Hq, pad=8)
    r.append(*slots_of([4, 0, 5], 45, 1, 16), Hq=Hq, pad=24, in_place=True)


@pytest.mark.parametrize("P", [16, 128])
def test_scales_grow_and_old_codes_follow(P):
    """Each token is larger than the last, then a smaller one: the scale grows, and stays."""
    r = Run(2, 2, 64, P)
    for i, mag in enumerate([1e-3, 1.0, 1.7, 1.9, 60.0, 5e4, 1.0, 0.0]):
        k = r.rng.standard_normal((1, 2, 64)) * mag
        v = r.rng.standard_normal((1, 2, 64)) * mag * np.array([1.0, 1e-2])[None, :, None]
        r.append([P + i], [i], k=k, v=v)
    assert (r.cpu.scales["k"][1] >= 2.0 ** 6).all()


def test_edges_of_the_scale():
    """Largest magnitudes at, just above and just below 448 * 2^e, zeros, and values past both ends."""
    r = Run(16, 1, 64, 16)
    for page, top in enumerate([448.0, 450.0, 446.0, 0.0, 1.75, 1.7578125, 2.0 ** -120, 3e38, 2.0 ** -92 * 1.75]):
        x = np.full((1, 1, 64), top)
        x[..., ::2] *= -0.3
        r.append([page * 16], [0], k=x, v=x, rot=0)
    # the subnormal steps of the code, and ties between two codes
    x = (np.arange(64) * 2.0 ** -10)[None, None]
    x[..., 63] = 448
    r.append([9 * 16], [0], k=x, v=-x, rot=0)


def test_padding_and_rows_out_of_range():
    import int4_grouped_expert_gb300 as st
    r = Run(8, 2, 128, 16)
    r.append([-1, 3 * 16, -1, -5, 5 * 16, 5 * 16 + 1, -1], [0, 0, -9, 1 << 30, 0, 1, 0])
    r.append([8 * 16, 3 * 16 + 1, 1 << 30], [0, 1, 2], expect_status=st.STRATA_DEV_BAD_SLOT)
    r.append([2 * 16, 6 * 16, 7 * 16], [-1, 5000, 4999], expect_status=st.STRATA_DEV_BAD_SLOT)
    r.append([2 * 16, 6 * 16], [1 << 30, -3], rot=0)                      # without rotation positions do not count
    r.append([-1] * 40, [0] * 40)


def test_many_single_rows_in_one_call():
    """More rows than one block starts runs for, each its own run, a page apart."""
    r = Run(700, 8, 64, 16)
    order = r.rng.permutation(700)[:600]
    r.append(order * 16, np.arange(600))
    r.append(order * 16 + 1, np.arange(600))


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("value", [0x7FC0, 0x7F80, 0xFF80, 0xFFC1])
def test_non_finite_rows(which, value):
    """A row with a nan or inf becomes nan keys and zero values, and the scales do not see it."""
    import int4_grouped_expert_gb300 as st
    r = Run(4, 3, 64, 16)
    s, p = slots_of([2, 1], 0, 20, 16)
    r.append(s, p, flaws=[(which, (5, 1, 40), value)], expect_status=st.STRATA_DEV_NONFINITE)
    r.append(*slots_of([2, 1], 20, 1, 16), flaws=[(which, (0, 2, 0), value)],
             expect_status=st.STRATA_DEV_NONFINITE)
    r.append(*slots_of([2, 1], 21, 3, 16), k=r.rng.standard_normal((3, 3, 64)) * 100)  # rescales the page


def test_keys_and_values_alone_on_another_stream():
    import torch
    import int4_grouped_expert_gb300 as st
    P, Hkv, D = 32, 2, 64
    c1, c2 = st.PagedKVCache(3, Hkv, D, P), st.PagedKVCache(3, Hkv, D, P)
    for t in (c1.k_codes, c1.v_codes, c2.k_codes, c2.v_codes):
        t.view(torch.uint8).zero_()
    for t in (c1.k_scales, c1.v_scales, c2.k_scales, c2.v_scales):
        t.zero_()
    k = torch.randn(40, Hkv * D, device="cuda").bfloat16()
    v = torch.randn(40, Hkv * D, device="cuda").bfloat16()
    slots = torch.arange(P, P + 40, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    st.check(st.strata_kv_append(c1.struct(), k, v, 40, slots), "append")
    st.check(st.strata_kv_append(c2.struct(), k, v, 40, slots, stream=side), "append")
    torch.cuda.synchronize()
    for name in ("k_codes", "v_codes"):
        assert torch.equal(getattr(c1, name).view(torch.uint8), getattr(c2, name).view(torch.uint8))
    assert torch.equal(c1.k_scales, c2.k_scales) and torch.equal(c1.v_scales, c2.v_scales)


def test_a_call_of_no_rows():
    import int4_grouped_expert_gb300 as st
    c = st.PagedKVCache(1, 1, 64, 16)
    assert st.strata_kv_append(c.struct(), None, None, 0, None) == 0
