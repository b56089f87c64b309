"""The cache append with norms of queries and keys against 64-bit norms, rotation and e4m3 rounding."""
import numpy as np
import pytest

import block_ref as ref
from helpers import bf16_tensor, bf16_to_np_bits
from test_gpu_kv_append import Run, bf16, slots_of

pytestmark = pytest.mark.gpu


class NormRun(Run):
    """A cache on the GPU and its 64-bit twin, appended to with norms."""

    def append(self, slots, positions, Hq=4, rot=None, neighbours=False, per_head=False, eps=1e-6, on="qk", k=None,
               q=None, in_place=False, expect_status=0, pad=0, flaws=()):
        import torch
        import int4_grouped_expert_gb300 as st
        T, D, Hkv, rng = len(slots), self.D, self.Hkv, self.rng
        rot = D if rot is None else rot
        q = 3 * rng.standard_normal((T, Hq, D)) if q is None else q
        k = 3 * rng.standard_normal((T, Hkv, D)) if k is None else k
        bits = {"q": bf16(q), "k": bf16(k), "v": bf16(rng.standard_normal((T, Hkv, D)))}
        for which, i, val in flaws:
            bits[which][i] = val
        a, b, c = Hq * D, (Hq + Hkv) * D, (Hq + 2 * Hkv) * D
        wide = np.zeros((T, c + pad), dtype=np.uint16)
        wide[:, :a], wide[:, a:b], wide[:, b:c] = (bits[i].reshape(T, -1) for i in "qkv")
        x = bf16_tensor(wide)
        weight = {i: rng.standard_normal((h if per_head else 1, D)).astype(np.float32)
                  for i, h in (("q", Hq), ("k", Hkv))}
        t = lambda z: torch.from_numpy(np.ascontiguousarray(z)).cuda()  # noqa: E731
        norm = st.QKNorm(*(t(weight[i]) if i in on else None for i in "qk"), D, eps=eps)
        h = max(rot // 2, 1)
        cs = np.concatenate([np.cos(self.rope[:, :h]), np.sin(self.rope[:, :h])], 1).astype(np.float32)
        q_out = x[:, :a] if in_place else torch.full((T, a), -7.0, dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        slots, positions = np.asarray(slots, dtype=np.int32), np.asarray(positions, dtype=np.int32)
        st.check(st.strata_kv_append_normed(
            self.gpu.struct(), norm.struct(), x[:, a:b], x[:, b:c], T, t(slots), t(positions) if rot else None,
            t(cs) if rot else None, self.n_pos, rot, q=x, n_heads=Hq, q_out=q_out, k_stride=x.stride(0),
            v_stride=x.stride(0), q_stride=x.stride(0), q_out_stride=q_out.stride(0),
            flags=st.STRATA_ROPE_NEIGHBOURS if neighbours else 0, dev_status=status), "strata_kv_append_normed")
        torch.cuda.synchronize()
        assert st.strata_read_status(status)[1] == expect_status
        n_slots = self.shape[0] * self.P
        good = (slots >= 0) & (slots < n_slots) & ((rot == 0) | ((positions >= 0) & (positions < self.n_pos)))
        at = np.where(good & (rot > 0), positions, 0)
        cos, sin = cs[at, :h].astype(np.float64), cs[at, h:].astype(np.float64)

        def turned(i):
            # The sum of D squares is off by 20 roundings at most (16 in a lane, 3 between lanes, the mean's with eps), its
            # root by half of that and its own two, and two products follow: 14 units of 2^-24, and 3 of the rotation.
            y = ref.bf16_bits_to_f64(bits[i])
            if i in on:
                y = y / np.sqrt((y * y).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * weight[i]
            r, mag = ref.rotate(y, cos, sin, rot, neighbours) if rot else (y, 0 * y)
            mag[..., rot:] = np.abs(y[..., rot:])
            return r, 18 * ref.U32 * mag

        with np.errstate(invalid="ignore"):
            qr, err = turned("q")
            got = ref.bf16_bits_to_f64(bf16_to_np_bits(q_out.contiguous())).reshape(T, Hq, D)
            fine = np.isfinite(qr).all(-1, keepdims=True) & good[:, None, None]
            assert (np.abs(got - qr) <= err + ref.half_ulp_bf16(np.abs(qr) + err))[np.broadcast_to(fine, qr.shape)].all()
            assert np.isnan(got).any(-1)[~np.isfinite(qr).all(-1) & good[:, None]].all()
            if not in_place:
                assert (got[~good] == -7).all()
            kr, kerr = turned("k")
            want = ref.append(self.cpu, kr, ref.bf16_bits_to_f64(bits["v"]), kerr, np.where(good, slots, -1), self.P)
        self.compare(want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_sequences_grow(P, D):
    r = NormRun(40, 3, D, P)
    order = r.rng.permutation(40)
    pages = [order[:12], order[12:24], order[24:36]]
    length = [0, 0, 0]
    for step in ([37, 5, 1], [P, 3, P + 1], [1, 1, 1], [1, 0, 1], [2, P - 1, 0]):
        parts = [slots_of(pages[s], length[s], n, P) for s, n in enumerate(step)]
        r.append(np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts]), per_head=sum(step) % 2)
        length = [a + b for a, b in zip(length, step)]


@pytest.mark.parametrize("rot", [0, 16, 48, 64, 128])
@pytest.mark.parametrize("neighbours", [False, True])
def test_rotations(rot, neighbours):
    r = NormRun(8, 2, 128, 32)
    s, p = slots_of(np.arange(8), 0, 100, 32)
    r.append(s, p * 37 % 5000, rot=rot, neighbours=neighbours, Hq=6)
    r.append(*slots_of(np.arange(8), 100, 1, 32), rot=rot, neighbours=neighbours, Hq=6, in_place=True, per_head=True)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 1), (28, 4), (5, 5), (64, 8), (66, 2)])
def test_head_counts_and_strides(Hq, Hkv):
    for D in (64, 128):
        r = NormRun(6, Hkv, D, 16)
        r.append(*slots_of([4, 0, 5], 0, 45, 16), Hq=Hq, pad=8, per_head=True)
        r.append(*slots_of([4, 0, 5], 45, 1, 16), Hq=Hq, pad=24, in_place=True)


@pytest.mark.parametrize("on", ["q", "k"])
def test_one_of_them(on):
    r = NormRun(8, 2, 128, 64)
    r.append(*slots_of(np.arange(8), 0, 130, 64), on=on, Hq=6)
    r.append(*slots_of(np.arange(8), 130, 2, 64), on=on, Hq=6, per_head=True)


@pytest.mark.parametrize("P", [16, 64, 128])
def test_rows_of_any_size(P):
    """Rows from the largest bf16 values to the smallest, zeros among them, and two sizes in one row."""
    r = NormRun(12, 2, 128, P)
    size = np.array([3e38, 1e30, 2.0 ** 64, 2.0 ** 60, 1e15, 1.0, 1e-3, 1e-6, 1e-15, 1e-30, 1e-38, 0.0])
    s, p = slots_of(np.arange(12), 0, len(size), P)
    x = r.rng.uniform(-1, 1, (len(size), 2, 128)) * size[:, None, None]
    r.append(s, p, q=x[:, :, ::-1], k=x, Hq=2)
    x[:, :, 3] *= 2.0 ** -40
    r.append(*slots_of(np.arange(12), len(size), len(size), P), q=x, k=x, Hq=2, per_head=True)


@pytest.mark.parametrize("eps", [2.0 ** -100, 1e-12, 1e-5, 1.0, 1e30])
def test_eps(eps):
    r = NormRun(8, 1, 64, 16)
    x = r.rng.standard_normal((30, 1, 64)) * np.exp2(r.rng.integers(-40, 8, (30, 1, 1)))
    r.append(*slots_of(np.arange(8), 0, 30, 16), q=x, k=x, Hq=1, eps=eps)


@pytest.mark.parametrize("rows", [1, 40])
def test_values_that_are_not_finite(rows):
    """A K row with inf or nan sets the status and gives nan codes and zeros; a Q row gives nan; no other row changes."""
    r = NormRun(8, 2, 128, 32)
    last = rows - 1
    flaws = [("k", (last, 0, 5), 0x7F80), ("q", (last, 3, 100), 0xFF80)]
    if rows > 1:
        flaws += [("k", (3, 1, 127), 0x7FC0), ("v", (7, 0, 0), 0x7F80), ("q", (3, 0, 0), 0x7FC0)]
    r.append(*slots_of(np.arange(8), 0, rows, 32), flaws=flaws, expect_status=1)


def test_rows_that_are_skipped():
    """Padding and slots out of range between the pages' rows, positions out of range inside a page."""
    r = NormRun(8, 2, 64, 16)
    s, p = slots_of(np.arange(8), 0, 50, 16)
    p[[19, 30]] = [5000, -1]
    for at, slot in ((48, 8 * 16), (32, -1), (16, -5), (0, 1 << 30)):
        s, p = np.insert(s, at, slot), np.insert(p, at, 7)
    r.append(s, p, Hq=5, expect_status=0x10)


def test_without_weights_it_is_the_plain_append():
    import torch
    import int4_grouped_expert_gb300 as st
    T, Hq, Hkv, D, P = 45, 6, 2, 128, 32
    x = torch.randn(T, (Hq + 2 * Hkv) * D, device="cuda").bfloat16()
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    rope = st.rope_table(100, D)
    got = []
    for norm in (None, st.QKNorm(None, None, D)):
        cache = st.PagedKVCache(2, Hkv, D, P, *(torch.zeros(2, Hkv, P, D, dtype=torch.uint8, device="cuda") for _ in "kv"))
        q = torch.empty(T, Hq * D, dtype=torch.bfloat16, device="cuda")
        args = dict(q=x, n_heads=Hq, q_out=q, k_stride=x.stride(0), v_stride=x.stride(0), q_stride=x.stride(0))
        rest = (x[:, Hq * D:], x[:, (Hq + Hkv) * D:], T, slots, slots, rope, 100, D)
        rc = (st.strata_kv_append(cache.struct(), *rest, **args) if norm is None else
              st.strata_kv_append_normed(cache.struct(), norm.struct(), *rest, **args))
        assert rc == 0
        got.append([q.view(torch.int16), cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_replayed_on_a_stream():
    """Captured once and replayed with new inputs: what the eager call gives, bit for bit."""
    import torch
    import int4_grouped_expert_gb300 as st
    T, Hq, Hkv, D, P = 3, 8, 2, 128, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    weight = [1 + 0.1 * torch.randn(h, D, device="cuda", generator=g) for h in (Hq, Hkv)]
    norm, rope = st.QKNorm(*weight, D), st.rope_table(200, D)
    x = torch.zeros(T, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, 64, 128], dtype=torch.int32, device="cuda")  # (each begins its page)
    zeros = lambda: [torch.zeros(3, Hkv, P, D, dtype=torch.uint8, device="cuda") for _ in "kv"]  # noqa: E731
    out = [torch.zeros(T, Hq * D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    caches = [st.PagedKVCache(3, Hkv, D, P, *zeros()) for _ in range(2)]

    def call(i):
        st.check(st.strata_kv_append_normed(
            caches[i].struct(), norm.struct(), x[:, Hq * D:], x[:, (Hq + Hkv) * D:], T, slots, slots, rope, 200, D, q=x,
            n_heads=Hq, q_out=out[i], k_stride=x.stride(0), v_stride=x.stride(0), q_stride=x.stride(0)), "append")

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(0)
    for _ in range(2):
        x.copy_(torch.randn(x.shape, device="cuda", generator=g))
        torch.cuda.synchronize()
        graph.replay()
        call(1)
        torch.cuda.synchronize()
        assert torch.equal(out[0].view(torch.int16), out[1].view(torch.int16))
        at = (slots // P, slice(None), slots % P)
        for name in ("k_codes", "v_codes"):
            a, b = (getattr(c, name).view(torch.uint8) for c in caches)
            assert torch.equal(a[at], b[at])
