"""Plain 64-bit implementations of the projections, the cache append and the attention over the cache
(NumPy), with the bounds that the GPU results are held to. Test infrastructure only."""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24


# ------------------------------------------------------------------------------- e4m3
def _e4m3_values():
    v = np.zeros(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            v[c] = np.nan
        elif e == 0:
            v[c] = m * 2.0 ** -9
        else:
            v[c] = (1 + m / 8) * 2.0 ** (e - 7)
        if s:
            v[c] = -v[c]
    return v


E4M3 = _e4m3_values()


def e4m3_step(x):
    """Spacing of e4m3 values at |x|."""
    _, e = np.frexp(np.abs(x))
    return np.where(x == 0, 2.0 ** -9, np.exp2(np.maximum(e - 4, -9).astype(np.float64)))


def round_e4m3(x):
    """Nearest e4m3 value, ties to even (|x| <= 448)."""
    s = e4m3_step(x)
    return np.rint(x / s) * s


def append_scale(absmax):
    """2^e, e the smallest integer >= -100 with absmax <= 448 * 2^e."""
    if absmax == 0:
        return 2.0 ** -100
    m, e = np.frexp(absmax / 448.0)
    return 2.0 ** max(int(e) - (1 if m == 0.5 else 0), -100)


# ------------------------------------------------------------------------------- bf16
def bf16_bits_to_f64(bits):
    return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def half_ulp_bf16(v):
    a = np.abs(np.asarray(v, dtype=np.float64))
    _, e = np.frexp(a)
    return np.where(a > 0, np.ldexp(1.0, np.maximum(e, -125) - 9), 0.0)


# ------------------------------------------------------------------------------- linear
def unpack(codes, bits):
    if bits == 8:
        return codes.view(np.int8).astype(np.float64)
    lo, hi = (codes & 15).astype(np.int8), (codes >> 4).astype(np.int8)
    q = np.stack([lo, hi], -1).reshape(codes.shape[0], -1)
    return np.where(q > 7, q - 16, q).astype(np.float64)


def linear(x, codes, scales, bits, group, bias=None, residual=None, rounded_weights=False):
    """Output in 64 bits, and the bound on a bf16 result's error. The sums run in fp32 (32 units
    in the last place of the sum of magnitudes: tens of additions to a partial sum, random in
    sign); with rounded_weights each weight is off by up to 2^-9 of itself, uniformly, so the sum
    by 2^-9 / sqrt(3) * ||x * w||_2 in the mean: 4 * 2^-9 is seven of those. The rounding of the
    output adds half a unit of a value that may itself be off by that much."""
    w = unpack(codes, bits) * np.repeat(scales.astype(np.float64), group, axis=1)
    y = x @ w.T
    b = 32 * U32 * (np.abs(x) @ np.abs(w).T)
    if rounded_weights:
        b += 4 * 2.0 ** -9 * np.sqrt((x * x) @ (w * w).T)
    if bias is not None:
        y = y + bias
        b += U32 * np.abs(y)
    if residual is not None:
        y = y + residual
        b += U32 * np.abs(y)
    return y, b + half_ulp_bf16(np.abs(y) + b)


# ------------------------------------------------------------------------------- append
def rotate(x, cos, sin, rot, neighbours):
    """x [T, H, D]; cos, sin [T, rot/2]. Returns the rotated rows and |a cos| + |b sin|."""
    y, mag = x.copy(), np.zeros_like(x)
    c, s = cos[:, None], sin[:, None]
    h = rot // 2
    i, j = ((slice(0, rot, 2), slice(1, rot, 2)) if neighbours else (slice(0, h), slice(h, rot)))
    a, b = x[..., i], x[..., j]
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    mag[..., i] = np.abs(a * c) + np.abs(b * s)
    mag[..., j] = np.abs(b * c) + np.abs(a * s)
    return y, mag


class Cache:
    """Values a cache holds: codes as numbers, scales."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        self.codes = {"k": E4M3[k_codes], "v": E4M3[v_codes]}
        self.scales = {"k": k_scales.astype(np.float64), "v": v_scales.astype(np.float64)}


def append(cache, k, v, kerr, slots, P):
    """Appends the rows k, v [T, Hkv, D] (64 bits) to the cache in place; kerr: the fp32 error that
    the caller's k may have. Returns, per kind, the values before the last rounding and the
    error allowed to the stored value (half a step of the code, plus that error), both laid out as
    the codes, with allowed = 0 where a code must not change."""
    out = {}
    slots = np.asarray(slots)
    good = slots >= 0
    bad_row = ~(np.isfinite(k).all(-1) & np.isfinite(v).all(-1))          # [T, Hkv]
    for kind, x, err in (("k", k, kerr), ("v", v, np.zeros_like(v))):
        codes, scales = cache.codes[kind], cache.scales[kind]
        want = codes * scales[:, :, None, None]
        allow = np.zeros_like(codes)
        for p in np.unique(slots[good] // P):
            rows = np.nonzero(good & (slots // P == p))[0]
            off = slots[rows] % P
            low = off.min()
            for h in range(x.shape[1]):
                fine = ~bad_row[rows, h]
                top = np.abs(x[rows[fine], h]).max() if fine.any() else 0.0
                now = append_scale(top)
                if low:
                    now = max(now, scales[p, h])
                    if now != scales[p, h]:
                        r = codes[p, h, :low] * (scales[p, h] / now)
                        want[p, h, :low] = r * now
                        allow[p, h, :low] = 0.5 * e4m3_step(r) * now
                        codes[p, h, :low] = round_e4m3(r)
                scales[p, h] = now
                r = np.where(fine[:, None], x[rows, h], 0.0) / now
                want[p, h, off] = r * now
                allow[p, h, off] = 0.5 * e4m3_step(r * (1 + 2.0 ** -20)) * now + err[rows, h]
                codes[p, h, off] = round_e4m3(r)
                if kind == "k":
                    want[p, h, off[~fine]] = codes[p, h, off[~fine]] = np.nan
        out[kind] = (want, allow)
    return out


# ------------------------------------------------------------------------------- attention
def attention(q, cache, table, seqs, P, scale, window=0):
    """q [T, Hq, D] 64 bits; seqs: (tokens in the cache, query rows) per sequence. Returns the output
    and the bound on a bf16 result's error: probabilities are rounded to f16 (2^-11 of themselves, or
    2^-25 where they are subnormal, against a largest one of 1), exponents carry the fp32 error of
    a D-term sum and of their own magnitude, and the output is rounded to bf16."""
    T, Hq, D = q.shape
    Hkv = cache.codes["k"].shape[1]
    out, bound = np.zeros_like(q), np.zeros_like(q)
    at = 0
    for s, (L, n) in enumerate(seqs):
        pages = np.asarray(table[s][:-(-L // P)], dtype=np.int64)
        for h in range(Hkv if n and L else 0):
            def rows(kind):
                x = cache.codes[kind][pages, h] * cache.scales[kind][pages, h][:, None, None]
                return x.reshape(-1, D)[:L]
            k, v = rows("k"), rows("v")
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = q[at:at + n, heads]
            pos = L - n + np.arange(n)
            j = np.arange(L)
            seen = j[None] <= pos[:, None]
            if window:
                seen &= j[None] > pos[:, None] - window
            t = np.einsum("ngd,ld->ngl", x, k) * scale
            mag = np.einsum("ngd,ld->ngl", np.abs(x), np.nan_to_num(np.abs(k))) * abs(scale)
            t = np.where(seen[:, None], t, -np.inf)
            top = t.max(-1, keepdims=True)
            top = np.where(np.isfinite(top), top, 0.0)
            p = np.exp(t - top)
            l = p.sum(-1, keepdims=True)
            empty = l == 0
            l = np.where(empty, 1.0, l)
            o = np.einsum("ngl,ld->ngd", p, v) / l
            rel = 2.0 ** -11 + 2.0 ** -21 + 16 * U32 * np.where(seen[:, None], mag + np.abs(np.where(seen[:, None], t, 0)) + np.abs(top), 0).max(-1, keepdims=True)
            b = 2 * rel * (np.einsum("ngl,ld->ngd", p, np.abs(v)) / l)
            b += 2.0 ** -24 * np.abs(v).sum(0) / l
            out[at:at + n, heads] = o
            bound[at:at + n, heads] = b + half_ulp_bf16(np.abs(o) + b)
        at += n
    return out, bound
