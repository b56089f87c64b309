"""Device storage of the attention half of a decoder block, and its C descriptors.

QuantLinear holds one projection's codes and scales, PagedKVCache the pages of
8-bit keys and values, PageTable who holds them, QKNorm the weights of the norms of queries and
keys, kv_batch the lengths and page tables of one call. All hold torch tensors (for device memory only) and fill the C structs with their
addresses, and the structs keep the tensors alive; the arithmetic runs in the library, which sees addresses only: element
types and layouts are checked here.
"""
from __future__ import annotations

from . import (GROUP, StrataError, check, ptr, strata_kv_batch, strata_kv_cache, strata_kv_pages,
               strata_linear, strata_linear_workspace_size, strata_qk_norm, strata_quantize_groups_bits, strata_read_status)


def _held(t, name: str, dtype: str, numel: int):
    """t: a tensor of `numel` elements that follow one another, of the dtype named ("codes": any of one byte), or an
    address, which cannot be checked."""
    if hasattr(t, "dtype"):
        kind = str(t.dtype).removeprefix("torch.")
        if t.element_size() != 1 if dtype == "codes" else kind != dtype:
            raise TypeError(f"{name} holds {kind}, not {'elements of one byte' if dtype == 'codes' else dtype}")
        if t.numel() != numel or not t.is_contiguous():
            raise ValueError(f"{name} {tuple(t.shape)} with strides {t.stride()}: {numel} consecutive elements expected")
    return t


class QuantLinear:
    """One projection [N, K] with 4- or 8-bit codes and an fp16 scale per `group` columns.

    codes and scales are outputs of strata_quantize_groups_bits, or come from fp16 weights
    (from_fp16). bias: fp32 [N] or None."""

    def __init__(self, codes, scales, N: int, K: int, bits: int = 4, group: int = GROUP, bias=None):
        _held(codes, "codes", "codes", N * K * (bits or 4) // 8)  # (0: the library's defaults)
        _held(scales, "scales", "float16", N * (K // (group or GROUP)))
        if bias is not None:
            _held(bias, "bias", "float32", N)
        self.codes, self.scales, self.bias = codes, scales, bias
        self.N, self.K, self.bits, self.group = N, K, bits, group
        s = strata_linear()
        s.N, s.K, s.group_size, s.bits = N, K, group, bits
        s.codes, s.scales, s.bias = ptr(codes), ptr(scales), ptr(bias)
        s.tensors = (codes, scales, bias)
        self._struct = s

    @classmethod
    def from_fp16(cls, w, bits: int = 4, group: int = GROUP, bias=None, stream=None):
        """Quantize fp16 weights [N, K] (host or device) on the device."""
        import torch
        src = torch.as_tensor(w).to("cuda", torch.float16).contiguous()
        N, K = src.shape
        codes = torch.empty(N, K * bits // 8, dtype=torch.uint8, device=src.device)
        scales = torch.empty(N, K // group, dtype=torch.float16, device=src.device)
        status = torch.zeros(1, dtype=torch.int32, device=src.device)
        if stream is not None:  # the copy and the cleared word were made on torch's current stream
            torch.cuda.current_stream(src.device).synchronize()
        check(strata_quantize_groups_bits(src, N, K, codes, scales, status, group_size=group,
                                          bits=bits, stream=stream), "strata_quantize_groups_bits")
        rc, v = strata_read_status(status, stream)
        if rc != 0:
            raise StrataError(rc, f"quantize device status 0x{v:x}")
        if bias is not None:
            bias = torch.as_tensor(bias).to("cuda", torch.float32).contiguous()
        return cls(codes, scales, N, K, bits, group, bias)

    def struct(self) -> strata_linear:
        return self._struct

    def workspace_size(self, T_max: int) -> int:
        return strata_linear_workspace_size(self._struct, T_max)


class PagedKVCache:
    """Pages of 8-bit keys and values of one layer: e4m3 codes [n_pages, n_kv_heads, page_size,
    head_dim] and fp32 scales [n_pages, n_kv_heads]. Storage may be given (any 1-byte dtype for
    the codes); it needs no initialisation."""

    def __init__(self, n_pages: int, n_kv_heads: int, head_dim: int, page_size: int, k_codes=None,
                 v_codes=None, k_scales=None, v_scales=None, device: str = "cuda"):
        import torch
        self.n_pages, self.n_kv_heads = n_pages, n_kv_heads
        self.head_dim, self.page_size = head_dim, page_size
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        n_scales = n_pages * n_kv_heads

        def codes(t, name):
            if t is None:
                return torch.empty(shape, dtype=torch.float8_e4m3fn, device=device)
            return _held(t, name, "codes", n_scales * page_size * head_dim)

        def scales(t, name):
            if t is None:
                return torch.empty(shape[:2], dtype=torch.float32, device=device)
            return _held(t, name, "float32", n_scales)

        self.k_codes, self.v_codes = codes(k_codes, "k_codes"), codes(v_codes, "v_codes")
        self.k_scales, self.v_scales = scales(k_scales, "k_scales"), scales(v_scales, "v_scales")
        s = strata_kv_cache()
        s.n_kv_heads, s.head_dim, s.page_size, s.n_pages = n_kv_heads, head_dim, page_size, n_pages
        s.k_codes, s.v_codes = ptr(self.k_codes), ptr(self.v_codes)
        s.k_scales, s.v_scales = ptr(self.k_scales), ptr(self.v_scales)
        s.tensors = (self.k_codes, self.v_codes, self.k_scales, self.v_scales)
        self._struct = s

    def struct(self) -> strata_kv_cache:
        return self._struct


def cache_array(caches):
    """A C array of the descriptors of several PagedKVCache (the layers of a model), which it keeps alive."""
    arr = (strata_kv_cache * len(caches))(*(c.struct() for c in caches))
    arr.tensors = list(caches)
    return arr


class PageTable:
    """Who holds which pages of a pool: page_table [n_seq, max_pages], kv_len [n_seq] and refs [n_pages], int32 on the
    device. Empty (-1, 0, 0) unless tensors are given; rows of a given page_table may lie apart."""

    def __init__(self, n_pages: int, n_seq: int, max_pages: int, page_size: int, page_table=None, kv_len=None, refs=None,
                 device: str = "cuda"):
        import torch
        self.n_pages, self.n_seq, self.max_pages, self.page_size = n_pages, n_seq, max_pages, page_size
        ints = dict(dtype=torch.int32, device=device)
        if page_table is None:
            page_table = torch.full((n_seq, max_pages), -1, **ints)
        elif tuple(page_table.shape) != (n_seq, max_pages):
            raise ValueError(f"page_table {tuple(page_table.shape)}: ({n_seq}, {max_pages}) expected")
        for row in page_table[:1]:
            _held(row, "page_table", "int32", max_pages)
        if n_seq > 1 and page_table.stride(0) < max_pages:
            raise ValueError(f"page_table: rows {page_table.stride(0)} apart, {max_pages} entries each")
        self.page_table = page_table
        self.kv_len = torch.zeros(n_seq, **ints) if kv_len is None else _held(kv_len, "kv_len", "int32", n_seq)
        self.refs = torch.zeros(n_pages, **ints) if refs is None else _held(refs, "refs", "int32", n_pages)
        s = strata_kv_pages()
        s.n_seq, s.page_size, s.n_pages, s.max_pages = n_seq, page_size, n_pages, max_pages
        s.table_stride = page_table.stride(0) if n_seq > 1 else max_pages
        s.page_table, s.kv_len, s.refs = ptr(self.page_table), ptr(self.kv_len), ptr(self.refs)
        s.tensors = (self.page_table, self.kv_len, self.refs)
        self._struct = s

    def struct(self) -> strata_kv_pages:
        return self._struct

    def batch(self, q_start, T: int, max_q: int, max_kv: int) -> strata_kv_batch:
        """kv_batch over these sequences: rows as strata_kv_pages_extend lays them out."""
        return kv_batch(q_start, self.kv_len, self.page_table, T, max_q, max_kv)


_ANY_HEADS = 1 << 30  # more than any call has


class QKNorm:
    """Norms of queries and keys for each head: fp32 weights, one row [head_dim] (or [1, head_dim]) for all heads
    or [heads, head_dim] with a row each, or None where there is no norm. eps is added to the mean of squares."""

    def __init__(self, q_weight, k_weight, head_dim: int, eps: float = 1e-6):
        self.q_weight, self.k_weight, self.eps = q_weight, k_weight, eps
        s = strata_qk_norm()
        s.eps = eps
        s.tensors = (q_weight, k_weight)
        serves = {"q": _ANY_HEADS, "k": _ANY_HEADS}
        for name, w in (("q", q_weight), ("k", k_weight)):
            if w is None:
                continue
            rows = 1 if w.dim() == 1 else w.shape[0]
            if w.dim() not in (1, 2) or w.shape[-1] != head_dim or w.numel() == 0:  # (nothing: an address that means no norm)
                raise ValueError(f"{name}_weight {tuple(w.shape)}: [{head_dim}] or [heads, {head_dim}] expected")
            _held(w, f"{name}_weight", "float32", rows * head_dim)
            setattr(s, f"{name}_weight", ptr(w))
            setattr(s, f"{name}_head_stride", head_dim if rows > 1 else 0)
            if rows > 1:
                serves[name] = rows
        if q_weight is not None or k_weight is not None:
            s.serves = (head_dim, serves["q"], serves["k"])  # width, and how many query and K/V heads
        self._struct = s

    def struct(self) -> strata_qk_norm:
        return self._struct


def kv_batch(q_start, kv_len, page_table, T: int, max_q: int, max_kv: int) -> strata_kv_batch:
    """Descriptor of one attention call: int32 device tensors q_start [n_seq + 1], kv_len [n_seq],
    page_table [n_seq, stride] (rows may lie apart), and the host's limits. It keeps the tensors alive."""
    n_seq = kv_len.shape[0]
    _held(kv_len, "kv_len", "int32", n_seq)
    _held(q_start[:n_seq + 1], "q_start", "int32", n_seq + 1)
    _held(page_table[:1, :1], "page_table", "int32", min(1, page_table.numel()))
    if page_table.shape[0] < n_seq or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError(f"page_table {tuple(page_table.shape)} with strides {page_table.stride()}: "
                         f"{n_seq} rows of consecutive elements expected")
    b = strata_kv_batch()
    b.n_seq, b.max_q, b.T, b.max_kv = n_seq, max_q, T, max_kv
    b.q_start, b.kv_len, b.page_table = ptr(q_start), ptr(kv_len), ptr(page_table)
    b.table_stride = page_table.stride(0)
    b.tensors = (q_start, kv_len, page_table)
    return b


def rope_table(n_pos: int, rot_dim: int, base: float = 10000.0, device: str = "cuda"):
    """[n_pos, rot_dim] fp32: cos of pos * base^(-2i / rot_dim) for i < rot_dim/2, then the sines,
    computed in 64 bits."""
    import torch
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    ang = torch.arange(n_pos, dtype=torch.float64)[:, None] * (base ** (-i / rot_dim))[None]
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous().to(device)


__all__ = ["QuantLinear", "PagedKVCache", "PageTable", "QKNorm", "cache_array", "kv_batch", "rope_table"]
