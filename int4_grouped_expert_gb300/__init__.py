"""Python binding of libstrata.so, the GB300 routed int4-g128 MoE layer (C ABI: include/strata.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. Functions carry the C names and take raw device pointers (ints) or
torch tensors (their data_ptr() is passed). The library must be built first
(`python -m int4_grouped_expert_gb300.build` or `__graft_entry__.build()`);
loading fails loudly when it is missing — there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libstrata.so")

STRATA_OK = 0
STATUS_NAMES = ["STRATA_OK", "STRATA_ERR_INVALID_ARG", "STRATA_ERR_SHAPE", "STRATA_ERR_UNSUPPORTED",
                "STRATA_ERR_WORKSPACE", "STRATA_ERR_CUDA", "STRATA_ERR_DEVICE_STATUS",
                "STRATA_ERR_TIMEOUT"]
STRATA_RENORM = 0x1
STRATA_ADD_RESIDUAL = 0x2
STRATA_ROUTER_FP16 = 0x4
STRATA_FORCE_WARP_PATH = 0x100
STRATA_FORCE_TC_PATH = 0x200
STRATA_WS_REUSE = 0x8
STRATA_ROPE_NEIGHBOURS = 0x1
STRATA_DEV_NONFINITE = 0x1
STRATA_DEV_BAD_ID = 0x2
STRATA_DEV_TIMEOUT = 0x4
STRATA_DEV_BAD_TOKENS = 0x8
STRATA_DEV_BAD_SLOT = 0x10
STRATA_DEV_NO_PAGES = 0x20
STRATA_ERR_DEVICE_STATUS = 6
STRATA_ERR_TIMEOUT = 7
GROUP_WORKSPACE_BYTES = 256
GROUP = 128
LINEAR_EXACT_T = 64  # STRATA_LINEAR_EXACT_T


class StrataError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else str(status)
        super().__init__(f"{where}: {name}")


class strata_moe_layer(ctypes.Structure):
    """Mirror of the C struct strata_moe_layer."""
    _fields_ = [
        ("H", ctypes.c_int64), ("I", ctypes.c_int64), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
        ("has_shared", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("w_router", ctypes.c_void_p), ("bias", ctypes.c_void_p),
        ("gate_codes", ctypes.c_void_p), ("gate_scales", ctypes.c_void_p),
        ("up_codes", ctypes.c_void_p), ("up_scales", ctypes.c_void_p),
        ("down_codes", ctypes.c_void_p), ("down_scales", ctypes.c_void_p),
        ("group_size", ctypes.c_int32), ("bits", ctypes.c_int32),
    ]


class strata_linear(ctypes.Structure):
    """Mirror of the C struct strata_linear."""
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64), ("group_size", ctypes.c_int32),
                ("bits", ctypes.c_int32), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("bias", ctypes.c_void_p)]


class strata_kv_cache(ctypes.Structure):
    """Mirror of the C struct strata_kv_cache."""
    _fields_ = [("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int64),
                ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p)]


class strata_qk_norm(ctypes.Structure):
    """Mirror of the C struct strata_qk_norm."""
    _fields_ = [("q_weight", ctypes.c_void_p), ("q_head_stride", ctypes.c_int64),
                ("k_weight", ctypes.c_void_p), ("k_head_stride", ctypes.c_int64),
                ("eps", ctypes.c_float)]


class strata_kv_batch(ctypes.Structure):
    """Mirror of the C struct strata_kv_batch."""
    _fields_ = [("n_seq", ctypes.c_int32), ("max_q", ctypes.c_int32), ("T", ctypes.c_int64),
                ("max_kv", ctypes.c_int64), ("q_start", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64)]


class strata_kv_pages(ctypes.Structure):
    """Mirror of the C struct strata_kv_pages."""
    _fields_ = [("n_seq", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int64),
                ("max_pages", ctypes.c_int64), ("table_stride", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("refs", ctypes.c_void_p)]


_lib = None
_byref = ctypes.byref
_P = ctypes.c_void_p
_F32 = ctypes.c_float
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_U32 = ctypes.c_uint32
_SZ = ctypes.c_size_t

_SIGNATURES = {
    "strata_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "strata_version": (ctypes.c_int, []),
    "strata_quantize_groups": (ctypes.c_int, [_P, _I64, _I64, _I32, _P, _P, _P, _P]),
    "strata_quantize_groups_bits": (ctypes.c_int, [_P, _I64, _I64, _I32, _I32, _P, _P, _P, _P]),
    "strata_route_workspace_size": (_SZ, [_I64, _I32, _I32]),
    "strata_route_topk": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I32, _I32, _U32,
                                         _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "strata_route_topk_noalloc": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I32, _I32, _U32,
                                                 _P, _P, _P, _P, _P, _P, _P]),
    "strata_moe_workspace_size": (_SZ, [ctypes.POINTER(strata_moe_layer), _I64]),
    "strata_moe_forward": (ctypes.c_int, [ctypes.POINTER(strata_moe_layer), _P, _I64, _P, _P, _SZ, _P]),
    "strata_moe_forward_padded": (ctypes.c_int, [ctypes.POINTER(strata_moe_layer), _P, _P, _I64,
                                                 _P, _P, _SZ, _P]),
    "strata_group_rows": (ctypes.c_int, [_P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _SZ, _P]),
    "strata_selftest_bounded_waits": (ctypes.c_int, [_P, _I64, _P]),
    "strata_moe_forward_ex": (ctypes.c_int, [ctypes.POINTER(strata_moe_layer), _P, _I64, _P,
                                             _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "strata_moe_forward_stats": (ctypes.c_int, [ctypes.POINTER(strata_moe_layer), _P, _I64, _P, _P,
                                                 _P, _SZ, _P]),
    "strata_moe_forward_profiled": (ctypes.c_int, [ctypes.POINTER(strata_moe_layer), _P, _I64, _P, _P,
                                                   _SZ, _P, ctypes.POINTER(_P), _I32]),
    "strata_moe_stack_workspace_size": (_SZ, [ctypes.POINTER(strata_moe_layer), _I32, _I64]),
    "strata_moe_stack_forward": (ctypes.c_int, [ctypes.POINTER(strata_moe_layer), _I32, _P, _I64,
                                                _P, _P, _SZ, _P]),
    "strata_moe_host_staging_size": (_SZ, [ctypes.POINTER(strata_moe_layer), _I64]),
    "strata_moe_forward_host": (ctypes.c_int, [ctypes.POINTER(strata_moe_layer), _P, _I64, _P, _P,
                                               _SZ, _P]),
    "strata_linear_workspace_size": (_SZ, [ctypes.POINTER(strata_linear), _I64]),
    "strata_linear_forward": (ctypes.c_int, [ctypes.POINTER(strata_linear), _P, _I64, _I64, _P, _I64,
                                             _P, _I64, _P, _SZ, _P]),
    "strata_kv_append": (ctypes.c_int, [ctypes.POINTER(strata_kv_cache), _P, _I64, _I32, _P, _I64, _P,
                                        _I64, _I64, _P, _P, _P, _I64, _I32, _U32, _P, _I64, _P, _P]),
    "strata_kv_append_normed": (ctypes.c_int, [ctypes.POINTER(strata_kv_cache), ctypes.POINTER(strata_qk_norm), _P,
                                               _I64, _I32, _P, _I64, _P, _I64, _I64, _P, _P, _P, _I64, _I32, _U32,
                                               _P, _I64, _P, _P]),
    "strata_attention_workspace_size": (_SZ, [ctypes.POINTER(strata_kv_cache),
                                              ctypes.POINTER(strata_kv_batch), _I32]),
    "strata_attention_forward": (ctypes.c_int, [ctypes.POINTER(strata_kv_cache),
                                                ctypes.POINTER(strata_kv_batch), _P, _I64, _I32,
                                                _F32, _I32, _U32, _P, _I64, _P, _SZ, _P]),
    "strata_attention_sinks_forward": (ctypes.c_int, [ctypes.POINTER(strata_kv_cache),
                                                      ctypes.POINTER(strata_kv_batch), _P, _I64, _I32,
                                                      _F32, _I32, _I32, _U32, _P, _I64, _P, _SZ, _P]),
    "strata_kv_pages_extend": (ctypes.c_int, [ctypes.POINTER(strata_kv_pages), _P, _I64, _P, _P, _P, _P, _P, _P, _P]),
    "strata_kv_pages_fork": (ctypes.c_int, [ctypes.POINTER(strata_kv_pages), _P, _P, _P]),
    "strata_kv_pages_release": (ctypes.c_int, [ctypes.POINTER(strata_kv_pages), _P, _I32, _I32, _P, _P]),
    "strata_kv_pages_compact_workspace_size": (_SZ, [ctypes.POINTER(strata_kv_pages)]),
    "strata_kv_pages_compact": (ctypes.c_int, [ctypes.POINTER(strata_kv_pages), ctypes.POINTER(strata_kv_pages), _P, _P,
                                               _P, _SZ, _P, _P]),
    "strata_kv_copy_pages": (ctypes.c_int, [ctypes.POINTER(strata_kv_cache), ctypes.POINTER(strata_kv_cache), _I32, _P,
                                            _P, _I64, _P, _P]),
    "strata_workspace_status": (ctypes.c_int, [_P, _P, ctypes.POINTER(_U32)]),
    "strata_read_status": (ctypes.c_int, [_P, _P, ctypes.POINTER(_U32)]),
}


def lib() -> ctypes.CDLL:
    """Load libstrata.so (raises when it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m int4_grouped_expert_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def ptr(t) -> int | None:
    """Device pointer of a torch tensor (or pass through an int / None)."""
    try:
        return t.data_ptr()
    except AttributeError:
        if t is None or isinstance(t, int):
            return t
        raise


_raw_stream = None      # (device index) -> handle of torch's current stream, once CUDA is in use
_current_device = None  # () -> device index


def stream_handle(stream) -> int | None:
    global _raw_stream, _current_device
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_current_device())
        try:
            import torch
            if torch.cuda.is_available():
                h = torch.cuda.current_stream().cuda_stream
                # the same lookup without building a Stream object: 0.3 us against 7 us a call
                if hasattr(torch._C, "_cuda_getCurrentRawStream") and hasattr(torch._C, "_cuda_getDevice"):
                    _current_device = torch._C._cuda_getDevice
                    _raw_stream = torch._C._cuda_getCurrentRawStream
                return h
        except Exception:  # pragma: no cover
            pass
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def check(status: int, where: str) -> None:
    if status != STRATA_OK:
        raise StrataError(status, where)


# ----------------------------------------------------------------------------- the C calls

def strata_status_string(status: int) -> str:
    return lib().strata_status_string(status).decode()


def strata_version() -> int:
    return lib().strata_version()


def strata_quantize_groups(w, n, k, codes, scales, dev_status=None, group_size=GROUP, stream=None):
    return lib().strata_quantize_groups(ptr(w), n, k, group_size, ptr(codes), ptr(scales),
                                        ptr(dev_status), stream_handle(stream))


def strata_quantize_groups_bits(w, n, k, codes, scales, dev_status=None, group_size=GROUP, bits=4,
                                stream=None):
    return lib().strata_quantize_groups_bits(ptr(w), n, k, group_size, bits, ptr(codes),
                                             ptr(scales), ptr(dev_status), stream_handle(stream))


def strata_route_workspace_size(T, E, k) -> int:
    return lib().strata_route_workspace_size(T, E, k)


def strata_route_topk(x, w_router, bias, T, H, E, k, flags, ids, gates, counts=None, offsets=None,
                      perm=None, inv=None, workspace=None, ws_bytes=0, stream=None):
    return lib().strata_route_topk(ptr(x), ptr(w_router), ptr(bias), T, H, E, k, flags, ptr(ids),
                                   ptr(gates), ptr(counts), ptr(offsets), ptr(perm), ptr(inv),
                                   ptr(workspace), ws_bytes, stream_handle(stream))


def strata_route_topk_noalloc(x, w_router, bias, T, H, E, k, flags, ids, gates, counts=None,
                              offsets=None, perm=None, inv=None, stream=None):
    """strata_route_topk with the library's own fixed scratch (no workspace, no allocation)."""
    return lib().strata_route_topk_noalloc(ptr(x), ptr(w_router), ptr(bias), T, H, E, k, flags,
                                           ptr(ids), ptr(gates), ptr(counts), ptr(offsets),
                                           ptr(perm), ptr(inv), stream_handle(stream))


NOALLOC_SCRATCH_BYTES = 8 << 20


def strata_moe_workspace_size(layer: strata_moe_layer, T_max: int) -> int:
    return lib().strata_moe_workspace_size(ctypes.byref(layer), T_max)


def strata_moe_forward(layer, x, T, out, workspace, ws_bytes, stream=None):
    return lib().strata_moe_forward(ctypes.byref(layer), ptr(x), T, ptr(out), ptr(workspace),
                                    ws_bytes, stream_handle(stream))


def strata_moe_forward_padded(layer, x, n_tokens, T_max, out, workspace, ws_bytes, stream=None):
    """n_tokens: a device int32 (tensor or pointer) holding the live token count."""
    return lib().strata_moe_forward_padded(ctypes.byref(layer), ptr(x), ptr(n_tokens), T_max, ptr(out),
                                           ptr(workspace), ws_bytes, stream_handle(stream))


def strata_group_rows(ids, T, k, E, counts, offsets, perm, inv, workspace, ws_bytes, stream=None):
    return lib().strata_group_rows(ptr(ids), T, k, E, ptr(counts), ptr(offsets), ptr(perm), ptr(inv),
                                   ptr(workspace), ws_bytes, stream_handle(stream))


def strata_selftest_bounded_waits(dev_words, limit_cycles, stream=None):
    return lib().strata_selftest_bounded_waits(ptr(dev_words), limit_cycles, stream_handle(stream))


def strata_moe_forward_stats(layer, x, T, out, expert_rows, workspace, ws_bytes, stream=None):
    return lib().strata_moe_forward_stats(ctypes.byref(layer), ptr(x), T, ptr(out), ptr(expert_rows),
                                          ptr(workspace), ws_bytes, stream_handle(stream))


def strata_moe_forward_ex(layer, x, T, out, ids=None, gates=None, counts=None, offsets=None,
                          perm=None, inv=None, workspace=None, ws_bytes=0, stream=None):
    return lib().strata_moe_forward_ex(ctypes.byref(layer), ptr(x), T, ptr(out), ptr(ids), ptr(gates),
                                       ptr(counts), ptr(offsets), ptr(perm), ptr(inv),
                                       ptr(workspace), ws_bytes, stream_handle(stream))


def strata_moe_forward_profiled(layer, x, T, out, workspace, ws_bytes, events, stream=None):
    """events: 6 torch.cuda.Event objects (or raw cudaEvent_t ints / None)."""
    handles = (_P * len(events))(*[None if e is None else (e if isinstance(e, int) else e.cuda_event)
                                   for e in events])
    return lib().strata_moe_forward_profiled(ctypes.byref(layer), ptr(x), T, ptr(out),
                                             ptr(workspace), ws_bytes, stream_handle(stream),
                                             handles, len(events))


def layer_array(structs):
    """A C array of strata_moe_layer from a list of descriptors."""
    arr = (strata_moe_layer * len(structs))(*structs)
    return arr


def strata_moe_stack_workspace_size(layers, T_max) -> int:
    arr = layers if not isinstance(layers, list) else layer_array(layers)
    return lib().strata_moe_stack_workspace_size(arr, len(arr), T_max)


def strata_moe_stack_forward(layers, x, T, out, workspace, ws_bytes, stream=None):
    arr = layers if not isinstance(layers, list) else layer_array(layers)
    return lib().strata_moe_stack_forward(arr, len(arr), ptr(x), T, ptr(out), ptr(workspace),
                                          ws_bytes, stream_handle(stream))


def strata_moe_host_staging_size(layer, T_max) -> int:
    return lib().strata_moe_host_staging_size(ctypes.byref(layer), T_max)


def strata_moe_forward_host(layer, x_host, T, out_host, workspace, ws_bytes, stream=None):
    return lib().strata_moe_forward_host(ctypes.byref(layer), ptr(x_host), T, ptr(out_host),
                                         ptr(workspace), ws_bytes, stream_handle(stream))


def strata_linear_workspace_size(lin: strata_linear, T_max: int) -> int:
    return lib().strata_linear_workspace_size(ctypes.byref(lin), T_max)


def strata_linear_forward(lin: strata_linear, x, T, out, workspace, ws_bytes, x_stride=None,
                          residual=None, residual_stride=None, out_stride=None, stream=None):
    """Strides in elements; None: rows follow one another."""
    return (_lib or lib()).strata_linear_forward(
        _byref(lin), ptr(x), lin.K if x_stride is None else x_stride, T,
        None if residual is None else ptr(residual), lin.N if residual_stride is None else residual_stride, ptr(out),
        lin.N if out_stride is None else out_stride, ptr(workspace), ws_bytes, stream_handle(stream))


def strata_kv_append(cache: strata_kv_cache, k, v, T, slots, positions=None, rope=None, n_pos=0,
                     rot_dim=0, q=None, n_heads=0, q_out=None, k_stride=None, v_stride=None,
                     q_stride=None, q_out_stride=None, flags=0, dev_status=None, stream=None):
    """Strides in elements; None: rows follow one another."""
    if k_stride is None or v_stride is None:
        kv = cache.n_kv_heads * cache.head_dim
        k_stride = kv if k_stride is None else k_stride
        v_stride = kv if v_stride is None else v_stride
    if q_stride is None or q_out_stride is None:
        qd = n_heads * cache.head_dim
        q_stride = qd if q_stride is None else q_stride
        q_out_stride = qd if q_out_stride is None else q_out_stride
    return (_lib or lib()).strata_kv_append(
        _byref(cache), None if q is None else ptr(q), q_stride, n_heads, ptr(k), k_stride, ptr(v), v_stride, T,
        ptr(slots), ptr(positions), ptr(rope), n_pos, rot_dim, flags, None if q_out is None else ptr(q_out),
        q_out_stride, None if dev_status is None else ptr(dev_status), stream_handle(stream))


def strata_kv_append_normed(cache: strata_kv_cache, norm: strata_qk_norm, k, v, T, slots, positions=None, rope=None,
                            n_pos=0, rot_dim=0, q=None, n_heads=0, q_out=None, k_stride=None, v_stride=None,
                            q_stride=None, q_out_stride=None, flags=0, dev_status=None, stream=None):
    """strata_kv_append with the norms that QKNorm describes. Strides in elements; None: rows follow one another."""
    serves = getattr(norm, "serves", None)  # (of a QKNorm: the library sees neither the width nor the rows of its weights)
    if serves and (serves[0] != cache.head_dim or serves[1] < n_heads or serves[2] < cache.n_kv_heads):
        raise ValueError(f"weights of {serves[0]} for {serves[1]} query and {serves[2]} K/V heads at most, but {n_heads} and "
                         f"{cache.n_kv_heads} heads of {cache.head_dim}")
    if k_stride is None or v_stride is None:
        kv = cache.n_kv_heads * cache.head_dim
        k_stride = kv if k_stride is None else k_stride
        v_stride = kv if v_stride is None else v_stride
    if q_stride is None or q_out_stride is None:
        qd = n_heads * cache.head_dim
        q_stride = qd if q_stride is None else q_stride
        q_out_stride = qd if q_out_stride is None else q_out_stride
    return (_lib or lib()).strata_kv_append_normed(
        _byref(cache), _byref(norm), None if q is None else ptr(q), q_stride, n_heads, ptr(k), k_stride, ptr(v),
        v_stride, T, ptr(slots), ptr(positions), ptr(rope), n_pos, rot_dim, flags,
        None if q_out is None else ptr(q_out), q_out_stride, None if dev_status is None else ptr(dev_status),
        stream_handle(stream))


def strata_attention_workspace_size(cache: strata_kv_cache, batch: strata_kv_batch, n_heads) -> int:
    return lib().strata_attention_workspace_size(ctypes.byref(cache), ctypes.byref(batch), n_heads)


def strata_attention_forward(cache: strata_kv_cache, batch: strata_kv_batch, q, n_heads, scale, out,
                             workspace, ws_bytes, window=0, flags=0, q_stride=None, out_stride=None,
                             stream=None):
    """Strides in elements; None: rows follow one another."""
    if q_stride is None or out_stride is None:
        qd = n_heads * cache.head_dim
        q_stride = qd if q_stride is None else q_stride
        out_stride = qd if out_stride is None else out_stride
    return (_lib or lib()).strata_attention_forward(
        _byref(cache), _byref(batch), ptr(q), q_stride, n_heads, scale, window, flags, ptr(out), out_stride,
        ptr(workspace), ws_bytes, stream_handle(stream))


def strata_attention_sinks_forward(cache: strata_kv_cache, batch: strata_kv_batch, q, n_heads, scale, out,
                                   workspace, ws_bytes, window=0, n_sinks=0, flags=0, q_stride=None, out_stride=None,
                                   stream=None):
    """strata_attention_forward with n_sinks first tokens that the window leaves visible."""
    if q_stride is None or out_stride is None:
        qd = n_heads * cache.head_dim
        q_stride = qd if q_stride is None else q_stride
        out_stride = qd if out_stride is None else out_stride
    return (_lib or lib()).strata_attention_sinks_forward(
        _byref(cache), _byref(batch), ptr(q), q_stride, n_heads, scale, window, n_sinks, flags, ptr(out), out_stride,
        ptr(workspace), ws_bytes, stream_handle(stream))


def strata_kv_pages_extend(pages: strata_kv_pages, new_tokens, T_max, slots, positions, q_start, copies, n_copies,
                           dev_status=None, stream=None):
    return (_lib or lib()).strata_kv_pages_extend(
        _byref(pages), ptr(new_tokens), T_max, ptr(slots), ptr(positions), ptr(q_start), ptr(copies), ptr(n_copies),
        None if dev_status is None else ptr(dev_status), stream_handle(stream))


def strata_kv_pages_fork(pages: strata_kv_pages, parent, dev_status=None, stream=None):
    return (_lib or lib()).strata_kv_pages_fork(_byref(pages), ptr(parent),
                                                None if dev_status is None else ptr(dev_status), stream_handle(stream))


def strata_kv_pages_release(pages: strata_kv_pages, keep=None, window=0, n_sinks=0, dev_status=None, stream=None):
    return (_lib or lib()).strata_kv_pages_release(_byref(pages), None if keep is None else ptr(keep), window, n_sinks,
                                                   None if dev_status is None else ptr(dev_status),
                                                   stream_handle(stream))


def strata_kv_pages_compact_workspace_size(src: strata_kv_pages) -> int:
    return lib().strata_kv_pages_compact_workspace_size(ctypes.byref(src))


def strata_kv_pages_compact(src: strata_kv_pages, dst: strata_kv_pages, copies, n_copies, workspace, ws_bytes,
                            dev_status=None, stream=None):
    return (_lib or lib()).strata_kv_pages_compact(
        _byref(src), _byref(dst), ptr(copies), ptr(n_copies), ptr(workspace), ws_bytes,
        None if dev_status is None else ptr(dev_status), stream_handle(stream))


def strata_kv_copy_pages(src, dst, copies, n_copies, max_copies, dev_status=None, stream=None):
    """src, dst: arrays of descriptors (cache_array), or one strata_kv_cache each."""
    n = 1 if isinstance(src, strata_kv_cache) else len(src)
    if n != (1 if isinstance(dst, strata_kv_cache) else len(dst)):
        raise ValueError("as many caches to copy to as to copy from expected")
    return (_lib or lib()).strata_kv_copy_pages(
        _byref(src) if isinstance(src, strata_kv_cache) else src,
        _byref(dst) if isinstance(dst, strata_kv_cache) else dst, n, ptr(copies),
        None if n_copies is None else ptr(n_copies), max_copies, None if dev_status is None else ptr(dev_status),
        stream_handle(stream))


def strata_workspace_status(workspace, stream=None):
    v = _U32(0)
    st = lib().strata_workspace_status(ptr(workspace), stream_handle(stream), ctypes.byref(v))
    return st, v.value


def strata_read_status(dev_status, stream=None):
    v = _U32(0)
    st = lib().strata_read_status(ptr(dev_status), stream_handle(stream), ctypes.byref(v))
    return st, v.value


from .layer import MoELayer  # noqa: E402,F401
from .attention import (PagedKVCache, PageTable, QKNorm, QuantLinear, cache_array,  # noqa: E402,F401
                        kv_batch, rope_table)  # noqa: E402,F401
