"""Python binding of the MISA indexer C ABI (``include/misa.h``).

Argument marshalling only: every function has the C entry point's name and
arguments, takes device tensors (torch) or raw device addresses (int), passes
their addresses and sizes to ``libmisa.so`` and raises :class:`MisaError` on a
non-OK status.  All computation happens in the library's HIP kernels; there is
no CPU fallback -- importing this package fails if the library is not built.

The serving calls at the end (attention over a paged cache, the cache's pages,
the norm) take contiguous tensors only, all on one device, and run there, on its
current stream unless one is given.  The integers that they read (tables, lengths,
lists) must be int32 tensors; other types and all sizes are the caller's to keep,
as in C.

MISA (Mixture of Indexer Sparse Attention) is the drop-in replacement for the
DeepSeek Sparse Attention token indexer described on the MISA summary page
("MISA: Mixture of Indexer Sparse Attention for Long-Context LLM Inference").
"""

from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmisa.so")

MISA_OK = 0
MISA_ERR_INVALID_ARG = -1
MISA_ERR_UNSUPPORTED = -2
MISA_ERR_WORKSPACE = -3
MISA_ERR_HIP = -4

MISA_F32, MISA_BF16, MISA_FP8_E4M3 = 0, 1, 2

EXPORTED = (
    "misa_workspace_bytes", "misa_pool_keys", "misa_pool_keys_range", "misa_route",
    "misa_score_topk", "misa_decode_step", "misa_decode_step_noalloc", "misa_rerank",
    "dsa_index_dense", "misa_hisa_workspace_bytes", "misa_hisa_score_topk", "misa_status_string",
    "misa_attend_workspace_bytes", "misa_attend", "misa_page_write", "misa_page_extend",
    "misa_page_fork", "misa_page_free", "misa_page_workspace_bytes", "misa_page_compact",
    "misa_page_copy", "misa_rms_norm",
)
MISA_NOALLOC_SCRATCH_BYTES = 64 << 20


class MisaError(RuntimeError):
    def __init__(self, status: int, fn: str):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")


class misa_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "L", "T", "H", "d", "B", "qk_dtype")]


class misa_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "row_pages", "pages", "page_tokens", "kv_heads",
                                              "dk", "dv", "kv_dtype")]


class misa_page_buffer(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("page_bytes", ctypes.c_int64), ("planes", ctypes.c_int32)]


if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the HIP library first "
        "(python -m long_context_pool_amd.build)")

_lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t
_SHP = ctypes.POINTER(misa_shape)

_lib.misa_workspace_bytes.argtypes = [_SHP, _I32, _I32, _I32]
_lib.misa_workspace_bytes.restype = _SZ
_lib.misa_pool_keys.argtypes = [_SHP, _P, _P, _P, _P]
_lib.misa_pool_keys_range.argtypes = [_SHP, _I32, _I32, _P, _P, _P, _P]
_lib.misa_route.argtypes = [_SHP, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
_lib.misa_score_topk.argtypes = [_SHP, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
_lib.misa_decode_step.argtypes = [_SHP, _I32, _I32] + [_P] * 11 + [_SZ, _P]
_lib.misa_decode_step_noalloc.argtypes = [_SHP, _I32, _I32] + [_P] * 11
_lib.misa_hisa_workspace_bytes.argtypes = [_SHP, _I32, _I32, _I32]
_lib.misa_hisa_workspace_bytes.restype = _SZ
_lib.misa_hisa_score_topk.argtypes = [_SHP, _I32, _I32, _I32] + [_P] * 12 + [_SZ, _P]
_lib.misa_rerank.argtypes = [_SHP, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
_lib.dsa_index_dense.argtypes = [_SHP, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
_CHE = ctypes.POINTER(misa_cache)
_F32 = ctypes.c_float
_lib.misa_attend_workspace_bytes.argtypes = [_CHE, _I32, _I32]
_lib.misa_attend_workspace_bytes.restype = _SZ
_lib.misa_attend.argtypes = [_CHE, _I32, _I32, _F32] + [_P] * 11 + [_SZ, _P]
_lib.misa_page_write.argtypes = [_CHE, _I32] + [_P] * 10
_lib.misa_page_extend.argtypes = [_CHE, _I32] + [_P] * 7
_lib.misa_page_fork.argtypes = [_CHE, _I32] + [_P] * 9
_lib.misa_page_free.argtypes = [_CHE, _I32] + [_P] * 5
_lib.misa_page_workspace_bytes.argtypes = [_CHE]
_lib.misa_page_workspace_bytes.restype = _SZ
_lib.misa_page_compact.argtypes = [_CHE] + [_P] * 9 + [_SZ, _P]
_lib.misa_page_copy.argtypes = [ctypes.POINTER(misa_page_buffer), _I32, _I32, _I32, _P, _P, _P]
_lib.misa_rms_norm.argtypes = [_I32] * 5 + [_F32] + [_P] * 7
for _f in ("misa_pool_keys", "misa_pool_keys_range", "misa_route", "misa_score_topk",
           "misa_decode_step", "misa_decode_step_noalloc", "misa_rerank", "dsa_index_dense",
           "misa_hisa_score_topk", "misa_attend", "misa_page_write", "misa_page_extend",
           "misa_page_fork", "misa_page_free", "misa_page_compact", "misa_page_copy",
           "misa_rms_norm"):
    getattr(_lib, _f).restype = ctypes.c_int
_lib.misa_status_string.argtypes = [ctypes.c_int]
_lib.misa_status_string.restype = ctypes.c_char_p


def lib() -> ctypes.CDLL:
    return _lib


def status_string(status: int) -> str:
    return _lib.misa_status_string(status).decode()


def shape(batch, L, T, H, d, B, qk_dtype) -> misa_shape:
    return misa_shape(batch, L, T, H, d, B, qk_dtype)


def _ptr(x):
    """Device address of a tensor (or an int address, or None -> NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_torch_device = _torch_stream = None


def _current_device() -> int:
    """torch's current device; its getters are looked up once (a Stream object for each call costs
    as much as the call)."""
    global _torch_device, _torch_stream
    if _torch_device is None:
        import torch
        torch.cuda.init()
        _torch_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda i: torch.cuda.current_stream(i).cuda_stream)
        _torch_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _torch_device()


def _stream(stream, device=None):
    """`device`: the current one, where the caller has looked it up."""
    if stream is None:
        if device is None:
            device = _current_device()
        return _torch_stream(device)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(ws) -> int:
    if ws is None:
        return 0
    return ws.numel() * ws.element_size()


def _check(status: int, fn: str):
    if status != MISA_OK:
        raise MisaError(status, fn)


def misa_workspace_bytes(shp: misa_shape, h: int, k: int, kprime: int) -> int:
    return int(_lib.misa_workspace_bytes(ctypes.byref(shp), h, k, kprime))


def misa_pool_keys(shp, k, k_scale, pooled, stream=None):
    _check(_lib.misa_pool_keys(ctypes.byref(shp), _ptr(k), _ptr(k_scale), _ptr(pooled),
                               _stream(stream)), "misa_pool_keys")


def misa_pool_keys_range(shp, block_begin, block_count, k, k_scale, pooled, stream=None):
    _check(_lib.misa_pool_keys_range(ctypes.byref(shp), block_begin, block_count, _ptr(k),
                                     _ptr(k_scale), _ptr(pooled), _stream(stream)),
           "misa_pool_keys_range")


def misa_route(shp, h, q, q_scale, w, pooled, k, k_scale, heads, E_out, ws, stream=None):
    _check(_lib.misa_route(ctypes.byref(shp), h, _ptr(q), _ptr(q_scale), _ptr(w), _ptr(pooled),
                           _ptr(k), _ptr(k_scale), _ptr(heads), _ptr(E_out), _ptr(ws),
                           _nbytes(ws), _stream(stream)), "misa_route")


def misa_score_topk(shp, h, k, q, q_scale, w, kk, k_scale, heads, idx, scores_out, ws,
                    stream=None):
    _check(_lib.misa_score_topk(ctypes.byref(shp), h, k, _ptr(q), _ptr(q_scale), _ptr(w),
                                _ptr(kk), _ptr(k_scale), _ptr(heads), _ptr(idx),
                                _ptr(scores_out), _ptr(ws), _nbytes(ws), _stream(stream)),
           "misa_score_topk")


def misa_decode_step(shp, h, k, q, q_scale, w, pooled, kk, k_scale, heads, E_out, idx,
                     scores_out, ws, stream=None):
    _check(_lib.misa_decode_step(ctypes.byref(shp), h, k, _ptr(q), _ptr(q_scale), _ptr(w),
                                 _ptr(pooled), _ptr(kk), _ptr(k_scale), _ptr(heads), _ptr(E_out),
                                 _ptr(idx), _ptr(scores_out), _ptr(ws), _nbytes(ws),
                                 _stream(stream)), "misa_decode_step")


def misa_decode_step_noalloc(shp, h, k, q, q_scale, w, pooled, kk, k_scale, heads, E_out, idx,
                             scores_out, stream=None):
    _check(_lib.misa_decode_step_noalloc(ctypes.byref(shp), h, k, _ptr(q), _ptr(q_scale), _ptr(w),
                                         _ptr(pooled), _ptr(kk), _ptr(k_scale), _ptr(heads),
                                         _ptr(E_out), _ptr(idx), _ptr(scores_out),
                                         _stream(stream)), "misa_decode_step_noalloc")


def misa_rerank(shp, kprime, k, q, q_scale, w, kk, k_scale, cand, idx, scores_out, ws,
                stream=None):
    _check(_lib.misa_rerank(ctypes.byref(shp), kprime, k, _ptr(q), _ptr(q_scale), _ptr(w),
                            _ptr(kk), _ptr(k_scale), _ptr(cand), _ptr(idx), _ptr(scores_out),
                            _ptr(ws), _nbytes(ws), _stream(stream)), "misa_rerank")


def dsa_index_dense(shp, k, q, q_scale, w, kk, k_scale, idx, scores_out, ws, stream=None):
    _check(_lib.dsa_index_dense(ctypes.byref(shp), k, _ptr(q), _ptr(q_scale), _ptr(w), _ptr(kk),
                                _ptr(k_scale), _ptr(idx), _ptr(scores_out), _ptr(ws),
                                _nbytes(ws), _stream(stream)), "dsa_index_dense")


def misa_hisa_workspace_bytes(shp: misa_shape, h: int, m: int, k: int) -> int:
    return int(_lib.misa_hisa_workspace_bytes(ctypes.byref(shp), h, m, k))


def misa_hisa_score_topk(shp, h, m, k, q, q_scale, w, pooled, kk, k_scale, heads, blocks_out,
                         block_scores_out, idx, scores_out, ws, stream=None):
    _check(_lib.misa_hisa_score_topk(ctypes.byref(shp), h, m, k, _ptr(q), _ptr(q_scale), _ptr(w),
                                     _ptr(pooled), _ptr(kk), _ptr(k_scale), _ptr(heads),
                                     _ptr(blocks_out), _ptr(block_scores_out), _ptr(idx),
                                     _ptr(scores_out), _ptr(ws), _nbytes(ws), _stream(stream)),
           "misa_hisa_score_topk")


# ------------------------------------------------------------------ serving


_int32 = None


def _device(x):
    """The device of a call's main tensor; None for an address."""
    if x is None or x.__class__ is int:
        return None
    device = x.get_device()
    if device < 0:
        raise ValueError("tensors must be contiguous and on the device")
    return device


def _dev(x, device):
    """Device address of a contiguous tensor on `device`, any one if None (or an int address, or
    None -> NULL)."""
    if x is None or x.__class__ is int:
        return x
    on = x.get_device()
    if (on != device and (device is not None or on < 0)) or not x.is_contiguous():
        raise ValueError("tensors must be contiguous and on the device, all on one")
    return x.data_ptr()


def _ints(x, device):
    """_dev for the integers a call reads: torch's own are 64-bit, and would be read as twice as
    many of 32."""
    if x is None or x.__class__ is int:
        return x
    if x.dtype is not _int32:
        _int32_only(x)
    on = x.get_device()
    if (on != device and (device is not None or on < 0)) or not x.is_contiguous():
        return _dev(x, device)
    return x.data_ptr()


def _int32_only(x):
    """torch.int32, looked up once; refuses x of another type."""
    global _int32
    import torch
    _int32 = torch.int32
    if x.dtype is not _int32:
        raise ValueError(f"integers must be torch.int32, not {x.dtype}")


def _call(f, device, args, stream):
    """Calls the entry point with `device` as the current one, on `stream` (by default that device's
    current one)."""
    if device is not None and device != (_torch_device or _current_device)():
        import torch
        with torch.cuda.device(device):
            status = f(*args, _stream(stream))
    elif stream is None:
        status = f(*args, _stream(None) if device is None else _torch_stream(device))
    else:
        status = f(*args, _stream(stream))
    if status:
        raise MisaError(status, f.__name__)


def cache(rows, row_pages, pages, page_tokens, kv_heads, dk, dv, kv_dtype) -> misa_cache:
    return misa_cache(rows, row_pages, pages, page_tokens, kv_heads, dk, dv, kv_dtype)


def page_buffers(buffers):
    """The `buffers` argument of misa_page_copy, from (data, planes, page_bytes) triples.  It holds
    addresses: the tensors must outlive it."""
    on = _device(buffers[0][0]) if buffers else None
    return (misa_page_buffer * len(buffers))(
        *(misa_page_buffer(_dev(d, on), b, p) for d, p, b in buffers))


def misa_attend_workspace_bytes(cache: misa_cache, heads: int, k: int) -> int:
    return int(_lib.misa_attend_workspace_bytes(ctypes.byref(cache), heads, k))


def misa_attend(cache, heads, k, scale, q, k_pages, k_scale, v_pages, v_scale, table, lengths, idx,
                out, lse, ws, stream=None):
    on = _device(q)
    _call(_lib.misa_attend, on, (
        ctypes.byref(cache), heads, k, scale, _dev(q, on), _dev(k_pages, on),
        _dev(k_scale, on), _dev(v_pages, on), _dev(v_scale, on),
        _ints(table, on), _ints(lengths, on), _ints(idx, on),
        _dev(out, on), _dev(lse, on), _dev(ws, on), _nbytes(ws)), stream)


def misa_page_write(cache, n, row, pos, k_new, v_new, k_pages, k_scale, v_pages, v_scale, table,
                    stream=None):
    on = _device(k_pages)
    _call(_lib.misa_page_write, on, (
        ctypes.byref(cache), n, _ints(row, on), _ints(pos, on),
        _dev(k_new, on), _dev(v_new, on), _dev(k_pages, on),
        _dev(k_scale, on), _dev(v_pages, on), _dev(v_scale, on),
        _ints(table, on)), stream)


def misa_page_extend(cache, n, row, count, table, lengths, refs, ok, stream=None):
    on = _device(table)
    _call(_lib.misa_page_extend, on, (
        ctypes.byref(cache), n, _ints(row, on), _ints(count, on),
        _ints(table, on), _ints(lengths, on), _ints(refs, on),
        _dev(ok, on)), stream)


def misa_page_fork(cache, n, parent, child, table, lengths, refs, src, dst, ok, stream=None):
    on = _device(table)
    _call(_lib.misa_page_fork, on, (
        ctypes.byref(cache), n, _ints(parent, on), _ints(child, on),
        _ints(table, on), _ints(lengths, on), _ints(refs, on),
        _dev(src, on), _dev(dst, on), _dev(ok, on)), stream)


def misa_page_free(cache, n, row, table, lengths, refs, stream=None):
    on = _device(table)
    _call(_lib.misa_page_free, on, (
        ctypes.byref(cache), n, _ints(row, on), _ints(table, on),
        _ints(lengths, on), _ints(refs, on)), stream)


def misa_page_workspace_bytes(cache: misa_cache) -> int:
    return int(_lib.misa_page_workspace_bytes(ctypes.byref(cache)))


def misa_page_compact(cache, table, refs, table_out, refs_out, map, live, src, dst, ws, stream=None):
    on = _device(table)
    _call(_lib.misa_page_compact, on, (
        ctypes.byref(cache), _ints(table, on), _ints(refs, on),
        _dev(table_out, on), _dev(refs_out, on), _dev(map, on),
        _dev(live, on), _dev(src, on), _dev(dst, on),
        _dev(ws, on), _nbytes(ws)), stream)


def misa_page_copy(buffers, pages, n, src, dst, stream=None):
    """`buffers`: what page_buffers() gives."""
    on = _device(src)
    _call(_lib.misa_page_copy, on, (
        buffers, len(buffers), pages, n, _dev(src, on), _dev(dst, on)), stream)


def misa_rms_norm(rows, n, groups, x_dtype, out_dtype, eps, x, residual, weight, sum_out, out,
                  out_scale, stream=None):
    on = _device(x)
    _call(_lib.misa_rms_norm, on, (
        rows, n, groups, x_dtype, out_dtype, eps, _dev(x, on), _dev(residual, on),
        _dev(weight, on), _dev(sum_out, on), _dev(out, on),
        _dev(out_scale, on)), stream)
