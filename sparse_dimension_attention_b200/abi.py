"""Thin ctypes binding of libaqua_b200.so (the C ABI declared in include/aqua.h).

Argument marshalling only: every step of the attention path runs in the CUDA
kernels behind these calls.  Functions carry the C names and raise AquaError
on a negative status.  There is no fallback: if the shared library is missing
or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_float, c_int, c_size_t, c_void_p

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libaqua_b200.so")

AQUA_OK = 0
AQUA_ERR_ARG = -1
AQUA_ERR_UNSUPPORTED = -2
AQUA_ERR_WORKSPACE = -3
AQUA_ERR_CUDA = -4
AQUA_ERR_TIMEOUT = -5
AQUA_F32 = 0
AQUA_BF16 = 1
AQUA_E4M3 = 2
AQUA_CTRL_WORDS = 16

EXPORTED = (
    "aqua_last_error", "aqua_version", "aqua_status",
    "aqua_calibrate_workspace_size", "aqua_calibrate",
    "aqua_project_keys",
    "aqua_decode_workspace_size", "aqua_decode_attn", "aqua_decode_select", "aqua_decode_attend",
    "aqua_decode_attn_static",
    "aqua_prefill_workspace_size", "aqua_prefill_attn",
    "aqua_h2o_update",
    "aqua_selftest_wait_timeout",
    "aqua_paged_status", "aqua_paged_append",
    "aqua_paged_decode_workspace_size", "aqua_paged_decode_attn",
    "aqua_paged_gather",
)


class AquaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"AQUA status {code}: {msg}")
        self.code = code


class aqua_cache(ctypes.Structure):
    """Mirror of struct aqua_cache in include/aqua.h."""
    device = None   # index of the GPU its buffers are on (-1: host); set by the Python objects, not part of the C struct
    _fields_ = [
        ("k_proj", c_void_p), ("v", c_void_p), ("len", c_void_p), ("n_abs", c_void_p),
        ("pos", c_void_p), ("score", c_void_p), ("ctrl", c_void_p),
        ("B", c_int), ("Hkv", c_int), ("d", c_int), ("d_store", c_int), ("Tcap", c_int),
        ("max_len", c_int), ("dtype", c_int), ("dv_store", c_int),
    ]


class aqua_paged_cache(ctypes.Structure):
    """Mirror of struct aqua_paged_cache in include/aqua.h."""
    device = None   # as in aqua_cache
    _fields_ = [
        ("k_pages", c_void_p), ("v_pages", c_void_p), ("k_scale", c_void_p), ("v_scale", c_void_p),
        ("block_table", c_void_p), ("ctrl", c_void_p),
        ("B", c_int), ("Hkv", c_int), ("d", c_int), ("d_store", c_int), ("page_size", c_int),
        ("n_pages", c_int), ("max_pages", c_int), ("dtype", c_int),
    ]


class aqua_rope(ctypes.Structure):
    """Mirror of struct aqua_rope in include/aqua.h."""
    _fields_ = [("cos_sin", c_void_p), ("n_pos", c_int), ("rot_dim", c_int), ("interleaved", c_int)]


_lib = None


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libaqua_b200.so once and declare the signatures; raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"AQUA CUDA library not built: {path} is missing "
                           "(run python -m sparse_dimension_attention_b200.build)")
    lib = ctypes.CDLL(path)
    P = c_void_p
    C = POINTER(aqua_cache)
    PC = POINTER(aqua_paged_cache)
    R = POINTER(aqua_rope)
    LL = ctypes.c_longlong
    sig = {
        "aqua_last_error": (ctypes.c_char_p, []),
        "aqua_version": (c_int, []),
        "aqua_status": (c_int, [C, POINTER(c_int), P]),
        "aqua_calibrate_workspace_size": (c_size_t, [c_int, c_int]),
        "aqua_calibrate": (c_int, [P, c_int, c_int, P, P, P, c_size_t, P]),
        "aqua_project_keys": (c_int, [C, P, P, P, c_int, P]),
        "aqua_decode_workspace_size": (c_size_t, [C, c_int]),
        "aqua_decode_attn": (c_int, [C, P, P, P, P, c_int, c_int, c_float, P, c_int, P, P, P, P, P, c_size_t, P]),
        "aqua_decode_select": (c_int, [C, P, P, P, P, c_int, c_int, c_float, P, P, P, c_size_t, P]),
        "aqua_decode_attend": (c_int, [C, P, c_int, c_int, P, c_int, P, P, P, c_size_t, P]),
        "aqua_decode_attn_static": (c_int, [C, P, P, P, P, c_int, c_int, c_float, P, c_int, P, P, P, P, P]),
        "aqua_selftest_wait_timeout": (c_int, [C, ctypes.c_ulonglong, P]),
        "aqua_prefill_workspace_size": (c_size_t, [C, c_int, c_int]),
        "aqua_prefill_attn": (c_int, [C, P, c_int, c_int, P, c_int, c_int, c_float, P, c_int, P, P, P, c_size_t, P]),
        "aqua_h2o_update": (c_int, [C, P, P, c_int, c_int, c_int, P, P]),
        "aqua_paged_status": (c_int, [PC, POINTER(c_int), P]),
        "aqua_paged_append": (c_int, [PC, P, P, c_int, LL, LL, LL, LL, c_int, P, P, P, R, P]),
        "aqua_paged_decode_workspace_size": (c_size_t, [PC, c_int]),
        "aqua_paged_decode_attn": (c_int, [PC, P, P, c_int, LL, LL, P, R, c_int, c_int, c_float, P, c_int, P, P, P, P,
                                           c_size_t, P]),
        "aqua_paged_gather": (c_int, [PC, P, P, C, c_int, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(t) -> int | None:
    """Device (or host) address of a tensor, None for None."""
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(rc: int) -> int:
    if rc != AQUA_OK:
        raise AquaError(rc, load_library().aqua_last_error().decode())
    return rc


# ------------------------------------------------------------------ entry points

def aqua_version() -> int:
    return load_library().aqua_version()


def aqua_last_error() -> str:
    return load_library().aqua_last_error().decode()


def aqua_selftest_wait_timeout(cache: aqua_cache, limit_ns: int, stream=None) -> None:
    """One CTA waits on a barrier nothing completes for limit_ns; the device
    records AQUA_ERR_TIMEOUT in the cache's status word (see aqua_status)."""
    _check(load_library().aqua_selftest_wait_timeout(ctypes.byref(cache), limit_ns, _stream(stream)))


def aqua_status(cache: aqua_cache, stream=None) -> int:
    out = c_int(0)
    _check(load_library().aqua_status(ctypes.byref(cache), ctypes.byref(out), _stream(stream)))
    return out.value


def aqua_calibrate_workspace_size(n: int, d: int) -> int:
    return load_library().aqua_calibrate_workspace_size(n, d)


def aqua_calibrate(X, P_out, sigma_out, workspace, stream=None) -> None:
    n, d = X.shape
    _check(load_library().aqua_calibrate(_ptr(X), n, d, _ptr(P_out), _ptr(sigma_out), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _stream(stream)))


def aqua_project_keys(cache: aqua_cache, k_new, v_new, P, L: int, stream=None) -> None:
    _check(load_library().aqua_project_keys(ctypes.byref(cache), _ptr(k_new), _ptr(v_new), _ptr(P), L,
                                            _stream(stream)))


def aqua_decode_workspace_size(cache: aqua_cache, Hq: int) -> int:
    return load_library().aqua_decode_workspace_size(ctypes.byref(cache), Hq)


def aqua_decode_attn(cache: aqua_cache, q, P, Hq: int, k: int, out, workspace, scale: float = 0.0,
                     k_new=None, v_new=None, sel_out=None, qproj_out=None, scores_out=None, lse_out=None,
                     stream=None) -> None:
    """One decode step; with k_new/v_new ([B, Hkv, d]) the step's token is appended first."""
    out_dtype = AQUA_BF16 if str(out.dtype) == "torch.bfloat16" else AQUA_F32
    _check(load_library().aqua_decode_attn(
        ctypes.byref(cache), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(P), Hq, k, scale, _ptr(out), out_dtype,
        _ptr(sel_out), _ptr(qproj_out), _ptr(scores_out), _ptr(lse_out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def aqua_decode_select(cache: aqua_cache, q, P, Hq: int, k: int, workspace, scale: float = 0.0, k_new=None,
                       v_new=None, sel_out=None, qproj_out=None, stream=None) -> None:
    """First half of a decode step: projection, top-k, group union (and the append)."""
    _check(load_library().aqua_decode_select(
        ctypes.byref(cache), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(P), Hq, k, scale, _ptr(sel_out),
        _ptr(qproj_out), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def aqua_decode_attend(cache: aqua_cache, Hq: int, out, workspace, appended: bool = False, P=None,
                       scores_out=None, lse_out=None, stream=None) -> None:
    """Second half of a decode step: attention over the selection aqua_decode_select left in the
    workspace (P is needed only with projected values)."""
    out_dtype = AQUA_BF16 if str(out.dtype) == "torch.bfloat16" else AQUA_F32
    _check(load_library().aqua_decode_attend(
        ctypes.byref(cache), _ptr(P), Hq, int(bool(appended)), _ptr(out), out_dtype, _ptr(scores_out),
        _ptr(lse_out), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def aqua_decode_attn_static(cache: aqua_cache, q, P, Hq: int, k: int, out, scale: float = 0.0, k_new=None,
                            v_new=None, sel_out=None, qproj_out=None, scores_out=None, lse_out=None,
                            stream=None) -> None:
    """The decode step without a workspace argument, for callers that cannot allocate
    device scratch: the library's built-in 8 MiB scratch array is used instead."""
    out_dtype = AQUA_BF16 if str(out.dtype) == "torch.bfloat16" else AQUA_F32
    _check(load_library().aqua_decode_attn_static(
        ctypes.byref(cache), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(P), Hq, k, scale, _ptr(out), out_dtype,
        _ptr(sel_out), _ptr(qproj_out), _ptr(scores_out), _ptr(lse_out), _stream(stream)))


def aqua_prefill_workspace_size(cache: aqua_cache, Hq: int, L: int) -> int:
    return load_library().aqua_prefill_workspace_size(ctypes.byref(cache), Hq, L)


def aqua_prefill_attn(cache: aqua_cache, q, pos0: int, L: int, P, Hq: int, k: int, out, workspace,
                      scale: float = 0.0, sel_out=None, qproj_out=None, stream=None) -> None:
    out_dtype = AQUA_BF16 if str(out.dtype) == "torch.bfloat16" else AQUA_F32
    _check(load_library().aqua_prefill_attn(
        ctypes.byref(cache), _ptr(q), pos0, L, _ptr(P), Hq, k, scale, _ptr(out), out_dtype, _ptr(sel_out),
        _ptr(qproj_out), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def aqua_h2o_update(cache: aqua_cache, scores, lse, Hq: int, budget: int, recent: int, evicted_out=None,
                    stream=None) -> None:
    _check(load_library().aqua_h2o_update(ctypes.byref(cache), _ptr(scores), _ptr(lse), Hq, budget, recent,
                                          _ptr(evicted_out), _stream(stream)))


# ------------------------------------------------------------------ paged 8-bit cache

# These wrappers run once per layer and token, so they are kept to a few microseconds: types compared by
# identity, the raw stream handle instead of a stream object.

def _torch():
    """torch, bound to this module at the first paged call (the module itself imports without it)."""
    global torch, _IO
    import torch
    _IO = {torch.bfloat16: AQUA_BF16, torch.float32: AQUA_F32}
    return torch


torch = None
_IO: dict = {}


def _io_dtype(t, what: str) -> int:
    io = (_IO or (_torch() and _IO)).get(t.dtype)
    if io is None:
        raise AquaError(AQUA_ERR_UNSUPPORTED, f"{what} must be bfloat16 or float32, not {t.dtype}")
    return io


def _want(t, shape, dtype, what: str) -> None:
    """A dense device tensor of this shape and type, or AquaError: the C side sees addresses only."""
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise AquaError(AQUA_ERR_ARG, f"{what} must be a contiguous {dtype} device tensor of shape {tuple(shape)}, "
                                      f"not {t.dtype} {tuple(t.shape)} on {t.device}")


def _rows(t, heads: int, what: str) -> tuple[int, int]:
    """Element strides between the rows and between the heads of t [n, heads, d] (0: there is only one)."""
    shape = t.shape
    if shape[1:] != (heads, 128) or not t.is_cuda:
        raise AquaError(AQUA_ERR_ARG, f"{what} must be a device tensor [rows, {heads}, 128], not {tuple(shape)}")
    n, (row, head, one) = shape[0], t.stride()
    if one != 1 or (n > 1 and row < 128) or (heads > 1 and head < 128):
        raise AquaError(AQUA_ERR_ARG, f"{what}: rows of 128 must be dense and apart, not strides {t.stride()}")
    return (row if n > 1 else 0), (head if heads > 1 else 0)


def _one_device(caches, t, *others) -> int:
    """Index of the one device all tensors and caches of a call are on (a descriptor made by hand does not say)."""
    dev = t.get_device()
    for o in others:
        if o is not None and o.get_device() != dev:
            raise AquaError(AQUA_ERR_ARG, f"tensors on device {o.get_device()} and {dev} in one call")
    for c in caches:
        if c.device is not None and c.device != dev:
            where = f"on device {c.device}" if c.device >= 0 else "on the host"
            raise AquaError(AQUA_ERR_ARG, f"a cache {where} and tensors on device {dev} in one call")
    return dev


def _call(fn, dev: int, stream, *args) -> None:
    """fn(*args, stream) with `dev` current (launches and default streams belong to a device)."""
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, raw)
    if rc != AQUA_OK:
        _check(rc)


def _rope(rope):
    return ctypes.byref(rope.desc) if rope is not None else None


def aqua_paged_status(cache: aqua_paged_cache, stream=None) -> int:
    out = c_int(0)
    dev = cache.device
    if dev is None:
        _check(load_library().aqua_paged_status(ctypes.byref(cache), ctypes.byref(out), _stream(stream)))
        return out.value
    if dev < 0:
        raise AquaError(AQUA_ERR_ARG, "the cache is on the host")
    if torch is None:
        _torch()
    _call(load_library().aqua_paged_status, dev, stream, ctypes.byref(cache), ctypes.byref(out))
    return out.value


def aqua_paged_append(cache: aqua_paged_cache, k_new, v_new, start, P, cu_new=None, rope=None, stream=None) -> None:
    """Rotate, project, quantise and append new tokens: k_new, v_new [n_tokens, Hkv, d] (bf16 or f32; tokens and
    heads may be strided), start [B] int32, cu_new [B + 1] int32 or None for one token of each sequence, rope an
    AquaRope."""
    io = _io_dtype(k_new, "k_new")
    ks, kh = _rows(k_new, cache.Hkv, "k_new")
    vs, vh = _rows(v_new, cache.Hkv, "v_new")
    if v_new.dtype is not k_new.dtype or v_new.shape != k_new.shape:
        raise AquaError(AQUA_ERR_ARG, "k_new and v_new must have the same type and shape")
    _want(start, (cache.B,), torch.int32, "start")
    _want(P, (cache.Hkv, cache.d, cache.d), torch.float32, "P")
    if cu_new is not None:
        _want(cu_new, (cache.B + 1,), torch.int32, "cu_new")
    _call((_lib or load_library()).aqua_paged_append,
          _one_device((cache,), k_new, v_new, start, P, cu_new, rope and rope.cos_sin), stream, ctypes.byref(cache),
          k_new.data_ptr(), v_new.data_ptr(), io, ks, kh, vs, vh, k_new.shape[0], start.data_ptr(), _ptr(cu_new),
          P.data_ptr(), _rope(rope))


def aqua_paged_decode_workspace_size(cache: aqua_paged_cache, Hq: int) -> int:
    return load_library().aqua_paged_decode_workspace_size(ctypes.byref(cache), Hq)


def aqua_paged_decode_attn(cache: aqua_paged_cache, q, len, P, Hq: int, k: int, out, workspace, rope=None,
                           scale: float = 0.0, sel_out=None, qproj_out=None, lse_out=None, stream=None) -> None:
    """One decode step over the pages: q [B, Hq, d] (rows and heads may be strided) at position len[b] - 1 of each
    sequence."""
    io = _io_dtype(q, "q")
    od = _io_dtype(out, "out")
    qs, qh = _rows(q, Hq, "q")
    B, d = cache.B, cache.d
    if q.shape[0] != B:
        raise AquaError(AQUA_ERR_ARG, f"q has {q.shape[0]} rows for {B} sequences")
    _want(out, (B, Hq, d), out.dtype, "out")
    _want(len, (B,), torch.int32, "len")
    _want(P, (cache.Hkv, d, d), torch.float32, "P")
    if sel_out is not None:
        _want(sel_out, (B, Hq, k), torch.int32, "sel_out")
    if qproj_out is not None:
        _want(qproj_out, (B, Hq, d), torch.float32, "qproj_out")
    if lse_out is not None:
        _want(lse_out, (B, Hq), torch.float32, "lse_out")
    if not workspace.is_contiguous():
        raise AquaError(AQUA_ERR_ARG, "workspace must be contiguous")
    _call((_lib or load_library()).aqua_paged_decode_attn,
          _one_device((cache,), q, len, P, out, workspace, sel_out, qproj_out, lse_out, rope and rope.cos_sin), stream,
          ctypes.byref(cache), len.data_ptr(), q.data_ptr(), io, qs, qh, P.data_ptr(), _rope(rope), Hq, k, scale,
          out.data_ptr(), od, _ptr(sel_out), _ptr(qproj_out), _ptr(lse_out), workspace.data_ptr(),
          workspace.nbytes)


def aqua_paged_gather(cache: aqua_paged_cache, len, dst: aqua_cache, max_len: int, seq_idx=None, stream=None) -> None:
    """Copy sequences out of the pages into a contiguous cache (dst.max_len becomes max_len)."""
    if torch is None:
        _torch()
    _want(len, (cache.B,), torch.int32, "len")
    if seq_idx is not None:
        _want(seq_idx, (dst.B,), torch.int32, "seq_idx")
    _call((_lib or load_library()).aqua_paged_gather, _one_device((cache, dst), len, seq_idx), stream, ctypes.byref(cache),
          len.data_ptr(), _ptr(seq_idx), ctypes.byref(dst), max_len)
