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
    _fields_ = [
        ("k_proj", c_void_p), ("v", c_void_p), ("len", c_void_p), ("n_abs", c_void_p),
        ("pos", c_void_p), ("score", c_void_p), ("ctrl", c_void_p),
        ("B", c_int), ("Hkv", c_int), ("d", c_int), ("d_store", c_int), ("Tcap", c_int),
        ("max_len", c_int), ("dtype", c_int), ("dv_store", c_int),
    ]


class aqua_paged_cache(ctypes.Structure):
    """Mirror of struct aqua_paged_cache in include/aqua.h."""
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

def _io_dtype(t, what: str) -> int:
    name = str(t.dtype)
    if name == "torch.bfloat16":
        return AQUA_BF16
    if name == "torch.float32":
        return AQUA_F32
    raise AquaError(AQUA_ERR_UNSUPPORTED, f"{what} must be bfloat16 or float32, not {name}")


def _want(t, shape, dtype: str, what: str) -> None:
    """A dense device tensor of this shape and type, or AquaError: the C side sees addresses only."""
    if str(t.dtype) != dtype or tuple(t.shape) != tuple(shape) or not t.is_cuda or not t.is_contiguous():
        raise AquaError(AQUA_ERR_ARG, f"{what} must be a contiguous {dtype} device tensor of shape {tuple(shape)}, "
                                      f"not {t.dtype} {tuple(t.shape)} on {t.device}")


def _rows(t, heads: int, what: str) -> tuple[int, int]:
    """Element strides between the rows and between the heads of t [n, heads, d] (0: there is only one)."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != 128 or not t.is_cuda:
        raise AquaError(AQUA_ERR_ARG, f"{what} must be a device tensor [rows, {heads}, 128], not {tuple(t.shape)}")
    row, head, one = t.stride()
    if one != 1 or (t.shape[0] > 1 and row < 128) or (heads > 1 and head < 128):
        raise AquaError(AQUA_ERR_ARG, f"{what}: rows of 128 must be dense and apart, not strides {t.stride()}")
    return (row if t.shape[0] > 1 else 0), (head if heads > 1 else 0)


class _on:
    """Makes the device of `t` current for a call (streams and launches belong to a device)."""

    def __init__(self, t, *others):
        import torch
        self.dev = t.device
        for o in others:
            if o is not None and o.device != self.dev:
                raise AquaError(AQUA_ERR_ARG, f"tensors on {o.device} and {self.dev} in one call")
        self.ctx = torch.cuda.device(self.dev) if torch.cuda.current_device() != self.dev.index else None

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _rope(rope):
    return ctypes.byref(rope.desc) if rope is not None else None


def aqua_paged_status(cache: aqua_paged_cache, stream=None) -> int:
    out = c_int(0)
    _check(load_library().aqua_paged_status(ctypes.byref(cache), ctypes.byref(out), _stream(stream)))
    return out.value


def aqua_paged_append(cache: aqua_paged_cache, k_new, v_new, start, P, cu_new=None, rope=None, stream=None) -> None:
    """Rotate, project, quantise and append new tokens: k_new, v_new [n_tokens, Hkv, d] (bf16 or f32; tokens and
    heads may be strided), start [B] int32, cu_new [B + 1] int32 or None for one token of each sequence, rope an AquaRope."""
    ks, kh = _rows(k_new, cache.Hkv, "k_new")
    vs, vh = _rows(v_new, cache.Hkv, "v_new")
    io = _io_dtype(k_new, "k_new")
    if v_new.dtype != k_new.dtype or v_new.shape != k_new.shape:
        raise AquaError(AQUA_ERR_ARG, "k_new and v_new must have the same type and shape")
    _want(start, (cache.B,), "torch.int32", "start")
    _want(P, (cache.Hkv, cache.d, cache.d), "torch.float32", "P")
    if cu_new is not None:
        _want(cu_new, (cache.B + 1,), "torch.int32", "cu_new")
    with _on(k_new, v_new, start, P, cu_new, rope):
        _check(load_library().aqua_paged_append(
            ctypes.byref(cache), _ptr(k_new), _ptr(v_new), io, ks, kh, vs, vh, k_new.shape[0], _ptr(start),
            _ptr(cu_new), _ptr(P), _rope(rope), _stream(stream)))


def aqua_paged_decode_workspace_size(cache: aqua_paged_cache, Hq: int) -> int:
    return load_library().aqua_paged_decode_workspace_size(ctypes.byref(cache), Hq)


def aqua_paged_decode_attn(cache: aqua_paged_cache, q, len, P, Hq: int, k: int, out, workspace, rope=None,
                           scale: float = 0.0, sel_out=None, qproj_out=None, lse_out=None, stream=None) -> None:
    """One decode step over the pages: q [B, Hq, d] (rows and heads may be strided) at position len[b] - 1 of each sequence."""
    qs, qh = _rows(q, Hq, "q")
    io = _io_dtype(q, "q")
    if q.shape[0] != cache.B:
        raise AquaError(AQUA_ERR_ARG, f"q has {q.shape[0]} rows for {cache.B} sequences")
    od = _io_dtype(out, "out")
    _want(out, (cache.B, Hq, cache.d), str(out.dtype), "out")
    _want(len, (cache.B,), "torch.int32", "len")
    _want(P, (cache.Hkv, cache.d, cache.d), "torch.float32", "P")
    if sel_out is not None:
        _want(sel_out, (cache.B, Hq, k), "torch.int32", "sel_out")
    if qproj_out is not None:
        _want(qproj_out, (cache.B, Hq, cache.d), "torch.float32", "qproj_out")
    if lse_out is not None:
        _want(lse_out, (cache.B, Hq), "torch.float32", "lse_out")
    with _on(q, len, P, out, workspace, rope):
        _check(load_library().aqua_paged_decode_attn(
            ctypes.byref(cache), _ptr(len), _ptr(q), io, qs, qh, _ptr(P), _rope(rope), Hq, k, scale, _ptr(out),
            od, _ptr(sel_out), _ptr(qproj_out), _ptr(lse_out), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream)))


def aqua_paged_gather(cache: aqua_paged_cache, len, dst: aqua_cache, max_len: int, seq_idx=None, stream=None) -> None:
    """Copy sequences out of the pages into a contiguous cache (dst.max_len becomes max_len)."""
    _want(len, (cache.B,), "torch.int32", "len")
    if seq_idx is not None:
        _want(seq_idx, (dst.B,), "torch.int32", "seq_idx")
    with _on(len, seq_idx):
        _check(load_library().aqua_paged_gather(ctypes.byref(cache), _ptr(len), _ptr(seq_idx), ctypes.byref(dst),
                                                max_len, _stream(stream)))
