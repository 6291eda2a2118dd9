"""ctypes binding of libtfa.so -- argument marshalling only.

Every entry point of ``include/tfa.h`` is exposed under the same name and
takes the same arguments (pointers as Python ints).  ``prefill`` is the
convenience wrapper a PyTorch user calls: it checks dtypes/devices, allocates
the output with PyTorch and passes raw pointers and the current stream to
``tfa_prefill``.  There is no fallback: if the library is missing or the call
fails, it raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import operator
import os
import re
import struct
import sys
import threading
import warnings

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtfa.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "tfa.h")

TFA_OK = 0
TFA_ERR_NULL = 1
TFA_ERR_HEADS = 2
TFA_ERR_SHORT_QUERY = 3
TFA_ERR_SHAPE = 4
TFA_ERR_HEAD_DIM = 5
TFA_ERR_WINDOW = 6
TFA_ERR_ALIGN = 7
TFA_ERR_CUDA = 8
TFA_ERR_TIMEOUT = 9
TFA_ERR_SCALE = 10
TFA_ERR_FLAGS = 11
TFA_ERR_CAPTURE = 12
TFA_ERR_SOFTCAP = 13
TFA_ERR_SEQLENS = 14
TFA_ERR_RING = 15
TFA_ERR_ROPE = 16
TFA_ERR_CACHE = 17
MAX_VARLEN_SEQS = 1024

TFA_DEBUG_NO_TILE_SKIP = 1
TFA_DEBUG_MASK_ALL = 2
TFA_DEBUG_SYNC = 4
TFA_DEBUG_NO_SPLIT = 8
TFA_DEBUG_FORCE_SPLIT = 16
TFA_DEBUG_SHORT_WAITS = 32

MIN_QUERY_ROWS = 9
MAX_DECODE_ROWS = 8
BLOCK_Q = 128
BLOCK_K = 128

_lock = threading.Lock()
_lib = None


class TfaError(RuntimeError):
    def __init__(self, code: int, where: str = "tfa_prefill"):
        self.code = code
        detail = f" [{last_error()}]" if code in (TFA_ERR_CUDA, TFA_ERR_CAPTURE) else ""
        super().__init__(f"{where} failed with status {code}: {status_string(code)}{detail}")


def lib():
    """Load libtfa.so; raise if it has not been built (no fallback path exists)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m sliding_window_gqa_tfa_b200.build`")
            L = ctypes.CDLL(LIB_PATH)
            P, i32, u32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_float
            common = [P, P, P, P, i32, i32, i32, i32, i32, i32, f32, i32, i32, P, P]
            L.tfa_prefill.argtypes = common
            L.tfa_prefill.restype = i32
            L.tfa_prefill_debug.argtypes = common + [u32]
            L.tfa_prefill_debug.restype = i32
            L.tfa_prefill_host.argtypes = common
            L.tfa_prefill_host.restype = i32
            L.tfa_prefill_noalloc.argtypes = common
            L.tfa_prefill_noalloc.restype = i32
            L.tfa_decode.argtypes = common
            L.tfa_decode.restype = i32
            L.tfa_attention_ex.argtypes = common[:14] + [f32, P, P]
            L.tfa_attention_ex.restype = i32
            L.tfa_prefill_backward.argtypes = [P] * 7 + [i32] * 6 + [f32, i32, i32, P, P]
            L.tfa_prefill_backward.restype = i32
            L.tfa_prefill_lse.argtypes = [P] * 5 + [i32] * 6 + [f32, i32, i32, P, P]
            L.tfa_prefill_lse.restype = i32
            L.tfa_prefill_backward_saved.argtypes = [P] * 9 + [i32] * 6 + [f32, i32, i32, P, P]
            L.tfa_prefill_backward_saved.restype = i32
            L.tfa_prefill_ring.argtypes = [P, P, P, P] + [i32] * 7 + [f32, i32, f32, P, P]
            L.tfa_prefill_ring.restype = i32
            L.tfa_prefill_varlen.argtypes = [P] * 6 + [i32] * 7 + [f32, i32, i32, f32, P, P]
            L.tfa_prefill_varlen.restype = i32
            L.tfa_check_status.argtypes = [P]
            L.tfa_check_status.restype = i32
            L.tfa_last_error.argtypes = []
            L.tfa_last_error.restype = ctypes.c_char_p
            L.tfa_status_string.argtypes = [i32]
            L.tfa_status_string.restype = ctypes.c_char_p
            L.tfa_plan_qtile.argtypes = [i32, i32, i32, i32, i32, i32, ctypes.POINTER(i32),
                                         ctypes.POINTER(i32), P, i32]
            L.tfa_plan_qtile.restype = i32
            L.tfa_plan_ktile.argtypes = [i32] * 5 + [ctypes.POINTER(i32), ctypes.POINTER(i32)]
            L.tfa_plan_ktile.restype = i32
            L.tfa_plan_first_cut.argtypes = [i32] * 8 + [ctypes.POINTER(i32), ctypes.POINTER(i32)]
            L.tfa_plan_first_cut.restype = i32
            L.tfa_plan_pieces.argtypes = [i32] * 9 + [P, i32, ctypes.POINTER(i32),
                                                      ctypes.POINTER(ctypes.c_longlong)]
            L.tfa_plan_pieces.restype = i32
            LL, dims = ctypes.c_char_p, [i32] * 7  # LL: host array of int64, packed
            L.tfa_qk_norm_rope.argtypes = [P] * 4 + [LL, P, P, P, P, i32, i32] + dims + [f32, f32, P]
            L.tfa_qk_norm_rope.restype = i32
            L.tfa_qk_norm_rope_backward.argtypes = [P] * 8 + [LL, P, P, P, P, i32, i32] + dims + [f32, f32, P, P]
            L.tfa_qk_norm_rope_backward.restype = i32
            L.tfa_prefill_first.argtypes = [P] * 5 + [i32] * 6 + [f32, i32, i32, P, f32, P, P]
            L.tfa_prefill_first.restype = i32
            L.tfa_prefill_first_backward.argtypes = [P] * 9 + [i32] * 6 + [f32, i32, i32, P, P]
            L.tfa_prefill_first_backward.restype = i32
            L.tfa_kv4_append.argtypes = [P, P, LL] + [P] * 5 + [i32] * 6 + [P]
            L.tfa_kv4_append.restype = i32
            L.tfa_kv4_read.argtypes = [P] * 7 + [i32] * 6 + [P]
            L.tfa_kv4_read.restype = i32
            L.tfa_kv4_decode.argtypes = [P] * 7 + [i32] * 6 + [f32, i32, i32, f32, P, P, P]
            L.tfa_kv4_decode.restype = i32
            L.tfa_kv4_prefill.argtypes = [P] * 6 + [i32] * 7 + [f32, i32, i32, f32, P, P, P]
            L.tfa_kv4_prefill.restype = i32
            L.tfa_kv4_prefill_workspace.argtypes = [i32] * 8
            L.tfa_kv4_prefill_workspace.restype = ctypes.c_size_t
            L.tfa_kv4_prefill_workspace_most.argtypes = [i32] * 8
            L.tfa_kv4_prefill_workspace_most.restype = ctypes.c_size_t
            L.tfa_kv4_decode_workspace.argtypes = [i32] * 4
            L.tfa_kv4_decode_workspace.restype = ctypes.c_size_t
            L.tfa_qk_norm_rope_workspace.argtypes = [i32]
            L.tfa_qk_norm_rope_workspace.restype = ctypes.c_size_t
            _load_calls(L)
            _lib = L
    return _lib


_calls = None  # csrc/calls.cpp's module, once the library is loaded


def _load_calls(L):
    """Only the way into the library depends on this module: without it, or where it was
    built for another torch (whose tensors it reads) or Python, the wrappers' own code
    makes the same calls, for some 10 us more each."""
    global _calls
    try:
        from . import _calls as module
    except ImportError as e:
        found = str(e)
    else:
        here = f"torch {torch.__version__}, Python {sys.version_info.major}.{sys.version_info.minor}"
        found = None if module.built_for == here else f"it was built for {module.built_for}, this is {here}"
    if found is not None:
        warnings.warn(f"_calls.so cannot be used ({found}): calls take longer; build it with "
                      "`python -m sliding_window_gqa_tfa_b200.build`", RuntimeWarning, stacklevel=3)
        return
    module.use(*(ctypes.cast(getattr(L, name), ctypes.c_void_p).value for name in (
        "tfa_qk_norm_rope", "tfa_qk_norm_rope_backward", "tfa_qk_norm_rope_workspace", "tfa_kv4_append",
        "tfa_kv4_read", "tfa_kv4_decode", "tfa_kv4_decode_workspace", "tfa_prefill_first",
        "tfa_prefill_first_backward", "tfa_kv4_prefill", "tfa_kv4_prefill_workspace")))
    _calls = module


def _native(result, where):
    """What a native call that was made returned: its status, if that is not TFA_OK."""
    if isinstance(result, int):
        raise TfaError(result, where)
    return result


def declared_symbols() -> list[str]:
    """Names of the functions include/tfa.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:int|size_t|const char \*)\s*(tfa_\w+)\s*\(", text, re.M)))


def last_error() -> str:
    return lib().tfa_last_error().decode()


def status_string(code: int) -> str:
    return lib().tfa_status_string(int(code)).decode()


# ----------------------------------------------------------- raw entry points
def tfa_attention_ex(q, k, v, o, B, Hq, Hkv, L, S, D, scale, causal, window, key_mask, softcap,
                     sinks, stream) -> int:
    return lib().tfa_attention_ex(q, k, v, o, B, Hq, Hkv, L, S, D, scale, causal, window, key_mask,
                                  softcap, sinks, stream)


def tfa_prefill_ring(q, k, v, o, B, Hq, Hkv, L, S, ring_rows, D, scale, window, softcap, sinks,
                     stream) -> int:
    return lib().tfa_prefill_ring(q, k, v, o, B, Hq, Hkv, L, S, ring_rows, D, scale, window,
                                  softcap, sinks, stream)


def tfa_prefill_varlen(q, k, v, o, cu_q, cu_k, B, Hq, Hkv, total_q, total_k, max_seqlen_q, D,
                       scale, causal, window, softcap, sinks, stream) -> int:
    return lib().tfa_prefill_varlen(q, k, v, o, cu_q, cu_k, B, Hq, Hkv, total_q, total_k,
                                    max_seqlen_q, D, scale, causal, window, softcap, sinks, stream)


def tfa_prefill(q, k, v, o, B, Hq, Hkv, L, S, D, scale, causal, window, key_mask, stream) -> int:
    return lib().tfa_prefill(q, k, v, o, B, Hq, Hkv, L, S, D, scale, causal, window, key_mask,
                             stream)


def tfa_prefill_debug(q, k, v, o, B, Hq, Hkv, L, S, D, scale, causal, window, key_mask, stream,
                      flags) -> int:
    return lib().tfa_prefill_debug(q, k, v, o, B, Hq, Hkv, L, S, D, scale, causal, window,
                                   key_mask, stream, flags)


def tfa_prefill_host(q, k, v, o, B, Hq, Hkv, L, S, D, scale, causal, window, key_mask,
                     stream) -> int:
    return lib().tfa_prefill_host(q, k, v, o, B, Hq, Hkv, L, S, D, scale, causal, window,
                                  key_mask, stream)


def tfa_decode(q, k, v, o, B, Hq, Hkv, L, S, D, scale, causal, window, key_mask, stream) -> int:
    return lib().tfa_decode(q, k, v, o, B, Hq, Hkv, L, S, D, scale, causal, window, key_mask,
                            stream)


def tfa_prefill_noalloc(q, k, v, o, B, Hq, Hkv, L, S, D, scale, causal, window, key_mask,
                        stream) -> int:
    return lib().tfa_prefill_noalloc(q, k, v, o, B, Hq, Hkv, L, S, D, scale, causal, window,
                                     key_mask, stream)


def tfa_check_status(stream) -> int:
    return lib().tfa_check_status(stream)


def tfa_plan_qtile(L, S, causal, window, has_key_mask, qtile):
    """Returns (status, kt_lo, kt_hi, needs_mask list)."""
    lo, hi = ctypes.c_int(0), ctypes.c_int(0)
    buf = (ctypes.c_ubyte * (S // BLOCK_K + 2))()
    rc = lib().tfa_plan_qtile(L, S, int(causal), window, int(has_key_mask), qtile,
                              ctypes.byref(lo), ctypes.byref(hi),
                              ctypes.cast(buf, ctypes.c_void_p), len(buf))
    if rc:
        return rc, None, None, None
    return rc, lo.value, hi.value, [bool(buf[i]) for i in range(hi.value - lo.value + 1)]


def tfa_plan_ktile(L, S, causal, window, ktile):
    """(status, first query tile, last query tile) that see key tile `ktile`."""
    lo, hi = ctypes.c_int(0), ctypes.c_int(0)
    rc = lib().tfa_plan_ktile(L, S, int(bool(causal)), window, ktile, ctypes.byref(lo), ctypes.byref(hi))
    return rc, lo.value, hi.value


def tfa_plan_first_cut(B, Hq, Hkv, L, S, window, first, sms):
    """(status, key tiles that the gradient with first tokens cuts, parts of each)."""
    tiles, parts = ctypes.c_int(0), ctypes.c_int(0)
    rc = lib().tfa_plan_first_cut(B, Hq, Hkv, L, S, window, first, sms, ctypes.byref(tiles), ctypes.byref(parts))
    return rc, tiles.value, parts.value


def tfa_plan_pieces(B, Hq, L, S, causal, window, grid, split, cta, max_pieces=4096):
    """Returns (status, total_steps, pieces) with pieces as tuples of 10 ints."""
    buf = (ctypes.c_int * (10 * max_pieces))()
    n = ctypes.c_int(0)
    w = ctypes.c_longlong(0)
    rc = lib().tfa_plan_pieces(B, Hq, L, S, int(causal), window, grid, int(split), cta,
                               ctypes.cast(buf, ctypes.c_void_p), max_pieces, ctypes.byref(n),
                               ctypes.byref(w))
    if rc:
        return rc, None, None
    return rc, w.value, [tuple(buf[10 * i:10 * i + 10]) for i in range(n.value)]


# ---------------------------------------------------------- torch wrapper
# the current stream's handle without the Stream object around it (3 us less a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream_handle(stream):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))


def _check(t, name, dtype, ndim):
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def prefill(q, k, v, *, scale=None, causal=True, window=0, key_mask=None, out=None, stream=None,
            debug_flags=0, softcap=0.0, sinks=None, first=0):
    """Attention output [B,Hq,L,D] bf16 for bf16 q [B,Hq,L,D], k/v [B,Hkv,S,D] on one GPU.

    L >= 9 goes to tfa_prefill, 1 <= L <= 8 to tfa_decode; a softcap > 0 or
    sinks (fp32 [Hq] on the device) go to tfa_attention_ex, first > 0 (first tokens
    that stay visible outside a causal window) to tfa_prefill_first.  key_mask: optional
    fp32 [B,S] (1 keep / 0 drop).  Raises TfaError on a nonzero status."""
    import torch

    if first:
        if debug_flags:
            raise ValueError("debug flags apply to tfa_prefill_debug only")
        return _prefill_first(q, k, v, scale, causal, window, first, key_mask, softcap, sinks, out, None, False,
                              stream)[0]
    _check(q, "q", torch.bfloat16, 4)
    _check(k, "k", torch.bfloat16, 4)
    _check(v, "v", torch.bfloat16, 4)
    B, Hq, L, D = q.shape
    Bk, Hkv, S, Dk = k.shape
    if tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must have the same shape")
    if Bk != B or Dk != D:
        raise ValueError("q and k disagree on batch or head dimension")
    if key_mask is not None:
        _check(key_mask, "key_mask", torch.float32, 2)
        if tuple(key_mask.shape) != (B, S):
            raise ValueError("key_mask must be [B, S]")
    if out is None:
        out = torch.empty_like(q)
    else:
        _check(out, "out", torch.bfloat16, 4)
        if tuple(out.shape) != tuple(q.shape):
            raise ValueError("out must have q's shape")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    args = (ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
            ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(out.data_ptr()), B, Hq, Hkv, L, S, D,
            float(scale), int(bool(causal)), int(window),
            ctypes.c_void_p(key_mask.data_ptr()) if key_mask is not None else None,
            _stream_handle(stream))
    if softcap or sinks is not None:
        if debug_flags:
            raise ValueError("debug flags apply to tfa_prefill_debug only")
        if sinks is not None:
            _check(sinks, "sinks", torch.float32, 1)
            if sinks.shape[0] != Hq:
                raise ValueError("sinks must hold one logit per query head")
        rc = tfa_attention_ex(*args[:14], float(softcap),
                              ctypes.c_void_p(sinks.data_ptr()) if sinks is not None else None,
                              args[14])
        if rc != TFA_OK:
            raise TfaError(rc, "tfa_attention_ex")
        return out
    if L <= MAX_DECODE_ROWS:
        if debug_flags:
            raise ValueError("debug flags apply to the prefill path only (L >= 9)")
        rc = tfa_decode(*args)
        if rc != TFA_OK:
            raise TfaError(rc, "tfa_decode")
        return out
    rc = tfa_prefill_debug(*args, debug_flags) if debug_flags else tfa_prefill(*args)
    if rc != TFA_OK:
        raise TfaError(rc)
    return out


def tfa_prefill_backward(q, k, v, dout, dq, dk, dv, B, Hq, Hkv, L, S, D, scale, causal, window,
                         key_mask, stream) -> int:
    return lib().tfa_prefill_backward(q, k, v, dout, dq, dk, dv, B, Hq, Hkv, L, S, D, scale, causal,
                                      window, key_mask, stream)


def prefill_lse(q, k, v, *, scale=None, causal=True, window=0, key_mask=None, out=None, lse=None,
                stream=None, first=0):
    """(o, lse): the forward of any L >= 1 and each row's base-2 log-sum-exp of
    its scaled scores, fp32 [B,Hq,L] (+inf for a row with no allowed key).  first: first
    tokens that stay visible outside a causal window."""
    import torch

    if first:
        return _prefill_first(q, k, v, scale, causal, window, first, key_mask, 0.0, None, out, lse, True, stream)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n, torch.bfloat16, 4)
    B, Hq, L, D = q.shape
    Bk, Hkv, S, Dk = k.shape
    if tuple(v.shape) != tuple(k.shape) or Bk != B or Dk != D:
        raise ValueError("q, k and v disagree")
    if key_mask is not None:
        _check(key_mask, "key_mask", torch.float32, 2)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, Hq, L), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(out, "out", torch.bfloat16, 4)
    _check(lse, "lse", torch.float32, 3)
    rc = lib().tfa_prefill_lse(*(ctypes.c_void_p(t.data_ptr()) for t in (q, k, v, out, lse)),
                               B, Hq, Hkv, L, S, D, float(scale), int(bool(causal)), int(window),
                               _ptr_or_none(key_mask), _stream_handle(stream))
    if rc != TFA_OK:
        raise TfaError(rc, "tfa_prefill_lse")
    return out, lse


def backward(q, k, v, dout, *, scale=None, causal=True, window=0, key_mask=None, out=None,
             saved=None, stream=None, first=0):
    """(dq, dk, dv) bf16 of the attention core for the upstream gradient dout
    [B,Hq,L,D]: recompute-based (the forward is re-run inside), or, given
    saved=(o, lse) from prefill_lse on the same inputs, from those.  first: as for
    prefill_lse, whose result is then needed in `saved`."""
    import torch

    if first:
        if saved is None:
            raise ValueError("the gradient with first tokens takes prefill_lse's result in `saved`")
        return _backward_first(q, k, v, dout, scale, causal, window, first, key_mask, out, saved, stream)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout")):
        _check(t, n, torch.bfloat16, 4)
    B, Hq, L, D = q.shape
    Bk, Hkv, S, Dk = k.shape
    if tuple(v.shape) != tuple(k.shape) or tuple(dout.shape) != tuple(q.shape) or Bk != B or Dk != D:
        raise ValueError("q, k, v and dout disagree")
    if key_mask is not None:
        _check(key_mask, "key_mask", torch.float32, 2)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    if out is None:
        out = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    dq, dk, dv = out
    for t, ref, n in ((dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv")):
        _check(t, n, torch.bfloat16, 4)
        if tuple(t.shape) != tuple(ref.shape):
            raise ValueError(f"{n} has the wrong shape")
    if saved is not None:
        o, lse = saved
        _check(o, "o", torch.bfloat16, 4)
        _check(lse, "lse", torch.float32, 3)
        if tuple(o.shape) != tuple(q.shape) or tuple(lse.shape) != (B, Hq, L):
            raise ValueError("saved (o, lse) have the wrong shape")
        rc = lib().tfa_prefill_backward_saved(
            *(ctypes.c_void_p(t.data_ptr()) for t in (q, k, v, o, lse, dout, dq, dk, dv)),
            B, Hq, Hkv, L, S, D, float(scale), int(bool(causal)), int(window), _ptr_or_none(key_mask),
            _stream_handle(stream))
        if rc != TFA_OK:
            raise TfaError(rc, "tfa_prefill_backward_saved")
        return dq, dk, dv
    rc = tfa_prefill_backward(*(ctypes.c_void_p(t.data_ptr()) for t in (q, k, v, dout, dq, dk, dv)),
                              B, Hq, Hkv, L, S, D, float(scale), int(bool(causal)), int(window),
                              _ptr_or_none(key_mask), _stream_handle(stream))
    if rc != TFA_OK:
        raise TfaError(rc, "tfa_prefill_backward")
    return dq, dk, dv


def _ptr_or_none(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def prefill_ring(q, k_ring, v_ring, *, S, window, scale=None, softcap=0.0, sinks=None, out=None,
                 stream=None):
    """Attention over a rotating K/V cache: k_ring/v_ring [B,Hkv,R,D] bf16 hold the
    last R positions, position j in row j mod R; q [B,Hq,L,D] are the newest L
    positions of S.  Causal with a window (R >= window - 1 + L, R a multiple of 64)."""
    import torch

    _check(q, "q", torch.bfloat16, 4)
    _check(k_ring, "k_ring", torch.bfloat16, 4)
    _check(v_ring, "v_ring", torch.bfloat16, 4)
    B, Hq, L, D = q.shape
    Bk, Hkv, R, Dk = k_ring.shape
    if tuple(v_ring.shape) != tuple(k_ring.shape) or Bk != B or Dk != D:
        raise ValueError("q, k_ring and v_ring disagree")
    if sinks is not None:
        _check(sinks, "sinks", torch.float32, 1)
    out = torch.empty_like(q) if out is None else out
    _check(out, "out", torch.bfloat16, 4)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    rc = tfa_prefill_ring(ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k_ring.data_ptr()),
                          ctypes.c_void_p(v_ring.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                          B, Hq, Hkv, L, int(S), R, D, float(scale), int(window), float(softcap),
                          _ptr_or_none(sinks), _stream_handle(stream))
    if rc != TFA_OK:
        raise TfaError(rc, "tfa_prefill_ring")
    return out


def prefill_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, *, max_seqlen_q, scale=None, causal=True,
                   window=0, softcap=0.0, sinks=None, out=None, stream=None):
    """Packed variable-length attention: q [Tq,Hq,D], k/v [Tk,Hkv,D] bf16, int32 device
    prefix sums cu_seqlens_* [B+1].  Returns out [Tq,Hq,D]."""
    import torch

    _check(q, "q", torch.bfloat16, 3)
    _check(k, "k", torch.bfloat16, 3)
    _check(v, "v", torch.bfloat16, 3)
    _check(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _check(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    Tq, Hq, D = q.shape
    Tk, Hkv, Dk = k.shape
    if tuple(v.shape) != tuple(k.shape) or Dk != D:
        raise ValueError("q, k and v disagree")
    B = cu_seqlens_q.shape[0] - 1
    if cu_seqlens_k.shape[0] != B + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    if sinks is not None:
        _check(sinks, "sinks", torch.float32, 1)
    out = torch.empty_like(q) if out is None else out
    _check(out, "out", torch.bfloat16, 3)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    rc = tfa_prefill_varlen(ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
                            ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                            ctypes.c_void_p(cu_seqlens_q.data_ptr()),
                            ctypes.c_void_p(cu_seqlens_k.data_ptr()), B, Hq, Hkv, Tq, Tk,
                            int(max_seqlen_q), D, float(scale), int(bool(causal)), int(window),
                            float(softcap), _ptr_or_none(sinks), _stream_handle(stream))
    if rc != TFA_OK:
        raise TfaError(rc, "tfa_prefill_varlen")
    return out


def check_status(stream=None) -> None:
    """Synchronize `stream` and raise TfaError if a kernel recorded a timed-out wait."""
    rc = tfa_check_status(_stream_handle(stream))
    if rc != TFA_OK:
        raise TfaError(rc, "tfa_check_status")


def prefill_host(q, k, v, *, scale=None, causal=True, window=0, key_mask=None, out=None,
                 stream=None):
    """The same operation on CPU tensors (pinned or pageable) through tfa_prefill_host."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 CPU tensor")
    B, Hq, L, D = q.shape
    _, Hkv, S, _ = k.shape
    if out is None:
        out = torch.empty_like(q)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    km = None
    if key_mask is not None:
        if key_mask.dtype != torch.float32 or key_mask.is_cuda or not key_mask.is_contiguous():
            raise ValueError("key_mask must be a contiguous fp32 CPU tensor")
        km = ctypes.c_void_p(key_mask.data_ptr())
    rc = tfa_prefill_host(ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
                          ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                          B, Hq, Hkv, L, S, D, float(scale), int(bool(causal)), int(window), km,
                          _stream_handle(stream))
    if rc != TFA_OK:
        raise TfaError(rc, "tfa_prefill_host")
    return out


# ------------------------------------------- norms and rotary positions of q and k
_NO_SCOPE = contextlib.nullcontext()
_BF16, _F32, _F64, _I32, _U8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8


def _scope(index, stream):
    """Makes device `index` current for a call, and `stream` where one is given, so
    that what the call allocates belongs to the stream that uses it."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError("stream belongs to another device than the tensors")
        return torch.cuda.stream(stream)
    return _NO_SCOPE if index == _current_device() else torch.cuda.device(index)


_current_device = torch.cuda.current_device


def _int32(x, name):
    """x (an int, or what stands for one) as a C call's int; ctypes would drop the bits
    that do not fit."""
    x = operator.index(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} must fit in 32 bits")
    return x


def _check_on(t, name, dtype, ndim, index=None, rows=False):
    """Checks a CUDA tensor's type, dimensions and device (`index`, or any); rows: any
    strides, as long as the last dimension is contiguous (else all of it must be)."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim
            and (t.get_device() == index if index is not None else t.is_cuda)
            and (t.is_contiguous() or (rows and (t.stride(-1) == 1 or t.shape[-1] == 1)))):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    raise ValueError(f"{name} must have a contiguous last dimension" if rows else f"{name} must be contiguous")


def _first_inputs(q, k, v, causal, key_mask):
    _check_on(q, "q", _BF16, 4)
    dev = q.get_device()
    _check_on(k, "k", _BF16, 4, dev)
    _check_on(v, "v", _BF16, 4, dev)
    B, Hq, L, D = q.shape
    kv = k.shape
    if v.shape != kv or kv[0] != B or kv[3] != D:
        raise ValueError("q, k and v disagree")
    if key_mask is not None:
        _check_on(key_mask, "key_mask", _F32, 2, dev)
        if key_mask.shape != (B, kv[2]):
            raise ValueError("key_mask must be [B, S]")
    if not causal:
        raise ValueError("first tokens need causal attention with a window")
    return dev, (B, Hq, kv[1], L, kv[2], D)


def _scale(scale, D):
    return D ** -0.5 if scale is None else float(scale)


def _prefill_first(q, k, v, scale, causal, window, first, key_mask, softcap, sinks, out, lse, want_lse, stream):
    """(out, lse): prefill and prefill_lse with first tokens that stay visible."""
    if _calls is not None and stream is None and causal:
        made = _calls.prefill_first(q, k, v, scale, window, first, key_mask, softcap, sinks, out, lse, want_lse)
        if made is not None:
            return _native(made, "tfa_prefill_first")
    dev, dims = _first_inputs(q, k, v, causal, key_mask)
    window, first = _int32(window, "window"), _int32(first, "first")
    if sinks is not None:
        _check_on(sinks, "sinks", _F32, 1, dev)
        if sinks.shape[0] != dims[1]:
            raise ValueError("sinks must hold one logit per query head")
    with _scope(dev, stream):
        if out is None:
            out = torch.empty_like(q)
        else:
            _check_on(out, "out", _BF16, 4, dev)
            if out.shape != q.shape:
                raise ValueError("out must have q's shape")
        if lse is not None:
            _check_on(lse, "lse", _F32, 3, dev)
            if lse.shape != q.shape[:3]:
                raise ValueError("lse must be [B,Hq,L]")
        elif want_lse:
            lse = torch.empty(q.shape[:3], dtype=_F32, device=q.device)
        rc = (_lib or lib()).tfa_prefill_first(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr() if lse is not None else None,
            *dims, _scale(scale, dims[5]), window, first,
            key_mask.data_ptr() if key_mask is not None else None, float(softcap),
            sinks.data_ptr() if sinks is not None else None, _raw_stream(dev))
    if rc != TFA_OK:
        raise TfaError(rc, "tfa_prefill_first")
    return out, lse


def _backward_first(q, k, v, dout, scale, causal, window, first, key_mask, out, saved, stream):
    """(dq, dk, dv): backward with first tokens that stay visible, from saved (o, lse)."""
    if _calls is not None and stream is None and out is None and causal:
        made = _calls.backward_first(q, k, v, dout, *saved, scale, window, first, key_mask)
        if made is not None:
            return _native(made, "tfa_prefill_first_backward")
    dev, dims = _first_inputs(q, k, v, causal, key_mask)
    window, first = _int32(window, "window"), _int32(first, "first")
    o, lse = saved
    for t, n in ((dout, "dout"), (o, "o")):
        _check_on(t, n, _BF16, 4, dev)
        if t.shape != q.shape:
            raise ValueError(f"{n} must have q's shape")
    _check_on(lse, "lse", _F32, 3, dev)
    if lse.shape != q.shape[:3]:
        raise ValueError("lse must be [B,Hq,L]")
    with _scope(dev, stream):
        if out is None:
            out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        else:
            for t, ref, n in zip(out, (q, k, v), ("dq", "dk", "dv")):
                _check_on(t, n, _BF16, 4, dev)
                if t.shape != ref.shape:
                    raise ValueError(f"{n} has the wrong shape")
        dq, dk, dv = out
        rc = (_lib or lib()).tfa_prefill_first_backward(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(), dq.data_ptr(),
            dk.data_ptr(), dv.data_ptr(), *dims, _scale(scale, dims[5]), window, first,
            key_mask.data_ptr() if key_mask is not None else None, _raw_stream(dev))
    if rc != TFA_OK:
        raise TfaError(rc, "tfa_prefill_first_backward")
    return dq, dk, dv


def rope_inv_freq(rot, base=10000.0, *, scaling=None, factor=1.0, original=8192, device=None):
    """(inv_freq, mscale) for qk_norm_rope: fp64 [rot/2] radians per position, base^(-2i/rot).

    scaling: None; "linear" (every pair's frequency divided by factor); "llama3" or
    "yarn": pairs that turn often within the `original` positions are kept, those that
    turn less than once are divided by factor, and a ramp lies between them.  llama3's
    ramp is linear in a pair's turns, from 1 to 4.  yarn's is linear in its index, from
    the last pair of at least 32 turns to the first of at most 1 (the ramp that
    published checkpoints use), and its mscale is 0.1 ln(factor) + 1."""
    if rot < 0 or rot % 2:
        raise ValueError("rot must be even and >= 0")
    if not (factor > 0 and original > 0 and base > 0):
        raise ValueError("base, factor and original must be positive")
    f = torch.tensor([float(base) ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    mscale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "llama3":
        keep = ((original * f / (2 * math.pi) - 1.0) / 3.0).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
    elif scaling == "yarn":
        if base <= 1:
            raise ValueError("yarn's ramp needs a base above 1")

        def place(turns):  # the index, not a whole number, of a pair with so many turns
            return rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))

        low, high = max(math.floor(place(32.0)), 0), min(math.ceil(place(1.0)), rot - 1)
        index = torch.arange(rot // 2, dtype=torch.float64)
        keep = 1 - ((index - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
        if factor > 1:
            mscale = 0.1 * math.log(factor) + 1.0
    elif scaling is not None:
        raise ValueError('scaling must be None, "linear", "llama3" or "yarn"')
    return f.to("cuda" if device is None else device), mscale


def _rope_arguments(q, k, positions, inv_freq, q_weight, k_weight):
    """Checks shared by the pass and its gradient; (device index, the C call's middle
    arguments, its sizes)."""
    _check_on(q, "q", _BF16, 4, rows=True)
    dev = q.get_device()
    _check_on(k, "k", _BF16, 4, dev, rows=True)
    B, L, Hq, D = q.shape
    Bk, Lk, Hkv, Dk = k.shape
    if Bk != B or Lk != L or Dk != D:
        raise ValueError("q and k disagree on batch, tokens or head dimension")
    _check_on(inv_freq, "inv_freq", _F64, 1, dev)
    wq = wk = None
    if q_weight is not None and k_weight is not None:
        _check_on(q_weight, "q_weight", _BF16, 1, dev)
        _check_on(k_weight, "k_weight", _BF16, 1, dev)
        if q_weight.shape[0] != D or k_weight.shape[0] != D:
            raise ValueError("q_weight and k_weight must hold one weight per channel")
        wq, wk = q_weight.data_ptr(), k_weight.data_ptr()
    elif q_weight is not k_weight:
        raise ValueError("q_weight and k_weight must be given together")
    per_row, first, ptr = 0, 0, None
    if not isinstance(positions, torch.Tensor):
        first = _int32(positions, "positions")
    else:
        per_row = 1 if positions.dim() == 2 else 0
        _check_on(positions, "positions", _I32, 1 + per_row, dev)
        if positions.shape != ((B, L) if per_row else (B,)):
            raise ValueError("positions must be an int, [B] or [B, L]")
        ptr = positions.data_ptr()
    return dev, (wq, wk, inv_freq.data_ptr(), ptr, per_row, first), (B, L, Hq, Hkv, D, 2 * inv_freq.shape[0])


_PACK6, _PACK12, _PACK18 = (struct.Struct(f"{n}q").pack for n in (6, 12, 18))


def _tokens(t):
    """(batch, token, head) element strides of a [B, L, H, D] tensor."""
    a = t.stride()
    return a[0], a[1], a[2]


def _heads(t):
    """(batch, token, head) element strides of a [B, H, L, D] tensor."""
    a = t.stride()
    return a[0], a[2], a[1]


def _check_rows(t, name, shape, dev):
    _check_on(t, name, _BF16, 4, dev, rows=True)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")


def qk_norm_rope(q, k, positions, inv_freq, *, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, mscale=1.0,
                 q_out=None, k_out=None, stream=None):
    """(q_out [B,Hq,L,D], k_out [B,Hkv,L,D]) bf16 of the projections q [B,L,Hq,D] and
    k [B,L,Hkv,D] (bf16, any strides with contiguous channels): RMS norms for each
    head (with q_weight and k_weight, bf16 [D]) and the rotary position, in one pass.

    positions: int32 [B] (of each sequence's first row) or [B,L] on the device, or
    an int.  inv_freq: fp64 [rot/2] on the device (rope_inv_freq), rot a multiple of
    16 up to D, the other channels pass through.  q_out and k_out may be views, e.g.
    a key cache's rows, in [B,H,L,D] order.  Raises TfaError on a nonzero status."""
    if _calls is not None and stream is None:
        made = _calls.rope(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, mscale, q_out, k_out)
        if made is not None:
            return _native(made, "tfa_qk_norm_rope")
    dev, mid, dims = _rope_arguments(q, k, positions, inv_freq, q_weight, k_weight)
    B, L, Hq, Hkv, D, rot = dims
    with _scope(dev, stream):
        if q_out is None:
            q_out = q.new_empty((B, Hq, L, D))
        else:
            _check_rows(q_out, "q_out", (B, Hq, L, D), dev)
        if k_out is None:
            k_out = k.new_empty((B, Hkv, L, D))
        else:
            _check_rows(k_out, "k_out", (B, Hkv, L, D), dev)
        (qb, ql, qh, _), (kb, kl, kh, _) = q.stride(), k.stride()
        (ob, oh, ol, _), (pb, ph, pl, _) = q_out.stride(), k_out.stride()
        rc = (_lib or lib()).tfa_qk_norm_rope(
            q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(),
            _PACK12(qb, ql, qh, kb, kl, kh, ob, ol, oh, pb, pl, ph), *mid, *dims, bool(interleaved), float(eps),
            float(mscale), _raw_stream(dev))
    if rc != TFA_OK:
        raise TfaError(rc, "tfa_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, positions, inv_freq, *, q_weight=None, k_weight=None, eps=1e-6,
                          interleaved=False, mscale=1.0, out=None, stream=None):
    """(dq, dk, dq_weight, dk_weight): the gradient of qk_norm_rope for upstream
    dq_out [B,Hq,L,D] and dk_out [B,Hkv,L,D] (bf16, any strides with contiguous
    channels).  dq [B,L,Hq,D] and dk [B,L,Hkv,D] are bf16 (views in `out` are fine);
    the weights' are fp32 [D], None without weights."""
    if _calls is not None and stream is None and out is None:
        made = _calls.rope_backward(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, mscale, dq_out,
                                    dk_out)
        if made is not None:
            return _native(made, "tfa_qk_norm_rope_backward")
    dev, mid, dims = _rope_arguments(q, k, positions, inv_freq, q_weight, k_weight)
    B, L, Hq, Hkv, D, rot = dims
    _check_rows(dq_out, "dq_out", (B, Hq, L, D), dev)
    _check_rows(dk_out, "dk_out", (B, Hkv, L, D), dev)
    with _scope(dev, stream):
        if out is None:
            dq, dk = q.new_empty((B, L, Hq, D)), k.new_empty((B, L, Hkv, D))
        else:
            dq, dk = out
            _check_rows(dq, "dq", (B, L, Hq, D), dev)
            _check_rows(dk, "dk", (B, L, Hkv, D), dev)
        L_ = _lib or lib()
        dwq = dwk = ws = pq = pk = pw = None
        if q_weight is not None:
            dwq, dwk = torch.empty((2, D), dtype=_F32, device=q.device).unbind(0)
            ws = torch.empty(L_.tfa_qk_norm_rope_workspace(D), dtype=_U8, device=q.device)
            pq, pk, pw = dwq.data_ptr(), dwk.data_ptr(), ws.data_ptr()
        rc = L_.tfa_qk_norm_rope_backward(
            dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), dq.data_ptr(), dk.data_ptr(), pq, pk,
            _PACK18(*_heads(dq_out), *_heads(dk_out), *_tokens(q), *_tokens(k), *_tokens(dq), *_tokens(dk)), *mid,
            *dims, bool(interleaved), float(eps), float(mscale), pw, _raw_stream(dev))
    if rc != TFA_OK:
        raise TfaError(rc, "tfa_qk_norm_rope_backward")
    return dq, dk, dwq, dwk


# ---------------------------------------------------- the 4-bit key/value cache
KV4_GROUP = 32


def kv4_cache(B, Hkv, capacity, D, device=None):
    """(k_codes, k_meta, v_codes, v_meta): an empty 4-bit cache (every value 0)."""
    if D not in (64, 128):
        raise ValueError("head dimension must be 64 or 128")
    dev = "cuda" if device is None else device
    out = []
    for _ in range(2):
        out.append(torch.zeros((B, Hkv, capacity, D // 2), dtype=torch.uint8, device=dev))
        out.append(torch.zeros((B, Hkv, capacity, D // KV4_GROUP, 2), dtype=torch.bfloat16, device=dev))
    return tuple(out)


def _kv4_check(k_codes, k_meta, v_codes, v_meta):
    """Checks a cache's tensors; (B, Hkv, capacity, D, device index)."""
    try:  # the usual case in one expression
        shape, mshape, dev = k_codes.shape, k_meta.shape, k_codes.get_device()
        B, Hkv, cap, half = shape
        if (k_codes.dtype is _U8 and v_codes.dtype is _U8 and k_meta.dtype is _BF16 and v_meta.dtype is _BF16
                and dev >= 0 and v_codes.get_device() == dev and k_meta.get_device() == dev
                and v_meta.get_device() == dev and v_codes.shape == shape and v_meta.shape == mshape
                and mshape == (B, Hkv, cap, half >> 4, 2) and k_codes.is_contiguous() and v_codes.is_contiguous()
                and k_meta.is_contiguous() and v_meta.is_contiguous()):
            return B, Hkv, cap, 2 * half, dev
    except (AttributeError, ValueError):
        pass
    _check_on(k_codes, "k_codes", _U8, 4)
    dev = k_codes.get_device()
    _check_on(v_codes, "v_codes", _U8, 4, dev)
    _check_on(k_meta, "k_meta", _BF16, 5, dev)
    _check_on(v_meta, "v_meta", _BF16, 5, dev)
    raise ValueError("a 4-bit cache is codes [B,Hkv,capacity,D/2] and meta [B,Hkv,capacity,D/32,2], twice")


def _kv4_start(start, B, dev):
    """(device pointer or None, first row) of an int or int32 [B]."""
    if not isinstance(start, torch.Tensor):
        return None, _int32(start, "start")
    _check_on(start, "start", _I32, 1, dev)
    if start.shape[0] != B:
        raise ValueError("start must hold one row per sequence")
    return start.data_ptr(), 0


def kv4_append(k, v, k_codes, k_meta, v_codes, v_meta, *, start, stream=None):
    """Writes k, v (bf16 [B,Hkv,L,D], any strides with contiguous channels) into the
    4-bit cache: row i of sequence b at cache row start[b] + i.  start: int32 [B] on
    the device (negative: nothing for that sequence), or an int for all."""
    if _calls is not None and stream is None:
        made = _calls.append(k, v, k_codes, k_meta, v_codes, v_meta, start)
        if made == TFA_OK:
            return
        if made is not None:
            raise TfaError(made, "tfa_kv4_append")
    B, Hkv, cap, D, dev = _kv4_check(k_codes, k_meta, v_codes, v_meta)
    _check_on(k, "k", _BF16, 4, dev, rows=True)
    _check_on(v, "v", _BF16, 4, dev, rows=True)
    L = k.shape[2]
    if k.shape != (B, Hkv, L, D) or v.shape != (B, Hkv, L, D):
        raise ValueError("k and v must be [B,Hkv,L,D] of the cache's B, Hkv and D")
    ptr, first = _kv4_start(start, B, dev)
    (kb, kh, kl, _), (vb, vh, vl, _) = k.stride(), v.stride()
    strides = _PACK6(kb, kh, kl, vb, vh, vl)
    with _scope(dev, stream):
        rc = (_lib or lib()).tfa_kv4_append(k.data_ptr(), v.data_ptr(), strides, k_codes.data_ptr(), k_meta.data_ptr(),
                                  v_codes.data_ptr(), v_meta.data_ptr(), ptr, first, B, Hkv, L, cap, D,
                                  _raw_stream(dev))
    if rc != TFA_OK:
        raise TfaError(rc, "tfa_kv4_append")


def kv4_read(k_codes, k_meta, v_codes, v_meta, *, start=0, rows=None, out=None, stream=None):
    """(k, v) bf16 [B,Hkv,rows,D]: the values of cached rows start[b] .. start[b] + rows - 1
    (start: int32 [B] on the device, or an int; rows: by default all from start on)."""
    if _calls is not None and stream is None and out is None:
        made = _calls.read(k_codes, k_meta, v_codes, v_meta, start, rows)
        if made is not None:
            return _native(made, "tfa_kv4_read")
    B, Hkv, cap, D, dev = _kv4_check(k_codes, k_meta, v_codes, v_meta)
    ptr, first = _kv4_start(start, B, dev)
    if rows is None:
        if ptr is not None:
            raise ValueError("rows must be given with a start for each sequence")
        rows = cap - first
    rows = _int32(rows, "rows")
    if rows < 1:
        raise TfaError(TFA_ERR_SHAPE, "tfa_kv4_read")
    if ptr is None and not 0 <= first <= cap - rows:  # before anything of that size is allocated
        raise TfaError(TFA_ERR_CACHE, "tfa_kv4_read")
    with _scope(dev, stream):
        if out is None:
            out = k_meta.new_empty((B, Hkv, rows, D)), k_meta.new_empty((B, Hkv, rows, D))
        else:
            for t, n in zip(out, ("k", "v")):
                _check_on(t, n, _BF16, 4, dev)
                if t.shape != (B, Hkv, rows, D):
                    raise ValueError(f"{n} must be [B,Hkv,rows,D]")
        rc = (_lib or lib()).tfa_kv4_read(k_codes.data_ptr(), k_meta.data_ptr(), v_codes.data_ptr(), v_meta.data_ptr(),
                                out[0].data_ptr(), out[1].data_ptr(), ptr, first, B, Hkv, rows, cap, D,
                                _raw_stream(dev))
    if rc != TFA_OK:
        raise TfaError(rc, "tfa_kv4_read")
    return out


def _kv4_query(q, B, D, dev, sinks, out):
    _check_on(q, "q", _BF16, 4, dev)
    if q.shape[0] != B or q.shape[3] != D:
        raise ValueError("q and the cache disagree")
    if sinks is not None:
        _check_on(sinks, "sinks", _F32, 1, dev)
        if sinks.shape[0] != q.shape[1]:
            raise ValueError("sinks must hold one logit per query head")
    if out is not None:
        _check_on(out, "out", _BF16, 4, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")


def _kv4_workspace(workspace, need, dev, like):
    if workspace is None:
        return like.new_empty(need)
    _check_on(workspace, "workspace", _U8, 1, dev)
    if workspace.shape[0] < need:
        raise ValueError(f"workspace must hold {need} bytes")
    return workspace


def kv4_decode(q, k_codes, k_meta, v_codes, v_meta, lens, *, scale=None, window=0, first=0, softcap=0.0, sinks=None,
               out=None, workspace=None, stream=None):
    """Decoding attention [B,Hq,L,D] (1 <= L <= 8) over the 4-bit cache: lens, int32 [B]
    on the device, holds each sequence's cached positions, its L new rows last among
    them.  window > 0: the last `window` positions and the `first` first ones.
    workspace: uint8 of tfa_kv4_decode_workspace bytes, by default allocated here."""
    if _calls is not None and stream is None:
        made = _calls.decode(q, k_codes, k_meta, v_codes, v_meta, lens, scale, window, first, softcap, sinks, out,
                             workspace)
        if made is not None:
            return _native(made, "tfa_kv4_decode")
    B, Hkv, cap, D, dev = _kv4_check(k_codes, k_meta, v_codes, v_meta)
    _kv4_query(q, B, D, dev, sinks, out)
    _check_on(lens, "lens", _I32, 1, dev)
    if lens.shape[0] != B:
        raise ValueError("lens must hold one length per sequence")
    Hq, L = q.shape[1], q.shape[2]
    window, first = _int32(window, "window"), _int32(first, "first")
    with _scope(dev, stream):
        if out is None:
            out = torch.empty_like(q)
        L_ = _lib or lib()
        workspace = _kv4_workspace(workspace, L_.tfa_kv4_decode_workspace(Hq, Hkv, L, D), dev, k_codes)
        rc = L_.tfa_kv4_decode(q.data_ptr(), k_codes.data_ptr(), k_meta.data_ptr(), v_codes.data_ptr(),
                                  v_meta.data_ptr(), lens.data_ptr(), out.data_ptr(), B, Hq, Hkv, L, cap, D,
                                  _scale(scale, D), window, first, float(softcap),
                                  sinks.data_ptr() if sinks is not None else None, workspace.data_ptr(),
                                  _raw_stream(dev))
    if rc != TFA_OK:
        raise TfaError(rc, "tfa_kv4_decode")
    return out


def kv4_prefill(q, k_codes, k_meta, v_codes, v_meta, *, S, scale=None, window=0, first=0, softcap=0.0, sinks=None,
                out=None, workspace=None, stream=None):
    """Causal attention [B,Hq,L,D] of chunks of any L >= 1 rows over the first S rows of
    the 4-bit cache (the chunk's own rows last among them); window and first as for
    kv4_decode.  workspace: uint8 of tfa_kv4_prefill_workspace bytes (or, for chunks of
    several sizes, tfa_kv4_prefill_workspace_most), by default allocated here."""
    if _calls is not None and stream is None:
        made = _calls.prefill(q, k_codes, k_meta, v_codes, v_meta, S, scale, window, first, softcap, sinks, out, workspace)
        if made is not None:
            return _native(made, "tfa_kv4_prefill")
    B, Hkv, cap, D, dev = _kv4_check(k_codes, k_meta, v_codes, v_meta)
    _kv4_query(q, B, D, dev, sinks, out)
    S = _int32(S, "S")
    Hq, L = q.shape[1], q.shape[2]
    window, first = _int32(window, "window"), _int32(first, "first")
    with _scope(dev, stream):
        if out is None:
            out = torch.empty_like(q)
        need = (_lib or lib()).tfa_kv4_prefill_workspace(B, Hq, Hkv, L, S, D, window, first)
        workspace = _kv4_workspace(workspace, max(need, 16), dev, k_codes)
        rc = (_lib or lib()).tfa_kv4_prefill(q.data_ptr(), k_codes.data_ptr(), k_meta.data_ptr(), v_codes.data_ptr(),
                                   v_meta.data_ptr(), out.data_ptr(), B, Hq, Hkv, L, S, cap, D,
                                   _scale(scale, D), window, first, float(softcap),
                                   sinks.data_ptr() if sinks is not None else None, workspace.data_ptr(),
                                   _raw_stream(dev))
    if rc != TFA_OK:
        raise TfaError(rc, "tfa_kv4_prefill")
    return out
