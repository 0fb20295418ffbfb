"""Python binding of libfa_rows: row-indexed flash attention over a unified KV pool.

Argument marshalling only.  Every step of the computation runs in the CUDA
kernels of ``libfa_rows.so``; torch supplies device memory, streams and
pointers.  If the library has not been built the calls raise instead of
computing anything another way.

The operation ("llama.cpp 0.9.0 inference boundaries", section 1): K/V rows of
all sequences share one pool; each query slice passes an int32 ``kv_rows``
list of the pool rows it attends to; a negative index is padding (mask minus
infinity); the result is exact attention over the listed rows.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import Optional, Tuple

import torch

__all__ = [
    "FaRowsError", "lib", "library_path", "fa_rows_args", "fa_rows_workspace_size", "fa_rows_workspace_init",
    "fa_rows_status", "fa_set_wait_limit_ns", "default_workspace", "FA_WS_WAIT_EXPIRED",
    "fa_rows_decode", "fa_rows_prefill", "fa_rows_decode_heads", "fa_rows_prefill_heads", "fa_rows_weights",
    "fa_kv_evict", "fa_kv_block_bounds", "fa_kv_block_scores", "fa_kv_block_rows", "fa_rows_validate", "fa_kv_page_table_to_rows", "fa_kv_quantize_int8",
    "fa_kv_dequantize_int8", "fa_kv_quantize_int4", "fa_kv_dequantize_int4", "fa_kv_quantize_fp8", "fa_kv_dequantize_fp8", "fa_kv_sparse_rows_workspace_size", "fa_kv_sparse_rows", "fa_kv_append", "fa_status_string", "fa_last_error", "fa_version",
    "FA_F16", "FA_BF16", "FA_F32", "FA_I8", "FA_I4", "FA_F8E4M3", "FA_MASK_NONE", "FA_MASK_DENSE", "FA_MASK_CAUSAL",
]

FA_F16, FA_BF16, FA_F32, FA_I8, FA_I4, FA_F8E4M3 = 0, 1, 2, 3, 4, 5
FA_MASK_NONE, FA_MASK_DENSE, FA_MASK_CAUSAL = 0, 1, 2
_STATUS = {0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED", 3: "FA_ERR_WORKSPACE",
           4: "FA_ERR_INDEX_OOB", 5: "FA_ERR_CUDA", 6: "FA_ERR_WAIT_EXPIRED"}
FA_ERR_WAIT_EXPIRED = 6
FA_WS_WAIT_EXPIRED = 1   # bit of the workspace status word (first uint32 of a workspace)

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libfa_rows.so")


class FaRowsError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_STATUS.get(status, status)}: {msg}")
        self.status = status


class fa_rows_args(ctypes.Structure):
    """Mirror of ``fa_rows_args`` in include/fa_rows.h."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("q_dtype", ctypes.c_int),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("kv_dtype", ctypes.c_int),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("n_pool_rows", ctypes.c_int64),
        ("kv_rows", ctypes.c_void_p), ("list_len", ctypes.c_int32),
        ("kv_len", ctypes.c_void_p),
        ("mask_kind", ctypes.c_int), ("mask", ctypes.c_void_p),
        ("scale", ctypes.c_float),
        ("out", ctypes.c_void_p), ("out_dtype", ctypes.c_int), ("lse", ctypes.c_void_p),
        ("S", ctypes.c_int32), ("Nq", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
        ("D", ctypes.c_int32),
        ("n_valid_hint", ctypes.c_int64),
    ]


_lib = None
_lib_lock = threading.Lock()

_P = ctypes.c_void_p
_SIGS = {
    "fa_rows_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(fa_rows_args), ctypes.c_int]),
    "fa_rows_decode_launches": (ctypes.c_int, [ctypes.POINTER(fa_rows_args)]),
    "fa_rows_workspace_init": (ctypes.c_int, [_P, ctypes.c_size_t, _P]),
    "fa_rows_status": (ctypes.c_int, [_P, ctypes.c_size_t, _P, ctypes.c_int, _P]),
    "fa_set_wait_limit_ns": (ctypes.c_int, [ctypes.c_uint64]),
    "fa_rows_decode": (ctypes.c_int, [ctypes.POINTER(fa_rows_args), _P, ctypes.c_size_t, _P]),
    "fa_rows_prefill": (ctypes.c_int, [ctypes.POINTER(fa_rows_args), _P, ctypes.c_size_t, _P]),
    "fa_rows_decode_static": (ctypes.c_int, [ctypes.POINTER(fa_rows_args), _P]),
    "fa_rows_validate": (ctypes.c_int, [ctypes.POINTER(fa_rows_args), _P, _P]),
    "fa_kv_page_table_to_rows": (ctypes.c_int, [_P, ctypes.c_int32, _P, ctypes.c_int32, ctypes.c_int32, _P,
                                                ctypes.c_int32, _P]),
    "fa_kv_quantize_int8": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P,
                                           _P, ctypes.c_int64, _P]),
    "fa_kv_dequantize_int8": (ctypes.c_int, [_P, _P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P]),
    "fa_kv_quantize_int4": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P,
                                           _P, ctypes.c_int64, _P]),
    "fa_kv_dequantize_int4": (ctypes.c_int, [_P, _P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P]),
    "fa_kv_quantize_fp8": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P,
                                          _P, ctypes.c_int64, _P]),
    "fa_kv_dequantize_fp8": (ctypes.c_int, [_P, _P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P]),
    "fa_kv_sparse_rows_workspace_size": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32]),
    "fa_kv_sparse_rows": (ctypes.c_int, [_P, ctypes.c_int32, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                         ctypes.c_int32, _P, _P, ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "fa_kv_append": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P,
                                    ctypes.c_int64, _P]),
    "fa_rows_decode_heads": (ctypes.c_int, [ctypes.POINTER(fa_rows_args), _P, ctypes.c_size_t, _P]),
    "fa_rows_prefill_heads": (ctypes.c_int, [ctypes.POINTER(fa_rows_args), _P, ctypes.c_size_t, _P]),
    "fa_rows_weights": (ctypes.c_int, [ctypes.POINTER(fa_rows_args), _P, ctypes.c_float, _P, _P, ctypes.c_size_t, _P]),
    "fa_kv_evict": (ctypes.c_int, [_P, _P, _P] + [ctypes.c_int32] * 6 + [_P, _P, _P, ctypes.c_int32, _P, _P, _P]),
    "fa_kv_block_bounds": (ctypes.c_int, [_P, ctypes.c_int, _P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P,
                                          ctypes.c_int32, _P, _P, ctypes.c_int, _P]),
    "fa_kv_block_scores": (ctypes.c_int, [_P, ctypes.c_int] + [ctypes.c_int32] * 5 + [_P, _P, ctypes.c_int64, _P,
                                          ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "fa_kv_block_rows": (ctypes.c_int, [_P, _P, ctypes.c_int32, ctypes.c_int32, _P, _P] + [ctypes.c_int32] * 5 +
                         [_P, _P, ctypes.c_int32, _P]),
    "fa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "fa_last_error": (ctypes.c_char_p, []),
    "fa_version": (ctypes.c_char_p, []),
}


def lib() -> ctypes.CDLL:
    """The loaded libfa_rows.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        with _lib_lock:
            if _lib is None:
                if not os.path.exists(library_path):
                    raise RuntimeError(f"libfa_rows.so is not built ({library_path}); "
                                       "run `python -m row_indexed_flash_gb300.build`")
                h = ctypes.CDLL(library_path)
                for name, (res, args) in _SIGS.items():
                    fn = getattr(h, name)
                    fn.restype = res
                    fn.argtypes = args
                _lib = h
    return _lib


def fa_status_string(s: int) -> str:
    return lib().fa_status_string(s).decode()


def fa_last_error() -> str:
    return lib().fa_last_error().decode()


def fa_version() -> str:
    return lib().fa_version().decode()


def _check(status: int):
    if status != 0:
        raise FaRowsError(status, fa_last_error())


# ---------------------------------------------------------------------------
# marshalling helpers

_DT = {torch.float16: FA_F16, torch.bfloat16: FA_BF16, torch.float32: FA_F32, torch.int8: FA_I8, torch.uint8: FA_I4,
       torch.float8_e4m3fn: FA_F8E4M3}


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


# The handle of a device's current stream without a Stream object (4 us less a call), where this torch
# has that function; it is not part of torch's public interface.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_NOTHING = contextlib.nullcontext()


def _stream(stream, device) -> int:
    if stream is None:
        if _raw_stream is not None and device.index is not None:
            return _raw_stream(device.index)
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _made_for(stream, device):
    """Context in which a call's new tensors are made: they belong to the stream that the call works on,
    so that they are zeroed before its kernels run and not handed out again while these still use them."""
    if stream is None:
        return _NOTHING
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream, device), device=device)
    return torch.cuda.stream(stream)


def _new(make, shape, dtype, device, stream):
    """A new tensor (make: torch.empty or torch.zeros) of the call's stream."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with _made_for(stream, device):
        return make(shape, dtype=dtype, device=device)


def _capturing(stream, device) -> bool:
    with _made_for(stream, device):
        return torch.cuda.is_current_stream_capturing()


def _captured_ws(nbytes: int, device, stream_handle: int, stream, counters: bool = False) -> torch.Tensor:
    """Scratch of one call that is being captured: of the graph alone, so that graphs may be replayed in any
    order and side by side.  Split counters (counters) are zeroed by the graph itself; nothing else of it has to
    be, as no one can read its status word."""
    buf = _new(torch.empty, max(nbytes, 256), torch.uint8, device, stream)
    if counters:
        _check(lib().fa_rows_workspace_init(buf.data_ptr(), min(buf.numel(), 16384), stream_handle))
    return buf


class _Workspace:
    """Caller-side scratch (status word, split counters, partials): grown on demand, zeroed once."""

    def __init__(self):
        self.buf: Optional[torch.Tensor] = None

    def get(self, nbytes: int, device, stream_handle: int, stream=None) -> torch.Tensor:
        if self.buf is None or self.buf.numel() < nbytes:
            if _capturing(stream, device):
                return _captured_ws(nbytes, device, stream_handle, stream)
            self.buf = _new(torch.empty, max(nbytes, 1 << 20), torch.uint8, device, stream)
            _check(lib().fa_rows_workspace_init(self.buf.data_ptr(), self.buf.numel(), stream_handle))
        return self.buf


_workspaces = {}


def _default_ws(device, stream_handle, is_prefill: bool) -> _Workspace:
    """The binding's own workspace for calls without one: one per (device, stream, decode or prefill).
    A call that is captured into a graph has one to itself instead."""
    key = (device, stream_handle, bool(is_prefill))
    if key not in _workspaces:
        _workspaces[key] = _Workspace()
    return _workspaces[key]


def default_workspace(device=None, stream=None, is_prefill: bool = False) -> Optional[torch.Tensor]:
    """The workspace tensor the binding uses for calls made without one (None before the first such call)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return _default_ws(device, _stream(stream, device), is_prefill).buf


def make_args(q, k, v, kv_rows, scale, *, kv_len=None, mask=None, causal=False, k_scale=None, v_scale=None,
              out=None, lse=None, out_dtype=torch.float32, want_lse=False, n_valid_hint=0, head_lists=False, stream=None):
    """Builds fa_rows_args from torch tensors; allocates ``out``/``lse`` (of ``stream``) if not given.

    head_lists: kv_rows is [S, Hkv, L] and kv_len [S, Hkv], one list per KV head.
    """
    S, Nq, Hq, D = q.shape
    R, Hkv, Dk = k.shape
    packed = k.dtype == torch.uint8   # INT4 pool: two codes per byte
    if tuple(v.shape) != (R, Hkv, Dk) or Dk * (2 if packed else 1) != D:
        raise ValueError(f"k {tuple(k.shape)} / v {tuple(v.shape)} do not match q {tuple(q.shape)}")
    lists = (S, Hkv) if head_lists else (S,)
    if kv_rows.dtype != torch.int32 or tuple(kv_rows.shape[:-1]) != lists:
        raise ValueError("kv_rows must be int32 [S, Hkv, L]" if head_lists else "kv_rows must be int32 [S, L]")
    if k.dtype != v.dtype:
        raise ValueError("k and v must share a dtype")
    if k.dtype in (torch.int8, torch.uint8, torch.float8_e4m3fn) and (k_scale is None or v_scale is None):
        raise ValueError("a quantised pool needs k_scale and v_scale")
    if kv_len is not None and (kv_len.dtype != torch.int32 or tuple(kv_len.shape) != lists):
        raise ValueError("kv_len must be int32 [S, Hkv]" if head_lists else "kv_len must be int32 [S]")
    if mask is not None and (mask.dtype != torch.float32 or tuple(mask.shape) != (S, Nq, kv_rows.shape[-1])):
        raise ValueError("mask must be float32 [S, Nq, L]")
    if out is None:
        out = _new(torch.empty, (S, Nq, Hq, D), out_dtype, q.device, stream)
    if lse is None and want_lse:
        lse = _new(torch.empty, (S, Nq, Hq), torch.float32, q.device, stream)
    a = fa_rows_args()
    a.q, a.q_dtype = _ptr(q), _DT[q.dtype]
    a.k, a.v, a.kv_dtype = _ptr(k), _ptr(v), _DT[k.dtype]
    a.k_scale, a.v_scale = _ptr(k_scale), _ptr(v_scale)
    a.n_pool_rows = R
    a.kv_rows, a.list_len = _ptr(kv_rows), kv_rows.shape[-1]
    a.kv_len = _ptr(kv_len)
    if mask is not None:
        a.mask_kind, a.mask = FA_MASK_DENSE, _ptr(mask)
    else:
        a.mask_kind = FA_MASK_CAUSAL if causal else FA_MASK_NONE
    a.scale = float(scale)
    a.out, a.out_dtype, a.lse = _ptr(out), _DT[out.dtype], _ptr(lse)
    a.S, a.Nq, a.Hq, a.Hkv, a.D = S, Nq, Hq, Hkv, D
    a.n_valid_hint = int(n_valid_hint)
    return a, out, lse


def fa_rows_workspace_size(args: fa_rows_args, is_prefill: bool = False) -> int:
    n = lib().fa_rows_workspace_size(ctypes.byref(args), int(is_prefill))
    err = fa_last_error()
    if err:
        raise FaRowsError(1, err)
    return n


def fa_rows_workspace_init(ws: torch.Tensor, stream=None):
    _check(lib().fa_rows_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream, ws.device)))


def fa_rows_status(ws: torch.Tensor, clear: bool = False, stream=None) -> int:
    """The workspace's status word (FA_WS_WAIT_EXPIRED set: a call on it had a
    pipeline wait run out).  Synchronises the stream to read it."""
    sh = _stream(stream, ws.device)
    with _made_for(stream, ws.device):   # and read on
        word = torch.empty(1, dtype=torch.int32, device=ws.device)
        _check(lib().fa_rows_status(_ptr(ws), ws.numel() * ws.element_size(), word.data_ptr(), int(clear), sh))
        return int(word.item()) & 0xffffffff


def fa_set_wait_limit_ns(limit_ns: int):
    """Limit of every bounded pipeline wait in kernels launched afterwards (0 = the 1 s default)."""
    _check(lib().fa_set_wait_limit_ns(int(limit_ns)))


def _attend(entry: str, is_prefill: bool, q, k, v, kv_rows, scale, *, workspace=None, stream=None,
            check_status=False, **kw):
    a, out, lse = make_args(q, k, v, kv_rows, scale, stream=stream, **kw)
    sh = _stream(stream, q.device)
    need = fa_rows_workspace_size(a, is_prefill)
    if workspace is None:
        if _capturing(stream, q.device):
            # one launch with partials: the splits are counted and merged in it
            counters = need > 256 and not is_prefill and lib().fa_rows_decode_launches(ctypes.byref(a)) == 1
            wtensor = _captured_ws(need, q.device, sh, stream, counters)
        else:
            wtensor = _default_ws(q.device, sh, is_prefill).get(need, q.device, sh, stream)
        wptr, wbytes = wtensor.data_ptr(), wtensor.numel()
    else:
        wptr, wbytes = _ptr(workspace), workspace.numel() * workspace.element_size()
        wtensor = workspace
    _check(getattr(lib(), entry)(ctypes.byref(a), wptr, wbytes, sh))
    if check_status:
        word = fa_rows_status(wtensor, clear=True, stream=stream)
        if word & FA_WS_WAIT_EXPIRED:
            raise FaRowsError(FA_ERR_WAIT_EXPIRED, f"{entry}: a pipeline wait ran out; the outputs are invalid")
    return out, lse


def fa_rows_decode(q, k, v, kv_rows, scale, **kw):
    """Decode (few query rows per slice).  Returns (out, lse or None).

    Keyword args: kv_len, mask (fp32 [S,Nq,L]), causal, k_scale/v_scale (int8
    pool, fp16 [R/64,Hkv,64]), out, lse, out_dtype, want_lse, n_valid_hint,
    workspace (zero-initialised uint8 tensor), stream (what the call allocates
    belongs to it; the current one if None), check_status (read the
    workspace status word after the call -- this synchronises -- and raise
    FA_ERR_WAIT_EXPIRED if a pipeline wait ran out, clearing the word).
    """
    return _attend("fa_rows_decode", False, q, k, v, kv_rows, scale, **kw)


def fa_rows_prefill(q, k, v, kv_rows, scale, **kw):
    """Prefill (many query rows per slice), tensor-core path.  Same arguments as decode."""
    return _attend("fa_rows_prefill", True, q, k, v, kv_rows, scale, **kw)


_ATTEND_TENSORS = ("kv_len", "k_scale", "v_scale", "out", "lse", "workspace")


def fa_rows_decode_heads(q, k, v, kv_rows, scale, **kw):
    """Decode over one list per (slice, KV head): kv_rows int32 [S, Hkv, L], kv_len int32 [S, Hkv].

    Keyword args as fa_rows_decode, without mask; n_valid_hint is the entries of
    all lists divided by Hkv.
    """
    _check_scale(k, kw.get("k_scale"))
    _check_scale(v, kw.get("v_scale"), "v_scale")
    _same_device(q.device, k, v, kv_rows, *(kw.get(x) for x in _ATTEND_TENSORS))
    with _on(q.device):
        return _attend("fa_rows_decode_heads", False, q, k, v, kv_rows, scale, head_lists=True, **kw)


def fa_rows_prefill_heads(q, k, v, kv_rows, scale, **kw):
    """Prefill over one list per (slice, KV head), as fa_rows_decode_heads; causal: each list
    ends with the slice's Nq newest positions."""
    _same_device(q.device, k, v, kv_rows, *(kw.get(x) for x in _ATTEND_TENSORS))
    with _on(q.device):
        return _attend("fa_rows_prefill_heads", True, q, k, v, kv_rows, scale, head_lists=True, **kw)


def _status_ws(workspace, device, sh, stream, need: int = 256):
    """(pointer, bytes, tensor) of the caller's workspace or the binding's own one for calls that
    need the status block alone."""
    if workspace is not None:
        return _ptr(workspace), workspace.numel() * workspace.element_size(), workspace
    buf = _default_ws(device, sh, True).get(need, device, sh, stream)
    return buf.data_ptr(), buf.numel(), buf


def _raise_expired(entry: str, wtensor, stream):
    word = fa_rows_status(wtensor, clear=True, stream=stream)
    if word & FA_WS_WAIT_EXPIRED:
        raise FaRowsError(FA_ERR_WAIT_EXPIRED, f"{entry}: a pipeline wait ran out; the outputs are invalid")


def _on(device):
    """Context that makes ``device`` the current one (nothing to do when it is)."""
    if device.index is None or device.index == torch.cuda.current_device():
        return _NOTHING
    return torch.cuda.device(device)


def _same_device(device, *tensors):
    if device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    index = device.index
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors must share one device ({t.device} and {device})")


def _ptrs(device, *tensors):
    """Pointers of tensors (None: None) that must be contiguous and on ``device``."""
    if device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    index = device.index
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        if t.get_device() != index:
            raise ValueError(f"tensors must share one device ({t.device} and {device})")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        out.append(t.data_ptr())
    return out


def fa_rows_weights(q, k, kv_rows, scale, lse, acc=None, *, decay: float = 1.0, kv_len=None, mask=None, causal=False,
                    k_scale=None, workspace=None, stream=None, check_status=False) -> torch.Tensor:
    """acc [S, Hkv, L] += the softmax weight each list entry received from the attention call that
    returned ``lse`` for the same arguments (acc None: a new zero accumulator; decay scales the old acc)."""
    S, Nq, Hq, D = q.shape
    R, Hkv, Dk = k.shape
    if Dk * (2 if k.dtype == torch.uint8 else 1) != D:
        raise ValueError(f"k {tuple(k.shape)} does not match q {tuple(q.shape)}")
    if kv_rows.dtype != torch.int32 or kv_rows.dim() != 2 or kv_rows.shape[0] != S:
        raise ValueError("kv_rows must be int32 [S, L]")
    L = kv_rows.shape[1]
    if lse.dtype != torch.float32 or lse.shape != (S, Nq, Hq):
        raise ValueError("lse must be float32 [S, Nq, Hq]")
    if kv_len is not None and (kv_len.dtype != torch.int32 or kv_len.shape != (S,)):
        raise ValueError("kv_len must be int32 [S]")
    if mask is not None and (mask.dtype != torch.float32 or mask.shape != (S, Nq, L)):
        raise ValueError("mask must be float32 [S, Nq, L]")
    if acc is None:
        acc = _new(torch.zeros, (S, Hkv, L), torch.float32, q.device, stream)
    elif acc.dtype != torch.float32 or acc.shape != (S, Hkv, L):
        raise ValueError("acc must be float32 [S, Hkv, L]")
    _check_scale(k, k_scale)
    dev = q.device
    a = fa_rows_args()
    a.q, a.k, a.k_scale, a.kv_rows, a.kv_len, a.mask, plse, pacc, _ = _ptrs(
        dev, q, k, k_scale, kv_rows, kv_len, mask, lse, acc, workspace)
    a.q_dtype, a.kv_dtype = _DT[q.dtype], _DT[k.dtype]
    a.n_pool_rows = R
    a.list_len = L
    a.mask_kind = FA_MASK_DENSE if mask is not None else FA_MASK_CAUSAL if causal else FA_MASK_NONE
    a.scale = float(scale)
    a.S, a.Nq, a.Hq, a.Hkv, a.D = S, Nq, Hq, Hkv, D
    with _on(dev):
        sh = _stream(stream, dev)
        wptr, wbytes, wtensor = _status_ws(workspace, dev, sh, stream)
        _check(lib().fa_rows_weights(ctypes.byref(a), plse, float(decay), pacc, wptr, wbytes, sh))
    if check_status:
        _raise_expired("fa_rows_weights", wtensor, stream)
    return acc


def fa_kv_evict(acc, kv_rows, kv_len, sinks: int, recent: int, k: int, *, out_len: Optional[int] = None, acc_out=None,
                rows_out=None, len_out=None, kept=None, freed=None, stream=None):
    """Keeps the sinks, the recent entries and the k heaviest of the others of each list.

    Returns (rows [S, out_len], length [S], acc [S, Hkv, out_len], kept positions [S, out_len],
    freed rows [S, L]); -1 (acc: 0) past the end.  out_len None: sinks + recent + k.
    """
    if acc.dtype != torch.float32 or acc.dim() != 3:
        raise ValueError("acc must be float32 [S, Hkv, L]")
    S, Hkv, L = acc.shape
    if kv_rows.dtype != torch.int32 or kv_rows.shape != (S, L):
        raise ValueError("kv_rows must be int32 [S, L]")
    if kv_len is not None and (kv_len.dtype != torch.int32 or kv_len.shape != (S,)):
        raise ValueError("kv_len must be int32 [S]")
    n = int(out_len) if out_len is not None else int(sinks) + int(recent) + int(k)
    dev = acc.device

    def dest(t, shape, dtype, name):
        if t is None:
            return _new(torch.empty, shape, dtype, dev, stream)
        if t.dtype != dtype or t.shape != shape:
            raise ValueError(f"{name} must be {dtype} {shape}")
        return t

    rows_out = dest(rows_out, (S, n), torch.int32, "rows_out")
    len_out = dest(len_out, (S,), torch.int32, "len_out")
    acc_out = dest(acc_out, (S, Hkv, n), torch.float32, "acc_out")
    kept = dest(kept, (S, n), torch.int32, "kept")
    freed = dest(freed, (S, L), torch.int32, "freed")
    pa, pr, pl, po, pro, plo, pk, pf = _ptrs(dev, acc, kv_rows, kv_len, acc_out, rows_out, len_out, kept, freed)
    with _on(dev):
        _check(lib().fa_kv_evict(pa, pr, pl, S, Hkv, L, int(sinks), int(recent), int(k), po, pro, plo, n, pk, pf,
                                 _stream(stream, dev)))
    return rows_out, len_out, acc_out, kept, freed


def fa_kv_block_bounds(k, pages, fill, kmin, kmax, *, k_scale=None, stream=None):
    """Updates kmin, kmax [R/64, Hkv, D] with the elementwise key bounds of the listed 64-row pages
    (the first fill[i] rows of each; fill None: 64).  Returns (kmin, kmax)."""
    R, Hkv, Dk = k.shape
    D = Dk * (2 if k.dtype == torch.uint8 else 1)
    if kmin.dtype != kmax.dtype or kmin.shape != (R // 64, Hkv, D) or kmax.shape != (R // 64, Hkv, D):
        raise ValueError(f"kmin and kmax must be [R/64, Hkv, D] = {(R // 64, Hkv, D)} of one dtype")
    for t, name in ((pages, "pages"), (fill, "fill")):
        if t is not None and (t.dtype != torch.int32 or t.shape != pages.shape or t.dim() != 1):
            raise ValueError(f"{name} must be int32 [n_pages]")
    _check_scale(k, k_scale)
    dev = k.device
    pk, ps, pp, pf, plo, phi = _ptrs(dev, k, k_scale, pages, fill, kmin, kmax)
    with _on(dev):
        _check(lib().fa_kv_block_bounds(pk, _DT[k.dtype], ps, R, Hkv, D, pp, pf, pages.shape[0], plo, phi,
                                        _DT[kmin.dtype], _stream(stream, dev)))
    return kmin, kmax


def _check_scale(pool, scale, name="k_scale"):
    if pool.dtype in (torch.int8, torch.uint8, torch.float8_e4m3fn):
        if scale is None:
            raise ValueError(f"a quantised pool needs {name}")
        if scale.dtype != torch.float16 or scale.shape != (pool.shape[0] // 64, pool.shape[1], 64):
            raise ValueError(f"{name} must be float16 [R/64, Hkv, 64]")


def _check_pages(S, page_table, seq_len, slice_seq):
    if page_table.dtype != torch.int32 or page_table.dim() != 2:
        raise ValueError("page_table must be int32 [n_seq, max_pages]")
    if seq_len.dtype != torch.int32 or seq_len.shape != (S,):
        raise ValueError("seq_len must be int32 [S]")
    if slice_seq is not None and (slice_seq.dtype != torch.int32 or slice_seq.shape != (S,)):
        raise ValueError("slice_seq must be int32 [S]")


def fa_kv_block_scores(q, kmin, kmax, page_table, seq_len, *, slice_seq=None, out=None, workspace=None, stream=None,
                       check_status=False) -> torch.Tensor:
    """Upper bounds [S, Hkv, max_pages] of the dot products of each slice's queries with the keys of
    each block of its sequence (page_table row slice_seq[s], or s)."""
    S, Nq, Hq, D = q.shape
    P, Hkv, Dk = kmin.shape
    if Dk != D or kmin.shape != kmax.shape or kmin.dtype != q.dtype or kmax.dtype != q.dtype:
        raise ValueError("kmin and kmax must be [pages, Hkv, D] of q's dtype")
    _check_pages(S, page_table, seq_len, slice_seq)
    n_seq, max_pages = page_table.shape
    if out is None:
        out = _new(torch.empty, (S, Hkv, max_pages), torch.float32, q.device, stream)
    elif out.dtype != torch.float32 or out.shape != (S, Hkv, max_pages):
        raise ValueError("out must be float32 [S, Hkv, max_pages]")
    dev = q.device
    pq, plo, phi, pt, pn, pseq, po, _ = _ptrs(dev, q, kmin, kmax, page_table, seq_len, slice_seq, out, workspace)
    with _on(dev):
        sh = _stream(stream, dev)
        wptr, wbytes, wtensor = _status_ws(workspace, dev, sh, stream)
        _check(lib().fa_kv_block_scores(pq, _DT[q.dtype], S, Nq, Hq, Hkv, D, plo, phi, P, pt, n_seq, max_pages, pn,
                                        pseq, po, wptr, wbytes, sh))
    if check_status:
        _raise_expired("fa_kv_block_scores", wtensor, stream)
    return out


def fa_kv_block_rows(score, page_table, seq_len, sink_blocks: int, recent_blocks: int, k: int, *, slice_seq=None,
                     list_len: Optional[int] = None, out=None, out_len=None, stream=None):
    """Row lists [S, Hkv, list_len] and lengths [S, Hkv] of the first sink_blocks, the last
    recent_blocks and the k best-scored other blocks (list_len None: 64 per block)."""
    if score.dtype != torch.float32 or score.dim() != 3:
        raise ValueError("score must be float32 [S, Hkv, max_pages]")
    S, Hkv, max_pages = score.shape
    _check_pages(S, page_table, seq_len, slice_seq)
    if page_table.shape[1] != max_pages:
        raise ValueError("page_table and score must have the same max_pages")
    L = 64 * (int(sink_blocks) + int(recent_blocks) + int(k)) if list_len is None else int(list_len)
    if out is None:
        out = _new(torch.empty, (S, Hkv, L), torch.int32, score.device, stream)
    elif out.dtype != torch.int32 or out.shape != (S, Hkv, L):
        raise ValueError("out must be int32 [S, Hkv, list_len]")
    if out_len is None:
        out_len = _new(torch.empty, (S, Hkv), torch.int32, score.device, stream)
    elif out_len.dtype != torch.int32 or out_len.shape != (S, Hkv):
        raise ValueError("out_len must be int32 [S, Hkv]")
    dev = score.device
    ps, pt, pn, pseq, po, pol = _ptrs(dev, score, page_table, seq_len, slice_seq, out, out_len)
    with _on(dev):
        _check(lib().fa_kv_block_rows(ps, pt, page_table.shape[0], max_pages, pn, pseq, S, Hkv, int(sink_blocks),
                                      int(recent_blocks), int(k), po, pol, L, _stream(stream, dev)))
    return out, out_len


def fa_rows_validate(kv_rows: torch.Tensor, n_pool_rows: int, kv_len=None, stream=None) -> Tuple[int, int]:
    """Range check of the lists; returns (entries >= n_pool_rows, first flat index or -1).  Synchronises."""
    a = fa_rows_args()
    a.kv_rows, a.list_len, a.S = _ptr(kv_rows), kv_rows.shape[1], kv_rows.shape[0]
    a.kv_len = _ptr(kv_len)
    a.n_pool_rows = int(n_pool_rows)
    with _made_for(stream, kv_rows.device):   # and read on
        status = torch.empty(2, dtype=torch.int64, device=kv_rows.device)
        _check(lib().fa_rows_validate(ctypes.byref(a), status.data_ptr(), _stream(stream, kv_rows.device)))
        c, f = status.tolist()
    return int(c), int(f)


def fa_kv_page_table_to_rows(page_table: torch.Tensor, seq_len: torch.Tensor, list_len: int, page_size: int = 64,
                             out=None, stream=None) -> torch.Tensor:
    n_seq, max_pages = page_table.shape
    if out is None:
        out = _new(torch.empty, (n_seq, list_len), torch.int32, page_table.device, stream)
    _check(lib().fa_kv_page_table_to_rows(_ptr(page_table), max_pages, _ptr(seq_len), n_seq, page_size, _ptr(out),
                                          list_len, _stream(stream, page_table.device)))
    return out


def fa_kv_quantize_int8(x: torch.Tensor, n_pool_rows: Optional[int] = None, dst_rows=None, q=None, scale=None,
                        stream=None):
    """Quantises x [n, Hkv, D] (bf16/f16) into an INT8 pool; returns (q [R,Hkv,D] int8, scale fp16 [R/64,Hkv,64])."""
    n, Hkv, D = x.shape
    R = n if n_pool_rows is None else int(n_pool_rows)
    if q is None:
        q = _new(torch.zeros, (R, Hkv, D), torch.int8, x.device, stream)
    if scale is None:
        scale = _new(torch.zeros, (R // 64, Hkv, 64), torch.float16, x.device, stream)
    _check(lib().fa_kv_quantize_int8(_ptr(x), _DT[x.dtype], n, Hkv, D, _ptr(dst_rows), _ptr(q), _ptr(scale),
                                     q.shape[0], _stream(stream, x.device)))
    return q, scale


def fa_kv_dequantize_int8(q: torch.Tensor, scale: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    R, Hkv, D = q.shape
    if out is None:
        out = _new(torch.empty, (R, Hkv, D), torch.float32, q.device, stream)
    _check(lib().fa_kv_dequantize_int8(_ptr(q), _ptr(scale), R, Hkv, D, _ptr(out), _stream(stream, q.device)))
    return out


def fa_kv_quantize_int4(x: torch.Tensor, n_pool_rows: Optional[int] = None, dst_rows=None, q=None, scale=None,
                        stream=None):
    """Quantises x [n, Hkv, D] (bf16/f16) into an INT4 pool; returns (q [R,Hkv,D/2] uint8, scale fp16 [R/64,Hkv,64])."""
    n, Hkv, D = x.shape
    R = n if n_pool_rows is None else int(n_pool_rows)
    if q is None:
        q = _new(torch.zeros, (R, Hkv, D // 2), torch.uint8, x.device, stream)
    if scale is None:
        scale = _new(torch.zeros, (R // 64, Hkv, 64), torch.float16, x.device, stream)
    _check(lib().fa_kv_quantize_int4(_ptr(x), _DT[x.dtype], n, Hkv, D, _ptr(dst_rows), _ptr(q), _ptr(scale),
                                     q.shape[0], _stream(stream, x.device)))
    return q, scale


def fa_kv_dequantize_int4(q: torch.Tensor, scale: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    R, Hkv, Dh = q.shape
    if out is None:
        out = _new(torch.empty, (R, Hkv, 2 * Dh), torch.float32, q.device, stream)
    _check(lib().fa_kv_dequantize_int4(_ptr(q), _ptr(scale), R, Hkv, 2 * Dh, _ptr(out), _stream(stream, q.device)))
    return out


def fa_kv_quantize_fp8(x: torch.Tensor, n_pool_rows: Optional[int] = None, dst_rows=None, q=None, scale=None,
                       stream=None):
    """Quantises x [n, Hkv, D] (bf16/f16) into an FP8 E4M3 pool; returns (q [R,Hkv,D] float8_e4m3fn, scale fp16)."""
    n, Hkv, D = x.shape
    R = n if n_pool_rows is None else int(n_pool_rows)
    if q is None:
        q = _new(torch.zeros, (R, Hkv, D), torch.float8_e4m3fn, x.device, stream)
    if scale is None:
        scale = _new(torch.zeros, (R // 64, Hkv, 64), torch.float16, x.device, stream)
    _check(lib().fa_kv_quantize_fp8(_ptr(x), _DT[x.dtype], n, Hkv, D, _ptr(dst_rows), _ptr(q), _ptr(scale),
                                    q.shape[0], _stream(stream, x.device)))
    return q, scale


def fa_kv_dequantize_fp8(q: torch.Tensor, scale: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    R, Hkv, D = q.shape
    if out is None:
        out = _new(torch.empty, (R, Hkv, D), torch.float32, q.device, stream)
    _check(lib().fa_kv_dequantize_fp8(_ptr(q), _ptr(scale), R, Hkv, D, _ptr(out), _stream(stream, q.device)))
    return out


def fa_kv_sparse_rows(score: torch.Tensor, sinks: int, recent: int, k: int, list_len: Optional[int] = None,
                      n_len=None, row_map=None, out=None, workspace="auto", stream=None) -> torch.Tensor:
    """Sorted kv_rows [S, list_len] of sinks + top-k(score) + recent per slice (score fp32 [S, n_max]).

    workspace: "auto" allocates the multi-block scratch, None runs one block
    per slice without scratch, or a uint8 tensor of at least
    fa_kv_sparse_rows_workspace_size(S, n_max) bytes.
    """
    if score.dtype != torch.float32 or score.dim() != 2:
        raise ValueError("score must be float32 [S, n_max]")
    S, n_max = score.shape
    L = sinks + recent + k if list_len is None else int(list_len)
    if out is None:
        out = _new(torch.empty, (S, L), torch.int32, score.device, stream)
    if isinstance(workspace, str):
        nbytes = lib().fa_kv_sparse_rows_workspace_size(S, n_max)
        workspace = _new(torch.empty, max(nbytes, 16), torch.uint8, score.device, stream)
    wptr = _ptr(workspace)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fa_kv_sparse_rows(_ptr(score), n_max, _ptr(n_len), S, sinks, recent, k, _ptr(row_map), _ptr(out),
                                   L, wptr, wbytes, _stream(stream, score.device)))
    return out


def fa_kv_append(x: torch.Tensor, dst_rows: torch.Tensor, pool: torch.Tensor, stream=None) -> torch.Tensor:
    n, Hkv, D = x.shape
    if pool.dtype != x.dtype or tuple(pool.shape[1:]) != (Hkv, D):
        raise ValueError("pool must be [R, Hkv, D] of x's dtype")
    _check(lib().fa_kv_append(_ptr(x), _DT[x.dtype], n, Hkv, D, _ptr(dst_rows), _ptr(pool), pool.shape[0],
                              _stream(stream, x.device)))
    return pool
