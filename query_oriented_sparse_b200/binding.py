"""ctypes binding over libquoka.so (argument marshalling only).

Every step of the selection and attention runs in the library's CUDA kernels; this
module turns torch tensors into pointers, host arrays and the current torch stream,
and turns non-OK statuses into exceptions.  torch provides device memory and streams.
If the library is missing the first call raises: there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import List, Optional, Sequence, Tuple, Union

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libquoka.so")

QUOKA_OK, QUOKA_ERR_INVALID_ARG, QUOKA_ERR_UNSUPPORTED, QUOKA_ERR_WORKSPACE, QUOKA_ERR_CUDA = range(5)
QUOKA_F32, QUOKA_BF16 = 0, 1
QUOKA_MAX_EVICT_LEN = 786432
STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "WORKSPACE", 4: "CUDA"}

# (name, restype, argtypes) of every symbol include/quoka.h declares
_P = ctypes.c_void_p
_I64P = ctypes.POINTER(ctypes.c_int64)
_I32P = ctypes.POINTER(ctypes.c_int32)


class QuokaShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("h_q", ctypes.c_int), ("h_kv", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("chunk", ctypes.c_int), ("dtype", ctypes.c_int)]


class QuokaPagedShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("h_q", ctypes.c_int), ("h_kv", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int), ("page_size", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("max_pages", ctypes.c_int)]


_SHAPE_P = ctypes.POINTER(QuokaShape)
_PAGED_P = ctypes.POINTER(QuokaPagedShape)

SIGNATURES = {
    "quoka_version": (ctypes.c_int, []),
    "quoka_last_error": (ctypes.c_char_p, []),
    "quoka_select_workspace_size": (ctypes.c_size_t, [_SHAPE_P, ctypes.c_int, ctypes.c_int]),
    "quoka_workspace_pooled_view": (ctypes.c_int, [_SHAPE_P, ctypes.c_int, ctypes.c_int,
                                                   ctypes.POINTER(ctypes.c_size_t),
                                                   ctypes.POINTER(ctypes.c_size_t)]),
    "quoka_select": (ctypes.c_int, [_SHAPE_P, _P, _P, _I64P, _I32P, ctypes.c_int, _I32P,
                                    ctypes.c_int, _P, _P, _P, ctypes.c_size_t, _P]),
    "sparse_chunk_attn": (ctypes.c_int, [_SHAPE_P, _P, _P, _P, _I64P, _I32P, _I32P, _P,
                                         ctypes.c_int, _P, _P, ctypes.c_size_t, _P]),
    "sparse_chunk_attn_workspace_size": (ctypes.c_size_t, [_SHAPE_P, ctypes.c_int]),
    "quoka_device_error": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint32), _P]),
    "quoka_select_noalloc": (ctypes.c_int, [_SHAPE_P, _P, _P, _I64P, _I32P, ctypes.c_int, _I32P,
                                            ctypes.c_int, _P, _P, _P]),
    "sparse_perq_attn": (ctypes.c_int, [_SHAPE_P, _P, _P, _P, _I64P, _P, ctypes.c_int, _P, _P,
                                        ctypes.c_size_t, _P]),
    "sparse_perq_attn_workspace_size": (ctypes.c_size_t, [_SHAPE_P, ctypes.c_int]),
    "sparse_perq_attn_tc": (ctypes.c_int, [_SHAPE_P, _P, _P, _P, _I64P, _P, ctypes.c_int, ctypes.c_int,
                                           _P, _P, ctypes.c_size_t, _P]),
    "sparse_perq_attn_tc_workspace_size": (ctypes.c_size_t, [_SHAPE_P, ctypes.c_int, ctypes.c_int]),
    "quoka_step": (ctypes.c_int, [_SHAPE_P, _P, _P, _P, _P, _P, _I64P, _I32P, ctypes.c_int,
                                  _I32P, ctypes.c_int, _P, _P, _P, ctypes.c_size_t, _P]),
    "quoka_step_workspace_size": (ctypes.c_size_t, [_SHAPE_P, ctypes.c_int, ctypes.c_int,
                                                    ctypes.c_int]),
    "quoka_prefill": (ctypes.c_int, [_SHAPE_P, ctypes.c_int, _P, _P, _P, _P, _P, _I64P,
                                     ctypes.c_int, _I32P, ctypes.c_int, _P, _P, _P,
                                     ctypes.c_size_t, _P]),
    "quoka_prefill_workspace_size": (ctypes.c_size_t, [_SHAPE_P, ctypes.c_int, ctypes.c_int,
                                                       ctypes.c_int]),
    "quoka_selcache_bytes": (ctypes.c_size_t, [_SHAPE_P, ctypes.c_int]),
    "quoka_selcache_workspace_size": (ctypes.c_size_t, [_SHAPE_P, ctypes.c_int]),
    "quoka_selcache_update": (ctypes.c_int, [_SHAPE_P, _P, _P, _I64P, _I32P, _I32P, _P, ctypes.c_int,
                                             _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "sparse_chunk_attn_selcache": (ctypes.c_int, [_SHAPE_P, _P, _I32P, _I32P, _P, ctypes.c_int, _P,
                                                  _P, ctypes.c_size_t, _P]),
    "window_chunk_attn_workspace_size": (ctypes.c_size_t, [_SHAPE_P, ctypes.c_int, ctypes.c_int]),
    "window_chunk_attn": (ctypes.c_int, [_SHAPE_P, _P, _P, _P, _I64P, _I32P, ctypes.c_int, ctypes.c_int,
                                         _P, _P, ctypes.c_size_t, _P]),
    "paged_append": (ctypes.c_int, [_PAGED_P, _P, _P, ctypes.c_int, _P, _P, _P, _P, _P, _P, _P]),
    "paged_decode_attn_workspace_size": (ctypes.c_size_t, [_PAGED_P, ctypes.c_int, ctypes.c_int]),
    "paged_decode_attn": (ctypes.c_int, [_PAGED_P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_int,
                                         ctypes.c_int, _P, _P, _P, ctypes.c_size_t, _P]),
    "paged_evict": (ctypes.c_int, [_PAGED_P, _P, _P, _P, _P, _P, ctypes.c_int, _P, ctypes.c_int,
                                   ctypes.c_int, ctypes.c_int, _P, ctypes.c_int, _P, _P, _P]),
    "quoka_profile_events": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]),
    "quoka_profile_marks": (ctypes.c_int, [ctypes.POINTER(ctypes.c_char_p), ctypes.c_int]),
}

_lib = None


class QuokaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Loads libquoka.so from the package directory (raises if it was never built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                               "`python -m query_oriented_sparse_b200.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _check(status: int) -> None:
    if status != QUOKA_OK:
        raise QuokaError(status, lib().quoka_last_error().decode())


def make_shape(batch: int, h_q: int, h_kv: int, head_dim: int, chunk: int,
               dtype: torch.dtype) -> QuokaShape:
    if dtype == torch.float32:
        dt = QUOKA_F32
    elif dtype == torch.bfloat16:
        dt = QUOKA_BF16
    else:
        raise QuokaError(QUOKA_ERR_UNSUPPORTED, f"dtype {dtype}")
    return QuokaShape(batch, h_q, h_kv, head_dim, chunk, dt)


def shape_of(q_chunk: torch.Tensor, k_cache: torch.Tensor) -> QuokaShape:
    batch, h_q, chunk, d = q_chunk.shape
    return make_shape(batch, h_q, k_cache.shape[0], d, chunk, q_chunk.dtype)


def _host_i64(xs: Sequence[int]):
    arr = (ctypes.c_int64 * len(xs))(*[int(x) for x in xs])
    return arr


def _host_i32(xs: Sequence[int]):
    return (ctypes.c_int32 * len(xs))(*[int(x) for x in xs])


# the current stream's handle without a Stream object around it, where torch has that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def version() -> int:
    return lib().quoka_version()


def select_workspace_size(shape: QuokaShape, max_prefix: int, nq: int) -> int:
    return int(lib().quoka_select_workspace_size(ctypes.byref(shape), max_prefix, nq))


def pooled_view(workspace: torch.Tensor, shape: QuokaShape, max_prefix: int, nq: int) -> torch.Tensor:
    """The pooled key scores inside a quoka_select workspace, [batch, h_kv, stride] fp32."""
    off, stride = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().quoka_workspace_pooled_view(ctypes.byref(shape), max_prefix, nq,
                                             ctypes.byref(off), ctypes.byref(stride)))
    n = shape.batch * shape.h_kv * stride.value
    return workspace[off.value:off.value + 4 * n].view(torch.float32).view(
        shape.batch, shape.h_kv, stride.value)


def quoka_select(q_chunk: torch.Tensor, k_cache: torch.Tensor, kv_off: Sequence[int],
                 prefix_len: Sequence[int], nq: int, budget: Sequence[int],
                 b_max: Optional[int] = None, idx_out: Optional[torch.Tensor] = None,
                 kept_out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """QUOKA selection for one chunk step; returns idx [batch, h_kv, b_max] int32."""
    shape = shape_of(q_chunk, k_cache)
    if b_max is None:
        b_max = max(max(int(b) for b in budget), 1)
    dev = q_chunk.device
    if idx_out is None:
        idx_out = torch.empty(shape.batch, shape.h_kv, b_max, dtype=torch.int32, device=dev)
    if workspace is None:
        ws = select_workspace_size(shape, max(int(p) for p in prefix_len), nq)
        workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=dev)
    _check(lib().quoka_select(
        ctypes.byref(shape), _ptr(q_chunk), _ptr(k_cache), _host_i64(kv_off),
        _host_i32(prefix_len), int(nq), _host_i32(budget), int(b_max), _ptr(idx_out),
        _ptr(kept_out), _ptr(workspace), workspace.numel() * workspace.element_size(),
        ctypes.c_void_p(_stream(stream))))
    return idx_out


def quoka_select_noalloc(q_chunk: torch.Tensor, k_cache: torch.Tensor, kv_off: Sequence[int],
                         prefix_len: Sequence[int], nq: int, budget: Sequence[int],
                         b_max: Optional[int] = None, idx_out: Optional[torch.Tensor] = None,
                         kept_out: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """quoka_select using the library's built-in scratch instead of a workspace (for
    callers that cannot allocate device memory); the outputs are still the caller's."""
    shape = shape_of(q_chunk, k_cache)
    if b_max is None:
        b_max = max(max(int(b) for b in budget), 1)
    if idx_out is None:
        idx_out = torch.empty(shape.batch, shape.h_kv, b_max, dtype=torch.int32,
                              device=q_chunk.device)
    _check(lib().quoka_select_noalloc(
        ctypes.byref(shape), _ptr(q_chunk), _ptr(k_cache), _host_i64(kv_off),
        _host_i32(prefix_len), int(nq), _host_i32(budget), int(b_max), _ptr(idx_out),
        _ptr(kept_out), ctypes.c_void_p(_stream(stream))))
    return idx_out


def attn_workspace_size(shape: QuokaShape, b_max: int) -> int:
    return int(lib().sparse_chunk_attn_workspace_size(ctypes.byref(shape), int(b_max)))


def sparse_chunk_attn(q_chunk: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      kv_off: Sequence[int], prefix_len: Sequence[int], budget: Sequence[int],
                      idx: torch.Tensor, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of the chunk over its compacted cache; returns out [batch, h_q, C, d]."""
    shape = shape_of(q_chunk, k_cache)
    if out is None:
        out = torch.empty_like(q_chunk)
    b_max = int(idx.shape[-1])
    if workspace is None:
        n = attn_workspace_size(shape, b_max)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q_chunk.device) if n else None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().sparse_chunk_attn(
        ctypes.byref(shape), _ptr(q_chunk), _ptr(k_cache), _ptr(v_cache), _host_i64(kv_off),
        _host_i32(prefix_len), _host_i32(budget), _ptr(idx), b_max, _ptr(out), _ptr(workspace),
        ws_bytes, ctypes.c_void_p(_stream(stream))))
    return out


def perq_workspace_size(shape: QuokaShape, S: int) -> int:
    return int(lib().sparse_perq_attn_workspace_size(ctypes.byref(shape), int(S)))


def sparse_perq_attn(q_chunk: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     kv_off: Sequence[int], sel: torch.Tensor, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Every query over its own key set, sel int32 [batch, h_q, C, S] (-1 = none);
    returns out [batch, h_q, C, d]."""
    shape = shape_of(q_chunk, k_cache)
    if out is None:
        out = torch.empty_like(q_chunk)
    S = int(sel.shape[-1])
    if workspace is None:
        n = perq_workspace_size(shape, S)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q_chunk.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().sparse_perq_attn(
        ctypes.byref(shape), _ptr(q_chunk), _ptr(k_cache), _ptr(v_cache), _host_i64(kv_off),
        _ptr(sel), S, _ptr(out), _ptr(workspace), ws_bytes, ctypes.c_void_p(_stream(stream))))
    return out


def perq_tc_workspace_size(shape: QuokaShape, S: int, max_union: int) -> int:
    return int(lib().sparse_perq_attn_tc_workspace_size(ctypes.byref(shape), int(S), int(max_union)))


def sparse_perq_attn_tc(q_chunk: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        kv_off: Sequence[int], sel: torch.Tensor, max_union: int,
                        out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """sparse_perq_attn on tensor cores over 256-row pair tiles whose key unions hold at
    most max_union keys; returns out [batch, h_q, C, d]."""
    shape = shape_of(q_chunk, k_cache)
    if out is None:
        out = torch.empty_like(q_chunk)
    S = int(sel.shape[-1])
    if workspace is None:
        n = perq_tc_workspace_size(shape, S, max_union)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q_chunk.device)
    _check(lib().sparse_perq_attn_tc(
        ctypes.byref(shape), _ptr(q_chunk), _ptr(k_cache), _ptr(v_cache), _host_i64(kv_off),
        _ptr(sel), S, int(max_union), _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), ctypes.c_void_p(_stream(stream))))
    return out


def step_workspace_size(shape: QuokaShape, max_prefix: int, nq: int, b_max: int) -> int:
    return int(lib().quoka_step_workspace_size(ctypes.byref(shape), int(max_prefix), int(nq),
                                               int(b_max)))


def quoka_step(q_chunk: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
               k_cache: torch.Tensor, v_cache: torch.Tensor, kv_off: Sequence[int],
               prefix_len: Sequence[int], nq: int, budget: Sequence[int], idx: torch.Tensor,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One chunk (or decode) step with the cache append: q_chunk [batch, h_q, C, d],
    k_new / v_new [batch, h_kv, C, d]; returns out [batch, h_q, C, d]."""
    shape = shape_of(q_chunk, k_cache)
    if out is None:
        out = torch.empty_like(q_chunk)
    b_max = int(idx.shape[-1])
    if workspace is None:
        n = step_workspace_size(shape, max(prefix_len), nq, b_max)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q_chunk.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().quoka_step(
        ctypes.byref(shape), _ptr(q_chunk), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
        _ptr(v_cache), _host_i64(kv_off), _host_i32(prefix_len), int(nq), _host_i32(budget),
        b_max, _ptr(idx), _ptr(out), _ptr(workspace), ws_bytes, ctypes.c_void_p(_stream(stream))))
    return out


def prefill_workspace_size(shape: QuokaShape, n_chunks: int, nq: int, b_max: int) -> int:
    return int(lib().quoka_prefill_workspace_size(ctypes.byref(shape), int(n_chunks), int(nq),
                                                  int(b_max)))


def quoka_prefill(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                  k_cache: torch.Tensor, v_cache: torch.Tensor, kv_off: Sequence[int], nq: int,
                  budgets: Sequence[int], idx: torch.Tensor, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """A whole prompt through chunked prefill, appending its K/V rows to the cache.

    q [n_chunks, batch, h_q, C, d]; k_new, v_new [n_chunks, batch, h_kv, C, d];
    budgets has one entry per chunk; returns out [n_chunks, batch, h_q, C, d].
    """
    n_chunks, batch, h_q, chunk, d = q.shape
    shape = make_shape(batch, h_q, k_cache.shape[0], d, chunk, q.dtype)
    if out is None:
        out = torch.empty_like(q)
    b_max = int(idx.shape[-1])
    if workspace is None:
        n = prefill_workspace_size(shape, n_chunks, nq, b_max)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().quoka_prefill(
        ctypes.byref(shape), int(n_chunks), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
        _ptr(v_cache), _host_i64(kv_off), int(nq), _host_i32(budgets), b_max, _ptr(idx),
        _ptr(out), _ptr(workspace), ws_bytes, ctypes.c_void_p(_stream(stream))))
    return out


_HERE_AND_NOW = contextlib.nullcontext()


def _on(dev: torch.device, stream: Optional[torch.cuda.Stream]):
    """Context of a call on tensors of `dev`: that device current, and `stream` (when given)
    the stream on which the call's outputs and scratch are allocated."""
    if dev.type != "cuda":             # the kernels would follow host pointers
        raise QuokaError(QUOKA_ERR_INVALID_ARG, f"the tensors are on {dev}, not on a CUDA device")
    if stream is not None:
        if stream.device != dev:
            raise QuokaError(QUOKA_ERR_INVALID_ARG, f"the stream is on {stream.device}, the tensors on {dev}")
        return torch.cuda.stream(stream)
    if dev.index != torch.cuda.current_device():
        return torch.cuda.device(dev)
    return _HERE_AND_NOW


def _need(name: str, t: torch.Tensor, shape: Tuple[int, ...], dtype: torch.dtype, dev: torch.device) -> None:
    if t.shape == shape and t.dtype is dtype and t.device == dev and t.is_contiguous():
        return
    if t.shape != shape:
        raise QuokaError(QUOKA_ERR_INVALID_ARG, f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.dtype != dtype:
        raise QuokaError(QUOKA_ERR_INVALID_ARG, f"{name} is {t.dtype}, not {dtype}")
    if t.device != dev:
        raise QuokaError(QUOKA_ERR_INVALID_ARG, f"{name} is on {t.device}, not {dev}")
    raise QuokaError(QUOKA_ERR_INVALID_ARG, f"{name} must be contiguous")


def _c_int(x: int) -> int:
    """x held to what a C int holds (ctypes would keep its low 32 bits: a window of 2^32 + 5 keys
    would be one of 5)."""
    x = int(x)
    return x if -2 ** 31 <= x < 2 ** 31 else 2 ** 31 - 1 if x > 0 else -2 ** 31


def _adr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _scratch(workspace: Optional[torch.Tensor], n: int, dev: torch.device):
    """(workspace, its bytes): the caller's, or a new one of n bytes (None for 0)."""
    if workspace is None:
        if n == 0:
            return None, 0
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise QuokaError(QUOKA_ERR_INVALID_ARG, f"workspace must be contiguous and on {dev}")
    return workspace, workspace.numel() * workspace.element_size()


def _dims(t: torch.Tensor, name: str, n: int) -> Tuple[int, ...]:
    if t.dim() != n:
        raise QuokaError(QUOKA_ERR_INVALID_ARG, f"{name} must have {n} dimensions, not {t.dim()}")
    return t.shape


def window_workspace_size(shape: QuokaShape, max_prefix: int, window: int) -> int:
    return int(lib().window_chunk_attn_workspace_size(ctypes.byref(shape), _c_int(max_prefix), _c_int(window)))


def window_chunk_attn(q_chunk: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      kv_off: Sequence[int], prefix_len: Sequence[int], window: int, n_sink: int = 0,
                      out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of the chunk over the latest `window` keys of each query and the first n_sink
    tokens, over the contiguous cache; returns out [batch, h_q, C, d]."""
    batch, _, _, d = _dims(q_chunk, "q_chunk", 4)
    h_kv, rows, _ = _dims(k_cache, "k_cache", 3)
    dev, dt = q_chunk.device, q_chunk.dtype
    shape = shape_of(q_chunk, k_cache)
    _need("q_chunk", q_chunk, q_chunk.shape, dt, dev)
    _need("k_cache", k_cache, (h_kv, rows, d), dt, dev)
    _need("v_cache", v_cache, (h_kv, rows, d), dt, dev)
    if len(kv_off) != batch + 1 or len(prefix_len) != batch:
        raise QuokaError(QUOKA_ERR_INVALID_ARG, "kv_off needs batch + 1 entries, prefix_len batch")
    if kv_off[batch] != rows:
        raise QuokaError(QUOKA_ERR_INVALID_ARG, f"the cache has {rows} rows, kv_off says {kv_off[batch]}")
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(q_chunk)
        else:
            _need("out", out, q_chunk.shape, dt, dev)
        n = window_workspace_size(shape, max(prefix_len), window) if workspace is None else 0
        workspace, ws_bytes = _scratch(workspace, n, dev)
        _check(lib().window_chunk_attn(
            ctypes.byref(shape), _adr(q_chunk), _adr(k_cache), _adr(v_cache), _host_i64(kv_off),
            _host_i32(prefix_len), _c_int(window), _c_int(n_sink), _adr(out), _adr(workspace), ws_bytes,
            _stream(stream)))
    return out


_DTYPES = {torch.float32: QUOKA_F32, torch.bfloat16: QUOKA_BF16}


def paged_shape(h_q: int, k_pages: torch.Tensor, block_table: torch.Tensor) -> QuokaPagedShape:
    """The shape of a paged cache: pools [num_pages, h_kv, page_size, d], block_table
    [batch, max_pages]."""
    num_pages, h_kv, page, d = _dims(k_pages, "k_pages", 4)
    batch, max_pages = _dims(block_table, "block_table", 2)
    dt = _DTYPES.get(k_pages.dtype)
    if dt is None:
        raise QuokaError(QUOKA_ERR_UNSUPPORTED, f"dtype {k_pages.dtype}")
    return QuokaPagedShape(batch, h_q, h_kv, d, dt, page, num_pages, max_pages)


def _need_pools(k_pages, v_pages, record, block_table, dev) -> None:
    _need("k_pages", k_pages, k_pages.shape, k_pages.dtype, dev)
    _need("v_pages", v_pages, k_pages.shape, k_pages.dtype, dev)
    if record is not None:
        _need("weight_pages", record, k_pages.shape[:3], torch.float32, dev)
    _need("block_table", block_table, block_table.shape, torch.int32, dev)


def paged_append(k_new: torch.Tensor, v_new: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                 block_table: torch.Tensor, start: torch.Tensor, n_new: Optional[torch.Tensor] = None,
                 weight_pages: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> None:
    """New K/V rows [batch, h_kv, n, d] of each sequence into its pages from position start[b]
    (int32 [batch]); n_new, int32 [batch], limits the rows per sequence."""
    dev = k_pages.device
    shape = paged_shape(k_pages.shape[1] if k_pages.dim() == 4 else 1, k_pages, block_table)
    _need_pools(k_pages, v_pages, weight_pages, block_table, dev)
    n = _dims(k_new, "k_new", 4)[2]
    want = (shape.batch, shape.h_kv, n, shape.head_dim)
    _need("k_new", k_new, want, k_pages.dtype, dev)
    _need("v_new", v_new, want, k_pages.dtype, dev)
    _need("start", start, (shape.batch,), torch.int32, dev)
    if n_new is not None:
        _need("n_new", n_new, (shape.batch,), torch.int32, dev)
    with _on(dev, stream):
        _check(lib().paged_append(
            ctypes.byref(shape), _adr(k_new), _adr(v_new), n, _adr(k_pages), _adr(v_pages),
            _adr(weight_pages), _adr(block_table), _adr(start), _adr(n_new),
            _stream(stream)))


def paged_decode_workspace_size(shape: QuokaPagedShape, max_len: int, with_record: bool) -> int:
    return int(lib().paged_decode_attn_workspace_size(ctypes.byref(shape), _c_int(max_len), int(with_record)))


def paged_decode_attn(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                      block_table: torch.Tensor, seq_len: torch.Tensor, max_len: int,
                      window: Optional[int] = None, n_sink: int = 0,
                      weight_pages: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of one new token per sequence, q [batch, h_q, 1, d], over its seq_len[b]
    (int32, at most max_len) keys, or the latest `window` and the first n_sink of them.  With
    weight_pages, each key's softmax weight, summed over its group's heads, is added there.
    Returns out [batch, h_q, 1, d]."""
    dev = k_pages.device
    h_q = _dims(q, "q", 4)[1]
    shape = paged_shape(h_q, k_pages, block_table)
    _need_pools(k_pages, v_pages, weight_pages, block_table, dev)
    _need("q", q, (shape.batch, h_q, 1, shape.head_dim), k_pages.dtype, dev)
    _need("seq_len", seq_len, (shape.batch,), torch.int32, dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(q)
        else:
            _need("out", out, q.shape, q.dtype, dev)
        workspace, ws_bytes = _scratch(
            workspace, paged_decode_workspace_size(shape, max_len, weight_pages is not None)
            if workspace is None else 0, dev)
        _check(lib().paged_decode_attn(
            ctypes.byref(shape), _adr(q), _adr(k_pages), _adr(v_pages), _adr(block_table), _adr(seq_len),
            _c_int(max_len), _c_int(max_len if window is None else window), _c_int(n_sink), _adr(weight_pages),
            _adr(out), _adr(workspace), ws_bytes, _stream(stream)))
    return out


def paged_evict(k_pages: torch.Tensor, v_pages: torch.Tensor, weight_pages: torch.Tensor,
                block_table: torch.Tensor, seq_len: torch.Tensor, max_len: int, budget: torch.Tensor,
                b_max: int, dst_table: torch.Tensor, n_sink: int = 0, n_recent: int = 0,
                idx_out: Optional[torch.Tensor] = None, new_len: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Copies, per sequence and KV head, the first n_sink, the n_recent latest and the heaviest
    (by weight_pages) rows, budget[b] in all, to the pages of dst_table; returns the kept
    positions [batch, h_kv, b_max] and the new lengths [batch]."""
    dev = k_pages.device
    shape = paged_shape(k_pages.shape[1] if k_pages.dim() == 4 else 1, k_pages, block_table)
    _need_pools(k_pages, v_pages, weight_pages, block_table, dev)
    _need("seq_len", seq_len, (shape.batch,), torch.int32, dev)
    _need("budget", budget, (shape.batch,), torch.int32, dev)
    dst_pages = _dims(dst_table, "dst_table", 2)[1]
    _need("dst_table", dst_table, (shape.batch, dst_pages), torch.int32, dev)
    with _on(dev, stream):
        if idx_out is None:
            idx_out = torch.empty(shape.batch, shape.h_kv, max(int(b_max), 1), dtype=torch.int32, device=dev)
        else:
            _need("idx_out", idx_out, (shape.batch, shape.h_kv, int(b_max)), torch.int32, dev)
        if new_len is None:
            new_len = torch.empty(shape.batch, dtype=torch.int32, device=dev)
        else:
            _need("new_len", new_len, (shape.batch,), torch.int32, dev)
        _check(lib().paged_evict(
            ctypes.byref(shape), _adr(k_pages), _adr(v_pages), _adr(weight_pages), _adr(block_table),
            _adr(seq_len), _c_int(max_len), _adr(budget), _c_int(b_max), _c_int(n_sink), _c_int(n_recent),
            _adr(dst_table), dst_pages, _adr(idx_out), _adr(new_len), _stream(stream)))
    return idx_out, new_len


class PagedCache:
    """A paged KV cache of one layer: pools, block table, lengths and free pages for a fixed
    batch, with the paged calls over them.  `record` adds the per-key weight record that
    evict() goes by.  Pages are handed out on the host; the calls are stream-ordered."""

    def __init__(self, batch: int, h_q: int, h_kv: int, head_dim: int, dtype: torch.dtype, num_pages: int,
                 page_size: int, max_pages: int, device, record: bool = False):
        self.h_q, self.page_size, self.max_pages = int(h_q), int(page_size), int(max_pages)
        dev = torch.empty(0, device=device).device
        self.k_pages = torch.zeros(num_pages, h_kv, page_size, head_dim, dtype=dtype, device=dev)
        self.v_pages = torch.zeros_like(self.k_pages)
        self.weight_pages = torch.zeros(num_pages, h_kv, page_size, device=dev) if record else None
        self.lens: List[int] = [0] * batch
        self.free: List[int] = list(range(num_pages - 1, -1, -1))
        self.pages: List[List[int]] = [[] for _ in range(batch)]
        self.block_table = torch.full((batch, max_pages), -1, dtype=torch.int32, device=dev)
        self.seq_len = torch.zeros(batch, dtype=torch.int32, device=dev)

    def _pick(self, counts: Sequence[int]) -> List[List[int]]:
        """The next free pages, counts[b] for each sequence.  They stay free until the call that
        writes to them has been accepted (_taken): a refused call leaves the cache as it was."""
        total = sum(counts)
        if total > len(self.free):
            raise QuokaError(QUOKA_ERR_INVALID_ARG, f"{total} pages needed, {len(self.free)} free")
        last = iter(self.free[len(self.free) - total:][::-1])
        return [[next(last) for _ in range(n)] for n in counts]

    def _taken(self, pages: Sequence[Sequence[int]]) -> None:
        del self.free[len(self.free) - sum(map(len, pages)):]

    def _table(self, pages: Sequence[Sequence[int]]) -> torch.Tensor:
        rows = [list(p) + [-1] * (self.max_pages - len(p)) for p in pages]
        return torch.tensor(rows, dtype=torch.int32).to(self.block_table.device)

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, counts: Optional[Sequence[int]] = None) -> None:
        """Appends k_new / v_new [batch, h_kv, n, d], or the first counts[b] rows of each."""
        n = _dims(k_new, "k_new", 4)[2]
        add = [n] * len(self.lens) if counts is None else [int(c) for c in counts]
        if len(add) != len(self.lens) or any(c < 0 or c > n for c in add):
            raise QuokaError(QUOKA_ERR_INVALID_ARG, "counts needs one entry in [0, n] per sequence")
        more = [-(-(l + c) // self.page_size) - len(p) for l, c, p in zip(self.lens, add, self.pages)]
        if any(len(p) + m > self.max_pages for p, m in zip(self.pages, more)):
            raise QuokaError(QUOKA_ERR_INVALID_ARG, "a sequence would need more than max_pages pages")
        pages, table, new = self.pages, self.block_table, []
        if any(more):
            new = self._pick(more)
            pages = [p + m for p, m in zip(pages, new)]
            table = self._table(pages)
        cnt = None if counts is None else torch.tensor(add, dtype=torch.int32).to(self.seq_len.device)
        paged_append(k_new, v_new, self.k_pages, self.v_pages, table, self.seq_len, n_new=cnt,
                     weight_pages=self.weight_pages)
        seq_len = self.seq_len + (n if cnt is None else cnt)
        self._taken(new)
        self.pages, self.block_table, self.seq_len = pages, table, seq_len
        self.lens = [l + c for l, c in zip(self.lens, add)]

    def attend(self, q: torch.Tensor, window: Optional[int] = None, n_sink: int = 0) -> torch.Tensor:
        """One new token per sequence, q [batch, h_q, 1, d]; adds to the record if there is one."""
        return paged_decode_attn(q, self.k_pages, self.v_pages, self.block_table, self.seq_len,
                                 max(max(self.lens), 1), window=window, n_sink=n_sink,
                                 weight_pages=self.weight_pages)

    def evict(self, budget: Union[int, Sequence[int]], n_sink: int = 0, n_recent: int = 0) -> torch.Tensor:
        """Shrinks every sequence to its budget; returns the kept positions of each KV head.  The
        records that it goes by are what attend() has added since a row was appended.  The kept rows
        go to free pages where those suffice for all sequences, else (a cache that is full) each
        sequence's go through a copy of its pages back into the first of them."""
        if self.weight_pages is None:
            raise QuokaError(QUOKA_ERR_INVALID_ARG, "this cache keeps no weight record")
        want = [int(budget)] * len(self.lens) if isinstance(budget, int) else [int(b) for b in budget]
        if len(want) != len(self.lens) or any(b < 0 for b in want):
            raise QuokaError(QUOKA_ERR_INVALID_ARG, "budget needs one entry >= 0 per sequence")
        keep = [min(l, b) for l, b in zip(self.lens, want)]
        need = [-(-k // self.page_size) for k in keep]
        if sum(need) > len(self.free):
            return self._evict_in_turn(keep, need, n_sink, n_recent)
        pages = self._pick(need)
        table = self._table(pages)
        dev = table.device
        idx, new_len = paged_evict(self.k_pages, self.v_pages, self.weight_pages, self.block_table, self.seq_len,
                                   max(max(self.lens), 1), torch.tensor(keep, dtype=torch.int32).to(dev),
                                   max(max(keep), 1), table, n_sink=n_sink, n_recent=n_recent)
        self._taken(pages)
        for p in self.pages:
            self.free.extend(p)
        self.pages, self.block_table, self.seq_len, self.lens = pages, table, new_len, keep
        return idx

    def _evict_in_turn(self, keep: Sequence[int], need: Sequence[int], n_sink: int, n_recent: int) -> torch.Tensor:
        """evict() without free pages, one sequence at a time (a sequence that keeps all of its rows
        stays as it is).  The books follow each sequence, should a later copy find no memory."""
        # what paged_evict would refuse, before the first sequence changes
        if n_sink < 0 or n_recent < 0:
            raise QuokaError(QUOKA_ERR_INVALID_ARG, f"n_sink={n_sink} and n_recent={n_recent} must be >= 0")
        if max(self.lens) > QUOKA_MAX_EVICT_LEN:
            raise QuokaError(QUOKA_ERR_UNSUPPORTED, f"length {max(self.lens)} exceeds {QUOKA_MAX_EVICT_LEN}")
        pools, dev = (self.k_pages, self.v_pages, self.weight_pages), self.k_pages.device
        budget = torch.tensor(keep, dtype=torch.int32).to(dev)
        idx = torch.full((len(keep), pools[0].shape[1], max(max(keep), 1)), -1, dtype=torch.int32, device=dev)
        self.block_table, self.seq_len = self.block_table.clone(), self.seq_len.clone()
        self.pages, self.lens = list(self.pages), list(self.lens)
        for b, (k, m) in enumerate(zip(keep, need)):
            n, old = self.lens[b], self.pages[b]
            if k == n:
                idx[b, :, :n] = torch.arange(n, dtype=torch.int32, device=dev)
                continue
            if k > 0:
                at = torch.tensor(old).to(dev)
                copies = [torch.cat([p[at], p.new_zeros(m, *p.shape[1:])]) for p in pools]
                table = torch.arange(len(old) + m, dtype=torch.int32, device=dev)[None]
                idx[b, :, :k] = paged_evict(*copies, table[:, :len(old)], self.seq_len[b:b + 1], n, budget[b:b + 1], k,
                                            table[:, len(old):], n_sink=n_sink, n_recent=n_recent)[0]
                for p, c in zip(pools, copies):
                    p[at[:m]] = c[len(old):]
            self.block_table[b, m:] = -1
            self.seq_len[b:b + 1] = budget[b:b + 1]
            self.pages[b], self.lens[b] = old[:m], k
            self.free.extend(old[m:])
        return idx


def device_error(stream: Optional[torch.cuda.Stream] = None) -> int:
    code = ctypes.c_uint32(0)
    _check(lib().quoka_device_error(ctypes.byref(code), ctypes.c_void_p(_stream(stream))))
    return code.value


class SelCache:
    """A selected-value cache (quoka_selcache_update / sparse_chunk_attn_selcache) for one
    shape and b_max: the K/V blocks, the slot map (all -1 at first) and a workspace, all
    torch device memory owned by this object."""

    def __init__(self, shape: QuokaShape, b_max: int, device):
        self.shape, self.b_max = shape, int(b_max)
        n = int(lib().quoka_selcache_bytes(ctypes.byref(shape), self.b_max))
        w = int(lib().quoka_selcache_workspace_size(ctypes.byref(shape), self.b_max))
        if n == 0 or w == 0:
            raise QuokaError(QUOKA_ERR_INVALID_ARG, "bad shape or b_max for a selected-value cache")
        self.cache = torch.zeros(n, dtype=torch.uint8, device=device)
        self.slot_rows = torch.full((shape.batch, shape.h_kv, self.b_max), -1, dtype=torch.int32,
                                    device=device)
        self.misses = torch.zeros(shape.batch, shape.h_kv, dtype=torch.int32, device=device)
        self.workspace = torch.empty(w, dtype=torch.uint8, device=device)

    def blocks(self, dtype: torch.dtype):
        """(K, V) views [batch, h_kv, kc_rows, head_dim] of the cache."""
        s = self.shape
        half = self.cache.numel() // 2
        esz = torch.empty((), dtype=dtype).element_size()
        rows = (self.b_max + s.chunk + 127) // 128 * 128
        n = s.batch * s.h_kv * rows * s.head_dim * esz
        k = self.cache[:n].view(dtype).view(s.batch, s.h_kv, rows, s.head_dim)
        v = self.cache[half:half + n].view(dtype).view(s.batch, s.h_kv, rows, s.head_dim)
        return k, v

    def update(self, k_cache: torch.Tensor, v_cache: torch.Tensor, kv_off: Sequence[int],
               prefix_len: Sequence[int], budget: Sequence[int], idx: torch.Tensor,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Brings the cache to the selection idx; returns the misses per (sequence, KV head)."""
        if int(idx.shape[-1]) != self.b_max:
            raise QuokaError(QUOKA_ERR_INVALID_ARG, "idx's last dimension must be the cache's b_max")
        _check(lib().quoka_selcache_update(
            ctypes.byref(self.shape), _ptr(k_cache), _ptr(v_cache), _host_i64(kv_off),
            _host_i32(prefix_len), _host_i32(budget), _ptr(idx), self.b_max, _ptr(self.cache),
            _ptr(self.slot_rows), _ptr(self.misses), _ptr(self.workspace),
            self.workspace.numel(), ctypes.c_void_p(_stream(stream))))
        return self.misses

    def attend(self, q_chunk: torch.Tensor, prefix_len: Sequence[int], budget: Sequence[int],
               out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """sparse_chunk_attn over the cache's rows; returns out [batch, h_q, C, d]."""
        if out is None:
            out = torch.empty_like(q_chunk)
        _check(lib().sparse_chunk_attn_selcache(
            ctypes.byref(self.shape), _ptr(q_chunk), _host_i32(prefix_len), _host_i32(budget),
            _ptr(self.cache), self.b_max, _ptr(out), _ptr(self.workspace), self.workspace.numel(),
            ctypes.c_void_p(_stream(stream))))
        return out


class KernelTimer:
    """Per-kernel device times of the library calls made inside a ``with`` block.

    Enqueues a short spin kernel and a start event on the stream, hands the library a pool
    of timing events (one is recorded after every kernel it launches from this thread,
    quoka_profile_events), and afterwards yields (kernel name, milliseconds) pairs in
    launch order.  The spin keeps the GPU busy while the host enqueues the calls, so each
    gap between events is one kernel's device time.  Eager calls only: not inside a
    stream capture.
    """

    def __init__(self, max_kernels: int = 64, stream: Optional[torch.cuda.Stream] = None):
        self.stream = stream if stream is not None else torch.cuda.current_stream()
        self.start = torch.cuda.Event(enable_timing=True)
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(max_kernels)]
        for e in [self.start] + self.events:          # torch creates events on first record
            e.record(self.stream)
        self.stream.synchronize()
        self._handles = (ctypes.c_void_p * max_kernels)(*[e.cuda_event for e in self.events])
        self.times = []

    def __enter__(self):
        # a spin kernel ahead of the calls keeps the GPU busy while the host enqueues them,
        # so no host gap sits between the start event and the first kernel
        with torch.cuda.stream(self.stream):
            torch.cuda._sleep(4_000_000)
        self.start.record(self.stream)
        _check(lib().quoka_profile_events(self._handles, len(self.events)))
        return self

    def __exit__(self, *exc):
        n = int(lib().quoka_profile_marks(None, 0))
        names = (ctypes.c_char_p * max(n, 1))()
        lib().quoka_profile_marks(names, n)
        _check(lib().quoka_profile_events(None, 0))
        if exc[0] is None:
            self.stream.synchronize()
            prev = self.start
            for i in range(n):
                self.times.append((names[i].decode(), prev.elapsed_time(self.events[i])))
                prev = self.events[i]
        return False
