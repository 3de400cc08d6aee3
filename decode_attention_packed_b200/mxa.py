"""Python binding of libmxa.so (the C ABI in include/mxa.h).

Argument marshalling only: every step of the decode path runs in the CUDA
kernels of libmxa.so.  Torch tensors supply device memory and the current
stream.  There is no fallback: if the library is missing this module raises
on import.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_HERE, "libmxa.so")

if not os.path.exists(LIBRARY):
    raise ImportError(f"libmxa.so is not built ({LIBRARY}); run "
                      "`python -m decode_attention_packed_b200.build`")

_lib = ctypes.CDLL(LIBRARY)

MXA_OK, MXA_ERR_INVALID_ARG, MXA_ERR_UNSUPPORTED, MXA_ERR_WORKSPACE, MXA_ERR_CUDA, MXA_ERR_TIMEOUT = range(6)
MXA_F16, MXA_BF16 = 0, 1
MXA_SCHED_UNIFORM, MXA_SCHED_BALANCED = 0, 1

EXPORTED = ("mxa_status_string", "mxa_should_pack_gqa", "mxa_num_splits_heuristic", "mxa_plan",
            "mxa_plan_balanced",
            "mxa_decode_fwd", "mxa_decode_fwd_with_plan", "mxa_combine", "mxa_device_error",
            "mxa_decode_fwd_noalloc", "mxa_decode_fwd_append", "mxa_decode_fwd_varlen",
            "mxa_decode_fwd_f32out", "mxa_decode_workspace_size", "mxa_plan_window", "mxa_decode_fwd_window",
            "mxa_extend_tables", "mxa_cache_write", "mxa_prefill_fwd", "mxa_prefill_workspace_size")

SIZE_MAX = ctypes.c_size_t(-1).value


class mxa_decode_params_t(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("q_len", ctypes.c_int), ("Hq", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("D", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("max_pages_per_seq", ctypes.c_int),
                ("max_seqlen_k", ctypes.c_int), ("dtype", ctypes.c_int)]


class mxa_plan_t(ctypes.Structure):
    _fields_ = [("num_splits", ctypes.c_int), ("schedule", ctypes.c_int), ("grid", ctypes.c_int),
                ("units", ctypes.c_int), ("rows_per_tile", ctypes.c_int),
                ("block_tokens", ctypes.c_int), ("ctas_per_sm", ctypes.c_int),
                ("sm_count", ctypes.c_int), ("needs_combine", ctypes.c_int),
                ("unit_cost", ctypes.c_int), ("workspace_bytes", ctypes.c_size_t)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


_P = ctypes.c_void_p
_I = ctypes.c_int
_lib.mxa_status_string.argtypes = [_I]
_lib.mxa_status_string.restype = ctypes.c_char_p
_lib.mxa_should_pack_gqa.argtypes = [_I, _I, _I, _I]
_lib.mxa_should_pack_gqa.restype = _I
_lib.mxa_num_splits_heuristic.argtypes = [_I, _I, _I, _I, _I, _I, _I, ctypes.c_double]
_lib.mxa_num_splits_heuristic.restype = _I
_lib.mxa_plan.argtypes = [ctypes.POINTER(mxa_decode_params_t), _I, _I, ctypes.POINTER(mxa_plan_t)]
_lib.mxa_plan.restype = _I
_lib.mxa_plan_balanced.argtypes = [ctypes.POINTER(mxa_decode_params_t), _I, _I, ctypes.POINTER(mxa_plan_t)]
_lib.mxa_plan_balanced.restype = _I
_lib.mxa_decode_fwd.argtypes = [_P, _P, _P, _P, _P, ctypes.POINTER(mxa_decode_params_t),
                                ctypes.c_float, _I, _I, _P, ctypes.c_size_t, _P, _P, _P]
_lib.mxa_decode_fwd.restype = _I
_lib.mxa_decode_fwd_with_plan.argtypes = [_P, _P, _P, _P, _P, ctypes.POINTER(mxa_decode_params_t),
                                          ctypes.c_float, _I, ctypes.POINTER(mxa_plan_t), _P,
                                          ctypes.c_size_t, _P, _P, _P]
_lib.mxa_decode_fwd_with_plan.restype = _I
_lib.mxa_decode_fwd_f32out.argtypes = _lib.mxa_decode_fwd_with_plan.argtypes
_lib.mxa_decode_fwd_f32out.restype = _I
_lib.mxa_decode_workspace_size.argtypes = [ctypes.POINTER(mxa_decode_params_t), _I]
_lib.mxa_decode_workspace_size.restype = ctypes.c_size_t
_lib.mxa_decode_fwd_append.argtypes = [_P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(mxa_decode_params_t),
                                       ctypes.c_float, _I, ctypes.POINTER(mxa_plan_t), _P, ctypes.c_size_t,
                                       _P, _P, _P]
_lib.mxa_decode_fwd_append.restype = _I
_lib.mxa_decode_fwd_varlen.argtypes = [_P, _P, _I, _P, _P, _P, _P, ctypes.POINTER(mxa_decode_params_t),
                                       ctypes.c_float, _I, ctypes.POINTER(mxa_plan_t), _P, ctypes.c_size_t,
                                       _P, _P, _P]
_lib.mxa_decode_fwd_varlen.restype = _I
_lib.mxa_decode_fwd_noalloc.argtypes = [_P, _P, _P, _P, _P, ctypes.POINTER(mxa_decode_params_t),
                                        ctypes.c_float, _I, _I, _P, _P, _P]
_lib.mxa_decode_fwd_noalloc.restype = _I
_lib.mxa_plan_window.argtypes = [ctypes.POINTER(mxa_decode_params_t), _I, _I, _I, _I, ctypes.POINTER(mxa_plan_t)]
_lib.mxa_plan_window.restype = _I
_lib.mxa_decode_fwd_window.argtypes = [_P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(mxa_decode_params_t),
                                       ctypes.c_float, _I, _I, ctypes.POINTER(mxa_plan_t), _P, ctypes.c_size_t,
                                       _P, _P, _P]
_lib.mxa_decode_fwd_window.restype = _I
_lib.mxa_prefill_fwd.argtypes = [_P, _P, _I, _P, _P, _P, _P, ctypes.POINTER(mxa_decode_params_t), ctypes.c_float,
                                 _I, _I, _I, _P, ctypes.c_size_t, _P, _P, _P]
_lib.mxa_prefill_fwd.restype = _I
_lib.mxa_prefill_workspace_size.argtypes = [ctypes.POINTER(mxa_decode_params_t), _I]
_lib.mxa_prefill_workspace_size.restype = ctypes.c_size_t
_lib.mxa_extend_tables.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P]
_lib.mxa_extend_tables.restype = _I
_lib.mxa_cache_write.argtypes = [_P, _P, ctypes.c_longlong, ctypes.c_longlong, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P]
_lib.mxa_cache_write.restype = _I
_lib.mxa_combine.argtypes = [_P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P]
_lib.mxa_combine.restype = _I
_lib.mxa_device_error.argtypes = [_I]
_lib.mxa_device_error.restype = _I


class MxaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {mxa_status_string(code)}")


def _check(code: int, where: str) -> None:
    if code != MXA_OK:
        raise MxaError(code, where)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# The current stream's handle without a Stream object around it, and the
# current device without the look at torch's initialisation before it: they
# cost more host time than the rest of a short call's marshalling.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(stream, like: torch.Tensor, shape=None, dtype=None) -> torch.Tensor:
    """A tensor as `like`, or of another shape and type, for a call on `stream`
    (None: the current one).  The memory comes from the pool of the stream that
    writes it, so nothing queued on the current stream still uses it and nothing
    allocated there gets it while the call runs.  It is lent to the current
    stream, where the caller waits for the call and reads it."""
    if stream is None or (handle := _stream(stream)) == _stream(None):  # by the calls of least host time
        return torch.empty_like(like) if shape is None else like.new_empty(*shape, dtype=dtype)
    if not isinstance(stream, torch.cuda.Stream):  # handles 0 and 1 name the legacy default stream
        stream = torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        t = _empty(None, like, shape, dtype)
    t.record_stream(torch.cuda.current_stream())
    return t


# --------------------------------------------------------------------------
# the C calls, same names
# --------------------------------------------------------------------------

def mxa_status_string(code: int) -> str:
    return _lib.mxa_status_string(code).decode()


def mxa_should_pack_gqa(varlen_q: int, seqlen_q: int, qhead_per_khead: int, block_m: int) -> int:
    return _lib.mxa_should_pack_gqa(varlen_q, seqlen_q, qhead_per_khead, block_m)


def mxa_num_splits_heuristic(tiles, sm_count, slots, num_n_blocks, max_splits, causal,
                             num_m_blocks, kv_head_bytes) -> int:
    return _lib.mxa_num_splits_heuristic(tiles, sm_count, slots, num_n_blocks, max_splits,
                                         int(causal), num_m_blocks, float(kv_head_bytes))


def mxa_plan(params: mxa_decode_params_t, num_splits: int = 0, sm_count: int = 0) -> mxa_plan_t:
    plan = mxa_plan_t()
    _check(_lib.mxa_plan(ctypes.byref(params), num_splits, sm_count, ctypes.byref(plan)), "mxa_plan")
    return plan


def mxa_plan_balanced(params: mxa_decode_params_t, grid: int, sm_count: int = 0) -> mxa_plan_t:
    plan = mxa_plan_t()
    _check(_lib.mxa_plan_balanced(ctypes.byref(params), grid, sm_count, ctypes.byref(plan)),
           "mxa_plan_balanced")
    return plan


def mxa_decode_fwd(q, k_cache, v_cache, block_table, cache_seqlens, params, scale, causal,
                   num_splits, workspace, out, lse, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.mxa_decode_fwd(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                               _ptr(cache_seqlens), ctypes.byref(params), float(scale), int(causal),
                               int(num_splits), _ptr(workspace), ws_bytes, _ptr(out), _ptr(lse),
                               _stream(stream)), "mxa_decode_fwd")


def mxa_decode_fwd_with_plan(q, k_cache, v_cache, block_table, cache_seqlens, params, scale, causal,
                             plan, workspace, out, lse, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.mxa_decode_fwd_with_plan(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                         _ptr(cache_seqlens), ctypes.byref(params), float(scale),
                                         int(causal), ctypes.byref(plan), _ptr(workspace), ws_bytes,
                                         _ptr(out), _ptr(lse), _stream(stream)),
           "mxa_decode_fwd_with_plan")


def mxa_decode_fwd_f32out(q, k_cache, v_cache, block_table, cache_seqlens, params, scale, causal,
                          plan, workspace, out, lse, stream=None) -> None:
    """As mxa_decode_fwd_with_plan with a float32 `out`: O before its rounding
    to the input type."""
    if out.dtype != torch.float32:
        raise TypeError("mxa_decode_fwd_f32out writes a float32 out")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.mxa_decode_fwd_f32out(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                      _ptr(cache_seqlens), ctypes.byref(params), float(scale),
                                      int(causal), ctypes.byref(plan), _ptr(workspace), ws_bytes,
                                      _ptr(out), _ptr(lse), _stream(stream)),
           "mxa_decode_fwd_f32out")


def mxa_decode_workspace_size(params: mxa_decode_params_t, num_splits: int = 0) -> int:
    """Workspace bytes of mxa_plan(params, num_splits); SIZE_MAX when refused."""
    return int(_lib.mxa_decode_workspace_size(ctypes.byref(params), int(num_splits)))


def mxa_decode_fwd_append(q, k_cache, v_cache, k_new, v_new, block_table, cache_seqlens, params, scale,
                          causal, plan, workspace, out, lse, stream=None) -> None:
    """Write k_new / v_new [B, q_len, Hkv, D] at positions cache_seqlens[b] + t of
    the cache, then decode over cache_seqlens[b] + q_len keys (see mxa.h)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.mxa_decode_fwd_append(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new),
                                      _ptr(block_table), _ptr(cache_seqlens), ctypes.byref(params),
                                      float(scale), int(causal), ctypes.byref(plan), _ptr(workspace), ws_bytes,
                                      _ptr(out), _ptr(lse), _stream(stream)), "mxa_decode_fwd_append")


def mxa_decode_fwd_varlen(q, cu_seqlens_q, k_cache, v_cache, block_table, cache_seqlens, params, scale,
                          causal, plan, workspace, out, lse, stream=None) -> None:
    """Decode rows with their own query counts: q [total_q, Hq, D], row b's
    queries at cu_seqlens_q[b] .. cu_seqlens_q[b + 1] - 1; params.q_len bounds
    every count.  out [total_q, Hq, D], lse [Hq, total_q] (see mxa.h)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.mxa_decode_fwd_varlen(_ptr(q), _ptr(cu_seqlens_q), int(q.shape[0]), _ptr(k_cache),
                                      _ptr(v_cache), _ptr(block_table), _ptr(cache_seqlens), ctypes.byref(params),
                                      float(scale), int(causal), ctypes.byref(plan), _ptr(workspace), ws_bytes,
                                      _ptr(out), _ptr(lse), _stream(stream)), "mxa_decode_fwd_varlen")


def mxa_decode_fwd_noalloc(q, k_cache, v_cache, block_table, cache_seqlens, params, scale, causal,
                           num_splits, out, lse, stream=None) -> None:
    """Decode with the library's fixed 16 MiB scratch array instead of a
    workspace, for callers that cannot allocate device memory (see
    include/mxa.h: first call per device before any stream capture; calls
    that overlap on the GPU race on the shared array)."""
    _check(_lib.mxa_decode_fwd_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                       _ptr(cache_seqlens), ctypes.byref(params), float(scale),
                                       int(causal), int(num_splits), _ptr(out), _ptr(lse),
                                       _stream(stream)), "mxa_decode_fwd_noalloc")


def _keys(n) -> int:
    """A count of keys as the library takes it, in 32 bits: more than that is
    more than any row holds, and what is negative is refused."""
    n = int(n)
    return n if 0 <= n <= 0x7fffffff else 0x7fffffff if n > 0 else -1


def mxa_plan_window(params: mxa_decode_params_t, window: int, sinks: int = 0, num_splits: int = 0,
                    sm_count: int = 0) -> mxa_plan_t:
    plan = mxa_plan_t()
    _check(_lib.mxa_plan_window(ctypes.byref(params), _keys(window), _keys(sinks), num_splits, sm_count,
                                ctypes.byref(plan)), "mxa_plan_window")
    return plan


def mxa_decode_fwd_window(q, k_cache, v_cache, k_new, v_new, block_table, cache_seqlens, params, scale, window,
                          sinks, plan, workspace, out, lse, stream=None) -> None:
    """Causal decode in which the query at position p sees its last `window`
    keys and the first `sinks` keys; k_new / v_new as in
    mxa_decode_fwd_append, or None (see mxa.h)."""
    ws, ws_bytes = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    code = _lib.mxa_decode_fwd_window(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                      None if k_new is None else k_new.data_ptr(),
                                      None if v_new is None else v_new.data_ptr(),
                                      None if block_table is None else block_table.data_ptr(),
                                      cache_seqlens.data_ptr(), ctypes.byref(params), float(scale), _keys(window), _keys(sinks),
                                      ctypes.byref(plan), ws, ws_bytes, out.data_ptr(),
                                      None if lse is None else lse.data_ptr(), _stream(stream))
    if code != MXA_OK:
        raise MxaError(code, "mxa_decode_fwd_window")


def mxa_prefill_workspace_size(params: mxa_decode_params_t, total_q: int) -> int:
    """Workspace bytes of mxa_prefill_fwd; SIZE_MAX when refused."""
    return int(_lib.mxa_prefill_workspace_size(ctypes.byref(params), int(total_q)))


def mxa_prefill_fwd(q, cu_seqlens_q, k_cache, v_cache, block_table, cache_seqlens, params, scale, causal, window,
                    sinks, workspace, out, lse, stream=None) -> None:
    """Attention of packed chunks q [total_q, Hq, D] over the cache; params.q_len
    bounds every row's queries (see mxa.h)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.mxa_prefill_fwd(_ptr(q), _ptr(cu_seqlens_q), q.shape[0], _ptr(k_cache), _ptr(v_cache),
                                _ptr(block_table), _ptr(cache_seqlens), ctypes.byref(params), float(scale),
                                int(causal), _keys(window), _keys(sinks), _ptr(workspace), ws_bytes, _ptr(out),
                                _ptr(lse), _stream(stream)), "mxa_prefill_fwd")


def mxa_extend_tables(block_table, cache_seqlens, cu_seqlens_q, free_pages, page_size, num_pages, slots,
                      new_seqlens, pages_used, stream=None) -> None:
    """Pages from the front of free_pages for the step's new tokens, written
    into block_table [B, width], and every new token's cache slot (see mxa.h)."""
    B, width = block_table.shape
    _check(_lib.mxa_extend_tables(_ptr(block_table), _ptr(cache_seqlens), _ptr(cu_seqlens_q), _ptr(free_pages), B,
                                  slots.numel(), free_pages.numel(), int(page_size), int(num_pages), width,
                                  _ptr(slots), _ptr(new_seqlens), _ptr(pages_used), _stream(stream)),
           "mxa_extend_tables")


def mxa_cache_write(k_new, v_new, slots, k_cache, v_cache, stream=None) -> None:
    """k_cache / v_cache [num_pages, page_size, Hkv, D] at slots[t] become
    k_new / v_new [total, Hkv, D] (tokens may be strided; see mxa.h)."""
    total, Hkv, D = k_new.shape
    num_pages, page_size = k_cache.shape[:2]
    dtype = MXA_BF16 if k_cache.dtype == torch.bfloat16 else MXA_F16
    ks, vs = (k_new.stride(0), v_new.stride(0)) if total > 1 else (Hkv * D, Hkv * D)
    _check(_lib.mxa_cache_write(_ptr(k_new), _ptr(v_new), ks, vs, _ptr(slots), total, Hkv, D, num_pages, page_size,
                                dtype, _ptr(k_cache), _ptr(v_cache), _stream(stream)), "mxa_cache_write")


def mxa_combine(o_part, lse_part, out, lse=None, stream=None) -> None:
    """o_part [S, B, q_len, Hq, D] fp32, lse_part [S, B, Hq, q_len] fp32 -> out [B, q_len, Hq, D]."""
    S, B, q_len, Hq, D = o_part.shape
    dtype = MXA_BF16 if out.dtype == torch.bfloat16 else MXA_F16
    _check(_lib.mxa_combine(_ptr(o_part), _ptr(lse_part), S, B, q_len, Hq, D, dtype, _ptr(out),
                            _ptr(lse), _stream(stream)), "mxa_combine")


def mxa_device_error(reset: bool = False) -> int:
    return _lib.mxa_device_error(int(reset))


# --------------------------------------------------------------------------
# convenience: shapes from tensors
# --------------------------------------------------------------------------

def params_for(q: torch.Tensor, k_cache: torch.Tensor, block_table: Optional[torch.Tensor],
               max_seqlen_k: Optional[int] = None) -> mxa_decode_params_t:
    """Problem shape from the tensors.  Without `max_seqlen_k` the bound is
    the cache capacity of a row (no device read)."""
    B, q_len, Hq, D = q.shape
    num_pages, page_size, Hkv, Dk = k_cache.shape
    assert Dk == D
    if block_table is None:
        mpps = 1
        cap = page_size
    else:
        mpps = block_table.shape[1]
        cap = mpps * page_size
    if max_seqlen_k is None:
        max_seqlen_k = cap
    if q.dtype == torch.bfloat16:
        dt = MXA_BF16
    elif q.dtype == torch.float16:
        dt = MXA_F16
    else:
        raise TypeError("q must be float16 or bfloat16")
    return mxa_decode_params_t(B, q_len, Hq, Hkv, D, num_pages, page_size, mpps, int(max_seqlen_k), dt)


@dataclass
class Prepared:
    """A planned call with its workspace: the two-phase use of the library."""
    params: mxa_decode_params_t
    plan: mxa_plan_t
    workspace: Optional[torch.Tensor]


def _widened(params: mxa_decode_params_t, max_seqlen_q, max_seqlen_k) -> mxa_decode_params_t:
    """The prepared shape with this call's bounds (None: none stated) where
    they go further, up to what a row of the cache holds; the library then
    checks that plan and workspace still do."""
    q_len = params.q_len if max_seqlen_q is None else max(params.q_len, int(max_seqlen_q))
    k_len = params.max_seqlen_k
    if max_seqlen_k is not None and max_seqlen_k > k_len:
        k_len = max(k_len, min(int(max_seqlen_k), params.max_pages_per_seq * params.page_size))
    if q_len == params.q_len and k_len == params.max_seqlen_k:
        return params
    wide = mxa_decode_params_t.from_buffer_copy(params)
    wide.q_len, wide.max_seqlen_k = q_len, k_len
    return wide


def prepare(q, k_cache, block_table, *, max_seqlen_k=None, num_splits=0, plan=None,
            device=None, window=0, sinks=0, stream=None) -> Prepared:
    """The plan and the workspace of decode calls, for a serving loop to keep:
    calls on `stream` (None: the current one)."""
    params = params_for(q, k_cache, block_table, max_seqlen_k)
    if plan is None:
        plan = mxa_plan_window(params, window, sinks, num_splits) if window else mxa_plan(params, num_splits)
    ws = None
    if plan.workspace_bytes:
        ws = _empty(stream, q if device is None else torch.empty(0, device=device), (plan.workspace_bytes,), torch.uint8)
    return Prepared(params, plan, ws)


def decode(q, k_cache, v_cache, block_table, cache_seqlens, *, scale=None, causal=False,
           num_splits=0, max_seqlen_k=None, out=None, lse=None, prepared: Optional[Prepared] = None,
           return_lse=True, stream=None, k_new=None, v_new=None, out_dtype=None, window=0, sinks=0):
    """out [B, q_len, Hq, D] (and lse [B, Hq, q_len] fp32) for one decode step.

    With k_new / v_new [B, q_len, Hkv, D] the step first writes them into the
    cache at positions cache_seqlens[b] + t and attends to cache_seqlens[b] +
    q_len keys; max_seqlen_k must then bound those lengths.  out_dtype =
    torch.float32 returns O before its rounding to q's type
    (mxa_decode_fwd_f32out).

    window > 0 (causal only) leaves each query its last `window` keys and the
    first `sinks` keys of its row (mxa_decode_fwd_window); the blocks between
    them are not read.

    All tensors are dense; a windowed call checks them against its
    preparation, a call without a window passes them on as they are."""
    if window < 0 or sinks < 0 or (sinks and not window):
        raise ValueError("window >= 0, and sinks >= 0 go with a window")
    if window and not causal:
        raise ValueError("a sliding window is causal: pass causal=True")
    if prepared is None:
        prepared = prepare(q, k_cache, block_table, max_seqlen_k=max_seqlen_k, num_splits=num_splits,
                           window=window, sinks=sinks, stream=stream)
    params = prepared.params if max_seqlen_k is None else _widened(prepared.params, None, max_seqlen_k)
    if scale is None:
        scale = params.D ** -0.5
    f32 = out_dtype == torch.float32 or (out is not None and out.dtype == torch.float32)
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new go together")
    if window and not f32:
        _want_decode(params, q, k_cache, v_cache, block_table, cache_seqlens, prepared.workspace, out, lse, k_new, v_new)
    elif k_new is not None and not (k_new.is_contiguous() and v_new.is_contiguous()):
        raise ValueError("k_new and v_new must be contiguous (write_cache takes slices of a fused projection)")
    if out is None:
        out = _empty(stream, q, q.shape, torch.float32) if f32 else _empty(stream, q)
    if lse is None and return_lse:
        B, q_len, Hq, _ = q.shape
        lse = _empty(stream, q, (B, Hq, q_len), torch.float32)
    if f32:
        if window:
            raise ValueError("a float32 output is not offered with a window")
        if k_new is not None:
            raise ValueError("a float32 output is not offered with k_new / v_new")
        mxa_decode_fwd_f32out(q, k_cache, v_cache, block_table, cache_seqlens, params, scale, causal,
                              prepared.plan, prepared.workspace, out, lse, stream)
    elif window:
        mxa_decode_fwd_window(q, k_cache, v_cache, k_new, v_new, block_table, cache_seqlens, params, scale,
                              window, sinks, prepared.plan, prepared.workspace, out, lse, stream)
    elif k_new is None:
        mxa_decode_fwd_with_plan(q, k_cache, v_cache, block_table, cache_seqlens, params, scale,
                                 causal, prepared.plan, prepared.workspace, out, lse, stream)
    else:
        mxa_decode_fwd_append(q, k_cache, v_cache, k_new, v_new, block_table, cache_seqlens, params,
                              scale, causal, prepared.plan, prepared.workspace, out, lse, stream)
    return out, lse


def decode_varlen(q, cu_seqlens_q, k_cache, v_cache, block_table, cache_seqlens, *, max_seqlen_q,
                  scale=None, causal=False, num_splits=0, max_seqlen_k=None, out=None, lse=None,
                  prepared: Optional[Prepared] = None, return_lse=True, stream=None):
    """out [total_q, Hq, D] (and lse [Hq, total_q] fp32) for rows with their
    own query counts: q [total_q, Hq, D], cu_seqlens_q [B + 1] int32 on the
    device, max_seqlen_q >= every row's count (it sizes the plan)."""
    total_q, Hq, D = q.shape
    B = cu_seqlens_q.shape[0] - 1
    if scale is None:
        scale = D ** -0.5
    if prepared is None:
        # planned as B rows of max_seqlen_q queries (a shape-only tensor)
        shape = torch.empty((B, int(max_seqlen_q), Hq, D), dtype=q.dtype, device="meta")
        params = params_for(shape, k_cache, block_table, max_seqlen_k)
        plan = mxa_plan(params, num_splits)
        ws = None
        if plan.workspace_bytes:
            ws = _empty(stream, q, (plan.workspace_bytes,), torch.uint8)
        prepared = Prepared(params, plan, ws)
    params = _widened(prepared.params, max_seqlen_q, max_seqlen_k)
    if out is None:
        out = _empty(stream, q)
    if lse is None and return_lse:
        lse = _empty(stream, q, (Hq, total_q), torch.float32)
    mxa_decode_fwd_varlen(q, cu_seqlens_q, k_cache, v_cache, block_table, cache_seqlens, params,
                          scale, causal, prepared.plan, prepared.workspace, out, lse, stream)
    return out, lse


# --------------------------------------------------------------------------
# chunks of new tokens, and the cache's bookkeeping
# --------------------------------------------------------------------------

def prepare_prefill(q, cu_seqlens_q, k_cache, block_table, *, max_seqlen_q, max_seqlen_k=None,
                    stream=None) -> Prepared:
    """The workspace of prefill calls with up to q.shape[0] packed tokens, for
    a serving loop to keep: calls on `stream` (None: the current one)."""
    total_q, Hq, D = q.shape
    B = cu_seqlens_q.shape[0] - 1
    shape = torch.empty((B, 1, Hq, D), dtype=q.dtype, device="meta")
    params = params_for(shape, k_cache, block_table, max_seqlen_k)
    params.q_len = int(max_seqlen_q) or 1  # 0: no row has a token
    size = mxa_prefill_workspace_size(params, total_q)
    if size == SIZE_MAX:  # the run call names the reason
        size = 0
    return Prepared(params, None, _empty(stream, q, (size,), torch.uint8))


def prefill(q, cu_seqlens_q, k_cache, v_cache, block_table, cache_seqlens, *, max_seqlen_q, scale=None, causal=True,
            window=0, sinks=0, max_seqlen_k=None, out=None, lse=None, prepared: Optional[Prepared] = None,
            return_lse=True, stream=None):
    """out [total_q, Hq, D] (and lse [Hq, total_q] fp32) for chunks of new
    tokens over the cache, which holds their keys and values already:
    q [total_q, Hq, D], row b's tokens at cu_seqlens_q[b] .. cu_seqlens_q[b + 1]
    - 1, its last ones among cache_seqlens[b] keys; max_seqlen_q >= every
    row's count.  Rows of one token and of thousands may be mixed, and
    tokens behind the last row are padding that is not written.

    causal: a token sees the keys up to its own position.  window > 0 (causal
    only) leaves it its last `window` keys and the first `sinks` keys."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    if prepared is None:
        prepared = prepare_prefill(q, cu_seqlens_q, k_cache, block_table, max_seqlen_q=max_seqlen_q,
                                   max_seqlen_k=max_seqlen_k, stream=stream)
    p, dev, dtype = _widened(prepared.params, max_seqlen_q, max_seqlen_k), _current_device(), q.dtype
    B = p.B
    _want_type(q, p)
    _want(dev, prepared.workspace, "the prepared workspace", torch.uint8)
    _want(dev, q, "q", dtype, (q.shape[0], p.Hq, p.D))
    _want(dev, cu_seqlens_q, "cu_seqlens_q", torch.int32, (B + 1,))
    _want(dev, k_cache, "k_cache", dtype, (p.num_pages, p.page_size, p.Hkv, p.D))
    _want(dev, v_cache, "v_cache", dtype, k_cache.shape)
    _want(dev, cache_seqlens, "cache_seqlens", torch.int32, (B,))
    if block_table is not None:
        _want(dev, block_table, "block_table", torch.int32, (B, p.max_pages_per_seq))
    if out is None:
        out = _empty(stream, q)
    else:
        _want(dev, out, "out", dtype, q.shape)
    if lse is None and return_lse:
        lse = _empty(stream, q, (q.shape[1], q.shape[0]), torch.float32)
    elif lse is not None:
        _want(dev, lse, "lse", torch.float32, (q.shape[1], q.shape[0]))
    mxa_prefill_fwd(q, cu_seqlens_q, k_cache, v_cache, block_table, cache_seqlens, p, scale, causal,
                    window, sinks, prepared.workspace, out, lse, stream)
    return out, lse


def _want_decode(p: mxa_decode_params_t, q, k_cache, v_cache, block_table, cache_seqlens, workspace, out, lse, k_new,
                 v_new) -> None:
    dev, dtype, B, q_len, Hq = _current_device(), q.dtype, p.B, p.q_len, p.Hq
    cache = (p.num_pages, p.page_size, p.Hkv, p.D)
    # All that a call always has in one condition: a short call is bound by the
    # host, which takes half as long for it as for the tests by name.
    if not (dtype is k_cache.dtype is v_cache.dtype is (torch.bfloat16 if p.dtype == MXA_BF16 else torch.float16)
            and cache_seqlens.dtype is torch.int32
            and q.get_device() == k_cache.get_device() == v_cache.get_device() == cache_seqlens.get_device() == dev
            and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous() and cache_seqlens.is_contiguous()
            and q.shape == (B, q_len, Hq, p.D) and k_cache.shape == cache and v_cache.shape == cache
            and cache_seqlens.shape == (B,)
            and (block_table is None or block_table.dtype is torch.int32 and block_table.get_device() == dev
                 and block_table.is_contiguous() and block_table.shape == (B, p.max_pages_per_seq))
            and (workspace is None or workspace.get_device() == dev)):
        _want_type(q, p)
        _want(dev, q, "q", dtype, (B, q_len, Hq, p.D))
        _want(dev, k_cache, "k_cache", dtype, cache)
        _want(dev, v_cache, "v_cache", dtype, cache)
        _want(dev, cache_seqlens, "cache_seqlens", torch.int32, (B,))
        if block_table is not None:
            _want(dev, block_table, "block_table", torch.int32, (B, p.max_pages_per_seq))
        if workspace is not None:
            _want(dev, workspace, "the prepared workspace", workspace.dtype)
    if out is not None:
        _want(dev, out, "out", dtype, q.shape)
    if lse is not None:
        _want(dev, lse, "lse", torch.float32, (B, Hq, q_len))
    if k_new is not None:
        _want(dev, k_new, "k_new", dtype, (B, q_len, p.Hkv, p.D))
        _want(dev, v_new, "v_new", dtype, k_new.shape)


def _want_type(q: torch.Tensor, p: mxa_decode_params_t) -> None:
    if q.dtype is not (torch.bfloat16 if p.dtype == MXA_BF16 else torch.float16):
        raise TypeError("q must have the type that the call was prepared for")


def _want(device: int, t: torch.Tensor, name: str, dtype, shape=None) -> None:
    """A dense tensor of `dtype` (and `shape`) on CUDA device `device`, the
    current one, or an error that names it."""
    if t.dtype is dtype and t.get_device() == device and t.is_contiguous() and (shape is None or t.shape == shape):
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != device:  # -1 for a tensor on the host
        raise ValueError(f"{name} must be on the current CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, not {tuple(t.shape)}")


def extend_tables(block_table, cache_seqlens, cu_seqlens_q, free_pages, *, page_size, num_pages, total_q,
                  slots=None, new_seqlens=None, pages_used=None, stream=None):
    """Pages and cache slots for a step's new tokens: row b holds
    cache_seqlens[b] keys and receives cu_seqlens_q[b + 1] - cu_seqlens_q[b]
    tokens, total_q in all.  The pages it needs besides those it holds are
    taken from the front of free_pages, in row order, and written into
    block_table [B, width] (all int32, on the device).

    Returns (slots [total_q], new_seqlens [B], pages_used [1]), int32.  Tokens
    behind the last row are padding with slot -1.  A row whose pages do not fit
    its table or the free list takes none: its slots are -1 and its length is
    unchanged."""
    dev, int32 = _current_device(), torch.int32
    _want(dev, block_table, "block_table", int32)
    B = block_table.shape[0]
    _want(dev, cache_seqlens, "cache_seqlens", int32, (B,))
    _want(dev, cu_seqlens_q, "cu_seqlens_q", int32, (B + 1,))
    _want(dev, free_pages, "free_pages", int32)
    if slots is None:
        slots = _empty(stream, block_table, (total_q,), int32)
    else:
        _want(dev, slots, "slots", int32, (total_q,))
    if new_seqlens is None:
        new_seqlens = _empty(stream, cache_seqlens)
    else:
        _want(dev, new_seqlens, "new_seqlens", int32, (B,))
    if pages_used is None:
        pages_used = _empty(stream, block_table, (1,), int32)
    else:
        _want(dev, pages_used, "pages_used", int32, (1,))
    if B and new_seqlens.data_ptr() == cache_seqlens.data_ptr():
        raise ValueError("new_seqlens must be another buffer than cache_seqlens")
    mxa_extend_tables(block_table, cache_seqlens, cu_seqlens_q, free_pages, page_size, num_pages, slots,
                      new_seqlens, pages_used, stream)
    return slots, new_seqlens, pages_used


def write_cache(k_new, v_new, k_cache, v_cache, slots, *, stream=None) -> None:
    """Copy k_new / v_new [total, Hkv, D] into the cache slots of
    extend_tables.  The tokens may be strided (slices of one fused
    projection); a token with slot -1 is left out; slots are distinct."""
    dev, dtype = _current_device(), k_cache.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError("the cache must be float16 or bfloat16")
    _want(dev, k_cache, "k_cache", dtype)
    _want(dev, v_cache, "v_cache", dtype, k_cache.shape)
    total, Hkv, D = k_new.shape
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        if t.dtype is not dtype:
            raise TypeError(f"{name} must have the cache's type")
        if t.get_device() != dev:
            raise ValueError(f"{name} must be on the current CUDA device")
        if t.shape != (total,) + k_cache.shape[2:]:
            raise ValueError(f"{name} must be [total, Hkv, D] with the cache's heads")
        if total and (t.stride(2) != 1 or (Hkv > 1 and t.stride(1) != D)):
            raise ValueError(f"a token of {name} must be contiguous")
    _want(dev, slots, "slots", torch.int32, (total,))
    mxa_cache_write(k_new, v_new, slots, k_cache, v_cache, stream)
