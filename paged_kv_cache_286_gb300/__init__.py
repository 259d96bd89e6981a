"""Paged-KV attention step for GB300: a thin PyTorch binding of libpagedattn.so.

The binding only marshals arguments: it checks devices, dtypes and contiguity of torch tensors
and passes their device pointers and the current CUDA stream to the C ABI (include/pa.h).  Every
step of the computation runs in the library's CUDA kernels; if the library is missing the calls
raise, there is no CPU fallback.

    import paged_kv_cache_286_gb300 as pa
    ws = pa.new_workspace(pa.attention_workspace_size(..., k_cache=k_cache), device="cuda")
    pa.cache_append(k, v, slot_mapping, k_cache, v_cache, ws)
    out = pa.attention(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, ws,
                       scale=..., max_context_len=..., max_query_len=...)

Smaller caches: pools of 4-bit floating point (``new_mxfp4_cache``, taken by every call), and
eviction of the keys that received the least attention:

    out = pa.attention_key_weights(q, k_cache, v_cache, block_tables, context_lens,
                                   query_start_loc, key_weights, ws, scale=..., ...)
    kept, context_lens = pa.evict_keys(k_cache, v_cache, block_tables, context_lens, keep_lens,
                                       key_weights, ws, recent=..., ...)
"""

from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import (PA_BF16, PA_FP8_E4M3, PA_FP32, PA_MXFP4,  # noqa: F401
                   PA_WORKSPACE_HEADER_BYTES, PagedAttnError)

__all__ = ["cache_append", "cache_read", "new_mxfp4_cache", "attention",
           "attention_key_weights", "attention_key_weights_workspace_size", "evict_keys",
           "evict_workspace_size", "attention_workspace_size", "new_workspace",
           "check_error", "library", "version", "PagedAttnError", "set_kernel_timing_events",
           "set_prefill_timing_events", "set_kernel_span_buffer"]


def library() -> ctypes.CDLL:
    return _lib.load()


def version() -> str:
    return _lib.load().pa_version().decode()


def _ptr(t: Optional[torch.Tensor]) -> int:
    return t.data_ptr() if t is not None else 0


def _stream(stream) -> int:
    """The stream's handle (None: the current device's current stream)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _need(t: torch.Tensor, name: str, dtypes, ndim: int):
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.dim() == ndim and \
            t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_FP8_DTYPES = (torch.uint8, torch.float8_e4m3fn)


def new_mxfp4_cache(num_blocks: int, num_kv_heads: int, head_dim: int, device="cuda"
                    ) -> torch.Tensor:
    """A zeroed MXFP4 pool for the keys or the values: uint8 [num_blocks, num_kv_heads, 17 *
    head_dim / 2], one tile of 16 rows of codes and their scale bytes per block and kv head."""
    if head_dim not in (64, 128):
        raise ValueError("MXFP4 pools are built for head_dim 64 and 128")
    return torch.zeros((num_blocks, num_kv_heads, head_dim * 17 // 2), dtype=torch.uint8,
                       device=device)


def _need_caches(k_cache: torch.Tensor, v_cache: torch.Tensor) -> None:
    """k_cache / v_cache: [NB, Hkv, 16, D] bf16 or E4M3, or [NB, Hkv, 17 D / 2] uint8 (MXFP4)."""
    mx = isinstance(k_cache, torch.Tensor) and k_cache.dim() == 3
    _need(k_cache, "k_cache", (torch.uint8,) if mx else (torch.bfloat16,) + _FP8_DTYPES,
          3 if mx else 4)
    _need(v_cache, "v_cache", (k_cache.dtype,), k_cache.dim())


def _same_shape(k_cache: torch.Tensor, v_cache: torch.Tensor) -> None:
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")


def cache_desc(k_cache: torch.Tensor, k_scale: float = 1.0, v_scale: float = 1.0):
    if k_cache.dim() == 3:
        nb, hkv, tile = k_cache.shape
        if tile % 17:
            raise ValueError("an MXFP4 pool has tiles of 17 * head_dim / 2 bytes")
        return _lib.CacheDesc(nb, 16, hkv, tile * 2 // 17, PA_MXFP4, 1.0, 1.0)
    nb, hkv, bs, d = k_cache.shape
    dt = PA_FP8_E4M3 if k_cache.dtype in _FP8_DTYPES else PA_BF16
    return _lib.CacheDesc(nb, bs, hkv, d, dt, float(k_scale), float(v_scale))


def new_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A workspace tensor with its error word cleared."""
    ws = torch.empty(max(int(nbytes), PA_WORKSPACE_HEADER_BYTES), dtype=torch.uint8,
                     device=device)
    ws[:PA_WORKSPACE_HEADER_BYTES].zero_()
    return ws


_HERE = contextlib.nullcontext()


def _on(stream, *tensors):
    """Checks that the tensors (None: absent) share one device and returns a context in which the
    call's allocations and its launch are on that device and on `stream` (None: the device's
    current stream)."""
    try:
        dev = tensors[0].get_device()
        for t in tensors:
            if t is not None and t.get_device() != dev:
                raise ValueError(
                    f"tensors on different devices: {t.device} and {tensors[0].device}")
    except AttributeError:
        raise TypeError("the call takes torch.Tensors") from None
    if stream is None:
        return _HERE if torch._C._cuda_getDevice() == dev else torch.cuda.device(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream of {stream.device} for tensors on {tensors[0].device}")
    return torch.cuda.stream(stream)


def cache_append(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                 k_cache: torch.Tensor, v_cache: torch.Tensor, workspace: torch.Tensor, *,
                 k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> None:
    """Write k/v [T, Hkv, D] (bf16) into the pools through slot_mapping [T] (int64)."""
    _need(k, "k", (torch.bfloat16,), 3)
    _need(v, "v", (torch.bfloat16,), 3)
    _need(slot_mapping, "slot_mapping", (torch.int64,), 1)
    _need_caches(k_cache, v_cache)
    _same_shape(k_cache, v_cache)
    desc = cache_desc(k_cache, k_scale, v_scale)
    if k.shape != v.shape or k.shape[0] != slot_mapping.shape[0] or \
            k.shape[1:] != (desc.num_kv_heads, desc.head_dim):
        raise ValueError("k/v/slot_mapping shapes do not match the cache")
    with _on(stream, k, v, slot_mapping, k_cache, v_cache, workspace):
        _lib.check(_lib.load().pa_cache_append(
            _ptr(k), _ptr(v), _ptr(slot_mapping), k.shape[0], _ptr(k_cache), _ptr(v_cache),
            ctypes.byref(desc), _ptr(workspace), _stream(stream)))


def attention_workspace_size(num_seqs: int, num_q_tokens: int, num_q_heads: int,
                             num_kv_heads: int, head_dim: int, max_context_len: int,
                             max_query_len: int, block_size: int = 16,
                             k_cache: Optional[torch.Tensor] = None) -> int:
    """Workspace bytes of a step of this shape over the pool `k_cache`.  Without one: enough for a
    pool of any type, which with runs of more than 32 (token x q head) rows is up to 256 MiB more
    than bf16 and E4M3 pools use."""
    return int(_lib.load().pa_attention_workspace_size_for(
        PA_MXFP4 if k_cache is None else cache_desc(k_cache).cache_dtype, num_seqs, num_q_tokens,
        num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, max_query_len))


def attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              block_tables: torch.Tensor, context_lens: torch.Tensor,
              query_start_loc: torch.Tensor, workspace: torch.Tensor, *, scale: float,
              max_context_len: int, max_query_len: int, out: Optional[torch.Tensor] = None,
              out_dtype: torch.dtype = torch.float32, k_scale: float = 1.0,
              v_scale: float = 1.0, stream=None) -> torch.Tensor:
    """Ragged paged attention: q [T, Hq, D] bf16 -> out [T, Hq, D] (fp32 or bf16)."""
    _need(q, "q", (torch.bfloat16,), 3)
    with _on(stream, q, k_cache, v_cache, block_tables, context_lens, query_start_loc, workspace, out):
        out, args = _step_args(q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                               workspace, scale, max_context_len, max_query_len, out, out_dtype,
                               k_scale, v_scale)
        _lib.check(_lib.load().pa_attention(*args, _ptr(workspace), workspace.numel(),
                                            _stream(stream)))
    return out


def _step_args(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, workspace, scale,
               max_context_len, max_query_len, out, out_dtype, k_scale, v_scale):
    """Checks one step's tensors; returns its output and the C arguments up to out_dtype."""
    _need_caches(k_cache, v_cache)
    _same_shape(k_cache, v_cache)
    _need(block_tables, "block_tables", (torch.int32,), 2)
    _need(context_lens, "context_lens", (torch.int32,), 1)
    _need(query_start_loc, "query_start_loc", (torch.int32,), 1)
    _need(workspace, "workspace", (torch.uint8,), 1)
    T, Hq, D = q.shape
    S = context_lens.size(0)
    Hkv = k_cache.size(1)
    if query_start_loc.size(0) != S + 1 or block_tables.size(0) != S:
        raise ValueError("query_start_loc must have num_seqs + 1 entries and block_tables "
                         "num_seqs rows")
    if out is None:
        out = torch.empty((T, Hq, D), dtype=out_dtype, device=q.device)
    else:
        _need(out, "out", (torch.float32, torch.bfloat16), 3)
        if tuple(out.shape) != (T, Hq, D):
            raise ValueError("out has the wrong shape")
    odt = PA_FP32 if out.dtype == torch.float32 else PA_BF16
    desc = cache_desc(k_cache, k_scale, v_scale)
    return out, (
        _ptr(q), T, _ptr(k_cache), _ptr(v_cache), ctypes.byref(desc), _ptr(block_tables),
        block_tables.size(1), _ptr(context_lens), _ptr(query_start_loc), S,
        int(max_context_len), int(max_query_len), Hq, Hkv, D, float(scale), _ptr(out), odt)


def _need_weights(key_weights, num_kv_heads, num_seqs, **rows):
    _need(key_weights, "key_weights", (torch.float32,), 3)
    if key_weights.size(1) != num_kv_heads:
        raise ValueError("key_weights must be [rows, num_kv_heads, max_keys]")
    for name, r in rows.items():
        if r is not None:
            _need(r, name, (torch.int32,), 1)
            if r.size(0) != num_seqs:
                raise ValueError(f"{name} must have num_seqs entries")


def attention_key_weights_workspace_size(num_seqs: int, num_q_tokens: int, num_q_heads: int,
                                         num_kv_heads: int, head_dim: int, max_context_len: int,
                                         max_query_len: int, block_size: int = 16,
                                         k_cache: Optional[torch.Tensor] = None) -> int:
    """The same for attention_key_weights."""
    return int(_lib.load().pa_attention_key_weights_workspace_size_for(
        PA_MXFP4 if k_cache is None else cache_desc(k_cache).cache_dtype, num_seqs, num_q_tokens,
        num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, max_query_len))


def attention_key_weights(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          block_tables: torch.Tensor, context_lens: torch.Tensor,
                          query_start_loc: torch.Tensor, key_weights: torch.Tensor,
                          workspace: torch.Tensor, *, scale: float, max_context_len: int,
                          max_query_len: int, weight_rows: Optional[torch.Tensor] = None,
                          decay: float = 1.0, out: Optional[torch.Tensor] = None,
                          out_dtype: torch.dtype = torch.float32, k_scale: float = 1.0,
                          v_scale: float = 1.0, stream=None) -> torch.Tensor:
    """`attention`, and key_weights [rows, Hkv, max_keys] (fp32) is updated in place: decayed,
    plus the softmax weights each cached key received from the step's queries and the q heads of
    its group.  weight_rows [num_seqs] (int32): the row of each sequence (None: row s)."""
    _need(q, "q", (torch.bfloat16,), 3)
    _need_caches(k_cache, v_cache)
    _need(context_lens, "context_lens", (torch.int32,), 1)
    _need_weights(key_weights, k_cache.size(1), context_lens.size(0), weight_rows=weight_rows)
    with _on(stream, q, k_cache, v_cache, block_tables, context_lens, query_start_loc, key_weights,
             workspace, weight_rows, out):
        out, args = _step_args(q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                               workspace, scale, max_context_len, max_query_len, out, out_dtype,
                               k_scale, v_scale)
        _lib.check(_lib.load().pa_attention_key_weights(
            *args, _ptr(key_weights), _ptr(weight_rows), key_weights.size(0),
            key_weights.size(2), float(decay), _ptr(workspace), workspace.numel(),
            _stream(stream)))
    return out


def evict_workspace_size(num_seqs: int, num_kv_heads: int, max_context_len: int,
                         max_keep_len: int) -> int:
    return int(_lib.load().pa_evict_workspace_size(num_seqs, num_kv_heads, max_context_len,
                                                   max_keep_len))


def evict_keys(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
               context_lens: torch.Tensor, keep_lens: torch.Tensor, key_weights: torch.Tensor,
               workspace: torch.Tensor, *, max_context_len: int, max_keep_len: int, recent: int,
               dst_tables: Optional[torch.Tensor] = None,
               weight_rows: Optional[torch.Tensor] = None,
               dst_weight_rows: Optional[torch.Tensor] = None,
               kept: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
               stream=None):
    """Keep keep_lens[s] keys of each sequence, per kv head: the last `recent` and those of the
    largest key_weights; they move to the front of dst_tables' blocks (None: in place), their
    weights with them.  Returns (kept [S, Hkv, max_keep_len] old positions, -1 past the kept ones;
    new_lens [S])."""
    _need_caches(k_cache, v_cache)
    _same_shape(k_cache, v_cache)
    _need(block_tables, "block_tables", (torch.int32,), 2)
    _need(context_lens, "context_lens", (torch.int32,), 1)
    _need(keep_lens, "keep_lens", (torch.int32,), 1)
    _need(workspace, "workspace", (torch.uint8,), 1)
    S, H = context_lens.size(0), k_cache.size(1)
    _need_weights(key_weights, H, S, weight_rows=weight_rows, dst_weight_rows=dst_weight_rows)
    if block_tables.size(0) != S or keep_lens.size(0) != S:
        raise ValueError("block_tables and keep_lens must have num_seqs rows")
    if dst_tables is not None:
        _need(dst_tables, "dst_tables", (torch.int32,), 2)
        if dst_tables.shape != block_tables.shape:
            raise ValueError("dst_tables must have block_tables' shape")
    if max_keep_len < 0:
        raise ValueError("max_keep_len must not be negative")
    with _on(stream, k_cache, v_cache, block_tables, context_lens, keep_lens, key_weights,
             workspace, dst_tables, weight_rows, dst_weight_rows, kept, new_lens):
        if kept is None:
            kept = torch.empty((S, H, max_keep_len), dtype=torch.int32, device=k_cache.device)
        else:
            _need(kept, "kept", (torch.int32,), 3)
            if tuple(kept.shape) != (S, H, max_keep_len):
                raise ValueError("kept has the wrong shape")
        if new_lens is None:
            new_lens = torch.empty((S,), dtype=torch.int32, device=k_cache.device)
        else:
            _need(new_lens, "new_lens", (torch.int32,), 1)
            if new_lens.shape[0] != S:
                raise ValueError("new_lens has the wrong shape")
        desc = cache_desc(k_cache)
        _lib.check(_lib.load().pa_evict_keys(
            _ptr(k_cache), _ptr(v_cache), ctypes.byref(desc), _ptr(block_tables),
            _ptr(dst_tables), block_tables.size(1), _ptr(context_lens), _ptr(keep_lens), S,
            int(max_context_len), int(max_keep_len), int(recent), _ptr(key_weights),
            _ptr(weight_rows), _ptr(dst_weight_rows), key_weights.size(0), key_weights.size(2),
            _ptr(kept), _ptr(new_lens), _ptr(workspace), workspace.numel(), _stream(stream)))
    return kept, new_lens


def cache_read(slot_mapping: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
               workspace: torch.Tensor, *, out_dtype: torch.dtype = torch.bfloat16,
               k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """The keys and values that the pools hold in slot_mapping [T] (int64): two tensors
    [T, Hkv, D] (bf16 or fp32); zeros for negative slots."""
    _need(slot_mapping, "slot_mapping", (torch.int64,), 1)
    _need_caches(k_cache, v_cache)
    _same_shape(k_cache, v_cache)
    _need(workspace, "workspace", (torch.uint8,), 1)
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out_dtype must be float32 or bfloat16")
    desc = cache_desc(k_cache, k_scale, v_scale)
    with _on(stream, slot_mapping, k_cache, v_cache, workspace):
        k = torch.empty((slot_mapping.shape[0], desc.num_kv_heads, desc.head_dim),
                        dtype=out_dtype, device=k_cache.device)
        v = torch.empty_like(k)
        _lib.check(_lib.load().pa_cache_read(
            _ptr(slot_mapping), slot_mapping.shape[0], _ptr(k_cache), _ptr(v_cache),
            ctypes.byref(desc), _ptr(k), _ptr(v),
            PA_FP32 if out_dtype == torch.float32 else PA_BF16, _ptr(workspace), _stream(stream)))
    return k, v


def check_error(workspace: torch.Tensor, stream=None, raise_on_error: bool = True) -> int:
    """Synchronise, read and clear the device error word; returns its PA_DEVERR_* bits."""
    word = ctypes.c_uint32(0)
    with _on(stream, workspace):
        st = _lib.load().pa_check_error(_ptr(workspace), _stream(stream), ctypes.byref(word))
    if raise_on_error and st != _lib.PA_OK:
        raise _lib.PagedAttnError(st, _lib.load().pa_last_error_string().decode())
    return int(word.value)


def set_kernel_timing_events(before: Optional[torch.cuda.Event],
                             after: Optional[torch.cuda.Event]) -> None:
    """Have later attention calls of this thread record `before`/`after` around their main
    kernel (benchmark hook); pass None to stop."""
    b = ctypes.c_void_p(before.cuda_event) if before is not None else ctypes.c_void_p(0)
    a = ctypes.c_void_p(after.cuda_event) if after is not None else ctypes.c_void_p(0)
    _lib.load().pa_set_kernel_timing_events(b, a)


def set_kernel_span_buffer(buf: Optional[torch.Tensor]) -> None:
    """Have later attention calls of this thread record the global-timer span (ns) of their
    split-KV kernel into buf[0:2] and of their prefill-tile kernel into buf[2:4] (int64 CUDA
    tensor preset to [-1, 0, -1, 0], read as unsigned); None stops (benchmark hook)."""
    if buf is not None:
        _need(buf, "span buffer", (torch.int64,), 1)
        if buf.numel() < 4:
            raise ValueError("the span buffer needs four entries")
    _lib.load().pa_set_kernel_span_buffer(_ptr(buf))


def set_prefill_timing_events(before: Optional[torch.cuda.Event],
                              after: Optional[torch.cuda.Event]) -> None:
    """Have later attention calls of this thread record `before`/`after` around their
    tensor-core prefill-tile kernel, when they launch one (benchmark hook); None stops."""
    b = ctypes.c_void_p(before.cuda_event) if before is not None else ctypes.c_void_p(0)
    a = ctypes.c_void_p(after.cuda_event) if after is not None else ctypes.c_void_p(0)
    _lib.load().pa_set_prefill_timing_events(b, a)
