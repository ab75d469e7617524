"""Binding of the attention layers beside the mixer (include/kdn.h): attention over whole
prompts, the paged 4-bit key/value cache, and attention of one new token per sequence
over it.  Argument marshalling only, as in :mod:`.binding`; forward only, outputs carry no
history.  What a call records on the GPU (a length or table entry out of range, a timeout) stands
in the status word of its workspace: pass ``workspace`` and read it with
``kdn_read_device_status``; one that the call makes for itself goes away with its status.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from .binding import KDN_BF16, KDN_F32, KDNError, library

_IO = {torch.bfloat16: KDN_BF16, torch.float32: KDN_F32}
_raw_stream = torch._C._cuda_getCurrentRawStream   # the handle alone, without a Stream object
_current_device = torch._C._cuda_getDevice          # CUDA is up: a tensor of its has been looked at


class CachePlan(NamedTuple):
    """Results of :func:`kdn_cache_plan` (device tensors, meanings in include/kdn.h)."""

    slot_map: torch.Tensor     # [capacity] int64
    position: torch.Tensor     # [capacity] int32
    cu_new: torch.Tensor       # [n_req + 1] int32
    seq_len: torch.Tensor      # [n_req] int32
    granted: torch.Tensor      # [n_req] int32
    free_left: torch.Tensor    # [1] int32


def _refuse(t, name, dtype, shape, device, dense):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous" if dense else f"the last axis of {name} must be contiguous")


def _tensor(t, name, dtype, shape, device):
    """Pointer of a dense tensor of this type and shape.  (Calls take a few microseconds on the GPU: the checks are few.)"""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device and t.is_cuda \
            and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, dtype, shape, device, True)


def _int(x, name):
    """A number for a 32-bit argument (ctypes would cut it off; negative ones are the library's to refuse)."""
    if -0x80000000 <= x <= 0x7fffffff:
        return x
    raise ValueError(f"{name} = {x} does not fit 32 bits")


def _io(t, name):
    if not isinstance(t, torch.Tensor) or t.dtype not in _IO:
        raise TypeError(f"{name} must be a bfloat16 or float32 CUDA tensor")
    return _IO[t.dtype]


def _rows(t, name, dtype, shape, device):
    """Pointer, row stride and head stride of a [rows, heads, d] operand."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device and t.is_cuda:
        row, head, one = t.stride()
        if one == 1 or shape[2] <= 1 or t.numel() == 0:
            return t.data_ptr(), row, head
    _refuse(t, name, dtype, shape, device, False)


def _call(fn, device, stream, args, scratch=()):
    """Run an entry point on `stream` (None: the device's current one).  `scratch`: tensors made here."""
    if stream is None:
        handle = _raw_stream(device.index)
    else:
        current = torch.cuda.current_stream(device)
        if stream != current:
            # the allocator made them for the current stream: their memory must not be reused before `stream` is
            # done, and `stream` must not write to it before what used it last
            stream.wait_stream(current)
            for t in scratch:
                t.record_stream(stream)
        handle = stream.cuda_stream
    if _current_device() == device.index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(*args, handle)
    if st != 0:
        raise KDNError(st, fn.__name__)


def _workspace(given, need, device, made):
    if given is None:
        given = torch.empty(need, dtype=torch.uint8, device=device)
        made.append(given)
        return given.data_ptr(), need
    if given.device != device:
        raise ValueError(f"workspace is on {given.device}, expected {device}")
    elif not given.is_contiguous():
        raise ValueError("workspace must be contiguous")
    elif given.numel() * given.element_size() < need:
        raise ValueError(f"workspace holds {given.numel() * given.element_size()} bytes, {need} needed")
    return given.data_ptr(), given.numel() * given.element_size()


def cache_alloc(n_pages, page, H_kv, d, device="cuda"):
    """A zeroed cache: uint8 [n_pages, H_kv, page / 16, 18 d] (its pages' blocks of 16 tokens)."""
    if library().kdn_cache_size(1, _int(page, "page"), 1, _int(d, "d")) == 0:
        raise KDNError(6, "kdn_cache_size rejected the arguments")
    return torch.zeros((n_pages, H_kv, page // 16, 18 * d), dtype=torch.uint8, device=device)


def _cache(cache, device):
    """Pointer, pages, tokens a page, key heads and head size of a cache tensor."""
    if not isinstance(cache, torch.Tensor) or cache.dim() != 4 or cache.shape[3] % 18:
        raise ValueError("cache must be a tensor of cache_alloc()")
    ptr = _tensor(cache, "cache", torch.uint8, cache.shape, device)
    return ptr, cache.shape[0], cache.shape[2] * 16, cache.shape[1], cache.shape[3] // 18


def kdn_cache_plan(context_len, new_len, block_table, free_pages, free_count, *, page, capacity, out=None,
                   workspace=None, stream=None):
    """Block tables and slot maps of one batch from its requests' lengths.  Returns a :class:`CachePlan`.

    context_len, new_len [n_req], free_pages [n_free], free_count [1] and block_table
    [n_req, table_width] are int32; the table gets the entries of the granted requests' new
    pages.  ``capacity`` is the length of the slot map (at least the new tokens).  ``out``: a
    CachePlan to write into.
    """
    device = context_len.device
    n, i32 = context_len.shape[0], torch.int32
    width, page, capacity = _int(block_table.shape[1], "table_width"), _int(page, "page"), _int(capacity, "capacity")
    n_free = _int(free_pages.shape[0], "n_free")
    made = []
    if out is None:
        empty = torch.empty
        out = CachePlan(empty(capacity, dtype=torch.int64, device=device), empty(capacity, dtype=i32, device=device),
                        empty(n + 1, dtype=i32, device=device), empty(n, dtype=i32, device=device),
                        empty(n, dtype=i32, device=device), empty(1, dtype=i32, device=device))
        made.extend(out)
        outs = [t.data_ptr() for t in out]
    else:
        outs = [_tensor(t, name, dt, shape, device) for t, name, dt, shape in zip(
            out, CachePlan._fields, (torch.int64, i32, i32, i32, i32, i32),
            ((capacity,), (capacity,), (n + 1,), (n,), (n,), (1,)))]
    ws, ws_bytes = _workspace(workspace, 256, device, made)
    _call(library().kdn_cache_plan, device, stream,
          (n, page, width, n_free, capacity,
           _tensor(context_len, "context_len", i32, (n,), device), _tensor(new_len, "new_len", i32, (n,), device),
           _tensor(block_table, "block_table", i32, (n, width), device),
           _tensor(free_pages, "free_pages", i32, (n_free,), device),
           _tensor(free_count, "free_count", i32, (1,), device), *outs, ws, ws_bytes), made)
    return out


def kdn_cache_write(k, v, slot_map, cache, *, stream=None):
    """Quantise k, v [n, H_kv, d] (fp32 or bf16) into the cache's slots slot_map [n] (int64; negative: skipped)."""
    device, io = k.device, _io(k, "k")
    ptr, pages, page, heads, d = _cache(cache, device)
    shape = (_int(k.shape[0], "n"), heads, d)
    _call(library().kdn_cache_write, device, stream,
          (shape[0], pages, page, heads, d, io, *_rows(k, "k", k.dtype, shape, device),
           *_rows(v, "v", k.dtype, shape, device), _tensor(slot_map, "slot_map", torch.int64, shape[:1], device), ptr))
    return cache


def kdn_cache_read(cache, slot_map, *, dtype=torch.bfloat16, out=None, stream=None):
    """The values that slots hold: (k, v) [n, H_kv, d]; zeros for negative slots.  ``out=(k, v)`` writes into tensors."""
    device = cache.device
    ptr, pages, page, heads, d = _cache(cache, device)
    shape = (_int(slot_map.shape[0], "n"), heads, d)
    made = []
    if out is None:
        made = [torch.empty(shape, dtype=dtype, device=device) for _ in range(2)]
        out = tuple(made)
    k, v = out
    io = _io(k, "k")
    _call(library().kdn_cache_read, device, stream,
          (shape[0], pages, page, heads, d, io, ptr, _tensor(slot_map, "slot_map", torch.int64, shape[:1], device),
           _tensor(k, "k", k.dtype, shape, device), _tensor(v, "v", k.dtype, shape, device)), made)
    return k, v


def cache_attention_workspace_size(n_seq, H, H_kv, d, max_len, window=0) -> int:
    names = ("n_seq", "H", "H_kv", "d", "max_len", "window")
    return int(library().kdn_cache_attention_workspace_size(*map(_int, (n_seq, H, H_kv, d, max_len, window), names)))


def kdn_cache_attention(q, cache, block_table, seq_len, *, max_len=None, window=0, scale=None, out=None, workspace=None,
                        stream=None):
    """Attention of one query token per sequence over the cache.  Returns (o, lse).

    q [n_seq, H, d] fp32 or bf16; block_table [n_seq, table_width], seq_len [n_seq] int32.
    ``max_len``: a bound on seq_len (None: what the table holds); ``window``: 0 or the number of
    last tokens that are seen; ``scale``: None (or 0) selects d^-1/2.  ``out=(o, lse)`` writes into tensors.
    """
    lib = library()
    device, io = q.device, _io(q, "q")
    width, window = _int(block_table.shape[1], "table_width"), _int(window, "window")
    if max_len is not None:
        _int(max_len, "max_len")
    ptr, pages, page, heads, d = _cache(cache, device)
    n, H = q.shape[0], q.shape[1]
    if max_len is None:
        max_len = min(width * page, 0x7fffffff)
    made = []
    if out is None:
        made = [torch.empty((n, H, d), dtype=q.dtype, device=device), torch.empty((n, H), dtype=torch.float32, device=device)]
        out = tuple(made)
    o, lse = out
    need = lib.kdn_cache_attention_workspace_size(n, H, heads, d, max_len, window)
    ws, ws_bytes = _workspace(workspace, need, device, made)
    _call(lib.kdn_cache_attention, device, stream,
          (n, H, heads, d, page, pages, width, max_len, window, 0.0 if scale is None else scale, io,
           *_rows(q, "q", q.dtype, (n, H, d), device), ptr,
           _tensor(block_table, "block_table", torch.int32, (n, width), device),
           _tensor(seq_len, "seq_len", torch.int32, (n,), device), _tensor(o, "o", q.dtype, (n, H, d), device),
           _tensor(lse, "lse", torch.float32, (n, H), device), ws, ws_bytes), made)
    return o, lse


def prompt_attention_workspace_size(n_seq, total_q, H, H_kv, d, io=KDN_BF16, flags=0) -> int:
    names = ("n_seq", "total_q", "H", "H_kv", "d", "io", "flags")
    return int(library().kdn_prompt_attention_workspace_size(*map(_int, (n_seq, total_q, H, H_kv, d, io, flags), names)))


def kdn_prompt_attention(q, k, v, cu_q, cu_k=None, *, window=0, scale=None, flags=0, out=None, workspace=None,
                         stream=None):
    """Causal attention over whole prompts packed one after another.  Returns (o, lse).

    q [total_q, H, d], k, v [total_k, H_kv, d] fp32 or bf16; cu_q, cu_k [n_seq + 1] int32
    (cu_k=None: as cu_q); with more keys than queries a prompt continues a prefix.  ``window``,
    ``scale`` and ``out`` as for :func:`kdn_cache_attention`.
    """
    lib = library()
    device, io = q.device, _io(q, "q")
    nq, H, d = q.shape
    nq, nk, heads = _int(nq, "total_q"), _int(k.shape[0], "total_k"), k.shape[1]
    n, window, flags = cu_q.shape[0] - 1, _int(window, "window"), _int(flags, "flags")
    made = []
    if out is None:
        made = [torch.empty((nq, H, d), dtype=q.dtype, device=device), torch.empty((nq, H), dtype=torch.float32, device=device)]
        out = tuple(made)
    o, lse = out
    need = lib.kdn_prompt_attention_workspace_size(n, nq, H, heads, d, io, flags)
    ws, ws_bytes = _workspace(workspace, need, device, made)
    _call(lib.kdn_prompt_attention, device, stream,
          (n, nq, nk, H, heads, d, window, 0.0 if scale is None else scale, io, flags,
           *_rows(q, "q", q.dtype, (nq, H, d), device), *_rows(k, "k", q.dtype, (nk, heads, d), device),
           *_rows(v, "v", q.dtype, (nk, heads, d), device), _tensor(cu_q, "cu_q", torch.int32, (n + 1,), device),
           None if cu_k is None else _tensor(cu_k, "cu_k", torch.int32, (n + 1,), device),
           _tensor(o, "o", q.dtype, (nq, H, d), device), _tensor(lse, "lse", torch.float32, (nq, H), device),
           ws, ws_bytes), made)
    return o, lse
