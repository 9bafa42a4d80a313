"""The 4-bit key/value cache: page tables, storing, loading and attention.

Argument marshalling for the calls of ``include/lt_kv4.h``, which documents the
cache's format and every argument. A serving step:

    kept, num_free = page_release(lengths, finished, table, free_pages, num_free, page_size)
    step = page_extend(kept, new_tokens, table, free_pages, num_free, page_size, max_tokens)
    kv4_store(k, v, cache, step.slots)
    out = kv4_attention(q, cache, table, step.lengths, starts=step.starts, max_new=max_new)

and, over the positions that the indexer's top-k kept,

    idx, _ = topk(scores, step.lengths, 512)
    out, lse = kv4_attention(q, cache, table, step.lengths, positions=idx, with_lse=True)
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import DTYPE_BF16, DTYPE_F32, LtError, _ptr, load

DTYPE_F16 = 2
_ALL = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}
_DIM_OF_ROW = {80: 64, 144: 128, 288: 256}


class PageStep(NamedTuple):
    """What page_extend places; see lt_page_extend."""
    slots: torch.Tensor      # int64 [max_tokens]
    positions: torch.Tensor  # int32 [max_tokens]
    starts: torch.Tensor     # int32 [requests + 1]
    lengths: torch.Tensor    # int32 [requests]
    num_free: torch.Tensor   # int32 [1]


def _stream(stream, dev):
    return ctypes.c_void_p((stream or torch.cuda.current_stream(dev)).cuda_stream)


def _want(name, t, dtype, dev=None, shape=None):
    """A contiguous CUDA tensor of this type (and shape), on this device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    if t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, has {tuple(t.shape)}")
    return t


def _result(name, t, shape, dtype, dev, stream):
    """The caller's output tensor, or a new one whose memory belongs to the stream that writes it."""
    if t is not None:
        return _want(name, t, dtype, dev, shape)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _int32(name, x, least):
    x = int(x)
    if x < least or x > 2 ** 31 - 1:
        raise ValueError(f"{name} must be from {least} to 2^31 - 1, got {x}")
    return x


def _check_page_size(page_size):
    page_size = int(page_size)
    if page_size < 1 or page_size > 1024 or page_size & (page_size - 1):
        raise ValueError(f"page_size must be a power of two from 1 to 1024, got {page_size}")
    return page_size


def kv4_row_bytes(head_dim: int) -> int:
    """Bytes of a cache row; raises for a head_dim that is not supported."""
    n = int(load().lt_kv4_row_bytes(int(head_dim)))
    if n == 0:
        raise ValueError(f"head_dim must be 64, 128 or 256, got {head_dim}")
    return n


def kv4_cache(pages: int, kv_heads: int, page_size: int, head_dim: int, device=None) -> torch.Tensor:
    """An empty cache: uint8 [pages, kv_heads, page_size, kv4_row_bytes(head_dim)]."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    return torch.zeros(pages, kv_heads, _check_page_size(page_size), kv4_row_bytes(head_dim), dtype=torch.uint8,
                       device=device)


def _check_cache(cache):
    """(pages, kv_heads, page_size, head_dim) of a cache."""
    _want("cache", cache, torch.uint8)
    if cache.dim() != 4 or cache.shape[3] not in _DIM_OF_ROW:
        raise ValueError("cache must be [pages, kv_heads, page_size, row bytes], as kv4_cache makes it")
    return cache.shape[0], cache.shape[1], _check_page_size(cache.shape[2]), _DIM_OF_ROW[cache.shape[3]]


def page_release(lengths: torch.Tensor, finished: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                 num_free: torch.Tensor, page_size: int, *, out_lengths: torch.Tensor | None = None,
                 out_num_free: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """Gives the pages of finished requests (bool or uint8 [requests]) back to free_pages (in place);
    returns (lengths, num_free): 0 for the finished requests, and the new number of free pages."""
    lib = load()
    _want("lengths", lengths, torch.int32)
    dev, n = lengths.device, lengths.numel()
    if not isinstance(finished, torch.Tensor) or finished.dtype not in (torch.bool, torch.uint8):
        raise TypeError("finished must be a bool or uint8 tensor")
    _want("finished", finished, finished.dtype, dev, (n,))
    _check_table(block_table, dev, n)
    _want("free_pages", free_pages, torch.int32, dev)
    _want("num_free", num_free, torch.int32, dev, (1,))
    out_lengths = _result("out_lengths", out_lengths, (n,), torch.int32, dev, stream)
    out_num_free = _result("out_num_free", out_num_free, (1,), torch.int32, dev, stream)
    with torch.cuda.device(dev):
        st = lib.lt_page_release(_ptr(lengths), _ptr(finished), n, _ptr(block_table), block_table.shape[1],
                                 _ptr(free_pages), free_pages.numel(), _ptr(num_free), _check_page_size(page_size),
                                 _ptr(out_lengths), _ptr(out_num_free), _stream(stream, dev))
    if st != 0:
        raise LtError("lt_page_release", st)
    return out_lengths, out_num_free


def _check_table(block_table, dev, n):
    _want("block_table", block_table, torch.int32, dev)
    if block_table.dim() != 2 or block_table.shape[0] != n or block_table.shape[1] < 1:
        raise ValueError("block_table must be [requests, pages a request]")


def page_extend(lengths: torch.Tensor, new_tokens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                num_free: torch.Tensor, page_size: int, max_tokens: int, *, out_slots: torch.Tensor | None = None,
                out_positions: torch.Tensor | None = None, out_starts: torch.Tensor | None = None,
                out_lengths: torch.Tensor | None = None, out_num_free: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None) -> PageStep:
    """Places the new tokens of a step: takes pages from the top of free_pages, writes them into
    block_table (in place) and returns slots, positions, starts, lengths and the pages left."""
    lib = load()
    _want("lengths", lengths, torch.int32)
    dev, n = lengths.device, lengths.numel()
    _want("new_tokens", new_tokens, torch.int32, dev, (n,))
    _check_table(block_table, dev, n)
    _want("free_pages", free_pages, torch.int32, dev)
    _want("num_free", num_free, torch.int32, dev, (1,))
    max_tokens = _int32("max_tokens", max_tokens, 0)
    step = PageStep(_result("out_slots", out_slots, (max_tokens,), torch.int64, dev, stream),
                    _result("out_positions", out_positions, (max_tokens,), torch.int32, dev, stream),
                    _result("out_starts", out_starts, (n + 1,), torch.int32, dev, stream),
                    _result("out_lengths", out_lengths, (n,), torch.int32, dev, stream),
                    _result("out_num_free", out_num_free, (1,), torch.int32, dev, stream))
    with torch.cuda.device(dev):
        st = lib.lt_page_extend(_ptr(lengths), _ptr(new_tokens), n, _ptr(block_table), block_table.shape[1],
                                _ptr(free_pages), free_pages.numel(), _ptr(num_free), _check_page_size(page_size),
                                max_tokens, _ptr(step.slots), _ptr(step.positions), _ptr(step.starts),
                                _ptr(step.lengths), _ptr(step.num_free), _stream(stream, dev))
    if st != 0:
        raise LtError("lt_page_extend", st)
    return step


def _check_slots(slots, dev, tokens):
    _want("slots", slots, torch.int64, dev)
    if slots.dim() != 1 or (tokens is not None and slots.numel() != tokens):
        raise ValueError("slots must be int64 [tokens]")


def kv4_store(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor, *,
              stream: torch.cuda.Stream | None = None) -> None:
    """Quantises k, v [tokens, kv_heads, head_dim] (float32, bfloat16 or float16; any strides of tokens
    and heads) into the cache rows that slots (int64 [tokens]; -1 skips) name."""
    lib = load()
    pages, heads, page_size, dim = _check_cache(cache)
    dev = cache.device
    for name, t in (("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.device != dev or t.dim() != 3 or tuple(t.shape[1:]) != (heads, dim):
            raise ValueError(f"{name} must be [tokens, {heads}, {dim}] on {dev}")
        if t.numel() > 0 and t.stride(2) != 1:
            raise ValueError(f"the channels of {name} must be contiguous")
    if k.dtype not in _ALL or v.dtype != k.dtype or v.shape != k.shape:
        raise ValueError("k and v must have one shape and one type: float32, bfloat16 or float16")
    tokens = k.shape[0]
    _check_slots(slots, dev, tokens)
    with torch.cuda.device(dev):
        st = lib.lt_kv4_store(_ptr(k), _ptr(v), _ALL[k.dtype], tokens, heads, dim, k.stride(0), k.stride(1),
                              v.stride(0), v.stride(1), _ptr(slots), _ptr(cache), pages, page_size,
                              _stream(stream, dev))
    if st != 0:
        raise LtError("lt_kv4_store", st)


def kv4_load(cache: torch.Tensor, slots: torch.Tensor, *, dtype: torch.dtype = torch.float16,
             out_k: torch.Tensor | None = None, out_v: torch.Tensor | None = None,
             stream: torch.cuda.Stream | None = None):
    """The numbers that the slots stand for: (k, v), each [tokens, kv_heads, head_dim]; zeros for a slot
    outside the cache."""
    lib = load()
    pages, heads, page_size, dim = _check_cache(cache)
    dev = cache.device
    if dtype not in _ALL:
        raise ValueError("dtype must be float32, bfloat16 or float16")
    _check_slots(slots, dev, None)
    shape = (slots.numel(), heads, dim)
    out_k = _result("out_k", out_k, shape, dtype, dev, stream)
    out_v = _result("out_v", out_v, shape, dtype, dev, stream)
    with torch.cuda.device(dev):
        st = lib.lt_kv4_load(_ptr(cache), pages, page_size, _ptr(slots), slots.numel(), heads, dim, _ptr(out_k),
                             _ptr(out_v), _ALL[dtype], _stream(stream, dev))
    if st != 0:
        raise LtError("lt_kv4_load", st)
    return out_k, out_v


def kv4_attention(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, lengths: torch.Tensor, *,
                  starts: torch.Tensor | None = None, max_new: int = 1, positions: torch.Tensor | None = None,
                  window: int = 0, scale: float | None = None, with_lse: bool = False,
                  out: torch.Tensor | None = None, out_lse: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """Attention of the requests' new tokens over the cache.

    q [tokens, q_heads, head_dim] (bfloat16 or float16) holds the queries of request r in rows
    starts[r] .. starts[r + 1] (starts int32 [requests + 1], at most max_new rows a request; None: one
    a request), the last of its lengths[r] cached positions. Causal; the last `window` positions only if
    window > 0; or the listed `positions` (int32 [tokens, n], -1 pads) instead. scale is
    1 / sqrt(head_dim) by default. Returns out, or (out, lse) with with_lse.

    workspace (uint8) replaces the scratch memory that a call takes from torch's allocator for its
    stream; see lt_kv4_workspace for its size.
    """
    lib = load()
    pages, heads, page_size, dim = _check_cache(cache)
    dev = cache.device
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise TypeError("q must be a CUDA tensor")
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("q must be bfloat16 or float16")
    if q.device != dev or q.dim() != 3 or q.shape[2] != dim or q.shape[1] % heads or q.shape[1] < 1:
        raise ValueError(f"q must be [tokens, a multiple of {heads} heads, {dim}] on {dev}")
    tokens, q_heads, _ = q.shape
    if q.numel() > 0 and (q.stride(2) != 1 or q.stride(0) % 8 or q.stride(1) % 8 or q.data_ptr() % 16):
        raise ValueError("q must have contiguous channels, strides that are multiples of 8 and a 16-byte aligned start")
    _want("lengths", lengths, torch.int32, dev)
    n = lengths.numel()
    _check_table(block_table, dev, n)
    max_new = _int32("max_new", max_new, 1)
    if starts is None:
        if tokens != n or max_new != 1:
            raise ValueError("without starts, q must have one row a request")
    else:
        _want("starts", starts, torch.int32, dev, (n + 1,))
    window = _int32("window", window, 0)
    if window and positions is not None:
        raise ValueError("window is not used with positions")
    list_len = 0
    if positions is not None:
        _want("positions", positions, torch.int32, dev)
        if positions.dim() != 2 or positions.shape[0] != tokens or positions.shape[1] < 1:
            raise ValueError("positions must be int32 [tokens, at least one]")
        list_len = positions.shape[1]
    out = _result("out", out, (tokens, q_heads, dim), q.dtype, dev, stream)
    lse = _result("out_lse", out_lse, (tokens, q_heads), torch.float32, dev, stream) if with_lse else None
    scale = dim ** -0.5 if scale is None else float(scale)
    with torch.cuda.device(dev):
        need = ctypes.c_int64(0)
        st = lib.lt_kv4_workspace(tokens, q_heads, heads, dim, n, max_new, list_len, ctypes.byref(need))
        if st != 0:
            raise LtError("lt_kv4_workspace", st)
        s = stream or torch.cuda.current_stream(dev)
        if workspace is None and need.value > 0:
            workspace = _result("workspace", None, (need.value,), torch.uint8, dev, stream)
        elif workspace is not None:
            _want("workspace", workspace, torch.uint8, dev)
            if workspace.numel() < need.value:
                raise ValueError(f"workspace must have at least {need.value} bytes")
        st = lib.lt_kv4_attention(_ptr(q), _ALL[q.dtype], tokens, q_heads, heads, dim, q.stride(0), q.stride(1),
                                  _ptr(cache), pages, page_size, _ptr(block_table), block_table.shape[1],
                                  _ptr(lengths), n, _ptr(starts), max_new, _ptr(positions), list_len, window,
                                  scale, _ptr(out), _ptr(lse), _ptr(workspace),
                                  0 if workspace is None else workspace.numel(), ctypes.c_void_p(s.cuda_stream))
    if st != 0:
        raise LtError("lt_kv4_attention", st)
    return (out, lse) if with_lse else out
