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
import functools
from typing import NamedTuple

import torch

from . import DTYPE_BF16, DTYPE_F32, LtError, load

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


# The checks are on the path of every decode step, whose kernels take a few microseconds: devices are
# compared by their index, the stream is taken by its handle.


def _raw_stream(stream, index):
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _call(name, index, *args):
    """Calls the library with the tensors' device current; raises on an error status."""
    fn = getattr(load(), name)
    if torch.cuda.current_device() == index:
        st = fn(*args)
    else:
        with torch.cuda.device(index):
            st = fn(*args)
    if st != 0:
        raise LtError(name, st)


def _want(name, t, dtype, index=None, shape=None):
    """A contiguous CUDA tensor of this type (and shape), on this device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}")
    if t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, has {tuple(t.shape)}")
    return t


def _result(name, t, shape, dtype, like, stream):
    """The caller's output tensor, or a new one whose memory belongs to the stream that writes it."""
    if t is not None:
        return _want(name, t, dtype, like.get_device(), shape)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


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
    """(pages, kv_heads, page_size, head_dim, device index) of a cache."""
    _want("cache", cache, torch.uint8)
    if cache.dim() != 4 or cache.shape[3] not in _DIM_OF_ROW:
        raise ValueError("cache must be [pages, kv_heads, page_size, row bytes], as kv4_cache makes it")
    pages, heads, page_size, row = cache.shape
    return pages, heads, _check_page_size(page_size), _DIM_OF_ROW[row], cache.get_device()


def _check_table(block_table, index, n):
    _want("block_table", block_table, torch.int32, index)
    if block_table.dim() != 2 or block_table.shape[0] != n or block_table.shape[1] < 1:
        raise ValueError("block_table must be [requests, pages a request]")
    return block_table.shape[1]


def page_release(lengths: torch.Tensor, finished: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                 num_free: torch.Tensor, page_size: int, *, out_lengths: torch.Tensor | None = None,
                 out_num_free: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """Gives the pages of finished requests (bool or uint8 [requests]) back to free_pages (in place; cells of
    block_table below 0 hold no page); returns (lengths, num_free): 0 for the finished requests, and the new number of free pages."""
    _want("lengths", lengths, torch.int32)
    index, n = lengths.get_device(), lengths.numel()
    if not isinstance(finished, torch.Tensor) or finished.dtype not in (torch.bool, torch.uint8):
        raise TypeError("finished must be a bool or uint8 tensor")
    _want("finished", finished, finished.dtype, index, (n,))
    width = _check_table(block_table, index, n)
    _want("free_pages", free_pages, torch.int32, index)
    _want("num_free", num_free, torch.int32, index, (1,))
    page_size = _check_page_size(page_size)
    out_lengths = _result("out_lengths", out_lengths, (n,), torch.int32, lengths, stream)
    out_num_free = _result("out_num_free", out_num_free, (1,), torch.int32, lengths, stream)
    _call("lt_page_release", index, lengths.data_ptr(), finished.data_ptr(), n, block_table.data_ptr(), width,
          free_pages.data_ptr(), free_pages.numel(), num_free.data_ptr(), page_size, out_lengths.data_ptr(),
          out_num_free.data_ptr(), _raw_stream(stream, index))
    return out_lengths, out_num_free


def page_extend(lengths: torch.Tensor, new_tokens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                num_free: torch.Tensor, page_size: int, max_tokens: int, *, out_slots: torch.Tensor | None = None,
                out_positions: torch.Tensor | None = None, out_starts: torch.Tensor | None = None,
                out_lengths: torch.Tensor | None = None, out_num_free: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None) -> PageStep:
    """Places the new tokens of a step: takes pages from the top of free_pages, writes them into
    block_table (in place) and returns slots, positions, starts, lengths and the pages left."""
    _want("lengths", lengths, torch.int32)
    index, n = lengths.get_device(), lengths.numel()
    _want("new_tokens", new_tokens, torch.int32, index, (n,))
    width = _check_table(block_table, index, n)
    _want("free_pages", free_pages, torch.int32, index)
    _want("num_free", num_free, torch.int32, index, (1,))
    page_size = _check_page_size(page_size)
    max_tokens = _int32("max_tokens", max_tokens, 0)
    slots = _result("out_slots", out_slots, (max_tokens,), torch.int64, lengths, stream)
    positions = _result("out_positions", out_positions, (max_tokens,), torch.int32, lengths, stream)
    starts = _result("out_starts", out_starts, (n + 1,), torch.int32, lengths, stream)
    out_lengths = _result("out_lengths", out_lengths, (n,), torch.int32, lengths, stream)
    out_num_free = _result("out_num_free", out_num_free, (1,), torch.int32, lengths, stream)
    _call("lt_page_extend", index, lengths.data_ptr(), new_tokens.data_ptr(), n, block_table.data_ptr(), width,
          free_pages.data_ptr(), free_pages.numel(), num_free.data_ptr(), page_size, max_tokens, slots.data_ptr(),
          positions.data_ptr(), starts.data_ptr(), out_lengths.data_ptr(), out_num_free.data_ptr(),
          _raw_stream(stream, index))
    return PageStep(slots, positions, starts, out_lengths, out_num_free)


def _check_slots(slots, index, tokens):
    _want("slots", slots, torch.int64, index)
    if slots.dim() != 1 or (tokens is not None and slots.numel() != tokens):
        raise ValueError("slots must be int64 [tokens]")


def kv4_store(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor, *,
              stream: torch.cuda.Stream | None = None) -> None:
    """Quantises k, v [tokens, kv_heads, head_dim] (float32, bfloat16 or float16; any strides of tokens
    and heads) into the cache rows that slots (int64 [tokens]; -1 skips) name."""
    pages, heads, page_size, dim, index = _check_cache(cache)
    for name, t in (("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.get_device() != index or t.dim() != 3 or t.shape[1:] != (heads, dim):
            raise ValueError(f"{name} must be [tokens, {heads}, {dim}] on cuda:{index}")
    dtype, tokens = _ALL.get(k.dtype), k.shape[0]
    if dtype is None or v.dtype != k.dtype or v.shape != k.shape:
        raise ValueError("k and v must have one shape and one type: float32, bfloat16 or float16")
    ks, vs = k.stride(), v.stride()
    if tokens > 0 and (ks[2] != 1 or vs[2] != 1):
        raise ValueError("the channels of k and v must be contiguous")
    _check_slots(slots, index, tokens)
    _call("lt_kv4_store", index, k.data_ptr(), v.data_ptr(), dtype, tokens, heads, dim, ks[0], ks[1], vs[0], vs[1],
          slots.data_ptr(), cache.data_ptr(), pages, page_size, _raw_stream(stream, index))


def kv4_load(cache: torch.Tensor, slots: torch.Tensor, *, dtype: torch.dtype = torch.float16,
             out_k: torch.Tensor | None = None, out_v: torch.Tensor | None = None,
             stream: torch.cuda.Stream | None = None):
    """The numbers that the slots stand for: (k, v), each [tokens, kv_heads, head_dim]; zeros for a slot
    outside the cache."""
    pages, heads, page_size, dim, index = _check_cache(cache)
    if dtype not in _ALL:
        raise ValueError("dtype must be float32, bfloat16 or float16")
    _check_slots(slots, index, None)
    tokens = slots.shape[0]
    out_k = _result("out_k", out_k, (tokens, heads, dim), dtype, cache, stream)
    out_v = _result("out_v", out_v, (tokens, heads, dim), dtype, cache, stream)
    _call("lt_kv4_load", index, cache.data_ptr(), pages, page_size, slots.data_ptr(), tokens, heads, dim,
          out_k.data_ptr(), out_v.data_ptr(), _ALL[dtype], _raw_stream(stream, index))
    return out_k, out_v


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(index, tokens, q_heads, kv_heads, head_dim, requests, max_new, list_len, positions, window):
    """lt_kv4_workspace's answer: it goes by these sizes and the device alone."""
    need = ctypes.c_int64(0)
    _call("lt_kv4_workspace", index, tokens, q_heads, kv_heads, head_dim, requests, max_new, list_len,
          positions, window, ctypes.byref(need))
    return need.value


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
    pages, heads, page_size, dim, index = _check_cache(cache)
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise TypeError("q must be a CUDA tensor")
    dtype = q.dtype
    if dtype != torch.bfloat16 and dtype != torch.float16:
        raise TypeError("q must be bfloat16 or float16")
    if q.get_device() != index or q.dim() != 3 or q.shape[2] != dim or q.shape[1] % heads or q.shape[1] < 1:
        raise ValueError(f"q must be [tokens, a multiple of {heads} heads, {dim}] on cuda:{index}")
    tokens, q_heads, _ = q.shape
    token_stride, head_stride, channel_stride = q.stride()
    q_ptr = q.data_ptr()
    if tokens > 0 and (channel_stride != 1 or token_stride % 8 or head_stride % 8 or q_ptr % 16):
        raise ValueError("q must have contiguous channels, strides that are multiples of 8 and a 16-byte aligned start")
    _want("lengths", lengths, torch.int32, index)
    n = lengths.numel()
    width = _check_table(block_table, index, n)
    max_new = _int32("max_new", max_new, 1)
    if starts is None:
        if tokens != n or max_new != 1:
            raise ValueError("without starts, q must have one row a request")
    else:
        _want("starts", starts, torch.int32, index, (n + 1,))
    window = _int32("window", window, 0)
    list_len = 0
    if positions is not None:
        if window:
            raise ValueError("window is not used with positions")
        _want("positions", positions, torch.int32, index)
        if positions.dim() != 2 or positions.shape[0] != tokens or positions.shape[1] < 1:
            raise ValueError("positions must be int32 [tokens, at least one]")
        list_len = positions.shape[1]
    out = _result("out", out, (tokens, q_heads, dim), dtype, q, stream)
    lse = _result("out_lse", out_lse, (tokens, q_heads), torch.float32, q, stream) if with_lse else None
    need = _workspace_bytes(index, tokens, q_heads, heads, dim, n, max_new, list_len, width * page_size, window)
    if workspace is not None:
        _want("workspace", workspace, torch.uint8, index)
        if workspace.numel() < need:
            raise ValueError(f"workspace must have at least {need} bytes")
    elif need > 0:
        workspace = _result("workspace", None, (need,), torch.uint8, q, stream)
    _call("lt_kv4_attention", index, q_ptr, _ALL[dtype], tokens, q_heads, heads, dim, token_stride, head_stride,
          cache.data_ptr(), pages, page_size, block_table.data_ptr(), width, lengths.data_ptr(), n,
          None if starts is None else starts.data_ptr(), max_new, None if positions is None else positions.data_ptr(),
          list_len, window, dim ** -0.5 if scale is None else scale, out.data_ptr(),
          None if lse is None else lse.data_ptr(), None if workspace is None else workspace.data_ptr(),
          0 if workspace is None else workspace.numel(), _raw_stream(stream, index))
    return (out, lse) if with_lse else out
