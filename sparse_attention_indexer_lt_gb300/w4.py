"""Products with 4-bit weights: argument marshalling for the calls of ``include/lt_w4.h``, which documents
the format and every argument.

    codes, scales = w4_quantise(weight)           # once
    y = w4_linear(x, codes, scales, bias=bias)    # x @ weight.T + bias
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import DTYPE_BF16
from .kv4 import _ALL, DTYPE_F16, _call, _raw_stream, _result, _want

_GROUP = 32
_KIND = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}


def w4_quantise(weight: torch.Tensor, *, out_codes: torch.Tensor | None = None, out_scales: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None):
    """Codes uint8 [n, k / 2] and scales float16 [n, k / 32] of weight [n, k] (float32, bfloat16 or float16; any
    stride of rows), with the rounding of kv4_store."""
    if not isinstance(weight, torch.Tensor) or not weight.is_cuda:
        raise TypeError("weight must be a CUDA tensor")
    dtype, index = _ALL.get(weight.dtype), weight.get_device()
    if dtype is None or weight.dim() != 2 or weight.shape[1] < _GROUP or weight.shape[1] % _GROUP:
        raise ValueError("weight must be [n, a multiple of 32] in float32, bfloat16 or float16")
    n, k = weight.shape
    if n > 0 and weight.stride(1) != 1:
        raise ValueError("the rows of weight must be contiguous")
    codes = _result("out_codes", out_codes, (n, k // 2), torch.uint8, weight, stream)
    scales = _result("out_scales", out_scales, (n, k // _GROUP), torch.float16, weight, stream)
    _call("lt_w4_quantise", index, weight.data_ptr(), dtype, n, k, weight.stride(0), codes.data_ptr(), scales.data_ptr(),
          _raw_stream(stream, index))
    return codes, scales


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(index, tokens, n, k):
    """lt_w4_workspace's answer: it goes by these sizes and the device alone."""
    need = ctypes.c_int64(0)
    _call("lt_w4_workspace", index, tokens, n, k, ctypes.byref(need))
    return need.value


def w4_linear(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, *, bias: torch.Tensor | None = None,
              out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
              stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """x [tokens, k] (bfloat16 or float16) times the weights that codes (uint8 [n, k / 2]) and scales (float16
    [n, k / 32]) hold, transposed, plus bias [n] in x's type: [tokens, n] in x's type.

    x may have any stride of rows that is a multiple of 8, out any stride of rows. workspace (uint8) replaces
    the scratch memory that a call takes from torch's allocator for its stream; see lt_w4_workspace.
    """
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    dtype, index = x.dtype, x.get_device()
    kind = _KIND.get(dtype)
    if kind is None:
        raise TypeError("x must be bfloat16 or float16")
    # (one look at each where all is as it should be; the reasons are found only where something is not)
    if not (isinstance(codes, torch.Tensor) and codes.dtype is torch.uint8 and codes.get_device() == index and codes.is_contiguous()):
        _want("codes", codes, torch.uint8, index)
    if not (isinstance(scales, torch.Tensor) and scales.dtype is torch.float16 and scales.get_device() == index and scales.is_contiguous()):
        _want("scales", scales, torch.float16, index)
    x_shape, shape = x.shape, codes.shape
    if len(x_shape) != 2 or len(shape) != 2 or x_shape[1] < _GROUP or x_shape[1] % _GROUP or shape[1] * 2 != x_shape[1]:
        raise ValueError("x must be [tokens, k] and codes [n, k / 2], k a multiple of 32")
    tokens, k = x_shape
    n = shape[0]
    if scales.shape != (n, k // _GROUP):
        raise ValueError(f"scales must have shape {(n, k // _GROUP)}, has {tuple(scales.shape)}")
    x_stride, one = x.stride()
    if tokens == 1:
        x_stride = k  # (of one token it says nothing)
    x_ptr, codes_ptr, scales_ptr = x.data_ptr(), codes.data_ptr(), scales.data_ptr()
    if tokens > 0 and (one != 1 or x_stride % 8 or x_ptr % 16):
        raise ValueError("x must have contiguous rows, a row stride that is a multiple of 8 and a 16-byte aligned start")
    if codes_ptr % 16 or scales_ptr % 16:
        raise ValueError("codes and scales must start on 16 bytes")
    if bias is not None:
        _want("bias", bias, dtype, index, (n,))
    out_stride = n
    if out is None:
        out = _result("out", None, (tokens, n), dtype, x, stream)
    else:
        if not isinstance(out, torch.Tensor) or not out.is_cuda or out.get_device() != index or out.dtype != dtype \
                or out.shape != (tokens, n) or (tokens > 0 and n > 0 and out.stride(1) != 1):
            raise ValueError(f"out must be a {dtype} tensor of shape {(tokens, n)} on cuda:{index}, its rows contiguous")
        out_stride = out.stride(0)
    need = _workspace_bytes(index, tokens, n, k)
    if workspace is not None:
        _want("workspace", workspace, torch.uint8, index)
        if workspace.numel() < need or workspace.data_ptr() % 16:
            raise ValueError(f"workspace must have at least {need} bytes and start on 16")
    elif need > 0:
        workspace = _result("workspace", None, (need,), torch.uint8, x, stream)
    _call("lt_w4_linear", index, x_ptr, kind, tokens, x_stride, codes_ptr, scales_ptr, n, k,
          None if bias is None else bias.data_ptr(), out.data_ptr(), out_stride,
          None if workspace is None else workspace.data_ptr(), need, _raw_stream(stream, index))
    return out
