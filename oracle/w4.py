"""Products with 4-bit weights in 64 bits, on the CPU. Shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

from . import kv4


def quantise(w):
    """(codes uint8 [n, k / 2], scales float16 [n, k / 32]) of weights, as the cache's keys are stored."""
    scales, codes = kv4.quantise(w)
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8), scales.astype(np.float16)


def weights(codes, scales):
    codes = np.asarray(codes)
    code = np.stack([codes & 15, codes >> 4], axis=-1).reshape(codes.shape[0], -1)
    return kv4.values(np.asarray(scales, dtype=np.float64), code)


def linear(x, codes, scales, bias=None):
    """(x W^T + bias, |x| |W|^T): the result and what its error bound goes by."""
    w, x = weights(codes, scales), np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        y = x @ w.T
        return (y if bias is None else y + np.asarray(bias, np.float64)), np.abs(x) @ np.abs(w).T
