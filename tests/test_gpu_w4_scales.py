"""Scales from elsewhere in products with 4-bit weights.

A weight code * scale is rounded to fp16 where the scale has more than 9 bits: by 2^-11 of itself, or 2^-25 where it is below
2^-14. Beside test_gpu_w4's bound a result is off by sum |x| times that.
"""
import numpy as np
import pytest
import torch

from oracle import w4 as ow
from test_gpu_w4 import TYPES, make, num

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_lt_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def foreign(n, k, size, seed):
    """Codes, and scales of 11 bits: around `size`, each group's a factor of up to 4 away, subnormal ones among small sizes."""
    codes, _ = make(n, k, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    scales = (size * 4.0 ** (2 * torch.rand(n, k // 32, generator=g, dtype=torch.float64) - 1)).clamp(2.0 ** -24, 10912.0).half()
    return codes, (scales.view(torch.int16) | 1).view(torch.float16).clamp(max=10912.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size", [0.1, 2.0 ** -14, 2.0 ** -17, 2.0 ** -23, 4000.0])
@pytest.mark.parametrize("tokens,n,k", [(1, 70, 512), (7, 130, 544), (40, 200, 512), (130, 300, 1056)])
def test_scales_of_eleven_bits(tokens, n, k, size, dtype):
    import sparse_attention_indexer_lt_gb300 as lt
    codes, scales = foreign(n, k, size, seed=tokens)
    x = (torch.randn(tokens, k, generator=torch.Generator().manual_seed(n)) * min(1.0, 0.1 / size)).to(TYPES[dtype])
    y = num(lt.w4_linear(x.cuda(), codes.cuda(), scales.cuda()))
    w = ow.weights(codes.numpy(), num(scales))
    want, reach = ow.linear(num(x), codes.numpy(), num(scales))
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    rounded = np.abs(num(x)) @ np.maximum(2.0 ** -11 * np.abs(w), 2.0 ** -25).T
    tiny = np.abs(num(x)).max(1, keepdims=True) * 2.0 ** -39 * np.abs(w).sum(1)[None]
    tol = (k + 16) * 2.0 ** -23 * (reach + rounded) + rounded + u * (np.abs(want) + rounded) + tiny + (2.0 ** -25 if dtype == "f16" else 2.0 ** -134)
    assert np.isfinite(y).all()
    err = np.abs(y - want)
    assert (err <= tol).all(), f"{int((err > tol).sum())} off, worst {float((err / tol).max()):.3g} of its bound"


@pytest.mark.parametrize("tokens", [1, 40])
def test_the_smallest_weights(tokens):
    """Of scales of 2^-24 the code 1/2 makes a weight that lies between two fp16 numbers, 0 and 2^-24: the even one is 0."""
    import sparse_attention_indexer_lt_gb300 as lt
    codes = torch.full((4, 32), 0x11, dtype=torch.uint8)
    codes[1] = 0x22
    codes[2] = 0x33
    scales = torch.full((4, 2), 2.0 ** -24).half()
    scales[3] = 3 * 2.0 ** -24  # half of it: 1.5 units, the even neighbour is 2
    y = lt.w4_linear(torch.ones(tokens, 64).cuda().half() * 1024, codes.cuda(), scales.cuda())
    assert y[0].tolist() == [0.0, 64 * 2.0 ** -14, 128 * 2.0 ** -14, 128 * 2.0 ** -14] and torch.equal(y, y[:1].expand_as(y))
