"""Products with 4-bit weights for long prompts, to the most tokens that a call takes: equal to 64 bits, rounded once.

Inputs of -1, 0 and 1 and weights that are multiples of 1/2, at most 6 in magnitude: sums of k of them are exact in 32 bits.
"""
import pytest
import torch

from oracle import w4 as ow

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_lt_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,n,k", [(1000, 700, 4096), (4096, 1030, 544), (8191, 4100, 256), (70001, 130, 96), (524280, 33, 64)])
def test_long_prompts(tokens, n, k, dtype):
    import sparse_attention_indexer_lt_gb300 as lt
    g = torch.Generator("cuda").manual_seed(tokens)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.ones(n, k // 32, device="cuda").half()
    x = (torch.randint(0, 3, (tokens, k), generator=g, device="cuda") - 1).to(dtype)
    w = torch.as_tensor(ow.weights(codes.cpu().numpy(), scales.cpu().double().numpy())).cuda()
    out = torch.full((tokens + 1, n), 3.0, device="cuda", dtype=dtype)
    y = lt.w4_linear(x, codes, scales, out=out[:tokens])
    for i in range(0, tokens, 65536):
        assert torch.equal(y[i:i + 65536], (x[i:i + 65536].double() @ w.T).to(dtype)), f"tokens from {i}"
    assert (out[tokens:] == 3.0).all()
