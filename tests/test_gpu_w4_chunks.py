"""Products of few tokens with more inputs than a CTA holds at a time: equal to the oracle, not near it.

The kernel for few tokens then takes its inputs in chunks, and every row block's again. Weights are whole multiples of 1/2 (codes
under scales of 1), so with inputs of -1, 0 and 1 every sum of some of the products, in whatever order, is a multiple of 1/2 of at
most 6 k = 3.2 million: 23 bits, exact in 32-bit sums. Tokens whose inputs are powers of two have two of them, with sums of 17
bits. What is compared is therefore rounded once, on both sides alike. That a mistake shows is looked at, too: with a group of
inputs left out the oracle's own results differ.
"""
import numpy as np
import pytest
import torch

from oracle import w4 as ow

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
# by the number of tokens: inputs of more than eight CTAs' shared memory. 16 (1 or 2 tokens), 32 (3 or 4) or 64 rows are a block,
# and 19 clusters run at once: the first, second and fourth sizes have more blocks than that.
SIZES = [(1, 330, 391968), (2, 340, 194656), (3, 45, 129120), (4, 690, 97024), (5, 70, 77952), (6, 100, 63520), (7, 90, 55424), (8, 650, 47136),
         (1, 37, 524384), (2, 20, 524384), (4, 90, 262240), (8, 30, 524384)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_lt_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def codes_of(n, k, seed):
    return torch.randint(0, 256, (n, k // 2), generator=torch.Generator().manual_seed(seed), dtype=torch.uint8), torch.ones(n, k // 32, dtype=torch.float16)


def exact(x, codes, scales):
    """x W^T, some rows at a time."""
    x = x.double().numpy()
    return np.concatenate([ow.linear(x, codes[i:i + 64].numpy(), scales[i:i + 64].double().numpy())[0] for i in range(0, codes.shape[0], 64)], 1)


def columns(codes, at):
    """The weights [n, len(at)] of inputs."""
    n, at = codes.shape[0], np.asarray(at)
    groups = codes.numpy().reshape(n, -1, 16)[:, at // 32].reshape(n, -1)
    return ow.weights(groups, np.ones((n, len(at)))).reshape(n, len(at), 32)[:, np.arange(len(at)), at % 32]


def rounded(y, dtype):
    return torch.as_tensor(y).float().to(dtype)  # (exact in float32)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,n,k", SIZES)
def test_dense_inputs(tokens, n, k, dtype):
    import sparse_attention_indexer_lt_gb300 as lt
    t = TYPES[dtype]
    codes, scales = codes_of(n, k, seed=k)
    x = (torch.randint(0, 3, (tokens, k), generator=torch.Generator().manual_seed(n)) - 1).to(t)
    want = exact(x, codes, scales)
    y = lt.w4_linear(x.cuda(), codes.cuda(), scales.cuda())
    assert torch.equal(y.cpu(), rounded(want, t))
    # a group of 32 inputs less, at the start, in the middle or at the end, is another result
    for g in (0, k // 64, k // 32 - 1):
        at = slice(g * 32, g * 32 + 32)
        part = x[:, at].double().numpy() @ ow.weights(codes[:, g * 16:g * 16 + 16].numpy(), scales[:, g:g + 1].double().numpy()).T
        assert not torch.equal(rounded(want - part, t), rounded(want, t))


@pytest.mark.parametrize("tokens,n,k", SIZES)
def test_inputs_at_the_borders_of_steps(tokens, n, k):
    """The first and last input of every 256 and of every 32 of some, a dozen a token: a result then is a sum of 12 weights."""
    import sparse_attention_indexer_lt_gb300 as lt
    n = min(n, 64)
    codes, scales = codes_of(n, k, seed=k + 1)
    device = codes.cuda(), scales.cuda()
    gen = torch.Generator().manual_seed(tokens)
    at = torch.arange(0, k, 256)
    at = torch.cat([at, torch.clamp(at + 255, max=k - 1), torch.randint(0, k // 32, (600,), generator=gen) * 32 + 31 * torch.randint(0, 2, (600,), generator=gen)])
    at = at[torch.randperm(len(at), generator=gen)]
    at = torch.cat([at, at[:-len(at) % (12 * tokens)]]).view(-1, tokens, 12)  # [call][token][input]
    sign = 1.0 - 2.0 * torch.randint(0, 2, at.shape, generator=gen)
    w = torch.as_tensor(columns(codes, at.flatten()))
    for i in range(at.shape[0]):
        x = torch.zeros(tokens, k)
        x.scatter_add_(1, at[i], sign[i])
        here = w[:, i * 12 * tokens:(i + 1) * 12 * tokens].view(n, tokens, 12)
        want = (here * sign[i][None].double()).sum(2).T
        assert torch.equal(lt.w4_linear(x.half().cuda(), *device).cpu(), rounded(want, torch.float16)), f"call {i}"


@pytest.mark.parametrize("tokens,n,k", SIZES)
def test_powers_of_two_along_the_inputs(tokens, n, k):
    """bf16 tokens are held as fp16 times a power of two, which goes down as larger inputs come: a small input and a large one somewhere
    before or behind it, or nothing before the last inputs. Half of the weights are zeros, so that the small input shows where
    the large one's weight is one."""
    import sparse_attention_indexer_lt_gb300 as lt
    codes, scales = codes_of(n, k, seed=k + 2)
    gen = torch.Generator().manual_seed(n + tokens)
    codes &= torch.tensor([0x00, 0x0F, 0xF0, 0xFF], dtype=torch.uint8)[torch.randint(0, 4, codes.shape, generator=gen)]
    device = codes.cuda(), scales.cuda()
    for turn in range(16):
        at = torch.sort(torch.randint(0, k // 2, (tokens, 2), generator=gen) * 2 + torch.tensor([0, 1]))[0]
        e = torch.randint(1, 12, (tokens, 1), generator=gen) * torch.tensor([-0.5, 0.5])
        for t in range(tokens):
            if (turn + t) % 4 == 1:
                e[t] = e[t].flip(0)
            elif (turn + t) % 4 == 2:
                at[t, 0] = turn
                at[t, 1] = k - 1 - t
            elif (turn + t) % 4 == 3:
                at[t] = k - 2 + torch.arange(2)
        value = 2.0 ** e.floor() * (1.0 - 2.0 * torch.randint(0, 2, e.shape, generator=gen))
        x = torch.zeros(tokens, k).scatter_(1, at, value).bfloat16()
        y = lt.w4_linear(x.cuda(), *device).cpu()
        for t in range(tokens):
            parts = columns(codes, at[t]) * value[t].double().numpy()
            want = rounded(parts.sum(1), torch.bfloat16)
            assert torch.equal(y[t], want), (turn, t)
            for c in range(2):  # each input alone makes a difference
                assert not torch.equal(rounded(parts[:, 1 - c], torch.bfloat16), want)
