"""GPU parity of the products with 4-bit weights against the 64-bit oracle.

Codes and scales are exact: they have to be equal. A product x * (code * scale) is exact in the
tensor core's sums for scales of 9 significant bits; a result adds k of them in fp32. Sums on the tensor core may be
cut instead of rounded: a unit 2^-23 an addition, of partial sums no larger than size = sum |x w|. With a few
additions more for the parts' join and the bias,

    |y - ref| <= (k + 16) 2^-23 size + u (|ref| + |bias|)

where u is the output's rounding: 2^-8 (bf16), 2^-11 (fp16; and 2^-25 where that is subnormal). bf16 inputs
below 2^-28 of their token's largest add 2^-39 of it for each weight. Inputs of one bit and whole weights make every sum
exact: such results are equal.
"""
import numpy as np
import pytest
import torch

from oracle import w4 as ow

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_lt_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def num(t):
    return t.detach().cpu().double().numpy()


def make(n, k, seed=0, size=0.1):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    s = size * torch.exp(0.3 * torch.randn(n, k // 32, generator=g))
    return codes, (s.half().view(torch.int16) & -4).view(torch.float16)


def check(y, x, codes, scales, bias=None):
    want, size = ow.linear(num(x), codes.cpu().numpy(), num(scales), None if bias is None else num(bias))
    k = x.shape[1]
    u = 2.0 ** -8 if y.dtype == torch.bfloat16 else 2.0 ** -11
    tiny = np.abs(num(x)).max(1, keepdims=True) * 2.0 ** -39 * np.abs(ow.weights(codes.cpu().numpy(), num(scales))).sum(1)[None]
    tol = (k + 16) * 2.0 ** -23 * size + u * (np.abs(want) + (0 if bias is None else np.abs(num(bias)))) + tiny + (2.0 ** -25 if y.dtype == torch.float16 else 2.0 ** -134)
    got = num(y)
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= tol).all(), f"{int((err > tol).sum())} off, worst {float((err / tol).max()):.3g} of its bound"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,k", [(1, 32), (3, 96), (17, 1056), (5, 8224)])
def test_quantise(n, k, dtype):
    import sparse_attention_indexer_lt_gb300 as lt
    torch.manual_seed(n + k)
    w = torch.randn(n, k) * 10.0 ** torch.randint(-7, 4, (n, k // 32, 1)).expand(n, k // 32, 32).reshape(n, k)
    w[0, :32] = 0.0
    w[-1, -1] = float("nan")
    w[n // 2, k // 2] = -float("inf")
    for extra in (0, 1):
        flat = torch.zeros(n, k + 9, dtype=TYPES[dtype])
        flat[:, extra:k + extra] = w.to(TYPES[dtype])
        view = flat.cuda()[:, extra:k + extra]
        codes, scales = lt.w4_quantise(view)
        want_codes, want_scales = ow.quantise(num(view))
        assert np.array_equal(codes.cpu().numpy(), want_codes)
        assert np.array_equal(scales.cpu().numpy(), want_scales, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,k", [(1, 32), (15, 64), (16, 128), (129, 160), (257, 1056), (1000, 2080), (40, 16384)])
@pytest.mark.parametrize("tokens", [1, 2, 3, 5, 8, 9, 16, 17, 33])
def test_linear(tokens, n, k, dtype):
    import sparse_attention_indexer_lt_gb300 as lt
    codes, scales = make(n, k, seed=n + k)
    torch.manual_seed(tokens + n)
    x = (torch.randn(tokens, k) * 10.0 ** torch.randint(-3, 2, (tokens, 1))).to(TYPES[dtype])
    bias = torch.randn(n).to(TYPES[dtype]) if n % 2 else None
    y = lt.w4_linear(x.cuda(), codes.cuda(), scales.cuda(), bias=None if bias is None else bias.cuda())
    check(y, x, codes, scales, bias)
    again = lt.w4_linear(x.cuda(), codes.cuda(), scales.cuda(), bias=None if bias is None else bias.cuda())
    assert torch.equal(y, again), "two runs differ"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,n,k", [(64, 200, 512), (100, 130, 4096), (256, 128, 96), (257, 300, 1056), (515, 1, 2048), (700, 144, 64)])
def test_many_tokens(tokens, n, k, dtype):
    import sparse_attention_indexer_lt_gb300 as lt
    codes, scales = make(n, k, seed=tokens)
    torch.manual_seed(tokens)
    x = torch.randn(tokens, k).to(TYPES[dtype])
    bias = torch.randn(n).to(TYPES[dtype])
    y = lt.w4_linear(x.cuda(), codes.cuda(), scales.cuda(), bias=bias.cuda())
    check(y, x, codes, scales, bias)
    assert torch.equal(y, lt.w4_linear(x.cuda(), codes.cuda(), scales.cuda(), bias=bias.cuda())), "two runs differ"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,n,k", [(1, 300, 8192), (7, 77, 992), (12, 130, 2048), (40, 333, 512), (130, 129, 288)])
def test_sums_that_are_exact_are_equal(tokens, n, k, dtype):
    """Inputs of -1, 0 and 1 and weights that are multiples of 1/2: every partial sum is a multiple of 1/2 below 2^18,
    and small outputs have no rounding either: any mistake of place shows."""
    import sparse_attention_indexer_lt_gb300 as lt
    g = torch.Generator().manual_seed(tokens)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    scales = 2.0 ** torch.randint(0, 2, (n, k // 32), generator=g).half()
    x = torch.zeros(tokens, k)
    for t in range(tokens):  # a few inputs each, the last ones among them
        at = torch.randperm(k, generator=g)[:9]
        x[t, at] = torch.where(torch.rand(9, generator=g) < 0.5, -1.0, 1.0)
        x[t, k - 1 - t % 32] = 1.0
    x = x.to(TYPES[dtype])
    want, _ = ow.linear(num(x), codes.numpy(), num(scales))
    y = lt.w4_linear(x.cuda(), codes.cuda(), scales.cuda())
    assert np.array_equal(num(y), num(torch.as_tensor(want).to(TYPES[dtype])))


@pytest.mark.parametrize("tokens", [1, 6, 20, 90])
def test_extremes(tokens):
    """Tokens of very large and very small inputs beside each other, zeros, infinities and NaN: each in its own outputs."""
    import sparse_attention_indexer_lt_gb300 as lt
    n, k = 70, 4160
    codes, scales = make(n, k, seed=tokens)
    torch.manual_seed(tokens)
    x = torch.randn(tokens, k)
    x *= 2.0 ** torch.tensor([[-120.0, 100.0, 0.0, -60.0, 30.0][t % 5] for t in range(tokens)]).unsqueeze(1)
    x = x.bfloat16()
    if tokens > 4:
        x[2] = 0.0
        x[3, :k // 2] *= 2.0 ** -20  # small inputs first, then large ones
    clean = lt.w4_linear(x.cuda(), codes.cuda(), scales.cuda())
    check(clean, x, codes, scales)
    if tokens > 4:
        assert not clean[2].any()
        x[0, 5], x[4, k - 1] = float("inf"), float("nan")
        y = lt.w4_linear(x.cuda(), codes.cuda(), scales.cuda())
        w = torch.as_tensor(ow.weights(codes.numpy(), num(scales)))
        up = torch.where(w[:, 5] == 0, float("nan"), w[:, 5] * float("inf"))
        assert torch.equal(torch.nan_to_num(y[0].cpu().double(), 7.0, 8.0, 9.0), torch.nan_to_num(up, 7.0, 8.0, 9.0))
        assert torch.isnan(y[4]).all()
        others = [t for t in range(tokens) if t not in (0, 4)]
        assert torch.equal(y[others], clean[others])


@pytest.mark.parametrize("tokens", [1, 2, 4, 5])
def test_inputs_beyond_shared_memory(tokens):
    """More inputs than a CTA holds at a time, a cluster's share of them among it: in chunks, whose powers of two go
    down as larger inputs come."""
    import sparse_attention_indexer_lt_gb300 as lt
    n, k = 37, 524288 + 96
    codes, scales = make(n, k, seed=tokens, size=0.01)
    torch.manual_seed(tokens)
    x = (torch.randn(tokens, k) * 2.0 ** torch.linspace(-12, 6, k)).bfloat16()
    y = lt.w4_linear(x.cuda(), codes.cuda(), scales.cuda())
    check(y, x, codes, scales)
    assert torch.equal(y, lt.w4_linear(x.cuda(), codes.cuda(), scales.cuda()))


@pytest.mark.parametrize("tokens,n,k", [(3, 4096, 8192), (4, 5000, 8192), (2, 9000, 64), (1, 30000, 256)])
def test_many_row_blocks(tokens, n, k):
    """More row blocks than CTAs that stay, on both sides of the choice of kernel."""
    import sparse_attention_indexer_lt_gb300 as lt
    codes, scales = make(n, k, seed=n)
    torch.manual_seed(n)
    x = torch.randn(tokens, k).half()
    y = lt.w4_linear(x.cuda(), codes.cuda(), scales.cuda())
    check(y, x, codes, scales)


@pytest.mark.parametrize("tokens", [1, 6, 40, 200])
def test_strides_and_what_lies_around_the_output(tokens):
    import sparse_attention_indexer_lt_gb300 as lt
    n, k = 45, 256
    codes, scales = (t.cuda() for t in make(n, k, seed=3))
    torch.manual_seed(1)
    wide = torch.randn(tokens, 3 * k, device="cuda").half()
    x = wide[:, k:2 * k]
    out = torch.full((tokens, n + 6), 3.0, device="cuda").half()
    got = lt.w4_linear(x, codes, scales, out=out[:, 2:2 + n])
    assert got.data_ptr() == out[:, 2:].data_ptr()
    assert torch.equal(out[:, 2:2 + n], lt.w4_linear(x.contiguous(), codes, scales))
    assert (out[:, :2] == 3.0).all() and (out[:, 2 + n:] == 3.0).all()
    check(out[:, 2:2 + n], x, codes, scales)


@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_streams_graphs_and_workspaces(tokens):
    import sparse_attention_indexer_lt_gb300 as lt
    n, k = 300, 1024
    codes, scales = (t.cuda() for t in make(n, k, seed=5))
    torch.manual_seed(2)
    x = torch.randn(tokens, k, device="cuda").bfloat16()
    want = lt.w4_linear(x, codes, scales)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lt.w4_linear(x, codes, scales, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    from sparse_attention_indexer_lt_gb300 import w4
    need = w4._workspace_bytes(0, tokens, n, k)
    space = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    assert torch.equal(lt.w4_linear(x, codes, scales, workspace=space), want)
    assert (space[need:] == 0x5A).all()
    if need:
        with pytest.raises(ValueError):
            lt.w4_linear(x, codes, scales, workspace=space[:need - 1])
    graphs, outs = [], []
    for _ in range(2):  # two graphs, their own scratch memory each
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(lt.w4_linear(x, codes, scales))
        graphs.append(g)
    x.normal_()
    for g in graphs:
        g.replay()
    want = lt.w4_linear(x, codes, scales)
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


@pytest.mark.parametrize("tokens,n,k", [(64, 8192, 10240), (509, 4096, 4096), (200, 2048, 8192), (16, 6144, 8192), (1, 8192, 10240),
                                        (8, 4096, 8192), (3, 4099, 5152)])
def test_weights_from_memory_and_from_the_cache(tokens, n, k):
    """A result does not go by how fast its weights come: as they are, and after a write of more than the L2 cache."""
    import sparse_attention_indexer_lt_gb300 as lt
    codes, scales = (t.cuda() for t in make(n, k, seed=n + k))
    x = torch.randn(tokens, k, generator=torch.Generator().manual_seed(tokens)).half().cuda()
    want = lt.w4_linear(x, codes, scales)
    check(want[:, :300], x, codes[:300].contiguous(), scales[:300].contiguous())
    flush, got = torch.empty(200 << 20, dtype=torch.uint8, device="cuda"), []
    for i in range(40):
        flush.fill_(i)
        got.append(lt.w4_linear(x, codes, scales))
    off = [i for i, y in enumerate(got) if not torch.equal(y, want)]
    assert not off, f"calls {off}"


def test_calls_of_all_kinds_at_once():
    # CTAs alone on their SMs and beside each other, in clusters and not, on four streams: each call has its own answer
    import sparse_attention_indexer_lt_gb300 as lt
    sizes = [(64, 8192, 4096), (16, 2048, 8192), (509, 1024, 4096), (128, 512, 8192), (5, 4096, 1024), (64, 8192, 10240)]
    calls = []
    for i, (tokens, n, k) in enumerate(sizes):
        codes, scales = lt.w4_quantise(torch.randn(n, k, device="cuda", generator=torch.Generator("cuda").manual_seed(i)) * 0.1)
        x = torch.randn(tokens, k, device="cuda", generator=torch.Generator("cuda").manual_seed(50 + i)).to(torch.float16)
        calls.append((x, codes, scales, lt.w4_linear(x, codes, scales)))
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for turn in range(60):
        for i, s in enumerate(streams):
            which = (turn + i * (1 + turn // 6)) % len(calls)
            x, codes, scales, _ = calls[which]
            got.append((which, lt.w4_linear(x, codes, scales, stream=s)))
    torch.cuda.synchronize()
    for which, y in got:
        assert torch.equal(y, calls[which][3]), which


def test_one_token_has_any_stride():
    import sparse_attention_indexer_lt_gb300 as lt
    codes, scales = (t.cuda() for t in make(40, 64))
    x = torch.randn(64, 1, generator=torch.Generator().manual_seed(0)).half().cuda().t()
    assert x.shape == (1, 64) and x.stride(0) == 1
    check(lt.w4_linear(x, codes, scales), x, codes, scales)


def test_weights_beyond_32_bit_offsets():
    """More than 2^32 bytes of codes, and a last row that is right."""
    import sparse_attention_indexer_lt_gb300 as lt
    n, k = 600000, 16384  # 4.9 GB of codes
    codes = torch.zeros(n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.ones(n, k // 32, dtype=torch.float16, device="cuda")
    few, fs = (t.cuda() for t in make(3, k, seed=1))
    codes[-3:], scales[-3:] = few, fs
    for tokens in (1, 20):
        x = torch.randn(tokens, k, device="cuda").half()
        y = lt.w4_linear(x, codes, scales)
        check(y[:, -3:], x, few, fs)
        assert not y[:, :-3].any()


def test_an_injected_launch_failure_writes_nothing():
    import sparse_attention_indexer_lt_gb300 as lt
    codes, scales = (t.cuda() for t in make(20, 64))
    x = torch.ones(2, 64, device="cuda").half()
    out = torch.full((2, 20), 3.0, device="cuda").half()
    lt.load().lt_test_inject(1, 1)
    with pytest.raises(lt.LtError):
        lt.w4_linear(x, codes, scales, out=out)
    assert (out == 3.0).all()
    lt.w4_linear(x, codes, scales, out=out)
    check(out, x, codes, scales)
    lt.load().lt_test_inject(1, 1)
    with pytest.raises(lt.LtError):
        lt.w4_quantise(x)


def test_nothing_and_refusals():
    import sparse_attention_indexer_lt_gb300 as lt
    codes, scales = (t.cuda() for t in make(20, 64))
    x = torch.ones(2, 64, device="cuda").half()
    assert lt.w4_linear(x[:0], codes, scales).shape == (0, 20)
    assert lt.w4_linear(x, codes[:0], scales[:0]).shape == (2, 0)
    assert lt.w4_quantise(x[:0])[0].shape == (0, 32)
    for bad in (dict(x=x.float()), dict(x=x[:, :32]), dict(x=x[0]), dict(x=torch.ones(2, 128, device="cuda").half()[:, ::2]),
                dict(x=torch.ones(2, 72, device="cuda").half()[:, 4:68]), dict(codes=codes.int()), dict(codes=codes[:, :16]),
                dict(scales=scales.float()), dict(scales=scales[:10]), dict(codes=codes.cpu()), dict(bias=torch.ones(20, device="cuda")),
                dict(bias=torch.ones(19, device="cuda").half()), dict(out=torch.ones(2, 21, device="cuda").half()),
                dict(out=torch.ones(20, 2, device="cuda").half().T), dict(out=torch.ones(2, 20, device="cuda").bfloat16())):
        args = {"x": x, "codes": codes, "scales": scales, **bad}
        with pytest.raises((TypeError, ValueError)):
            lt.w4_linear(args.pop("x"), args.pop("codes"), args.pop("scales"), **args)
    for bad in (x[:, :40], x.double(), x[0], torch.ones(64, 64, device="cuda").T[:, ::2]):
        with pytest.raises((TypeError, ValueError)):
            lt.w4_quantise(bad)
