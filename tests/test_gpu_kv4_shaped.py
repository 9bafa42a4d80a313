"""GPU parity of caps, slopes and prefixes in the 4-bit cache's attention against the 64-bit oracle.

The bound is that of the plain attention (a logit off by (D + 8) eps reach, eps = 2^-24, and what follows from
it), with what shaping adds to a logit: a capped logit is off by 2^-22 of a cap up to 64 and by 2^-20 of itself with
larger ones (a hyperbolic tangent's slope is at most 1, so that errors before it do not grow); a
slope's term is rounded twice and carries the rounding of the slope's factor, 4 eps of the term; and the sum once, eps of the
largest part. Logits then lie anywhere below the row's largest, so eps |logit| is bounded by eps times the largest
magnitudes among the visible: cap or reach, and slope * distance. fp16 numbers below 2^-14 are multiples of 2^-24, so
that the output's rounding is 2^-25 there, whatever the output (one position with nearly all the weight and a value of zero
leaves outputs of 2^-25 and less).
"""
import numpy as np
import pytest
import torch

from oracle import kv4 as ok
from test_gpu_kv4 import EPS, Problem, num

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_lt_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def check(p, window=0, scale=None, softcap=0.0, slopes=None, prefix=None, **kw):
    pre = None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device="cuda")
    slo = None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda")
    out, lse = p.run(window=window, scale=scale, softcap=softcap, slopes=slo, prefix=pre, **kw)
    s32 = None if slopes is None else np.asarray(slopes, np.float32).astype(np.float64)
    want, want_lse, size, reach = ok.attention(num(p.q), p.rows_at, p.lengths, p.starts, p.heads, p.dim ** -0.5 if scale is None else scale,
                                               window, p.positions, softcap, s32, prefix)
    n = max(p.lengths + [1]) if p.positions is None else np.shape(p.positions)[1]
    held = [p.rows_at(r, h, x) for r, n_r in enumerate(p.lengths) for h in range(p.heads) for x in range(n_r)]
    vmax = max([float(np.abs(x[1]).max()) for x in held if x is not None] + [0.0])
    far = 0.0 if slopes is None else np.abs(s32)[None] * (max(p.lengths + [1]) + max(p.starts))
    top = reach + far if not softcap else np.minimum(reach, softcap) + far
    d = (p.dim + 8) * EPS * reach + 5 * EPS * far + EPS * top + EPS * np.where(np.isfinite(want_lse), np.abs(want_lse), 0) + 2.0 ** -21
    if softcap:
        d = d + (2.0 ** -22 * softcap if softcap <= 64 else 2.0 ** -20 * np.minimum(reach, softcap))
    u = 2.0 ** -8 if p.q.dtype == torch.bfloat16 else 2.0 ** -11
    tol = size * (2 * d[..., None] + 2.0 ** -11 + 2 * n * EPS) + n * 2.0 ** -33 * vmax + u * np.abs(want)
    if p.q.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    got = num(out)
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= tol).all(), f"out: {int((err > tol).sum())} off, worst {float((err / tol).max()):.3g} of its bound"
    got = num(lse)
    empty = np.isinf(want_lse)
    assert np.array_equal(np.isinf(got) & (got < 0), empty) and not num(out)[empty].any()
    err = np.abs(got[~empty] - want_lse[~empty])
    tol = (d + n * EPS + 2.0 ** -21 * (1 + np.abs(np.where(empty, 0, want_lse))))[~empty]
    assert (err <= tol).all(), f"lse: worst {float((err / tol).max()):.3g} of its bound"
    return out, lse


def slopes_of(heads):
    return [2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)]


SHAPES = [dict(softcap=2.0), dict(softcap=50.0), dict(softcap=300.0), dict(slopes=True), dict(softcap=5.0, slopes=True)]


def shape_of(kw, heads):
    return {**kw, "slopes": slopes_of(heads)} if kw.get("slopes") else kw


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,heads,group", [(64, 2, 1), (64, 1, 3), (128, 2, 4), (128, 1, 16), (128, 1, 33), (256, 1, 8), (256, 1, 20)])
@pytest.mark.parametrize("kw", SHAPES)
def test_decode(dim, heads, group, dtype, kw):
    p = Problem([1, 2, 31, 32, 33, 63, 64, 65, 200], [1] * 9, heads, group, dim, 16, dtype, seed=dim + group, spread=4.0)
    check(p, **shape_of(kw, heads * group))


@pytest.mark.parametrize("dim,window", [(128, 0), (128, 1), (64, 5), (64, 100), (256, 32)])
@pytest.mark.parametrize("kw", SHAPES)
def test_ragged_queries_and_windows(dim, window, kw):
    p = Problem([0, 5, 40, 130, 3, 70, 0], [1, 5, 0, 9, 6, 1, 0], 2, 3, dim, 8, "bf16", seed=window, extra_width=3, spread=3.0)
    check(p, window=window, **shape_of(kw, 6))


@pytest.mark.parametrize("page", [1, 16, 128])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=5.0), dict(slopes=True), dict(softcap=500.0, slopes=True)])
@pytest.mark.parametrize("dim,lengths,new,group", [(64, [5, 40, 130, 3, 70, 0], [5, 2, 9, 6, 1, 0], 3), (128, [200, 64, 300], [4, 4, 1], 4),
                                                   (256, [33, 90], [3, 1], 8)])
def test_prefixes_of_few_rows(dim, lengths, new, group, kw, page):
    """Prefixes of nothing, of less and of more than a query's position, past the request's end, below zero."""
    n = len(lengths)
    p = Problem(lengths, new, 2, group, dim, page, "f16", seed=dim + page, extra_width=1, spread=2.0)
    for prefix in ([0] * n, [x // 2 for x in lengths], lengths, [2 ** 31 - 1] * n, [-3] * n, [x - 2 for x in lengths]):
        check(p, prefix=prefix, **shape_of(kw, 2 * group))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kw", SHAPES)
@pytest.mark.parametrize("dim,lengths,new,group,window", [
    (64, [64], [64], 1, 0), (128, [300], [129], 1, 0), (128, [129, 5, 400], [70, 0, 33], 5, 0), (64, [700, 90, 1], [100, 90, 1], 3, 50),
    (128, [640], [90], 3, 200), (64, [1500], [40], 4, 0), (128, [50], [80], 4, 0), (256, [300, 0, 5, 33], [129, 70, 0, 33], 1, 0),
    (256, [700, 64], [40, 17], 4, 150), (256, [1300], [33], 2, 0)])
def test_prefill(dim, lengths, new, group, window, kw, dtype):
    p = Problem(lengths, new, 2, group, dim, 16, dtype, seed=sum(lengths) + dim, extra_width=1, spread=4.0)
    kw = shape_of(kw, 2 * group)
    out, _ = check(p, window=window, **kw)
    assert torch.equal(out, check(p, window=window, **kw)[0]), "two runs differ"


@pytest.mark.parametrize("kw", [dict(), dict(softcap=5.0), dict(slopes=True)])
@pytest.mark.parametrize("dim,lengths,new,group", [(64, [130, 90], [100, 90], 2), (128, [300, 33], [129, 33], 1), (128, [50], [80], 4),
                                                   (256, [300, 64], [129, 60], 1), (64, [1500], [40], 4)])
def test_prefixes_of_many_rows(dim, lengths, new, group, kw):
    n = len(lengths)
    p = Problem(lengths, new, 2, group, dim, 16, "bf16", seed=dim, extra_width=1, spread=2.0)
    for prefix in ([x - y // 2 for x, y in zip(lengths, new)], lengths, [2 ** 31 - 1] * n, [-1] * n, [7] * n):
        check(p, prefix=prefix, **shape_of(kw, 2 * group))


@pytest.mark.parametrize("kw", SHAPES)
@pytest.mark.parametrize("dim,heads,group,list_len", [(64, 2, 4, 1), (128, 1, 16, 33), (128, 2, 8, 512), (256, 1, 4, 100), (128, 1, 40, 130)])
def test_listed(dim, heads, group, list_len, kw):
    rng = np.random.default_rng(list_len)
    lengths, new = [400, 1, 90, 0], [3, 1, 2, 1]
    pos = np.full((sum(new), list_len), -1)
    t = 0
    for n, c in zip(lengths, new):
        for i in range(c):
            pos[t] = rng.integers(-3, n + 9, list_len) if i != 1 else -1  # pads, positions past the end, repeats; an empty list
            t += 1
    p = Problem(lengths, new, heads, group, dim, 16, "bf16", seed=list_len, positions=pos, spread=3.0)
    check(p, **shape_of(kw, heads * group))


@pytest.mark.parametrize("lengths,new", [([20000], [1]), ([17000, 3, 0, 9000], [2, 1, 1, 0]), ([300] * 40 + [17001], [1] * 41)])
def test_long_tables_are_cut_into_chunks(lengths, new):
    p = Problem(lengths, new, 1, 2, 64, 64, "bf16", seed=len(lengths))
    check(p, softcap=20.0, slopes=[0.01, 0.0001])
    check(p, prefix=[x // 3 for x in lengths])


@pytest.mark.parametrize("spread,magnitude,scale,softcap,slopes", [
    (30.0, 1.0, None, 30.0, None), (1.0, 1.0, -0.2, 1.0, [0.1, 0.2, 0.3, 0.4]), (1.0, 1.0, 0.0, 10.0, None), (1.0, 1e-4, 300.0, 2.0 ** -10, None),
    (1.0, 3000.0, 1e-4, 2.0 ** 20, None), (1.0, 1.0, None, 1e4, [0.0, -0.01, 5.0, 1e-6]), (1.0, 1.0, None, 64.0, [3.0, 0.5, 0.0, 1e30])])
@pytest.mark.parametrize("new", [1, 40])
def test_scales_caps_and_bad_pages(new, spread, magnitude, scale, softcap, slopes):
    p = Problem([300], [new], 1, 4, 64, 16, "bf16", seed=21, spread=spread, magnitude=magnitude)
    p.table[0, 3] = -1
    p.table[0, 17] = 2 ** 31 - 1
    if slopes is not None and max(slopes) > 100:
        slopes = slopes[:3] + [100.0]
    check(p, scale=scale, softcap=softcap, slopes=slopes)


@pytest.mark.parametrize("dim,new", [(128, 3), (64, 80), (256, 80)])
def test_nan_where_nothing_looks(dim, new):
    """Hidden keys, values and scales that are no numbers have no effect, with caps, slopes and a prefix."""
    p = Problem([200], [new], 1, 2, dim, 16, "bf16", seed=22)
    slopes = torch.tensor([0.1, 0.01], device="cuda")
    kw = dict(softcap=3.0, slopes=slopes, prefix=torch.tensor([150], dtype=torch.int32, device="cuda"))
    clean, clean_lse = p.run(**kw)
    nan = torch.tensor([0x7FFF], dtype=torch.int16).view(torch.uint8)
    for byte in range(dim, dim + dim // 8, 2):
        p.cache[p.table[0, 199 // 16], 0, 199 % 16, byte:byte + 2] = nan
    out, lse = p.run(**kw)
    assert torch.equal(out[:-1], clean[:-1]) and torch.equal(lse[:-1], clean_lse[:-1])
    assert torch.isnan(out[-1]).all()


@pytest.mark.parametrize("new", [3, 70])
@pytest.mark.parametrize("slope", [4.0, 30.0, 1e5, -2.0])
def test_steep_slopes(new, slope):
    """The nearest positions keep their logits whatever the far ones' terms are: with a steep slope a query sees itself (with
    a steep one of the other sign, the first position), and `lse` is that logit."""
    p = Problem([260], [new], 1, 2, 64, 16, "f16", seed=3)
    out, lse = p.run(slopes=torch.full((2,), slope, device="cuda"))
    for i in (0, new - 1):
        own = 260 - new + i
        for h in range(2):
            q = num(p.q)[i, h]
            k, v = (np.stack([p.rows_at(0, 0, x)[j] for x in range(own + 1)]) for j in (0, 1))
            s = k @ q / 8.0 - slope * np.abs(own - np.arange(own + 1))
            want = s.max() + np.log(np.exp(s - s.max()).sum())
            w = np.exp(s - want)
            # 64-term sums and a few roundings of the logit, of the slope's term at the largest term's distance, and of the result
            far = abs(slope) * (0 if slope > 0 else own)
            assert abs(num(lse)[i, h] - want) <= 80 * EPS * np.abs(k * q).sum(1).max() / 8 + 8 * EPS * far + 70 * EPS * min(abs(slope), 4.0) + 2.0 ** -20 + 4 * EPS * abs(want)
            assert np.abs(num(out)[i, h] - w @ v).max() <= 2.0 ** -9 * (w @ np.abs(v)).max() + 2.0 ** -9 * np.abs(v).max() * 2.0 ** -6


def test_nan_queries():
    """A NaN query gives NaN, in its own row, whatever the cap makes of its logits."""
    p = Problem([70], [40], 1, 1, 64, 16, "bf16", seed=5)
    for rows in (1, 40):
        q = p.q[-rows:].clone().cuda()
        table, lengths = p.table.cuda(), torch.tensor([70], dtype=torch.int32, device="cuda")
        starts = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        import sparse_attention_indexer_lt_gb300 as lt
        call = lambda x: lt.kv4_attention(x, p.cache.cuda(), table, lengths, starts=starts, max_new=rows, softcap=5.0)  # noqa: E731
        clean = call(q)
        q[-1, 0, 3] = float("nan")
        out = call(q)
        assert torch.isnan(out[-1]).all() and torch.equal(out[:-1], clean[:-1])


def test_plain_calls_and_shapes_that_change_nothing():
    """Slopes of zero and a prefix of nothing give what the plain call gives, up to the order of roundings."""
    for new in (1, 60):
        p = Problem([300, 80], [new, new], 2, 2, 128, 16, "f16", seed=9)
        out, lse = p.run()
        for kw in (dict(slopes=torch.zeros(4, device="cuda")), dict(prefix=torch.zeros(2, dtype=torch.int32, device="cuda"))):
            got, got_lse = p.run(**kw)
            assert (got - out).abs().max() <= 2.0 ** -10 * out.abs().max() and (got_lse - lse).abs().max() <= 1e-5


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page_size", [1, 16, 128])
@pytest.mark.parametrize("new", [1, 4, 8, 300])
def test_rows_from_memory_and_from_the_cache(dim, page_size, new):
    """A result does not go by how fast the rows come: as they are, and after a write of more than the L2 cache."""
    import sparse_attention_indexer_lt_gb300 as lt
    requests, width, heads, group = 20, 2048 // page_size, 4, 4
    gen = torch.Generator("cuda").manual_seed(dim + new)
    cache = lt.kv4_cache(requests * width, heads, page_size, dim)
    k, v = (torch.randn(requests * 2048, heads, dim, device="cuda", generator=gen).half() for _ in range(2))
    lt.kv4_store(k, v, cache, torch.arange(requests * 2048, device="cuda"))
    table = torch.randperm(requests * width, device="cuda", generator=gen).int().view(requests, width)
    lengths = torch.randint(new, 2048, (requests,), device="cuda", generator=gen).int()
    starts = torch.arange(requests + 1, device="cuda").int() * new
    q = torch.randn(requests * new, heads * group, dim, device="cuda", generator=gen).bfloat16()
    slopes = torch.tensor(slopes_of(heads * group), device="cuda")
    flush = torch.empty(200 << 20, dtype=torch.uint8, device="cuda")
    ways = [{}, dict(softcap=20.0, prefix=lengths // 3), dict(slopes=slopes, window=900)]
    if new < 300:
        ways.append(dict(slopes=slopes, positions=torch.randint(0, new, (requests * new, 500), device="cuda", generator=gen).int()))
    for kw in ways:
        call = lambda: lt.kv4_attention(q, cache, table, lengths, starts=starts, max_new=new, **kw)  # noqa: E731
        want, got = call(), []
        for i in range(15):
            flush.fill_(i)
            got.append(call())
        assert all(torch.equal(y, want) for y in got), kw


def test_graphs_and_streams():
    p = Problem([300, 80], [2, 1], 2, 2, 128, 16, "bf16", seed=9)
    import sparse_attention_indexer_lt_gb300 as lt
    q, cache, table = p.q.cuda(), p.cache.cuda(), p.table.cuda()
    lengths, starts = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (p.lengths, p.starts))
    slopes, prefix = torch.tensor(slopes_of(4), device="cuda"), torch.tensor([300, 0], dtype=torch.int32, device="cuda")
    call = lambda **kw: lt.kv4_attention(q, cache, table, lengths, starts=starts, max_new=2, softcap=9.0, slopes=slopes, prefix=prefix, **kw)  # noqa: E731
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    slopes *= 2.0
    prefix -= 150
    q.normal_()
    graph.replay()
    assert torch.equal(out, call()) and not torch.equal(out, want)


def test_binding_refuses():
    p = Problem([30], [1], 1, 2, 64, 16, "bf16", seed=1)
    one, two = torch.ones(1, dtype=torch.int32, device="cuda"), torch.ones(2, device="cuda")
    for bad in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=1e9), dict(softcap=1e-9), dict(slopes=two[:1]), dict(slopes=two.half()),
                dict(slopes=two.cpu()), dict(prefix=one.long()), dict(prefix=two.int()), dict(prefix=one, window=3)):
        with pytest.raises((TypeError, ValueError)):
            p.run(**bad)
    p.positions = np.zeros((1, 4), np.int64)
    with pytest.raises(ValueError):
        p.run(prefix=one)
