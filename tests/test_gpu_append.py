"""GPU parity of the rotated append: queries, codes and scales are equal to the oracle's bit for bit, since every
rounding of the rotation is part of its definition."""
import numpy as np
import pytest
import torch

from oracle import kv4 as ok

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_lt_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def num(t):
    return t.detach().cpu().double().numpy()


def tables(most, pairs, seed=0):
    g = torch.Generator().manual_seed(seed)
    angle = torch.rand(most, pairs, generator=g, dtype=torch.float64) * 6.3
    return torch.cos(angle).float(), torch.sin(angle).float()


def turned(x, positions, cos, sin, interleaved):
    """float32 [tokens, heads, D] by the oracle."""
    at = positions.cpu().long().clamp(0, cos.shape[0] - 1)
    return torch.from_numpy(ok.rotate(num(x), num(cos[at]), num(sin[at]), interleaved))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary,heads,group,page", [(64, 64, 1, 1, 1), (64, 32, 3, 2, 16), (128, 128, 2, 4, 32), (128, 16, 5, 1, 64),
                                                         (128, 80, 1, 3, 8), (256, 256, 1, 2, 8), (256, 64, 2, 3, 16)])
def test_rows_and_queries(dim, rotary, heads, group, page, interleaved, dtype):
    import sparse_attention_indexer_lt_gb300 as lt
    torch.manual_seed(dim + rotary + heads)
    t, tokens, most = TYPES[dtype], 29, 50
    pages = 64 if page == 1 else 9
    qh = heads * group
    cos, sin = tables(most, rotary // 2, seed=rotary)
    joint = torch.randn(tokens, qh + 2 * heads, dim) * 10.0 ** torch.randint(-6, 3, (tokens, qh + 2 * heads, 1))
    joint[3, qh, :8] = 0.0
    joint[4, qh] = 0.0
    joint[5, qh, 3] = float("inf")
    joint[6, qh + heads, 5] = float("nan")
    joint = joint.to(t)
    positions = torch.randint(0, most, (tokens,), dtype=torch.int32)
    positions[7], positions[8], positions[9], positions[10], positions[11] = -1, most, 2 ** 31 - 1, 0, most - 1
    slots = torch.randperm(pages * page)[:tokens].long()
    slots[12], slots[13], slots[14] = -1, pages * page, -2 ** 40
    for wide in (True, False):
        # views of one projection, its channels at an odd offset for the scalar accesses
        extra = 0 if wide else 1
        flat = torch.full((tokens, (qh + 2 * heads) * dim + extra), 7.0, dtype=t)
        flat[:, extra:] = joint.flatten(1)
        view = flat.cuda()[:, extra:].unflatten(1, (qh + 2 * heads, dim))
        q, k, v = view[:, :qh], view[:, qh:qh + heads], view[:, qh + heads:]
        want_q = turned(joint[:, :qh], positions, cos, sin, interleaved).to(t)
        want_k = turned(joint[:, qh:qh + heads], positions, cos, sin, interleaved)
        cache = torch.full((pages, heads, page, lt.kv4_row_bytes(dim)), 0xA5, dtype=torch.uint8, device="cuda")
        out = torch.full((tokens, qh, dim), 5.0, dtype=t, device="cuda")
        got = lt.kv4_append(q, k, v, cache, slots.cuda(), positions.cuda(), cos.cuda(), sin.cuda(), interleaved=interleaved, out_q=out)
        assert got is out
        there = ((positions >= 0) & (positions < most)).numpy()
        res = out.cpu()
        assert torch.equal(torch.nan_to_num(res[there], 99.0), torch.nan_to_num(want_q[there], 99.0))
        assert (res[~there] == 5.0).all(), "a token without a position was turned"
        c = cache.cpu().numpy()
        written = np.zeros((pages, page), bool)
        for i, s in enumerate(slots.tolist()):
            if 0 <= s < pages * page and there[i]:
                written[s // page, s % page] = True
                row = c[s // page, :, s % page]
                want = ok.rows_of(num(want_k[i]), num(joint[i, qh + heads:]))
                scales, pad = slice(dim, dim + dim // 8), slice(dim + dim // 8, None)
                g, w = row[:, scales].copy().view(np.float16), want[:, scales].copy().view(np.float16)
                assert np.array_equal(g, w, equal_nan=True) and np.array_equal(row[:, pad], want[:, pad]), f"scales of token {i}"
                assert np.array_equal(row[:, :dim], want[:, :dim]), f"codes of token {i}"
        assert (c.transpose(0, 2, 1, 3)[~written] == 0xA5).all(), "rows without a slot were written"
        # in place, the queries a view of the projection
        lt.kv4_append(q, k, v, cache, slots.cuda(), positions.cuda(), cos.cuda(), sin.cuda(), interleaved=interleaved, out_q=q)
        assert torch.equal(torch.nan_to_num(q.cpu()[there], 99.0), torch.nan_to_num(want_q[there], 99.0))
        assert torch.equal(torch.nan_to_num(q.cpu()[~there], 99.0), torch.nan_to_num(joint[:, :qh][~there], 99.0))
        assert torch.equal(torch.nan_to_num(view[:, qh:].cpu(), 99.0), torch.nan_to_num(joint[:, qh:], 99.0))
        assert np.array_equal(cache.cpu().numpy(), c)


def reference(q, k, v, cache, slots, positions, cos, sin, interleaved):
    """The same by torch's 32-bit products and sums and the store."""
    import sparse_attention_indexer_lt_gb300 as lt
    r = 2 * cos.shape[1]
    c, s = cos[positions.long()][:, None], sin[positions.long()][:, None]

    def turn(x):
        x = x.float()
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
        a, b = a * c - b * s, b * c + a * s
        y = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
        return torch.cat([y, x[..., r:]], -1)
    lt.kv4_store(turn(k), v.float(), cache, slots)
    return turn(q).to(q.dtype)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,dim,rotary,tokens,heads,group", [("bf16", 128, 128, 3001, 8, 4), ("f16", 64, 64, 1, 1, 1),
                                                                 ("bf16", 256, 64, 777, 3, 7), ("f32", 128, 96, 1025, 2, 1)])
def test_many_tokens(dtype, dim, rotary, tokens, heads, group, interleaved):
    import sparse_attention_indexer_lt_gb300 as lt
    torch.manual_seed(tokens)
    t, page = TYPES[dtype], 16
    cos, sin = (x.cuda() for x in tables(2 * tokens + 8, rotary // 2))
    x = torch.randn(tokens, heads * (group + 2), dim, device="cuda").to(t)
    q, k, v = x.split([heads * group, heads, heads], 1)
    positions = torch.arange(tokens, device="cuda", dtype=torch.int32) + 7
    pages = tokens // page + 2
    slots = torch.randperm(pages * page, device="cuda")[:tokens]
    want, got = (lt.kv4_cache(pages, heads, page, dim) for _ in range(2))
    want_q = reference(q, k, v, want, slots, positions, cos, sin, interleaved)
    got_q = lt.kv4_append(q, k, v, got, slots, positions, cos, sin, interleaved=interleaved)
    assert torch.equal(got_q, want_q) and torch.equal(got, want)
    alone = lt.kv4_cache(pages, heads, page, dim)
    assert lt.kv4_append(None, k, v, alone, slots, positions, cos, sin, interleaved=interleaved) is None
    assert torch.equal(alone, want)


def test_beyond_32_bit_offsets():
    """A cache of more than 2^32 bytes, tables of more than 2^32 bytes, query rows more than 2^32 bytes apart."""
    import sparse_attention_indexer_lt_gb300 as lt
    torch.manual_seed(2)
    pages, page, dim = 300000, 64, 256  # 5.5 GB
    cache = torch.zeros(pages, 1, page, 288, dtype=torch.uint8, device="cuda")
    most = 2 ** 23 + 5  # 4.3 GB each
    cos, sin = torch.zeros(most, 128, device="cuda"), torch.zeros(most, 128, device="cuda")
    c, s = (x.cuda() for x in tables(2, 128))
    cos[0], sin[0], cos[-1], sin[-1] = c[0], s[0], c[1], s[1]
    far = torch.empty(2, 2 ** 31 + 256, dtype=torch.bfloat16, device="cuda")
    q = far[:, :256].unflatten(1, (1, 256))
    q.normal_()
    k, v = torch.randn(2, 2, 1, dim, device="cuda").bfloat16()
    positions = torch.tensor([0, most - 1], dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, pages * page - 1], device="cuda")
    small = lt.kv4_cache(1, 1, 64, dim)
    near = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    want = reference(q, k, v, small, torch.arange(2, device="cuda"), near, c, s, False)
    assert torch.equal(lt.kv4_append(q, k, v, cache, slots, positions, cos, sin), want)
    flat = cache.view(-1, 288)
    assert torch.equal(flat[slots], small.view(-1, 288)[:2])
    assert int(flat[4:-1].any(1).sum()) == 0


def test_on_other_streams_and_in_graphs():
    import sparse_attention_indexer_lt_gb300 as lt
    torch.manual_seed(4)
    cos, sin = (x.cuda() for x in tables(40, 64))
    x = torch.randn(9, 6, 128, device="cuda").bfloat16()
    q, k, v = x.split([2, 2, 2], 1)
    positions, slots = torch.arange(9, dtype=torch.int32, device="cuda"), torch.arange(9, device="cuda")
    want = lt.kv4_cache(1, 2, 16, 128)
    want_q = lt.kv4_append(q, k, v, want, slots, positions, cos, sin)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lt.kv4_cache(1, 2, 16, 128)
    side.wait_stream(torch.cuda.current_stream())
    got_q = lt.kv4_append(q, k, v, got, slots, positions, cos, sin, stream=side)
    side.synchronize()
    assert torch.equal(got_q, want_q) and torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lt.kv4_append(q, k, v, got, slots, positions, cos, sin)
    positions += 20
    x.normal_()
    graph.replay()
    again = lt.kv4_cache(1, 2, 16, 128)
    assert torch.equal(out, lt.kv4_append(q, k, v, again, slots, positions, cos, sin)) and torch.equal(again[:, :, :9], got[:, :, :9])


def test_an_injected_launch_failure_writes_nothing():
    import sparse_attention_indexer_lt_gb300 as lt
    cos, sin = (x.cuda() for x in tables(4, 64))
    x = torch.ones(1, 1, 128, device="cuda")
    cache, out = lt.kv4_cache(1, 1, 16, 128), torch.zeros(1, 1, 128, device="cuda")
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    lt.load().lt_test_inject(1, 1)
    with pytest.raises(lt.LtError):
        lt.kv4_append(x, x, x, cache, z.long(), z, cos, sin, out_q=out)
    assert not cache.any() and not out.any()
    lt.kv4_append(x, x, x, cache, z.long(), z, cos, sin, out_q=out)
    assert cache.any() and out.any()


def test_binding_refuses():
    import sparse_attention_indexer_lt_gb300 as lt
    cos, sin = (x.cuda() for x in tables(4, 64))
    x = torch.ones(2, 1, 128, device="cuda").half()
    cache = lt.kv4_cache(1, 1, 16, 128)
    pos, slots = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.arange(2, device="cuda")

    def call(q=x, k=x, v=x, slots=slots, positions=pos, cos=cos, sin=sin, **kw):
        return lt.kv4_append(q, k, v, cache, slots, positions, cos, sin, **kw)
    call()
    for bad in (dict(q=x.float()), dict(k=x[:1]), dict(v=x.bfloat16()), dict(q=x.double(), k=x.double(), v=x.double()),
                dict(q=x.expand(2, 3, 128).transpose(1, 2)), dict(k=x.repeat(1, 2, 1)), dict(k=torch.ones(2, 1, 256, device="cuda").half()[..., ::2]),
                dict(slots=slots.int()), dict(slots=slots[:1]), dict(positions=pos.long()), dict(positions=pos[:1]), dict(cos=cos[:, :32]),
                dict(cos=cos[:, :60].contiguous(), sin=sin[:, :60].contiguous()), dict(cos=cos[:0, :0], sin=sin[:0, :0]), dict(cos=cos.half()),
                dict(cos=cos.repeat(1, 2), sin=sin.repeat(1, 2)), dict(out_q=x[:1]), dict(out_q=x.float()), dict(q=None, out_q=x)):
        with pytest.raises((TypeError, ValueError)):
            call(**bad)
