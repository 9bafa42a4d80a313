"""Attention over a full GPU, its rows from memory and from the cache: the same bits.

The rings' places are handed back by what was read from them; a copy that came too early would show where rows come quickly
and the rest of a step slowly, so each call is made with a cold and a warm cache, and beside another stream's.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_lt_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("shaped", [False, True])
@pytest.mark.parametrize("dim,heads,group,new,list_len", [
    (128, 4, 8, 1, 0), (128, 2, 16, 1, 0), (128, 2, 8, 4, 0), (64, 8, 4, 1, 0), (64, 4, 12, 2, 0), (64, 2, 4, 8, 0), (256, 4, 8, 1, 0),
    (256, 2, 16, 1, 0), (128, 4, 8, 1, 512), (64, 2, 16, 1, 512), (256, 2, 8, 1, 512), (128, 1, 32, 1, 512),
    (64, 2, 4, 256, 0), (128, 2, 4, 256, 0), (256, 2, 4, 256, 0)])
def test_the_same_bits_however_fast_the_rows_come(dim, heads, group, new, list_len, shaped):
    import sparse_attention_indexer_lt_gb300 as lt
    requests, most, page = 32, 4096, 64
    gen = torch.Generator("cuda").manual_seed(dim + heads + group + new)
    pages = requests * most // page
    cache = lt.kv4_cache(pages, heads, page, dim)
    for at in range(0, requests * most, 32768):  # a part of the slots at a time
        k, v = (torch.randn(32768, heads, dim, device="cuda", generator=gen).half() for _ in range(2))
        lt.kv4_store(k, v, cache, torch.arange(at, at + 32768, device="cuda"))
    table = torch.randperm(pages, device="cuda", generator=gen).int().view(requests, -1)
    lengths = torch.randint(most // 2, most + 1, (requests,), device="cuda", generator=gen).int()
    starts = torch.arange(requests + 1, device="cuda").int() * new
    q = torch.randn(requests * new, heads * group, dim, device="cuda", generator=gen).bfloat16()
    kw = {}
    if list_len:
        kw["positions"] = torch.randint(0, most // 2, (requests * new, list_len), device="cuda", generator=gen).int()
    if shaped:
        kw.update(softcap=20.0, slopes=2.0 ** (-8.0 * torch.arange(1, heads * group + 1, device="cuda") / (heads * group)))
    call = lambda **s: lt.kv4_attention(q, cache, table, lengths, starts=starts, max_new=new, **kw, **s)  # noqa: E731
    want, got = call(), []
    assert torch.isfinite(want).all()
    flush, side = torch.empty(200 << 20, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    for i in range(12):
        flush.fill_(i)
        got.append(call())
        got.append(call())
        side.wait_stream(torch.cuda.current_stream())
        got += [call(stream=side), call()]
        torch.cuda.current_stream().wait_stream(side)
    off = [i for i, y in enumerate(got) if not torch.equal(y, want)]
    assert not off, f"calls {off}"
