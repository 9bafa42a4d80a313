"""A compressed sparse attention layer's cache work, run with the library's operators together.

A prefill compresses the tokens' keys and values (4:1), takes pages for the
entries, stores them in the 4-bit cache; then decode steps bring the compressor
token by token, store an entry whenever one is complete, and attend: the
indexer's scores pick k entries a request, attention reads just those. At the
end the requests give their pages back.

    python examples/sparse_step.py          # on a GB300, with the built library

The projections and the indexer belong to a model: random numbers stand in for them.
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import sparse_attention_indexer_lt_gb300 as lt  # noqa: E402


def run(requests: int = 4, tokens: int = 2048, steps: int = 8, ratio: int = 4, kv_heads: int = 2, group: int = 8,
        head_dim: int = 128, k: int = 64, page_size: int = 16, seed: int = 0):
    """Runs the prefill and the decode steps; returns each step's (out, lse, picked positions) and the values
    that the cache holds, [requests, entries, kv_heads, head_dim] each, for a check."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    dim = kv_heads * head_dim
    bias = rand(ratio, dim, dtype=torch.float32)
    entries = tokens // ratio
    width = (entries + steps // ratio + 1 + page_size - 1) // page_size
    cache = lt.kv4_cache(requests * width, kv_heads, page_size, head_dim)
    table = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
    free_pages = torch.arange(requests * width, dtype=torch.int32, device="cuda")
    num_free = torch.tensor([requests * width], dtype=torch.int32, device="cuda")
    lengths = torch.zeros(requests, dtype=torch.int32, device="cuda")

    # prefill: entries for all tokens, pages for the entries
    new = torch.full((requests,), entries, dtype=torch.int32, device="cuda")
    step = lt.page_extend(lengths, new, table, free_pages, num_free, page_size, requests * entries)
    pair = [lt.compress(rand(requests, tokens, dim), rand(requests, tokens, dim), bias, ratio).view(-1, kv_heads, head_dim)
            for _ in range(2)]
    lt.kv4_store(*pair, cache, step.slots)

    # decode: the compressor's state in rings, an entry every `ratio` tokens (the requests run in phase here)
    rings = [rand(requests, ratio, dim) for _ in range(4)]
    entry = [torch.empty(requests, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    results = []
    for i in range(steps):
        at = tokens + i
        pos = torch.full((requests,), at, dtype=torch.int32, device="cuda")
        for j in range(2):
            lt.compress_decode(rand(requests, dim), rand(requests, dim), bias, rings[2 * j], rings[2 * j + 1], pos, entry[j])
        new = torch.full((requests,), 1 if (at + 1) % ratio == 0 else 0, dtype=torch.int32, device="cuda")
        step = lt.page_extend(step.lengths, new, table, free_pages, step.num_free, page_size, requests)
        lt.kv4_store(entry[0].view(-1, kv_heads, head_dim), entry[1].view(-1, kv_heads, head_dim), cache, step.slots)
        scores = rand(requests, width * page_size, dtype=torch.float32)
        picked, _ = lt.topk(scores, step.lengths, k, with_values=False)
        q = rand(requests, kv_heads * group, head_dim)
        out, lse = lt.kv4_attention(q, cache, table, step.lengths, positions=picked, with_lse=True)
        results.append((q, out, lse, picked))

    count = int(step.lengths.max())
    p = torch.arange(count, device="cuda")
    slots = table.long()[:, p // page_size] * page_size + p % page_size
    held = [t.view(requests, count, kv_heads, head_dim) for t in lt.kv4_load(cache, slots.reshape(-1), dtype=torch.float32)]

    done = torch.ones(requests, dtype=torch.bool, device="cuda")
    lengths, num_free = lt.page_release(step.lengths, done, table, free_pages, step.num_free, page_size)
    return results, held, int(num_free), requests * width


def check(results, held) -> float:
    """The largest difference of any output from attention over the held values in 64 bits."""
    keys, values = (t.double() for t in held)
    worst = 0.0
    for q, out, _, picked in results:
        requests, heads, dim = q.shape
        group = heads // keys.shape[2]
        at = picked.long()
        for r in range(requests):
            mine = at[r][at[r] >= 0]
            kk, vv = keys[r, mine].repeat_interleave(group, 1), values[r, mine].repeat_interleave(group, 1)
            s = torch.einsum("hd,lhd->hl", q[r].double(), kk) / dim ** 0.5
            want = torch.einsum("hl,lhd->hd", torch.softmax(s, -1), vv)
            worst = max(worst, float((out[r].double() - want).abs().max()))
    return worst


if __name__ == "__main__":
    results, held, free, pages = run()
    torch.cuda.synchronize()
    print(f"{len(results)} decode steps over {held[0].shape[1]} entries a request; largest difference from 64 bits "
          f"{check(results, held):.2e}; {free} of {pages} pages free at the end")
