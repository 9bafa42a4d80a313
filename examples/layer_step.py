"""An attention layer whose weights and cache are held in 4 bits, run with the library's operators together.

A prefill of ragged prompts, then decode steps. Each: queries, keys and values by one
product with 4-bit weights, pages for the new tokens, queries and keys turned by their
positions on the way into the 4-bit cache, attention over it, and the output product.
The prompts' tokens all see each other (a prefix mask), logits are capped, and
every head has a slope.

    python examples/layer_step.py           # on a GB300, with the built library

The weights and the tokens are random numbers.
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import sparse_attention_indexer_lt_gb300 as lt  # noqa: E402


def run(prompts=(70, 1, 33), steps: int = 3, hidden: int = 256, kv_heads: int = 2, group: int = 4, head_dim: int = 64,
        rotary: int = 32, softcap: float = 20.0, page_size: int = 16, seed: int = 0, dtype=torch.bfloat16):
    """Runs the steps; returns each one's tokens and outputs with what the layer holds, for a check."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    n, heads = len(prompts), kv_heads * group
    joint = (heads + 2 * kv_heads) * head_dim
    qkv, out = lt.w4_quantise(rand(joint, hidden) / hidden ** 0.5), lt.w4_quantise(rand(hidden, heads * head_dim) / (heads * head_dim) ** 0.5)
    bias = rand(joint)
    most = max(prompts) + steps
    angle = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** -(
        torch.arange(rotary // 2, device="cuda", dtype=torch.float64) / (rotary // 2))
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    slopes = 2.0 ** (-8.0 * torch.arange(1, heads + 1, device="cuda") / heads)
    width = (most + page_size - 1) // page_size
    cache = lt.kv4_cache(n * width, kv_heads, page_size, head_dim)
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(n * width, dtype=torch.int32, device="cuda")
    num_free = torch.tensor([n * width], dtype=torch.int32, device="cuda")
    lengths = torch.zeros(n, dtype=torch.int32, device="cuda")
    prefix = torch.tensor(prompts, dtype=torch.int32, device="cuda")

    seen = []
    for i in range(steps + 1):
        new = prefix if i == 0 else torch.ones_like(prefix)
        tokens, max_new = (sum(prompts), max(prompts)) if i == 0 else (n, 1)
        x = rand(tokens, hidden)
        step = lt.page_extend(lengths, new, table, free, num_free, page_size, tokens)
        q, k, v = lt.w4_linear(x, *qkv, bias=bias).view(tokens, -1, head_dim).split([heads, kv_heads, kv_heads], 1)
        q = lt.kv4_append(q, k, v, cache, step.slots, step.positions, cos, sin)
        a = lt.kv4_attention(q, cache, table, step.lengths, starts=step.starts, max_new=max_new, softcap=softcap, slopes=slopes,
                             prefix=prefix)
        y = lt.w4_linear(a.view(tokens, -1), *out)
        seen.append((x, y, step))
        lengths, num_free = step.lengths, step.num_free
    held = dict(qkv=qkv, out=out, bias=bias, cos=cos, sin=sin, slopes=slopes, prefix=prefix, cache=cache, table=table, softcap=softcap,
                page_size=page_size, kv_heads=kv_heads, group=group, head_dim=head_dim)
    return seen, held


def weights(codes, scales):
    """The numbers that codes and scales stand for, in 64 bits."""
    level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=codes.device)
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    return level[code & 7] * (1 - 2 * (code >> 3)) * scales.double().repeat_interleave(32, 1)


def check(seen, held) -> float:
    """The largest difference of any output from the layer in 64 bits over the values that the cache holds, relative to the
    outputs' size."""
    h, d, group, page = held["kv_heads"], held["head_dim"], held["group"], held["page_size"]
    w, wo = weights(*held["qkv"]), weights(*held["out"])
    half, worst, size = held["cos"].shape[1], 0.0, 0.0
    for x, y, step in seen:
        starts, lengths = step.starts.tolist(), step.lengths.tolist()
        q = (x.double() @ w.T + held["bias"].double()).view(x.shape[0], -1, d)[:, :h * group]
        for r, length in enumerate(lengths):
            rows = slice(starts[r], starts[r + 1])
            own = step.positions[rows].long()
            c, s = held["cos"][own].double()[:, None], held["sin"][own].double()[:, None]
            a, b = q[rows, :, :half], q[rows, :, half:2 * half]
            qr = torch.cat([a * c - b * s, b * c + a * s, q[rows, :, 2 * half:]], -1)
            p = torch.arange(length, device=x.device)
            slots = held["table"][r].long()[p // page] * page + p % page
            k, v = (t.double().repeat_interleave(group, 1) for t in lt.kv4_load(held["cache"], slots, dtype=torch.float32))
            logits = torch.einsum("thd,lhd->thl", qr, k) / d ** 0.5
            logits = held["softcap"] * torch.tanh(logits / held["softcap"])
            logits -= held["slopes"].double()[None, :, None] * (own[:, None] - p).abs().double()[:, None]
            visible = (p <= own[:, None]) | (p < held["prefix"][r])
            logits.masked_fill_(~visible[:, None], -torch.inf)
            want = torch.einsum("thl,lhd->thd", torch.softmax(logits, -1), v).flatten(1) @ wo.T
            if want.numel():
                worst, size = max(worst, float((y[rows].double() - want).abs().max())), max(size, float(want.abs().max()))
    return worst / size


if __name__ == "__main__":
    seen, held = run()
    torch.cuda.synchronize()
    print(f"a prefill and {len(seen) - 1} decode steps of {len(held['prefix'])} requests; largest difference from 64 bits "
          f"{check(seen, held):.2e} of the outputs' size")
