"""What is measured of the operators on either side of the 4-bit key/value cache.

A layer's step projects its tokens with 4-bit weights (``w4_linear``), rotates the
queries and keys by their positions while the keys and values go into the cache
(``kv4_append``; ``kv4_load`` reads back what it stored) and attends over the cache
with logits that are capped by a tanh, lowered with the distance, or seen through a
prefix mask (``kv4_attention`` with ``softcap``, ``slopes`` and ``prefix``).

4-bit values. A code is an e2m1 number: sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6. A
group of 32 channels shares an fp16 scale. What is stored: the scale is the smallest
number at least amax / 6 that has 9 significant bits and is a multiple of 2^-23 (at
most 10912; NaN for a group with a NaN or an infinity), a value the code nearest to
x / scale, ties to the even code. A cache row, one for each (page, kv head, token),
holds D/2 bytes of key codes, D/2 of value codes (low nibble first), D/32 key scales
and D/32 value scales, and is padded to a multiple of 16 bytes. Weights [n, k] are
codes [n, k/2] and scales [n, k/32].

Rotation. Channels (i, i + R/2), or (2i, 2i + 1) where interleaved, of the first R
channels turn by the angle of (position, i): x c - y s and y c + x s, with the
cosine and the sine from fp32 tables, each product and each sum rounded to 32 bits.
Queries are rounded to their type then; keys are quantised from the 32-bit numbers.
"""
import math

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
#: borders between neighbouring levels, and whether a value on the border goes up (to the even code)
BORDERS = ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False))
GROUP = 32
SCALE_MAX = 10912.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---- cases

def _append(name, **kw):
    return {"name": name, "kind": "append", "page": 64, "dim": 128, "rotary": 128, "interleaved": False, "type": "bf16", **kw}


def _linear(name, **kw):
    return {"name": name, "kind": "linear", "bias": False, "type": "bf16", **kw}


def _attend(name, **kw):
    base = {"kind": "attend", "requests": 1, "window": 0, "listed": 0, "page": 64, "dim": 128, "type": "bf16", "softcap": 0.0,
            "slopes": False, "prefix": 0}
    return {"name": name, **base, **kw}


def listed():
    return [
        # the new token of each of 64 requests
        _append("append_decode", tokens=64, kv_heads=4, group=8, longest=65536),
        # a prefill of an odd number of tokens, the layout of the 4-bit store's
        _append("append_prefill", tokens=8191, kv_heads=8, group=4, longest=131072),
        # wide heads of which the first 64 channels turn, neighbours paired; small pages
        _append("append_partial", tokens=1021, kv_heads=2, group=8, dim=256, rotary=64, interleaved=True, type="f16", page=16, longest=16384),
        # one token through a square projection: the smallest call
        _linear("linear_token", tokens=1, n=4096, k=4096),
        # one token through the wide projection of a large layer
        _linear("linear_wide", tokens=1, n=28672, k=8192),
        # odd sizes: seven tokens, rows that end inside every tile, with a bias
        _linear("linear_odd", tokens=7, n=4099, k=5152, bias=True, type="f16"),
        # the tokens of a decode batch of 64 requests through a joint query, key and value projection
        _linear("linear_batch", tokens=64, n=10240, k=8192),
        # a prefill chunk of an odd number of tokens
        _linear("linear_chunk", tokens=509, n=14336, k=4096),
        # the smallest attention call: one request's next token over a short context, capped
        _attend("capped_decode", min_len=4096, max_len=4096, max_new=1, kv_heads=4, group=4, softcap=30.0),
        # a decode batch of ragged contexts, a slope for each head
        _attend("biased_decode", requests=64, min_len=2048, max_len=65536, max_new=1, kv_heads=4, group=8, slopes=True),
        # a ragged prefill of six requests whose first tokens all see each other, capped, small heads
        _attend("prefix_prefill", requests=6, min_len=1501, max_len=5003, max_new=1500, kv_heads=4, group=4, dim=64, type="f16",
                page=16, softcap=50.0, prefix=4000),
        # a prefill chunk behind a cached context, capped and with slopes
        _attend("capped_chunk", min_len=16384, max_len=16384, max_new=2048, kv_heads=8, group=4, softcap=30.0, slopes=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "linear", "linear", "decode", "decode", "prefill", "listed"])
    if kind == "append":
        dim = rng.choice([64, 128, 256])
        return {"kind": "append", "tokens": _log_int(rng, 1, 8191), "kv_heads": rng.choice([1, 2, 3, 4, 8]), "group": rng.choice([1, 3, 4]),
                "dim": dim, "rotary": rng.choice([dim, dim, dim // 2, 32]), "interleaved": rng.random() < 0.4, "page": rng.choice([16, 32, 64]),
                "type": rng.choice(["bf16", "f16"]), "longest": _log_int(rng, 8192, 262144)}
    if kind == "linear":
        tokens, k = _log_int(rng, 1, 600), 32 * _log_int(rng, 2, 512)
        n = _log_int(rng, 64, min(32768, 30_000_000_000 // (tokens * k)))
        return {"kind": "linear", "tokens": tokens, "n": n, "k": k, "bias": rng.random() < 0.5, "type": rng.choice(["bf16", "f16"])}
    case = {"kind": "attend", "window": 0, "listed": 0, "page": rng.choice([16, 32, 64]), "dim": rng.choice([64, 128]),
            "type": rng.choice(["bf16", "f16"]), "kv_heads": rng.choice([1, 2, 4]), "group": rng.choice([1, 3, 4, 8]), "prefix": 0}
    case["softcap"], case["slopes"] = rng.choice([(20.0, False), (50.0, False), (0.0, True), (30.0, True)])
    if kind == "decode":
        requests = _log_int(rng, 1, 64)
        longest = _log_int(rng, 300, min(262144, 2097152 // requests))
        return {**case, "requests": requests, "min_len": max(4, longest // 32), "max_len": longest,
                "max_new": rng.choice([1, 1, 1, 2, 3, 4]), "window": rng.choice([0, 0, 0, 1000]), "dim": rng.choice([64, 128, 256])}
    if kind == "prefill":
        requests = _log_int(rng, 1, 6)
        new = _log_int(rng, 17, 2048 // requests)
        longest = new + _log_int(rng, 1, 8000)
        return {**case, "requests": requests, "min_len": max(new, longest // 4), "max_len": longest, "max_new": new,
                "dim": rng.choice([64, 128, 256]), "prefix": rng.choice([0, longest // 2, longest])}
    tokens = _log_int(rng, 1, 1021)
    if rng.random() < 0.5:
        tokens, requests = 1, min(tokens, 64)
    else:
        requests = 1
    return {**case, "requests": requests, "min_len": max(tokens, 700), "max_len": max(tokens, _log_int(rng, 1400, 32768)),
            "max_new": tokens, "listed": rng.choice([64, 100, 512, 1024]), "group": rng.choice([4, 8, 16]), "kv_heads": rng.choice([1, 2])}


def _row_bytes(dim):
    return (dim + dim // 8 + 15) // 16 * 16


def _lengths(case):
    """The requests' lengths after the step, their new tokens and prefixes, spread over the case's range: the same for every seed."""
    n = case["requests"]
    if n == 1:
        return [case["max_len"]], [case["max_new"]], [case["prefix"]]
    lens, new, prefix = [], [], []
    for r in range(n):
        # a low-discrepancy walk: any number of requests covers the range
        u, w, x = (0.5 + r * 0.6180339887498949) % 1.0, (0.25 + r * 0.7548776662466927) % 1.0, (0.75 + r * 0.5698402909980532) % 1.0
        lens.append(case["min_len"] + int(u * (case["max_len"] - case["min_len"] + 1)))
        new.append(1 + int(w * case["max_new"]))
        prefix.append(int(x * (case["prefix"] + 1)))
    new[n // 2] = case["max_new"]
    return lens, [min(a, b) for a, b in zip(new, lens)], prefix


# ---- inputs

def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed(seed * 1000003 + salt)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _scales(shape, size, g):
    """fp16 scales of the format, 9 significant bits, log-normal around `size`."""
    s = size * torch.exp(0.3 * torch.randn(shape, device="cuda", generator=g))
    return (s.half().view(torch.int16) & -4).view(torch.float16)


def prepare(case, seed):
    return {"append": _prepare_append, "linear": _prepare_linear, "attend": _prepare_attend}[case["kind"]](case, seed)


def _prepare_append(case, seed):
    g = _gen(seed, 1)
    t, h, d, page = case["tokens"], case["kv_heads"], case["dim"], case["page"]
    heads = h * case["group"]
    # a joint projection's output: queries, keys and values are views of it
    joint = torch.randn(t, heads + 2 * h, d, device="cuda", generator=g)
    joint[:, heads:heads + h, ::17] *= 6.0  # keys have a few large channels
    joint = joint.to(TYPES[case["type"]])
    pages = (t + page - 1) // page + 3
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:t]
    # a decode step's requests are anywhere in their contexts; a chunk's tokens follow each other
    if t <= 64:
        positions = torch.randint(0, case["longest"], (t,), device="cuda", generator=g, dtype=torch.int32)
    else:
        positions = torch.arange(t, device="cuda", dtype=torch.int32) + (case["longest"] - t) // 2
    half = case["rotary"] // 2
    angle = torch.arange(case["longest"], device="cuda", dtype=torch.float64)[:, None] * \
        10000.0 ** -(torch.arange(half, device="cuda", dtype=torch.float64) / half)
    cache = torch.zeros(pages, h, page, _row_bytes(d), dtype=torch.uint8, device="cuda")
    return {"case": case, "q": joint[:, :heads], "k": joint[:, heads:heads + h], "v": joint[:, heads + h:], "slots": slots,
            "positions": positions, "cos": torch.cos(angle).float(), "sin": torch.sin(angle).float(), "cache": cache,
            "interleaved": case["interleaved"]}


def _prepare_linear(case, seed):
    g = _gen(seed, 2)
    t, n, k, dtype = case["tokens"], case["n"], case["k"], TYPES[case["type"]]
    # uniform codes are what normal weights quantise to; a weight's size is about 1 / sqrt(k)
    codes = torch.randint(0, 256, (n, k // 2), device="cuda", generator=g, dtype=torch.uint8)
    scales = _scales((n, k // GROUP), 0.35 / math.sqrt(k), g)
    x = torch.randn(t, k, device="cuda", generator=g)
    x[:, ::61] *= 8.0  # activations have a few large channels
    bias = torch.randn(n, device="cuda", generator=g).to(dtype) if case["bias"] else None
    return {"case": case, "x": x.to(dtype), "codes": codes, "scales": scales, "bias": bias}


def _prepare_attend(case, seed):
    g = _gen(seed, 3)
    h, d, page, group = case["kv_heads"], case["dim"], case["page"], case["group"]
    lens, new, prefix = _lengths(case)
    n, tokens = len(lens), sum(new)
    width = (max(lens) + page - 1) // page
    held = [(x + page - 1) // page for x in lens]
    pages = sum(held) + 1
    order = torch.randperm(pages, device="cuda", generator=g, dtype=torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    cells = torch.arange(width, device="cuda")[None, :] < _int32(held)[:, None]
    table[cells] = order[:sum(held)]
    # uniform codes are what normal values quantise to (16 levels of about equal share); scales of about 0.35 give values of unit size
    cache = torch.randint(0, 256, (pages, h, page, _row_bytes(d)), device="cuda", generator=g, dtype=torch.uint8)
    cache[..., d:d + d // 8] = _scales((pages, h, page, 2 * d // GROUP), 0.35, g).view(torch.uint8)
    # queries a few times the unit size, so that logits come near the caps
    q = (4.0 * torch.randn(tokens, h * group, d, device="cuda", generator=g)).to(TYPES[case["type"]])
    starts = [0]
    for x in new:
        starts.append(starts[-1] + x)
    # slopes fall geometrically over the heads, 2^-8 at the last
    slopes = 2.0 ** (-8.0 * torch.arange(1, h * group + 1, device="cuda") / (h * group)) if case["slopes"] else None
    state = {"case": case, "q": q, "cache": cache, "table": table, "lengths": _int32(lens), "starts": _int32(starts),
             "max_new": max(new), "window": case["window"], "positions": None, "page": page, "dim": d, "group": group,
             "softcap": case["softcap"], "slopes": slopes, "prefix": _int32(prefix) if case["prefix"] else None}
    if case["listed"]:
        owner = torch.repeat_interleave(torch.arange(n, device="cuda"), _int32(new))
        last = state["lengths"][owner] - state["starts"][1:][owner] + torch.arange(tokens, device="cuda")  # each token's position
        picks = []
        for part in torch.arange(tokens, device="cuda").split(128):
            w = torch.rand(part.numel(), max(max(lens), case["listed"]), device="cuda", generator=g)
            w[torch.arange(w.shape[1], device="cuda")[None, :] > last[part][:, None]] = -1.0
            val, idx = w.topk(case["listed"], dim=1)
            picks.append(torch.where(val >= 0, idx, -1).int())
        state["positions"] = torch.cat(picks)
    return state


# ---- one pass

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _OWN[kind](state)
    return _PLAIN[kind](state)


def _own_append(st):
    import sparse_attention_indexer_lt_gb300 as lt
    q = lt.kv4_append(st["q"], st["k"], st["v"], st["cache"], st["slots"], st["positions"], st["cos"], st["sin"],
                      interleaved=st["interleaved"])
    k, v = lt.kv4_load(st["cache"], st["slots"])
    return {"q": q, "k": k, "v": v}


def _own_linear(st):
    import sparse_attention_indexer_lt_gb300 as lt
    return lt.w4_linear(st["x"], st["codes"], st["scales"], bias=st["bias"])


def _own_attend(st):
    import sparse_attention_indexer_lt_gb300 as lt
    return lt.kv4_attention(st["q"], st["cache"], st["table"], st["lengths"], starts=st["starts"], max_new=st["max_new"],
                            positions=st["positions"], window=st["window"], softcap=st["softcap"], slopes=st["slopes"],
                            prefix=st["prefix"], with_lse=True)


def _power(e):
    """2^e in 64 bits, exactly (exp2 and pow may be off by one unit on a GPU)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _plain_quantised(x):
    """The numbers that x is stored as, in 32 bits."""
    g = x.float().unflatten(-1, (-1, GROUP))
    size = g.abs()
    amax = size.amax(-1, keepdim=True).double()
    low = amax / 6
    step = _power(torch.clamp(torch.frexp(low).exponent - 9, min=-23))
    scale = torch.clamp(torch.ceil(low / step) * step, max=SCALE_MAX)
    edges = (scale[..., None] * torch.tensor([b for b, _ in BORDERS], dtype=torch.float64, device="cuda")).float()  # 12 bits at most: exact
    up = torch.tensor([u for _, u in BORDERS], device="cuda")
    code = torch.where(up, size[..., None] >= edges, size[..., None] > edges).sum(-1)
    value = torch.tensor(LEVELS, device="cuda")[code] * scale.float() * torch.sign(g)
    return torch.where(torch.isfinite(amax), value, math.nan).flatten(-2)


def _plain_rotated(x, cos, sin, interleaved):
    """x [tokens, heads, D] turned by the tokens' angles, in 32 bits."""
    r = 2 * cos.shape[-1]
    head, rest = x[..., :r].float(), x[..., r:].float()
    a, b = (head[..., 0::2], head[..., 1::2]) if interleaved else head.chunk(2, -1)
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, rest], -1)


def _plain_append(st):
    at = st["positions"].long()
    cos, sin = st["cos"][at][:, None], st["sin"][at][:, None]
    q = _plain_rotated(st["q"], cos, sin, st["interleaved"])
    k = _plain_rotated(st["k"], cos, sin, st["interleaved"])
    return {"q": q.to(st["q"].dtype), "k": _plain_quantised(k).half(), "v": _plain_quantised(st["v"]).half()}


def _plain_levels():
    """Of a byte of two codes: what its low and its high nibble stand for."""
    signed = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device="cuda")
    return torch.stack([signed.repeat(16), signed.repeat_interleave(16)], -1)


def _plain_linear(st):
    w = _plain_levels()[st["codes"].int()].flatten(-2).unflatten(-1, (-1, GROUP)) * st["scales"].float()[..., None]
    y = st["x"].float() @ w.flatten(-2).T
    if st["bias"] is not None:
        y = y + st["bias"].float()
    return y.to(st["x"].dtype)


def _plain_values(rows, d):
    """Keys and values, in 32 bits, of cache rows [..., row bytes]."""
    scales = rows[..., d:d + d // 8].contiguous().view(torch.float16).float().unflatten(-1, (2, d // GROUP))
    values = _plain_levels()[rows[..., :d].int()].flatten(-2).unflatten(-1, (2, d // GROUP, GROUP)) * scales[..., None]
    values = values.flatten(-2)
    return values[..., 0, :], values[..., 1, :]


def _plain_softmax(q, k, v, seen, st, slopes, distance):
    """q [..., rows, D], k and v [..., L, D]; slopes [..., rows, 1], distance and seen [..., rows, L] (broadcast): outputs and the
    logarithm of the sums."""
    s = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(st["dim"]))
    if st["softcap"]:
        s = st["softcap"] * torch.tanh(s / st["softcap"])
    if slopes is not None:
        s = s - slopes * distance
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), 0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, (p @ v) / total, 0)
    return o, (torch.log(total) + torch.where(torch.isinf(top), 0, top))[..., 0]


def _plain_attend(st):
    d, page, group, q = st["dim"], st["page"], st["group"], st["q"]
    h = st["cache"].shape[1]
    lengths, starts = st["lengths"].long(), st["starts"].long()
    n, tokens, new = lengths.numel(), q.shape[0], st["max_new"]
    token = torch.arange(tokens, device="cuda")
    owner = torch.searchsorted(starts[1:], token, right=True)
    qf = q.float().unflatten(1, (h, group))
    slopes = None if st["slopes"] is None else st["slopes"].view(h, group)
    if st["positions"] is not None:
        at = st["positions"].long()
        seen = (at >= 0) & (at < lengths[owner][:, None])
        at = torch.where(seen, at, 0)
        own_at = lengths[owner] - starts[1:][owner] + token
        rows = st["cache"][st["table"].long()[owner[:, None], at // page].clamp(min=0), :, at % page]  # [T, list, H, bytes]
        k, v = _plain_values(rows.transpose(1, 2), d)
        distance = (own_at[:, None] - at).abs().float()[:, None, None, :]
        o, lse = _plain_softmax(qf, k, v, seen[:, None, None, :], st, None if slopes is None else slopes[..., None], distance)
        return o.flatten(1, 2).to(q.dtype), lse.flatten(1, 2)
    longest = st["table"].shape[1] * page
    rows = st["cache"][st["table"].long().clamp(min=0)].transpose(2, 3).flatten(1, 2).transpose(1, 2)  # [R, H, L, bytes]
    k, v = _plain_values(rows, d)
    nth = token - starts[owner]
    wide = qf.new_zeros(n, new, h, group, d)
    wide[owner, nth] = qf
    wide = wide.permute(0, 2, 1, 3, 4).flatten(2, 3)  # [R, H, new * group, D]
    last = lengths[:, None] - (starts[1:] - starts[:-1])[:, None] + torch.arange(new, device="cuda")
    last = last.repeat_interleave(group, 1)[:, None, :, None]
    cell = torch.arange(longest, device="cuda")
    seen = cell <= last
    if st["prefix"] is not None:
        seen = seen | (cell < st["prefix"].long()[:, None, None, None])
    seen = seen & (cell < lengths[:, None, None, None])
    if st["window"]:
        seen = seen & (cell > last - st["window"])
    by_row, distance = None, None
    if slopes is not None:
        by_row, distance = slopes.repeat(1, new)[None, :, :, None], (last - cell).abs().float()
    o, lse = _plain_softmax(wide, k, v, seen, st, by_row, distance)
    o = o.unflatten(2, (new, group)).permute(0, 2, 1, 3, 4)[owner, nth]
    lse = lse.unflatten(2, (new, group)).permute(0, 2, 1, 3)[owner, nth]
    return o.flatten(1, 2).to(q.dtype), lse.flatten(1, 2)


_OWN = {"append": _own_append, "linear": _own_linear, "attend": _own_attend}
_PLAIN = {"append": _plain_append, "linear": _plain_linear, "attend": _plain_attend}


# ---- the definition in 64 bits

def _exact_quantised(x):
    """By the definition: the smallest scale of the grid, then the nearest of the signed levels by distance."""
    g = x.double().reshape(*x.shape[:-1], -1, GROUP)
    need = g.abs().max(-1).values / 6
    bits = torch.floor(torch.log2(torch.where(need > 0, need, 1.0)))
    scale = torch.full_like(need, SCALE_MAX)
    for finer in (1, 0, -1):  # the finest grid of 9 bits that reaches it; the logarithm may be off by one
        step = _power(torch.clamp(bits + finer - 8, min=-23.0))
        number = torch.ceil(need / step)
        scale = torch.where(number < 512, number * step, scale)
    scale = torch.clamp(scale, max=SCALE_MAX)[..., None]
    best, dist = torch.zeros_like(g), g.abs()
    for code, level in enumerate(LEVELS):
        away = (g.abs() - level * scale).abs()
        take = (away < dist) | ((away == dist) & (code % 2 == 0))
        best, dist = torch.where(take, level * scale.expand_as(g), best), torch.where(take, away, dist)
    return torch.copysign(best, g).reshape(x.shape)


def _exact_codes(raw):
    """What bytes of two codes stand for, in 64 bits, from the bits."""
    code = torch.stack([raw & 15, raw >> 4], -1).flatten(-2).long()
    two, one = (code >> 1) & 3, (code & 1).double()
    size = torch.where(two == 0, 0.5 * one, (1 + 0.5 * one) * _power(two - 1))
    return torch.where(code >= 8, -size, size)


def _exact_half(word):
    """fp16 numbers from their bits, in 64 bits (none is negative)."""
    exponent, fraction = (word >> 10) & 31, (word & 1023).double()
    return torch.where(exponent == 0, fraction * 2.0 ** -24, (1024 + fraction) * _power(exponent - 25))


def _exact_rows(st, pages, offsets, head):
    """Keys and values in 64 bits of one head's cache rows."""
    d = st["dim"]
    raw = st["cache"][pages, head, offsets].long()
    word = raw[:, d:d + d // 8:2] | (raw[:, d + 1:d + d // 8:2] << 8)
    value = _exact_codes(raw[:, :d]) * _exact_half(word).repeat_interleave(GROUP, 1)
    return value[:, :d], value[:, d:]


def _exact_rotated(x, st, round32):
    """The rotation as complex numbers' products; round32: each product and sum rounded to 32 bits, as the stored keys are defined."""
    r32 = (lambda y: y.float().double()) if round32 else (lambda y: y)
    out = x.double().clone()
    at, half = st["positions"].long(), st["cos"].shape[1]
    for i in range(half):
        c, s = st["cos"][at, i].double()[:, None], st["sin"][at, i].double()[:, None]
        m, n = (2 * i, 2 * i + 1) if st["interleaved"] else (i, i + half)
        a, b = x[..., m].double(), x[..., n].double()
        out[..., m] = r32(r32(a * c) - r32(b * s))
        out[..., n] = r32(r32(b * c) + r32(a * s))
    return out


def _exact_append(st):
    return {"q": _exact_rotated(st["q"], st, False), "k": _exact_quantised(_exact_rotated(st["k"], st, True)),
            "v": _exact_quantised(st["v"])}


def _exact_linear(st):
    y = torch.empty(st["x"].shape[0], st["codes"].shape[0], dtype=torch.float64, device="cuda")
    for rows in torch.arange(st["codes"].shape[0], device="cuda").split(4096):
        w = _exact_codes(st["codes"][rows]) * _exact_half(st["scales"][rows].view(torch.int16).long()).repeat_interleave(GROUP, 1)
        y[:, rows] = torch.einsum("tk,nk->tn", st["x"].double(), w)
    return y if st["bias"] is None else y + st["bias"].double()


def _exact_attend(st):
    q, page, group, d = st["q"].double(), st["page"], st["group"], st["dim"]
    lens, starts = st["lengths"].tolist(), st["starts"].tolist()
    prefix = [0] * len(lens) if st["prefix"] is None else st["prefix"].tolist()
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for r, length in enumerate(lens):
        new = starts[r + 1] - starts[r]
        cells = torch.arange(length, device="cuda")
        pages = st["table"][r].long()[cells // page]
        for head in range(st["cache"].shape[1]):
            k, v = _exact_rows(st, pages, cells % page, head)
            heads = slice(head * group, (head + 1) * group)
            for first in range(0, new, 256):
                count = min(256, new - first)
                rows = slice(starts[r] + first, starts[r] + first + count)
                last = length - new + first + torch.arange(count, device="cuda")[:, None]
                if st["positions"] is None:
                    seen = cells <= last
                    if st["window"]:
                        seen &= cells > last - st["window"]
                    seen |= cells < prefix[r]
                else:
                    at = st["positions"][rows].long()
                    hits = torch.zeros(count, length + 1, device="cuda")
                    hits.scatter_(1, torch.where((at < 0) | (at >= length), length, at), 1.0)
                    seen = hits[:, :length] > 0
                s = torch.einsum("thd,ld->thl", q[rows, heads], k) / math.sqrt(d)
                if st["softcap"]:
                    s = st["softcap"] * torch.tanh(s / st["softcap"])
                if st["slopes"] is not None:
                    s -= st["slopes"][heads].double()[None, :, None] * (cells - last).abs().double()[:, None, :]
                s.masked_fill_(~seen[:, None, :], -math.inf)
                lse[rows, heads] = torch.logsumexp(s, -1)
                out[rows, heads] = torch.softmax(s, -1) @ v
    return out, lse


def exact(case, seed):
    return {"append": _exact_append, "linear": _exact_linear, "attend": _exact_attend}[case["kind"]](prepare(case, seed))


# ---- what a pass cannot do without

def work(case):
    if case["kind"] == "append":
        t, kv = case["tokens"], case["tokens"] * case["kv_heads"] * case["dim"]
        tables = min(t, case["longest"]) * case["rotary"] * 4
        # queries, keys and values in, queries out; 4.5 bits a value written and read, fp16 values out; positions and slots
        return {"bytes": 2 * 2 * kv * case["group"] + 2 * 2 * kv + 2 * 2 * kv * 9 // 16 + 2 * 2 * kv + tables + 12 * t,
                "flops": 3 * case["rotary"] * t * case["kv_heads"] * (case["group"] + 1) + 4 * kv}
    if case["kind"] == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        return {"bytes": n * k * 9 // 16 + 2 * t * (n + k) + (2 * n if case["bias"] else 0), "flops": 2 * t * n * k}
    lens, new, prefix = _lengths(case)
    heads, tokens = case["kv_heads"] * case["group"], sum(new)
    if case["listed"]:
        pairs = sum(b * min(case["listed"], a) for a, b in zip(lens, new))
        cells = sum(min(a, b * case["listed"]) for a, b in zip(lens, new))
    else:
        span = case["window"] or max(lens)
        cells = sum(min(a, span + b - 1) for a, b in zip(lens, new))
        pairs = sum(max(min(a - b + i + 1, span), min(a, x)) for a, b, x in zip(lens, new, prefix) for i in range(b))
    once = 2 * 2 * tokens * heads * case["dim"] + 4 * tokens * case["listed"] + 4 * tokens * heads
    return {"bytes": cells * case["kv_heads"] * case["dim"] * 9 // 8 + once, "flops": 4 * case["dim"] * heads * pairs}
