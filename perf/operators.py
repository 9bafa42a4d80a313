"""What is measured of the operators around a key/value cache held in 4 bits.

A serving step over such a cache runs: page tables and slot maps from the
requests' lengths (``page_release``, ``page_extend``), the new tokens' keys and
values quantised into their slots (``kv4_store``; ``kv4_load`` reads them back),
and attention over the cached positions (``kv4_attention``), all of a request's
or those that an indexer's top-k lists.

The cache. One row for each (page, kv head, token): D/2 bytes of key codes, D/2
of value codes (low nibble first), then D/32 fp16 key scales and D/32 fp16 value
scales, the row padded to a multiple of 16 bytes. A code is an e2m1 number: sign,
then 0, 0.5, 1, 1.5, 2, 3, 4, 6. A group of 32 channels shares a scale: the
smallest number at least amax / 6 that has 9 significant bits and is a multiple
of 2^-23 (at most 10912; NaN for a group with a NaN or an infinity). A value is
the code nearest to x / scale, ties to the even code, times the scale.
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

def _pages(name, **kw):
    return {"name": name, "kind": "pages", **kw}


def _store(name, **kw):
    return {"name": name, "kind": "store", **kw}


def _attend(name, **kw):
    base = {"kind": "attend", "requests": 1, "window": 0, "listed": 0, "page": 64, "dim": 128, "type": "bf16"}
    return {"name": name, **base, **kw}


def listed():
    return [
        # a decode step of 64 requests whose lengths are those of the ragged top-k batch; four requests have ended
        _pages("pages_decode", requests=64, page=64, min_len=2048, max_len=65536, max_new=1, ended=4),
        # a mixed step of many short requests: prefill chunks of 0 to 128 tokens beside ended ones
        _pages("pages_mixed", requests=1000, page=16, min_len=0, max_len=4000, max_new=128, ended=50),
        # the new token of each of 64 requests
        _store("store_decode", tokens=64, kv_heads=4, dim=128, page=64, type="bf16"),
        # a prefill of an odd number of tokens
        _store("store_prefill", tokens=8191, kv_heads=8, dim=128, page=64, type="bf16"),
        # the smallest attention call: one request's next token over a short context
        _attend("decode_short", min_len=4096, max_len=4096, max_new=1, kv_heads=4, group=4),
        # a decode batch of ragged contexts
        _attend("decode_ragged", requests=64, min_len=2048, max_len=65536, max_new=1, kv_heads=4, group=8),
        # one request at a million tokens compressed 4:1, the decode row of the top-k, on wide heads
        _attend("decode_long", min_len=262144, max_len=262144, max_new=1, kv_heads=4, group=8, dim=256, type="f16"),
        # a step that checks up to 4 drafted tokens a request, small heads, a sliding window
        _attend("decode_drafted", requests=32, min_len=5, max_len=9001, max_new=4, kv_heads=8, group=4, dim=64, type="f16",
                page=32, window=4096),
        # a prefill chunk behind a cached context
        _attend("prefill_chunk", min_len=16384, max_len=16384, max_new=2048, kv_heads=8, group=4),
        # a ragged prefill of odd lengths
        _attend("prefill_ragged", requests=6, min_len=1501, max_len=5003, max_new=1500, kv_heads=4, group=4, dim=64, type="f16",
                page=16),
        # the later half of a sparse decode step: each request attends to the 512 positions its top-k kept
        _attend("listed_decode", requests=64, min_len=2048, max_len=65536, max_new=1, kv_heads=1, group=16, listed=512),
        # the same for the tokens of a prefill chunk, one list a token
        _attend("listed_prefill", min_len=32768, max_len=32768, max_new=1021, kv_heads=1, group=16, listed=512),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["pages", "store", "decode", "decode", "prefill", "listed"])
    if kind == "pages":
        return {"kind": "pages", "requests": _log_int(rng, 1, 2000), "page": rng.choice([16, 32, 64, 128]), "min_len": 0,
                "max_len": _log_int(rng, 100, 65536), "max_new": _log_int(rng, 1, 200), "ended": rng.randrange(0, 3)}
    if kind == "store":
        return {"kind": "store", "tokens": _log_int(rng, 1, 8191), "kv_heads": rng.choice([1, 2, 3, 4, 8]),
                "dim": rng.choice([64, 128]), "page": rng.choice([16, 32, 64]), "type": rng.choice(["bf16", "f16"])}
    case = {"kind": "attend", "window": 0, "listed": 0, "page": rng.choice([16, 32, 64]), "dim": rng.choice([64, 128]),
            "type": rng.choice(["bf16", "f16"]), "kv_heads": rng.choice([1, 2, 4]), "group": rng.choice([1, 3, 4, 8])}
    if kind == "decode":
        requests = _log_int(rng, 1, 64)
        longest = _log_int(rng, 300, min(262144, 2097152 // requests))
        return {**case, "requests": requests, "min_len": max(4, longest // 32), "max_len": longest,
                "max_new": rng.choice([1, 1, 1, 2, 3, 4]), "window": rng.choice([0, 0, 0, 1000]), "dim": rng.choice([64, 128, 256])}
    if kind == "prefill":
        requests = _log_int(rng, 1, 6)
        new = _log_int(rng, 17, 2048 // requests)
        longest = new + _log_int(rng, 1, 8000)
        return {**case, "requests": requests, "min_len": max(new, longest // 4), "max_len": longest, "max_new": new}
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
    """The requests' lengths after the step and their new tokens, spread over the case's range: the same for every seed."""
    n = case["requests"]
    if n == 1:
        return [case["max_len"]], [case["max_new"]]
    lens, new = [], []
    for r in range(n):
        # a low-discrepancy walk: any number of requests covers the range
        u, w = (0.5 + r * 0.6180339887498949) % 1.0, (0.25 + r * 0.7548776662466927) % 1.0
        lens.append(case["min_len"] + int(u * (case["max_len"] - case["min_len"] + 1)))
        new.append(1 + int(w * case["max_new"]))
    new[n // 2] = case["max_new"]
    return lens, [min(a, b) for a, b in zip(new, lens)]


# ---- inputs

def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed(seed * 1000003 + salt)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    return {"pages": _prepare_pages, "store": _prepare_store, "attend": _prepare_attend}[case["kind"]](case, seed)


def _prepare_pages(case, seed):
    g = _gen(seed, 1)
    n, page = case["requests"], case["page"]
    lengths = torch.randint(case["min_len"], case["max_len"] + 1, (n,), device="cuda", generator=g, dtype=torch.int32)
    new = torch.randint(0 if case["max_new"] > 1 else 1, case["max_new"] + 1, (n,), device="cuda", generator=g, dtype=torch.int32)
    finished = torch.zeros(n, dtype=torch.bool, device="cuda")
    if case["ended"] and n > case["ended"]:
        finished[torch.randperm(n, device="cuda", generator=g)[:case["ended"]]] = True
        new[finished] = 0
    width = (case["max_len"] + case["max_new"] + page - 1) // page
    pages = n * width
    order = torch.randperm(pages, device="cuda", generator=g, dtype=torch.int32)
    table = order.view(n, width).clone()
    held = (lengths + page - 1) // page
    spare = torch.arange(width, device="cuda")[None, :] >= held[:, None]
    loose = table[spare]
    table[spare] = -1
    free = torch.zeros(pages, dtype=torch.int32, device="cuda")
    free[:loose.numel()] = loose
    return {"case": case, "lengths": lengths, "new": new, "finished": finished, "table": table, "free": free,
            "num_free": _int32([loose.numel()]), "page": page, "max_tokens": n * case["max_new"]}


def _prepare_store(case, seed):
    g = _gen(seed, 2)
    t, h, d, page = case["tokens"], case["kv_heads"], case["dim"], case["page"]
    # a fused projection's output: the keys and values are views of it
    kv = torch.randn(t, 2, h, d, device="cuda", generator=g)
    kv[:, 0, :, ::17] *= 6.0  # keys have a few large channels
    kv = kv.to(TYPES[case["type"]])
    pages = (t + page - 1) // page + 3
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:t]
    cache = torch.zeros(pages, h, page, _row_bytes(d), dtype=torch.uint8, device="cuda")
    return {"case": case, "k": kv[:, 0], "v": kv[:, 1], "slots": slots, "cache": cache, "page": page, "dim": d}


def _prepare_attend(case, seed):
    g = _gen(seed, 3)
    h, d, page = case["kv_heads"], case["dim"], case["page"]
    lens, new = _lengths(case)
    n, tokens = len(lens), sum(new)
    width = (max(lens) + page - 1) // page
    held = [(x + page - 1) // page for x in lens]
    pages = sum(held) + 1
    order = torch.randperm(pages, device="cuda", generator=g, dtype=torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    cells = torch.arange(width, device="cuda")[None, :] < _int32(held)[:, None]
    table[cells] = order[:sum(held)]
    # uniform codes are what normal values quantise to (16 levels of about equal share);
    # scales of about 0.35 with 9 significant bits give values of unit size
    cache = torch.randint(0, 256, (pages, h, page, _row_bytes(d)), device="cuda", generator=g, dtype=torch.uint8)
    scales = 0.35 * torch.exp(0.3 * torch.randn(pages, h, page, 2 * d // GROUP, device="cuda", generator=g))
    cache[..., d:d + d // 8] = (scales.half().view(torch.int16) & -4).view(torch.uint8)
    q = torch.randn(tokens, h * case["group"], d, device="cuda", generator=g).to(TYPES[case["type"]])
    starts = [0]
    for x in new:
        starts.append(starts[-1] + x)
    state = {"case": case, "q": q, "cache": cache, "table": table, "lengths": _int32(lens), "starts": _int32(starts),
             "max_new": max(new), "window": case["window"], "positions": None, "page": page, "dim": d, "group": case["group"]}
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


def _own_pages(st):
    import sparse_attention_indexer_lt_gb300 as lt
    kept, num_free = lt.page_release(st["lengths"], st["finished"], st["table"], st["free"], st["num_free"], st["page"])
    step = lt.page_extend(kept, st["new"], st["table"], st["free"], num_free, st["page"], st["max_tokens"])
    return {"slots": step.slots, "positions": step.positions, "starts": step.starts, "lengths": step.lengths,
            "num_free": step.num_free, "table": st["table"], "free": st["free"], "after_release": num_free}


def _own_store(st):
    import sparse_attention_indexer_lt_gb300 as lt
    lt.kv4_store(st["k"], st["v"], st["cache"], st["slots"])
    return lt.kv4_load(st["cache"], st["slots"], dtype=st["k"].dtype)


def _own_attend(st):
    import sparse_attention_indexer_lt_gb300 as lt
    if st["positions"] is not None:
        return lt.kv4_attention(st["q"], st["cache"], st["table"], st["lengths"], starts=st["starts"], max_new=st["max_new"],
                                positions=st["positions"], with_lse=True)
    return lt.kv4_attention(st["q"], st["cache"], st["table"], st["lengths"], starts=st["starts"], max_new=st["max_new"],
                            window=st["window"])


def _plain_pages(st):
    page, free, table = st["page"], st["free"].clone(), st["table"].clone()
    cells = torch.arange(table.shape[1], device="cuda")[None, :]
    # release: the pages of the ended requests go on top of the free ones, in request and then table order
    held = (st["lengths"].long() + page - 1) // page
    back = table[(cells < held[:, None]) & st["finished"][:, None]]
    at = st["num_free"].long() + torch.arange(back.numel(), device="cuda")
    free[at] = back
    top = st["num_free"].long() + back.numel()
    lengths = torch.where(st["finished"], 0, st["lengths"]).long()
    # extend: pages from the top of the free ones, request by request, until one does not fit
    new = st["new"].long().clamp(min=0)
    have, want = (lengths + page - 1) // page, (lengths + new + page - 1) // page
    page_end, token_end = (want - have).cumsum(0), new.cumsum(0)
    fits = (page_end <= top) & (token_end <= st["max_tokens"]) & (want <= table.shape[1])
    fits = fits.int().cummin(0).values.bool()
    new, want = torch.where(fits, new, 0), torch.where(fits, want, have)
    page_end, token_end = (want - have).cumsum(0), new.cumsum(0)
    fresh = (cells >= have[:, None]) & (cells < want[:, None])
    nth = (page_end - want)[:, None] + cells  # of a fresh cell: how many pages were taken before it
    table[fresh] = free[top - 1 - nth[fresh]]
    token = torch.arange(st["max_tokens"], device="cuda")
    owner = torch.searchsorted(token_end, token, right=True).clamp(max=new.numel() - 1)
    real = token < token_end[-1]
    position = lengths[owner] + token - (token_end - new)[owner]
    position = torch.where(real, position, 0)
    slot = table[owner, position // page].long() * page + position % page
    return {"slots": torch.where(real, slot, -1), "positions": torch.where(real, position, -1).int(),
            "starts": torch.cat([token_end.new_zeros(1), token_end]).int(), "lengths": (lengths + new).int(),
            "num_free": (top - page_end[-1]).int(), "table": table, "free": free, "after_release": top.int()}


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
    code = torch.zeros_like(size, dtype=torch.int32)
    for border, up in BORDERS:
        edge = (scale * border).float()  # 12 bits at most: exact
        code += (size >= edge) if up else (size > edge)
    value = torch.tensor(LEVELS, device="cuda")[code] * scale.float() * torch.sign(g)
    return torch.where(torch.isfinite(amax), value, math.nan).flatten(-2)


def _plain_store(st):
    return _plain_quantised(st["k"]).to(st["k"].dtype), _plain_quantised(st["v"]).to(st["k"].dtype)


def _plain_values(rows, d):
    """Keys and values, in 32 bits, of cache rows [..., row bytes]."""
    signed = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device="cuda")
    pair = torch.stack([signed.repeat(16), signed.repeat_interleave(16)], -1)  # of a byte: low nibble, high nibble
    scales = rows[..., d:d + d // 8].contiguous().view(torch.float16).float().unflatten(-1, (2, d // GROUP))
    values = pair[rows[..., :d].int()].flatten(-2).unflatten(-1, (2, d // GROUP, GROUP)) * scales[..., None]
    values = values.flatten(-2)
    return values[..., 0, :], values[..., 1, :]


def _plain_softmax(q, k, v, seen, scale):
    """q [..., rows, D], k and v [..., L, D], seen (broadcast) [..., rows, L]: outputs and the logarithm of the sums."""
    s = (q @ k.transpose(-1, -2)) * scale
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), 0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, (p @ v) / total, 0)
    return o, (torch.log(total) + torch.where(torch.isinf(top), 0, top))[..., 0]


def _plain_attend(st):
    d, page, group, q = st["dim"], st["page"], st["group"], st["q"]
    h = st["cache"].shape[1]
    scale = 1.0 / math.sqrt(d)
    lengths, starts = st["lengths"].long(), st["starts"].long()
    n, tokens = lengths.numel(), q.shape[0]
    token = torch.arange(tokens, device="cuda")
    owner = torch.searchsorted(starts[1:], token, right=True)
    qf = q.float().unflatten(1, (h, group))
    if st["positions"] is not None:
        at = st["positions"].long()
        seen = (at >= 0) & (at < lengths[owner][:, None])
        at = torch.where(seen, at, 0)
        rows = st["cache"][st["table"].long()[owner[:, None], at // page].clamp(min=0), :, at % page]  # [T, list, H, bytes]
        k, v = _plain_values(rows.transpose(1, 2), d)
        o, lse = _plain_softmax(qf, k, v, seen[:, None, None, :], scale)
        return o.flatten(1, 2).to(q.dtype), lse.flatten(1, 2)
    longest = st["table"].shape[1] * page
    rows = st["cache"][st["table"].long().clamp(min=0)].transpose(2, 3).flatten(1, 2).transpose(1, 2)  # [R, H, L, bytes]
    k, v = _plain_values(rows, d)
    nth = token - starts[owner]
    wide = qf.new_zeros(n, st["max_new"], h, group, d)
    wide[owner, nth] = qf
    wide = wide.permute(0, 2, 1, 3, 4).flatten(2, 3)  # [R, H, new * group, D]
    last = lengths[:, None] - (starts[1:] - starts[:-1])[:, None] + torch.arange(st["max_new"], device="cuda")
    last = last.repeat_interleave(group, 1)[:, None, :, None]
    cell = torch.arange(longest, device="cuda")
    seen = (cell <= last) & (cell < lengths[:, None, None, None])
    if st["window"]:
        seen &= cell > last - st["window"]
    o, _ = _plain_softmax(wide, k, v, seen, scale)
    o = o.unflatten(2, (st["max_new"], group)).permute(0, 2, 1, 3, 4)[owner, nth]
    return o.flatten(1, 2).to(q.dtype)


_OWN = {"pages": _own_pages, "store": _own_store, "attend": _own_attend}
_PLAIN = {"pages": _plain_pages, "store": _plain_store, "attend": _plain_attend}


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


def _exact_rows(st, pages, offsets, head):
    """Keys and values in 64 bits of one head's cache rows."""
    d = st["dim"]
    raw = st["cache"][pages, head, offsets].long()
    code = torch.stack([raw[:, :d] & 15, raw[:, :d] >> 4], -1).reshape(-1, 2 * d)
    value = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")[code & 7] * (1 - 2 * (code >> 3)).double()
    word = raw[:, d:d + d // 8:2] | (raw[:, d + 1:d + d // 8:2] << 8)
    exponent, fraction = (word >> 10) & 31, (word & 1023).double()
    scale = torch.where(exponent == 0, fraction * 2.0 ** -24, (1024 + fraction) * _power(exponent - 25))
    value = value * scale.repeat_interleave(GROUP, 1)
    return value[:, :d], value[:, d:]


def exact(case, seed):
    if case["kind"] == "pages":
        return None
    st = prepare(case, seed)
    if case["kind"] == "store":
        return _exact_quantised(st["k"]), _exact_quantised(st["v"])
    q, page, group, d = st["q"].double(), st["page"], st["group"], st["dim"]
    lens, starts = st["lengths"].tolist(), st["starts"].tolist()
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for r, length in enumerate(lens):
        new = starts[r + 1] - starts[r]
        cells = torch.arange(length, device="cuda")
        pages = st["table"][r].long()[cells // page]
        for head in range(st["cache"].shape[1]):
            k, v = _exact_rows(st, pages, cells % page, head)
            for first in range(0, new, 256):
                count = min(256, new - first)
                rows = slice(starts[r] + first, starts[r] + first + count)
                last = length - new + first + torch.arange(count, device="cuda")[:, None]
                if st["positions"] is None:
                    seen = cells <= last
                    if st["window"]:
                        seen &= cells > last - st["window"]
                else:
                    at = st["positions"][rows].long()
                    hits = torch.zeros(count, length + 1, device="cuda")
                    hits.scatter_(1, torch.where((at < 0) | (at >= length), length, at), 1.0)
                    seen = hits[:, :length] > 0
                heads = slice(head * group, (head + 1) * group)
                s = torch.einsum("thd,ld->thl", q[rows, heads], k) / math.sqrt(d)
                s = s.masked_fill(~seen[:, None, :], -math.inf)
                lse[rows, heads] = torch.logsumexp(s, -1)
                out[rows, heads] = torch.softmax(s, -1) @ v
    return out if st["positions"] is None else (out, lse)


# ---- what a pass cannot do without

def work(case):
    if case["kind"] == "pages":
        n = case["requests"]
        tokens = n * case["max_new"]
        fresh = min(n, tokens // case["page"] + n)
        gone = case["ended"] * (case["max_len"] // 2 // case["page"])
        # lengths, new tokens, flags; slots and positions; starts and new lengths; the fresh and the returned cells
        return {"bytes": n * 9 + tokens * 12 + n * 8 + fresh * 8 + gone * 8, "flops": 0}
    if case["kind"] == "store":
        values = case["tokens"] * case["kv_heads"] * case["dim"] * 2
        # 16-bit values in and out again, 4.5 bits a value written and read
        return {"bytes": 4 * values + 2 * values * 9 // 16 + 8 * case["tokens"], "flops": 4 * values}
    lens, new = _lengths(case)
    heads, tokens = case["kv_heads"] * case["group"], sum(new)
    if case["listed"]:
        pairs = sum(b * min(case["listed"], a) for a, b in zip(lens, new))
        cells = sum(min(a, b * case["listed"]) for a, b in zip(lens, new))
    else:
        span = case["window"] or max(lens)
        cells = sum(min(a, span + b - 1) for a, b in zip(lens, new))
        pairs = sum(min(a - b + i + 1, span) for a, b in zip(lens, new) for i in range(b))
    once = 2 * 2 * tokens * heads * case["dim"] + 4 * tokens * case["listed"]
    return {"bytes": cells * case["kv_heads"] * case["dim"] * 9 // 8 + once, "flops": 4 * case["dim"] * heads * pairs}
