"""The 4-bit cache's definition in 64 bits, on the CPU: quantisation by exact
fractions, rows as bytes, page tables request by request, attention by explicit
sums. Shares no code with the GPU path."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GROUP = 32
SCALE_MAX = 10912


def row_bytes(d):
    return -(-(d + d // 8) // 16) * 16


def scale_of(amax: float) -> float:
    """The smallest number >= amax / 6 with 9 significant bits that is a multiple of 2^-23, at most 10912."""
    need = Fraction(float(amax)) / 6
    if need == 0:
        return 0.0
    if need > SCALE_MAX:
        return float(SCALE_MAX)
    step = Fraction(1, 2 ** 23)
    while -(-need // step) >= 512:  # too many bits at this step: the next coarser one
        step *= 2
    return float(min(Fraction(SCALE_MAX), -(-need // step) * step))


def code_of(x: float, scale: float) -> int:
    """The sign and code nearest to x / scale, ties to the even code (finite x)."""
    a, s = abs(Fraction(float(x))), Fraction(scale)
    best = min(range(8), key=lambda c: (abs(a - Fraction(LEVELS[c]) * s), c % 2, c)) if s else 0
    return best | (8 if math.copysign(1.0, x) < 0 else 0)


def quantise(x):
    """(scales [..., D / 32] float64 with NaN for a group that holds NaN or infinity, codes [..., D])."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(-1, GROUP)
    scales = np.empty(len(g))
    codes = np.zeros(g.shape, dtype=np.uint8)
    for i, row in enumerate(g):
        if not np.isfinite(row).all():
            scales[i] = math.nan
            continue
        scales[i] = scale_of(np.abs(row).max())
        codes[i] = [code_of(v, scales[i]) for v in row]
    return scales.reshape(*x.shape[:-1], -1), codes.reshape(x.shape)


def values(scales, codes):
    with np.errstate(invalid="ignore"):  # NaN scales
        return _values(scales, codes)


def _values(scales, codes):
    level = np.asarray(LEVELS)[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return level * np.repeat(scales, GROUP, axis=-1)


def rows_of(k, v):
    """Cache rows uint8 [..., row bytes] of keys and values [..., D]."""
    d = np.shape(k)[-1]
    parts, tail = [], []
    for x in (k, v):
        s, c = quantise(x)
        parts.append((c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8))
        tail.append(np.ascontiguousarray(s.astype(np.float16)).view(np.uint8))
    row = np.concatenate(parts + tail, axis=-1)
    pad = row_bytes(d) - row.shape[-1]
    return np.concatenate([row, np.zeros(row.shape[:-1] + (pad,), np.uint8)], axis=-1) if pad else row


def values_of(rows, d):
    """(k, v) in 64 bits of cache rows."""
    out = []
    for i in range(2):
        b = rows[..., i * (d // 2):(i + 1) * (d // 2)]
        codes = np.stack([b & 15, b >> 4], axis=-1).reshape(*b.shape[:-1], d)
        s = np.ascontiguousarray(rows[..., d + i * (d // 16):d + (i + 1) * (d // 16)]).view(np.float16)
        with np.errstate(invalid="ignore"):
            out.append(values(s.astype(np.float64), codes))
    return tuple(out)


def release(lengths, finished, table, free, num_free, page):
    free, lengths = free.copy(), np.array(lengths, np.int64)
    n = min(max(int(num_free), 0), len(free))
    for r, done in enumerate(finished):
        if done:
            for j in range(min(-(-max(int(lengths[r]), 0) // page), table.shape[1])):
                if n < len(free) and table[r, j] >= 0:  # (a cell below 0 holds no page)
                    free[n] = table[r, j]
                    n += 1
            lengths[r] = 0
    return lengths, free, n


def extend(lengths, new, table, free, num_free, page, max_tokens):
    table, out_lengths = table.copy(), np.array(lengths, np.int64)
    n = min(max(int(num_free), 0), len(free))
    slots, positions, starts, stopped = [], [], [0], False
    for r in range(len(lengths)):
        have, add = max(int(lengths[r]), 0), max(int(new[r]), 0)
        old, want = -(-have // page), -(-(have + add) // page)
        if want - old > n or len(slots) + add > max_tokens or want > table.shape[1] or have + add > 2 ** 31 - 1:
            stopped = True
        if not stopped:
            for j in range(old, want):
                n -= 1
                table[r, j] = free[n]
            for p in range(have, have + add):
                positions.append(p)
                slots.append(int(table[r, p // page]) * page + p % page if table[r, p // page] >= 0 else -1)
            out_lengths[r] = have + add
        starts.append(len(slots))
    pad = max_tokens - len(slots)
    return {"slots": np.array(slots + [-1] * pad, np.int64), "positions": np.array(positions + [-1] * pad, np.int32),
            "starts": np.array(starts, np.int32), "lengths": out_lengths, "num_free": n, "table": table}


def attention(q, rows_at, lengths, starts, kv_heads, scale, window=0, positions=None):
    """out, lse, and for error bounds: the weighted |v| and the largest sum of |q k| over the visible positions.

    q [tokens, heads, D]; rows_at(request, head, p) gives (k, v) of one position in 64 bits, or None where
    its page is outside the cache."""
    tokens, heads, d = q.shape
    group = heads // kv_heads
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    lse, reach = np.full((tokens, heads), -math.inf), np.zeros((tokens, heads))
    for r, length in enumerate(lengths):
        count = starts[r + 1] - starts[r]
        for h in range(kv_heads):
            known = {p: rows_at(r, h, p) for p in range(length)}
            for i in range(count):
                t, at = starts[r] + i, length - count + i
                if positions is None:
                    seen = [p for p in range(max(0, at - window + 1 if window else 0), at + 1)]
                else:
                    seen = [int(p) for p in positions[t] if 0 <= p < length]
                seen = [p for p in seen if known[p] is not None]
                if not seen:
                    continue
                k = np.stack([known[p][0] for p in seen])
                v = np.stack([known[p][1] for p in seen])
                for g in range(h * group, (h + 1) * group):
                    s = scale * (k @ q[t, g])
                    top = s.max()
                    w = np.exp(s - top)
                    out[t, g] = w @ v / w.sum()
                    size[t, g] = w @ np.abs(v) / w.sum()
                    lse[t, g] = top + math.log(w.sum())
                    reach[t, g] = abs(scale) * (np.abs(k) @ np.abs(q[t, g])).max()
    return out, lse, size, reach
