"""GPU parity of the 4-bit cache against its 64-bit oracle.

Page tables, slots, codes and scales are whole numbers or exact: they have to be
equal. Attention is compared within a bound derived from its arithmetic, eps =
2^-24: a logit is a sum of D exact products in fp32 on the tensor core, off by at most
D eps reach (reach: the largest sum of |scale q k| over the visible positions) and a
few roundings of factors (8 eps reach, and eps of the logit), so a weight by that much
relative and 2^-21 from the exponential: together d. The weights are rounded to fp16
(2^-11 relative, or 2^-33 of the largest where they become subnormal), the sums of n
terms add n eps. Numerator and denominator carry d each, so, with |v| averaged by
the weights in `size`,

    |out - ref| <= size (2 d + 2^-11 + 2 n eps) + n 2^-33 max|v| + u |ref|,   |lse - ref| <= d + n eps + 2^-21 (1 + |ref|)

where u is the output's rounding: 2^-8 (bf16), 2^-11 (fp16).
"""
import numpy as np
import pytest
import torch

from oracle import kv4 as ok

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_lt_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def num(t):
    return t.detach().cpu().double().numpy()


# ---- page tables

def check_extend(lengths, new, table, free, num_free, page, max_tokens):
    import sparse_attention_indexer_lt_gb300 as lt
    want = ok.extend(lengths, new, table, free, num_free, page, max_tokens)
    dev = [torch.as_tensor(np.asarray(x, np.int32)).cuda() for x in (lengths, new, table, free, [num_free])]
    got = lt.page_extend(*dev[:2], dev[2], dev[3], dev[4], page, max_tokens)
    torch.cuda.synchronize()
    assert np.array_equal(got.starts.cpu().numpy(), want["starts"])
    assert np.array_equal(got.lengths.cpu().numpy(), want["lengths"])
    assert int(got.num_free) == want["num_free"]
    assert np.array_equal(dev[2].cpu().numpy(), want["table"])
    assert np.array_equal(got.slots.cpu().numpy(), want["slots"])
    assert np.array_equal(got.positions.cpu().numpy(), want["positions"])
    return want


@pytest.mark.parametrize("requests", [0, 1, 2, 33, 1024, 1025, 3000])
@pytest.mark.parametrize("page", [1, 16, 1024])
def test_extend(requests, page):
    rng = np.random.default_rng(requests * 7 + page)
    lengths = rng.integers(-1, 40 if page < 1024 else 3000, requests).astype(np.int32)
    new = rng.integers(-2, 9, requests).astype(np.int32)
    width = max(1, (3008 if page == 1024 else 48) // page + 1)
    pages = requests * width + 5
    order = rng.permutation(pages).astype(np.int32)
    table = order[:requests * width].reshape(requests, width).copy()
    free = np.concatenate([order[requests * width:], order[:requests * width]])
    plenty = len(free)
    total = int(np.maximum(new, 0).sum())
    for num_free, room in ((plenty, total + 11), (plenty, total), (plenty, max(0, total - 3)), (plenty // 9, total + 300), (0, total),
                           (plenty + 100, total)):
        if requests == 0 and num_free > plenty:
            continue
        check_extend(lengths, new, table.reshape(requests, width), free, num_free, page, room)


def test_extend_stops_at_the_first_that_does_not_fit():
    table = np.full((4, 2), -1, np.int32)
    free = np.arange(10, dtype=np.int32)
    # request 1 wants three pages of a table two wide: nothing for it and the later ones
    want = check_extend([0, 5, 0, 0], [4, 6, 1, 1], table, free, 10, 4, 20)
    assert want["lengths"].tolist() == [4, 5, 0, 0] and want["starts"].tolist() == [0, 4, 4, 4, 4]
    check_extend([0, 2 ** 31 - 2, 0, 0], [4, 6, 1, 1], table, free, 10, 4, 20)
    # a hole in an old page gives slots of -1 (nothing is stored there)
    check_extend([2, 0, 0, 0], [2, 0, 0, 0], table, free, 10, 4, 20)


@pytest.mark.parametrize("requests", [0, 1, 5, 1023, 2500])
def test_release(requests):
    import sparse_attention_indexer_lt_gb300 as lt
    rng = np.random.default_rng(requests)
    page, width = 8, 7
    lengths = rng.integers(-2, 70, requests).astype(np.int32)  # some longer than their row of the table
    done = rng.random(requests) < 0.4
    table = rng.permutation(requests * width).astype(np.int32).reshape(requests, width)
    for capacity, num_free in ((requests * width + 9, 3), (requests * width // 3 + 4, 1), (5, 9)):
        free = np.full(capacity, -7, np.int32)
        want_l, want_f, want_n = ok.release(lengths, done, table, free, num_free, page)
        d = [torch.as_tensor(x).cuda() for x in (lengths, done, table, free, np.array([num_free], np.int32))]
        got_l, got_n = lt.page_release(*d[:4], d[4], page)
        torch.cuda.synchronize()
        assert np.array_equal(got_l.cpu().numpy(), want_l) and int(got_n) == want_n
        assert np.array_equal(d[3].cpu().numpy(), want_f)


# ---- storing and loading

def special(x):
    """Values at the quantiser's edges in the first groups."""
    x[0, 0, :32] = 0.0
    x[0, 0, 32:64] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4) * torch.tensor([1.0, -1.0] * 16)
    x[1, 0, :32] = 1e-9 * torch.arange(32)
    x[1, 0, 32:64] = 60000.0
    x[2, 0, 5] = float("inf")
    x[2, 0, 40] = float("nan")
    x[3, 0, :32] = torch.linspace(-6.0, 6.0, 32) * 2.0 ** -17
    x[3, 0, 32:64] = -x[0, 0, 32:64] * 11 / 16
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim,heads,page", [(64, 1, 1), (64, 3, 16), (128, 2, 32), (256, 1, 8)])
def test_store_and_load(dtype, dim, heads, page):
    import sparse_attention_indexer_lt_gb300 as lt
    torch.manual_seed(dim + heads)
    tokens, pages = 37, 64 if page == 1 else 9
    t = TYPES[dtype]
    k = special(torch.randn(tokens, heads, dim) * 10.0 ** torch.randint(-6, 3, (tokens, heads, 1))).to(t)
    v = special(torch.randn(tokens, heads, dim)).to(t)
    # keys and values as views of one projection, its channels at an odd offset for the scalar loads
    for wide in (True, False):
        extra = 0 if wide else 1
        both = torch.full((tokens, 2 * heads * dim + extra), 7.0, dtype=t)
        both[:, extra:] = torch.cat([k.flatten(1), v.flatten(1)], 1)
        both = both.cuda()
        kd, vd = both[:, extra:extra + heads * dim].unflatten(1, (heads, dim)), both[:, extra + heads * dim:].unflatten(1, (heads, dim))
        slots = torch.randperm(pages * page)[:tokens].long()
        slots[4], slots[5], slots[6] = -1, pages * page, -2 ** 40
        cache = torch.full((pages, heads, page, lt.kv4_row_bytes(dim)), 0xA5, dtype=torch.uint8, device="cuda")
        lt.kv4_store(kd, vd, cache, slots.cuda())
        c = cache.cpu().numpy()
        written = np.zeros((pages, page), bool)
        for i, s in enumerate(slots.tolist()):
            if 0 <= s < pages * page:
                written[s // page, s % page] = True
                row = c[s // page, :, s % page]
                want = ok.rows_of(num(k[i]), num(v[i]))
                scales = slice(dim, dim + dim // 8)
                g, w = row[:, scales].copy().view(np.float16), want[:, scales].copy().view(np.float16)
                assert np.array_equal(g, w, equal_nan=True), f"scales of token {i}"
                gk, wk = ok.values_of(row, dim), ok.values_of(want, dim)
                assert np.array_equal(gk, wk, equal_nan=True), f"values of token {i}"
        assert (c.transpose(0, 2, 1, 3)[~written] == 0xA5).all(), "rows without a slot were written"
        for out_type in TYPES.values():
            gk, gv = lt.kv4_load(cache, slots.cuda(), dtype=out_type)
            for i, s in enumerate(slots.tolist()):
                if 0 <= s < pages * page:
                    wk, wv = ok.values_of(c[s // page, :, s % page], dim)
                    for got, want in ((gk, wk), (gv, wv)):
                        want = torch.as_tensor(want).to(out_type)
                        assert torch.equal(torch.nan_to_num(got[i].cpu(), 99.0), torch.nan_to_num(want, 99.0))
                else:
                    assert not gk[i].any() and not gv[i].any()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_16_bit_magnitude_as_the_largest_of_a_group(dtype):
    """The scale of each finite magnitude, and codes of values spread below it, on either side of the borders."""
    import sparse_attention_indexer_lt_gb300 as lt
    t = TYPES[dtype]
    bits = torch.arange(0x7F80 if dtype == "bf16" else 0x7C00, dtype=torch.int32).to(torch.int16)
    top = bits.view(t)
    rows = (top.numel() + 7) // 8  # eight groups a token: key and value of D = 128
    top = torch.cat([top, top.new_zeros(rows * 8 - top.numel())]).view(rows, 8, 1)
    x = (top.float() * torch.linspace(-1.0, 1.0, 32)).to(t)
    x[..., 31] = top[..., 0]
    k, v = x[:, :4].reshape(rows, 1, 128), x[:, 4:].reshape(rows, 1, 128)
    cache = lt.kv4_cache((rows + 63) // 64, 1, 64, 128)
    slots = torch.arange(rows, device="cuda")
    lt.kv4_store(k.cuda(), v.cuda(), cache, slots)
    got = cache.view(-1, 144)[:rows].cpu().numpy()
    for i in range(0, rows, 7 if dtype == "bf16" else 5):
        want = ok.rows_of(num(k[i, 0]), num(v[i, 0]))
        assert np.array_equal(got[i, 128:], want[128:]), f"scales of row {i}"
        assert np.array_equal(ok.values_of(got[i], 128), ok.values_of(want, 128)), f"values of row {i}"


def test_store_of_many_tokens_and_a_repeat():
    import sparse_attention_indexer_lt_gb300 as lt
    torch.manual_seed(5)
    tokens, heads, dim, page = 5001, 3, 128, 64
    k, v = torch.randn(2, tokens, heads, dim, dtype=torch.bfloat16)
    cache = lt.kv4_cache(100, heads, page, dim)
    slots = torch.randperm(6400)[:tokens].cuda()
    lt.kv4_store(k.cuda(), v.cuda(), cache, slots)
    first = cache.clone()
    lt.kv4_store(k.cuda(), v.cuda(), cache, slots)
    assert torch.equal(first, cache)
    gk, gv = lt.kv4_load(cache, slots, dtype=torch.float32)
    for i in range(0, tokens, 499):
        for got, x in ((gk, k), (gv, v)):
            s, c = ok.quantise(num(x[i]))
            assert np.array_equal(num(got[i]), ok.values(s, c))
    lt.kv4_store(k[:0].cuda(), v[:0].cuda(), cache, slots[:0])
    assert torch.equal(first, cache) and lt.kv4_load(cache, slots[:0])[0].shape == (0, heads, dim)


# ---- attention

class Problem:
    """A filled cache with a random block table, and the oracle's view of it."""

    def __init__(self, lengths, new, heads, group, dim, page, dtype, seed=0, spread=1.0, extra_width=0, positions=None, magnitude=1.0):
        import sparse_attention_indexer_lt_gb300 as lt
        g = torch.Generator().manual_seed(seed)
        self.lengths, self.heads, self.dim, self.page = lengths, heads, dim, page
        self.starts = [0]
        for n in new:
            self.starts.append(self.starts[-1] + n)
        self.max_new = max(new + [1])
        held = [-(-n // page) for n in lengths]
        width = max(held + [1]) + extra_width
        order = torch.randperm(sum(held) + 3, generator=g).int()
        table = torch.full((len(lengths), width), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(held):
            table[r, :n] = order[at:at + n]
            at += n
        rows = lt.kv4_row_bytes(dim)
        shape = (sum(held) + 3, heads, page)
        # every byte random first: what no request holds is garbage, NaN scales among it
        cache = torch.randint(0, 256, shape + (rows,), generator=g, dtype=torch.uint8)
        scales = magnitude * 0.35 * torch.exp(0.3 * torch.randn(shape + (dim // 16,), generator=g))
        good = (scales.half().view(torch.int16) & -4).view(torch.uint8)
        for r, n in enumerate(lengths):
            for p in range(n):
                cache[table[r, p // page], :, p % page, dim:dim + dim // 8] = good[table[r, p // page], :, p % page]
        self.table, self.cache = table, cache
        self.q = (spread * torch.randn(self.starts[-1], heads * group, dim, generator=g)).to(TYPES[dtype])
        self.positions = positions

    def rows_at(self, r, h, p):
        page = int(self.table[r, p // self.page])
        if not 0 <= page < self.cache.shape[0]:
            return None
        if not hasattr(self, "_values"):
            self._values = ok.values_of(self.cache.numpy(), self.dim)
        return self._values[0][page, h, p % self.page], self._values[1][page, h, p % self.page]

    def run(self, **kw):
        import sparse_attention_indexer_lt_gb300 as lt
        pos = None if self.positions is None else torch.as_tensor(self.positions).int().cuda()
        starts = torch.tensor(self.starts, dtype=torch.int32).cuda()
        args = dict(starts=starts, max_new=self.max_new, positions=pos, with_lse=True)
        args.update(kw)
        q = args.pop("q", None)
        return lt.kv4_attention(self.q.cuda() if q is None else q, self.cache.cuda(), self.table.cuda(),
                                torch.tensor(self.lengths, dtype=torch.int32).cuda(), **args)

    def check(self, out, lse, window=0, scale=None):
        want, want_lse, size, reach = ok.attention(num(self.q), self.rows_at, self.lengths, self.starts, self.heads,
                                                   self.dim ** -0.5 if scale is None else scale, window, self.positions)
        n = max(self.lengths + [1]) if self.positions is None else np.shape(self.positions)[1]
        held = [self.rows_at(r, h, x) for r, n_r in enumerate(self.lengths) for h in range(self.heads) for x in range(n_r)]
        vmax = max([float(np.abs(x[1]).max()) for x in held if x is not None] + [0.0])
        d = (self.dim + 8) * EPS * reach + EPS * np.where(np.isfinite(want_lse), np.abs(want_lse), 0) + 2.0 ** -21
        u = 2.0 ** -8 if self.q.dtype == torch.bfloat16 else 2.0 ** -11
        tol = size * (2 * d[..., None] + 2.0 ** -11 + 2 * n * EPS) + n * 2.0 ** -33 * vmax + u * np.abs(want)
        err = np.abs(num(out) - want)
        assert np.isfinite(num(out)).all(), "not finite"
        assert (err <= tol).all(), f"out: {int((err > tol).sum())} off, worst {float((err - tol).max()):.3g} over its bound"
        got = num(lse)
        empty = np.isinf(want_lse)
        assert np.array_equal(np.isinf(got) & (got < 0), empty)
        assert not num(out)[empty].any()
        err = np.abs(got[~empty] - want_lse[~empty])
        tol = (d + n * EPS + 2.0 ** -21 * (1 + np.abs(np.where(empty, 0, want_lse))))[~empty]
        assert (err <= tol).all(), f"lse: worst {float((err / tol).max()):.3g} of its bound"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,heads,group", [(64, 2, 1), (64, 1, 3), (128, 2, 4), (128, 1, 16), (128, 1, 33), (256, 1, 8), (256, 1, 20)])
def test_decode(dim, heads, group, dtype):
    """One query a request: lengths of one, around the tile's 32 and a page's end, and longer."""
    p = Problem([1, 2, 31, 32, 33, 63, 64, 65, 200], [1] * 9, heads, group, dim, 16, dtype, seed=dim + group)
    p.check(*p.run())
    p.check(*p.run(starts=None))


@pytest.mark.parametrize("page", [1, 2, 8, 32, 64, 256, 1024])
def test_page_sizes(page):
    p = Problem([1, 77, 300], [1, 2, 3], 2, 4, 128, page, "bf16", seed=page)
    p.check(*p.run())


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64), ("bf16", 256)])
@pytest.mark.parametrize("window", [0, 1, 5, 32, 100, 10 ** 9])
def test_ragged_queries_and_windows(dtype, dim, window):
    """Requests of no, one and several new tokens; more queries than positions leave the first ones empty;
    a request without positions."""
    p = Problem([0, 5, 40, 130, 3, 70, 0], [1, 5, 0, 9, 6, 1, 0], 2, 3, dim, 8, dtype, seed=window % 97, extra_width=3)
    p.check(*p.run(window=window), window=window)


def test_many_query_rows():
    """More query rows than one CTA takes: several row tiles a request."""
    p = Problem([90, 150], [50, 33], 1, 5, 128, 32, "bf16", seed=3)
    p.check(*p.run())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,lengths,new,group,window", [
    (64, [64], [64], 1, 0), (128, [64], [64], 1, 0), (64, [130], [100], 2, 0), (128, [300], [129], 1, 0), (128, [129, 5, 400], [70, 0, 33], 5, 0),
    (64, [700, 90, 1], [100, 90, 1], 3, 50), (128, [640], [90], 3, 200), (64, [1500], [40], 4, 0), (128, [50], [80], 4, 0),
    (256, [100], [70], 1, 0), (256, [300, 0, 5, 33], [129, 70, 0, 33], 1, 0), (256, [700, 64], [40, 17], 4, 150), (256, [1300], [33], 2, 0)])
def test_prefill(dim, lengths, new, group, window, dtype):
    """Many query rows a request: one and two row tiles, ragged ends, windows, requests cut into parts, more
    queries than positions."""
    p = Problem(lengths, new, 2, group, dim, 16, dtype, seed=sum(lengths) + dim, extra_width=1)
    out, lse = p.run(window=window)
    p.check(out, lse, window=window)
    again, _ = p.run(window=window)
    assert torch.equal(out, again), "two runs differ"


@pytest.mark.parametrize("page", [1, 32, 64, 128, 1024])
def test_prefill_page_sizes_with_parts_and_windows(page):
    """Parts and windows that start inside a page, runs of positions longer and shorter than a page."""
    for window, dim in ((0, 64), (77, 64), (300, 64), (77, 256)):
        p = Problem([1100, 161], [33, 20], 1, 3, dim, page, "f16", seed=page + window)
        p.check(*p.run(window=window), window=window)


def test_prefill_of_empty_and_of_many_requests():
    p = Problem([0, 200, 0], [90, 70, 64], 1, 1, 64, 16, "f16", seed=31, extra_width=1)
    p.check(*p.run())
    p = Problem([64 + (r * 7) % 40 for r in range(40)], [64 + r % 3 for r in range(40)], 1, 1, 64, 16, "bf16", seed=32)
    p.check(*p.run())


def test_prefill_scales_and_bad_pages():
    for spread, magnitude, scale in ((30.0, 1.0, None), (1.0, 1.0, -0.2), (1.0, 1.0, 0.0), (1.0, 1e-4, 300.0), (1.0, 3000.0, 1e-4)):
        p = Problem([300], [40], 1, 4, 64, 16, "bf16", seed=21, spread=spread, magnitude=magnitude)
        p.table[0, 3] = -1
        p.table[0, 17] = 2 ** 31 - 1
        p.check(*p.run(scale=scale), scale=scale)


@pytest.mark.parametrize("dim", [128, 256])
def test_prefill_nan_where_nothing_looks(dim):
    p = Problem([200], [80], 1, 2, dim, 16, "bf16", seed=22)
    clean, clean_lse = p.run()
    nan = torch.tensor([0x7FFF], dtype=torch.int16).view(torch.uint8)
    for position, byte in ((150, dim + dim // 16 + 2), (199, dim)):  # value group 1 of position 150, key group 0 of the last
        p.cache[p.table[0, position // 16], 0, position % 16, byte:byte + 2] = nan
    out, lse = p.run()
    assert torch.equal(out[:30], clean[:30]) and torch.equal(lse[:79], clean_lse[:79])
    assert torch.isnan(out[30:79, :, 32:64]).all()
    assert torch.equal(out[30:79, :, :32], clean[30:79, :, :32]) and torch.equal(out[30:79, :, 64:], clean[30:79, :, 64:])
    assert torch.isnan(out[79]).all() and torch.isnan(lse[79]).all()


@pytest.mark.parametrize("dim,group,most", [(64, 5, 5), (128, 5, 5), (64, 10, 6), (256, 10, 3)])
def test_many_requests_of_some_query_rows(dim, group, most):
    """Row tiles of 32 (16 for D = 256), two of them for some requests, where there are CTAs for every SM."""
    p = Problem([1 + (r * 11) % 70 for r in range(45)], [1 + r % most for r in range(45)], 1, group, dim, 16, "bf16", seed=dim + most)
    for window in (0, 9):
        p.check(*p.run(window=window), window=window)


@pytest.mark.parametrize("dim,heads,group,list_len", [(64, 2, 4, 1), (128, 1, 16, 33), (128, 2, 8, 512), (256, 1, 4, 100), (128, 1, 40, 130)])
def test_listed(dim, heads, group, list_len):
    rng = np.random.default_rng(list_len)
    lengths, new = [400, 1, 90, 0], [3, 1, 2, 1]
    pos = np.full((sum(new), list_len), -1)
    t = 0
    for n, c in zip(lengths, new):
        for i in range(c):
            take = rng.integers(-3, n + 9, list_len)  # pads, positions past the end, repeats
            pos[t] = take if i != 1 else -1           # (one list is empty)
            t += 1
    p = Problem(lengths, new, heads, group, dim, 16, "bf16", seed=list_len, positions=pos)
    p.check(*p.run())


@pytest.mark.parametrize("requests", [1, 3, 130, 300])
def test_split_requests_join_to_the_same(requests):
    """Long requests are cut into parts and joined; more requests than a CTA's threads scan at once."""
    lengths = [(r * 389) % 1500 + 1 if requests < 100 else (r * 37) % 90 for r in range(requests)]
    p = Problem(lengths, [1] * requests, 1, 2, 64, 64, "f16", seed=requests)
    out, lse = p.run(starts=None)
    p.check(out, lse)
    again, lse2 = p.run(starts=None)
    assert torch.equal(out, again) and torch.equal(lse, lse2), "two runs differ"


@pytest.mark.parametrize("lengths,new", [([20000], [1]), ([17000, 3, 0, 9000], [2, 1, 1, 0]), ([300] * 40 + [17001], [1] * 41)])
def test_long_tables_are_cut_into_chunks(lengths, new):
    """Tables too long for parts of one size: chunks of like work over all requests, and a second launch."""
    p = Problem(lengths, new, 1, 2, 64, 64, "bf16", seed=len(lengths))
    out, lse = p.run()
    p.check(out, lse)
    assert torch.equal(out, p.run()[0])


def test_a_great_many_requests_stay_whole():
    """More requests than chunks would serve, of tables longer than a part: rows against the same rows alone."""
    import sparse_attention_indexer_lt_gb300 as lt
    torch.manual_seed(3)
    n, heads, page, width = 700, 8, 64, 40
    cache = torch.randint(0, 256, (300, heads, page, 80), dtype=torch.uint8, device="cuda")
    scales = (0.35 * torch.exp(0.3 * torch.randn(300, heads, page, 4, device="cuda"))).half().view(torch.int16) & -4
    cache[..., 64:72] = scales.view(torch.uint8)
    table = torch.randint(0, 300, (n, width), dtype=torch.int32, device="cuda")
    lengths = torch.randint(0, width * page + 1, (n,), dtype=torch.int32, device="cuda")
    lengths[:3] = torch.tensor([0, 1, width * page])
    q = torch.randn(n, heads * 2, 64, device="cuda").half()
    out, lse = lt.kv4_attention(q, cache, table, lengths, with_lse=True)
    for r in (0, 1, 2, 350, 699):
        one, one_lse = lt.kv4_attention(q[r:r + 1], cache, table[r:r + 1], lengths[r:r + 1].clone(), with_lse=True)
        # the same sums in another order: fp32 sums of up to 2560 terms, outputs rounded to fp16
        assert (one.float() - out[r:r + 1].float()).abs().max() <= 2.0 ** -10 * 6 and torch.allclose(one_lse, lse[r:r + 1], atol=1e-4, rtol=0)
    assert not out[0].any() and torch.isinf(lse[0]).all()


def test_scales_and_spreads():
    """Peaked and flat rows, a negative and a zero scale, small and large stored values."""
    for spread, magnitude, scale in ((30.0, 1.0, None), (1e-3, 1.0, None), (1.0, 1.0, -0.2), (1.0, 1.0, 0.0), (1.0, 1e-4, 300.0), (1.0, 3000.0, 1e-4)):
        for dtype in ("bf16", "f16"):
            p = Problem([50, 200], [1, 2], 1, 4, 64, 16, dtype, seed=11, spread=spread, magnitude=magnitude)
            p.check(*p.run(scale=scale), scale=scale)


def test_large_and_small_bf16_queries():
    """bf16 queries outside fp16's range."""
    for power in (-100, 100):
        p = Problem([70], [1], 1, 4, 64, 16, "bf16", seed=12)
        p.q = (p.q.float() * 2.0 ** power).bfloat16()
        scale = 2.0 ** -power / 8
        p.check(*p.run(scale=scale), scale=scale)


def test_strided_queries_and_given_outputs():
    import sparse_attention_indexer_lt_gb300 as lt
    p = Problem([33, 100], [2, 3], 2, 4, 128, 16, "bf16", seed=4)
    out, lse = p.run()
    wide = torch.randn(5, 16 + 3, 128 + 8, device="cuda").bfloat16()
    q = wide[:, 2:10, :128]
    q.copy_(p.q)
    given, given_lse = torch.empty_like(out), torch.empty_like(lse)
    space = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    got, got_lse = p.run(q=q, out=given, out_lse=given_lse, workspace=space)
    assert got.data_ptr() == given.data_ptr() and torch.equal(out, got) and torch.equal(lse, got_lse)
    with pytest.raises(ValueError):
        p.run(q=wide[:, 2:10, 4:132])  # not 16-byte aligned
    assert torch.equal(out, p.run(q=q, workspace=space[:16])[0])  # (short requests need none)
    long = Problem([40000], [1], 1, 4, 64, 64, "bf16", seed=4)
    with pytest.raises(ValueError):
        long.run(workspace=space[:16])
    with pytest.raises(ValueError):
        p.run(starts=None)
    with pytest.raises(ValueError):
        p.run(out=given[:1])
    with pytest.raises(ValueError):
        p.run(window=-1)
    with pytest.raises(TypeError):
        p.run(q=q.float())
    with pytest.raises(ValueError):
        p.run(positions=torch.zeros(5, 0, dtype=torch.int32, device="cuda"))
    assert lt.kv4_attention(q[:0], p.cache.cuda(), p.table.cuda(), torch.tensor([3, 3], dtype=torch.int32, device="cuda"),
                            starts=torch.zeros(3, dtype=torch.int32, device="cuda")).shape == (0, 8, 128)


def test_rows_past_the_last_request_are_not_touched():
    p = Problem([40, 20], [2, 1], 1, 4, 64, 16, "bf16", seed=5)
    q = torch.cat([p.q, p.q]).cuda()
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    p.run(q=q, out=out, out_lse=lse)
    assert (out[3:] == 7.0).all() and (lse[3:] == 7.0).all()
    p.check(out[:3], lse[:3])


@pytest.mark.parametrize("bad_page", [-1, -2 ** 31, 2 ** 31 - 1, None])
def test_positions_on_pages_outside_the_cache_are_not_seen(bad_page):
    p = Problem([100, 64], [3, 1], 1, 4, 128, 16, "bf16", seed=6)
    p.table[0, 2] = p.cache.shape[0] if bad_page is None else bad_page
    p.table[0, 6] = -1  # the last page, partly filled
    p.check(*p.run())
    pos = np.tile(np.arange(100), (4, 1))
    p.positions = pos
    p.check(*p.run())


def test_nan_where_nothing_looks():
    """NaN stored at positions that a row's mask hides leaves the row as it is; a row that sees one gets NaN
    in that group (value) or everywhere (key)."""
    for window in (0, 20):
        p = Problem([70], [6], 1, 2, 128, 16, "bf16", seed=7)
        clean, clean_lse = p.run(window=window)
        nan = torch.tensor([0x7FFF], dtype=torch.int16).view(torch.uint8)

        def poison(position, byte):
            p.cache[p.table[0, position // 16], 0, position % 16, byte:byte + 2] = nan
        poison(67, 128 + 8 + 2)      # value group 1 of position 67: queries 3, 4, 5 see it
        poison(69, 128)              # key group 0 of position 69: the last query alone
        if window:
            poison(45, 128 + 8)      # value group 0 of position 45: queries 0 (position 64) sees it, later ones do not
        out, lse = p.run(window=window)
        first = 1 if window else 0
        assert torch.equal(out[first:3], clean[first:3]) and torch.equal(lse[first:5], clean_lse[first:5])
        if window:
            assert torch.isnan(out[0, :, :32]).all() and torch.equal(out[0, :, 32:], clean[0, :, 32:])
        assert torch.isnan(out[3:5, :, 32:64]).all()
        assert torch.equal(out[3:5, :, :32], clean[3:5, :, :32]) and torch.equal(out[3:5, :, 64:], clean[3:5, :, 64:])
        assert torch.isnan(out[5]).all() and torch.isnan(lse[5]).all()


def test_cache_beyond_32_bit_offsets():
    import sparse_attention_indexer_lt_gb300 as lt
    page, heads, dim = 64, 1, 128
    pages = (5 << 30) // (page * lt.kv4_row_bytes(dim))
    cache = lt.kv4_cache(pages, heads, page, dim)
    table = torch.tensor([[pages - 1, 3, pages - 7]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([150], dtype=torch.int32, device="cuda")
    k, v = torch.randn(2, 150, heads, dim, device="cuda").half()
    p = torch.arange(150, device="cuda")
    slots = table[0].long()[p // page] * page + p % page
    lt.kv4_store(k, v, cache, slots)
    lk, lv = lt.kv4_load(cache, slots, dtype=torch.float32)
    q = torch.randn(1, 4, dim, device="cuda").half()
    for kw in ({}, {"positions": torch.arange(150, dtype=torch.int32, device="cuda")[None]}):
        out = lt.kv4_attention(q, cache, table, lengths, **kw)
        s = torch.einsum("hd,ld->hl", q[0].double(), lk[:, 0].double()) / dim ** 0.5
        want = torch.softmax(s, -1) @ lv[:, 0].double()
        assert (out[0].double() - want).abs().max() < 4e-3
    del cache


def test_streams_and_graphs():
    import sparse_attention_indexer_lt_gb300 as lt
    p = Problem([500, 90], [1, 1], 2, 4, 128, 16, "bf16", seed=9)
    want, _ = p.run(starts=None)
    q, cache, table = p.q.cuda(), p.cache.cuda(), p.table.cuda()
    lengths = torch.tensor(p.lengths, dtype=torch.int32).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lt.kv4_attention(q, cache, table, lengths, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    with torch.cuda.stream(side):
        lt.kv4_attention(q, cache, table, lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lt.kv4_attention(q, cache, table, lengths)
    lengths.copy_(torch.tensor([90, 33], dtype=torch.int32))
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, lt.kv4_attention(q, cache, table, lengths)) and not torch.equal(out, want)


def test_injected_launch_failures():
    import sparse_attention_indexer_lt_gb300 as lt
    lib = lt.load()
    p = Problem([50], [1], 1, 4, 64, 16, "bf16", seed=10)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv, cache, slots = torch.zeros(1, 1, 64, device="cuda"), p.cache.cuda(), torch.zeros(1, dtype=torch.int64, device="cuda")
    for call in (p.run, lambda: lt.kv4_store(kv, kv, cache, slots), lambda: lt.kv4_load(cache, slots),
                 lambda: lt.page_release(z, z.bool(), z[None], z, z, 16), lambda: lt.page_extend(z, z, z[None], z, z, 16, 4)):
        assert lib.lt_test_inject(1, 1) == 0
        with pytest.raises(lt.LtError):
            call()
        call()
    torch.cuda.synchronize()


def test_a_serving_step_end_to_end():
    """Extend, store, attend and release over several steps against a dense copy of what was stored."""
    import sparse_attention_indexer_lt_gb300 as lt
    torch.manual_seed(1)
    n, page, width, heads, group, dim = 3, 16, 12, 2, 4, 128
    cache = lt.kv4_cache(n * width, heads, page, dim)
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(n * width).int().cuda()
    num_free = torch.tensor([n * width], dtype=torch.int32, device="cuda")
    lengths = torch.zeros(n, dtype=torch.int32, device="cuda")
    kept = [([], []) for _ in range(n)]
    for new in ([40, 1, 7], [1, 1, 1], [0, 5, 1], [1, 30, 2]):
        tokens = sum(new) + 2  # two rows of padding
        k, v = torch.randn(2, tokens, heads, dim, device="cuda").bfloat16()
        q = torch.randn(tokens, heads * group, dim, device="cuda").bfloat16()
        step = lt.page_extend(lengths, torch.tensor(new, dtype=torch.int32).cuda(), table, free, num_free, page, tokens)
        lt.kv4_store(k, v, cache, step.slots)
        out = lt.kv4_attention(q, cache, table, step.lengths, starts=step.starts, max_new=max(new))
        lk, lv = lt.kv4_load(cache, step.slots, dtype=torch.float32)
        lengths, num_free = step.lengths, step.num_free
        at = 0
        for r, count in enumerate(new):
            kept[r][0].append(lk[at:at + count])
            kept[r][1].append(lv[at:at + count])
            kk, vv = torch.cat(kept[r][0]).double(), torch.cat(kept[r][1]).double()
            for i in range(count):
                upto = len(kk) - count + i + 1
                for h in range(heads * group):
                    s = kk[:upto, h // group] @ q[at + i, h].double() / dim ** 0.5
                    want = torch.softmax(s, -1) @ vv[:upto, h // group]
                    assert (out[at + i, h].double() - want).abs().max() < 3e-2
            at += count
    before = int(num_free)
    lengths, num_free = lt.page_release(lengths, torch.tensor([True, False, True], device="cuda"), table, free, num_free, page)
    held = [-(-sum(x) // page) for x in ([40, 1, 0, 1], [7, 1, 1, 2])]
    assert int(num_free) == before + sum(held) and lengths.tolist() == [0, 37, 0]


def test_the_example_runs_and_is_right():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_step.py")
    spec = importlib.util.spec_from_file_location("sparse_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    for kw in ({"tokens": 400, "steps": 9}, {"tokens": 64, "steps": 4, "k": 100, "head_dim": 64, "kv_heads": 1}):
        results, held, free, pages = example.run(**kw)
        # outputs are averages of values of unit size, rounded to bf16 and with fp16 weights
        assert example.check(results, held) < 2.0 ** -8 * 4 + 2.0 ** -9 * 4
        assert free == pages and len(results) == kw["steps"]


@pytest.mark.parametrize("bits", [0x7C00, 0xFC00, 0x7BFF, 0x7155])
@pytest.mark.parametrize("dim,new,group,window", [(64, 6, 2, 0), (64, 6, 2, 20), (128, 6, 2, 0), (128, 6, 2, 20), (128, 3, 10, 20), (256, 6, 2, 20),
                                                  (64, 80, 2, 0), (64, 80, 2, 90), (128, 80, 2, 0), (128, 80, 2, 90), (256, 80, 2, 0), (256, 80, 2, 90)])
def test_scales_outside_the_format_where_nothing_looks(bits, dim, new, group, window):
    """Infinite scales, and finite ones above 10912 (whose product with a code overflows fp16), at positions that a
    row's mask hides leave the row as it is: later than the row's own, before its window, before every row's."""
    p = Problem([200], [new], 1, group, dim, 16, "bf16", seed=dim + new + window)
    clean, clean_lse = p.run(window=window)
    scale = torch.tensor([bits - 0x10000 if bits > 0x7FFF else bits], dtype=torch.int16).view(torch.uint8)
    codes = torch.tensor([0x00, 0x77, 0x70, 0xF7] * 4, dtype=torch.uint8)  # 0 * inf and 6 * 10920 both

    def put(position, value_group=None, key_group=None):
        row = p.cache[p.table[0, position // 16], 0, position % 16]
        if value_group is not None:
            row[dim + dim // 16 + 2 * value_group:][:2] = scale
            row[dim // 2 + 16 * value_group:][:16] = codes
        if key_group is not None:
            row[dim + 2 * key_group:][:2] = scale
            row[16 * key_group:][:16] = codes
    first, late = 0, new // 2
    put(200 - new + late, value_group=1)       # seen by the queries from `late` on
    if window:
        first = 1
        lowest = 200 - new - window + 1        # the lowest position of query 0, which no later one sees
        put(lowest, value_group=0)
        put(lowest - 1, value_group=1, key_group=0)  # seen by none
    out, lse = p.run(window=window)
    assert torch.equal(lse, clean_lse)
    assert torch.equal(out[first:late], clean[first:late])
    keep = [c for c in range(dim) if not 32 <= c < 64]
    assert torch.equal(out[late:, :, keep], clean[late:, :, keep])
    put(199, key_group=1)                      # the last query's own position
    out, lse = p.run(window=window)
    # (one row's logits may move when the others' maximum is taken: two results within their bounds of the same)
    vmax = 6 * 0.35 * 2.72
    assert ((out[first:late] - clean[first:late]).float().abs() <= 2 * (2.0 ** -8 * clean[first:late].float().abs() + 2.0 ** -10 * vmax)).all()
    assert (lse[:-1] - clean_lse[:-1]).abs().max() <= 1e-4


@pytest.mark.parametrize("requests,width", [(1, 1), (1, 5000), (3, 40), (33, 300), (1500, 7), (2500, 40)])
def test_release_takes_no_cell_that_holds_no_page(requests, width):
    """Cells below 0 in an ended request's row (pages dropped behind a window, or never given) are not pages."""
    import sparse_attention_indexer_lt_gb300 as lt
    rng = np.random.default_rng(requests + width)
    page = 8
    lengths = rng.integers(-2, width * page + 20, requests).astype(np.int32)
    done = rng.random(requests) < 0.5
    done[0] = True
    if requests == 2500:
        done[1:1500] = False  # (few cells first, many later)
    table = rng.permutation(requests * width).astype(np.int32).reshape(requests, width)
    table[rng.random((requests, width)) < 0.3] = -1
    table[rng.random((requests, width)) < 0.05] = -2 ** 31
    if requests > 2:
        table[1] = -1
    for capacity, num_free in ((requests * width + 9, 3), (requests * width // 5 + 4, 1)):
        free = np.full(capacity, -7, np.int32)
        free[:num_free] = requests * width + np.arange(num_free)
        held = [int(x) for r in range(requests) if done[r] for x in table[r, :-(-max(int(lengths[r]), 0) // page)] if x >= 0]
        want = np.concatenate([free[:num_free], np.array(held, np.int32)])[:capacity]
        d = [torch.as_tensor(x).cuda() for x in (lengths, done, table, free, np.array([num_free], np.int32))]
        got_l, got_n = lt.page_release(*d[:4], d[4], page)
        torch.cuda.synchronize()
        assert np.array_equal(got_l.cpu().numpy(), np.where(done, 0, lengths))
        assert int(got_n) == len(want)
        got = d[3].cpu().numpy()
        assert np.array_equal(got[:len(want)], want) and (got[len(want):] == -7).all()
        oracle = ok.release(lengths, done, table, free, num_free, page)
        assert oracle[2] == len(want) and np.array_equal(oracle[1], got)
        # what is taken next are pages
        few = min(len(want), 50)
        rows = torch.full((1, 64), -1, dtype=torch.int32, device="cuda")
        zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        step = lt.page_extend(zero, zero + few * page, rows, d[3], got_n, page, few * page)
        assert int(step.lengths) == few * page and (step.slots >= 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_stored_rows_are_the_oracles_byte_for_byte(dtype, dim):
    """Codes with the sign of zeros, and the padding; scales of groups with NaN are some NaN."""
    import sparse_attention_indexer_lt_gb300 as lt
    torch.manual_seed(dim)
    t = TYPES[dtype]
    x = special(torch.randn(24, 2, dim) * 10.0 ** torch.randint(-6, 3, (24, 2, 1)))
    x[5, :, :32] = torch.tensor([0.0, -0.0] * 16)                   # a group of zeros alone
    x[6, :, :32] = torch.tensor([-0.0, 3.0, 0.0, -1e-6, 1e-6, -6.0, -0.0, 1.0] * 4)
    x[7, :, 32:64] = torch.tensor([-0.0, -1e-9, 1e-9, 0.0] * 8)
    x[8:16][x[8:16].abs() < 0.5] = -0.0
    x = x.to(t)
    for k, v in ((x, x.flip(0)), (x.flip(0), x)):
        cache = torch.full((3, 2, 8, lt.kv4_row_bytes(dim)), 0xA5, dtype=torch.uint8, device="cuda")
        lt.kv4_store(k.cuda(), v.cuda(), cache, torch.arange(24, device="cuda"))
        got = cache.cpu().transpose(1, 2).reshape(24, 2, -1).numpy()
        for i in range(24):
            want = ok.rows_of(num(k[i]), num(v[i]))
            scales = slice(dim, dim + dim // 8)
            assert np.array_equal(got[i, :, :dim], want[:, :dim]), f"codes of token {i}"
            assert np.array_equal(got[i, :, scales].copy().view(np.float16), want[:, scales].copy().view(np.float16), equal_nan=True)
            assert np.array_equal(got[i, :, dim + dim // 8:], want[:, dim + dim // 8:]), f"padding of token {i}"


def _workspace(tokens, q_heads, kv_heads, dim, requests, max_new, positions, window=0):
    import ctypes

    import sparse_attention_indexer_lt_gb300 as lt
    need = ctypes.c_int64(-1)
    assert lt.load().lt_kv4_workspace(tokens, q_heads, kv_heads, dim, requests, max_new, 0, positions, window, ctypes.byref(need)) == 0
    return need.value


@pytest.mark.parametrize("tokens,q_heads,kv_heads,dim,requests,max_new", [
    (1215, 32, 8, 128, 64, 1152), (1407, 32, 8, 128, 256, 1152), (5000, 32, 8, 128, 1000, 500), (768, 128, 8, 256, 256, 3),
    (320, 64, 8, 128, 64, 5), (4000, 16, 4, 64, 6, 1500)])
def test_workspace_is_for_the_parts_that_can_be(tokens, q_heads, kv_heads, dim, requests, max_new):
    """With c chunks wanted for all the requests a chunk has at least a cth of their positions, so the requests that
    are longer than a chunk are cut into fewer than 2 c parts, each of the most query rows that a request has: the
    scratch memory does not grow with the requests that stay whole."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = max_new * (q_heads // kv_heads)
    tile = 128 if dim == 256 else 256
    wanted = -(-sms // (kv_heads * -(-rows // tile)))
    parts = 2 * wanted * kv_heads * rows
    assert _workspace(tokens, q_heads, kv_heads, dim, requests, max_new, 65536) <= parts * (dim + 1) * 4 + 8 * requests + 64


@pytest.mark.parametrize("lengths,new,dim,group", [
    ([5, 2600, 40, 1700, 0, 1300, 7], [3, 20, 1, 33, 0, 17, 7], 64, 1),           # many rows, several requests in parts among whole ones
    ([700, 1, 1300, 9], [19, 1, 40, 2], 128, 2), ([9, 900, 3, 700], [2, 17, 3, 30], 256, 1),
    ([2100, 30, 1600], [150, 3, 90], 64, 3),                                      # (more than one row tile)
    ([40] * 20 + [3000] + [50] * 60 + [2500, 1, 600] + [60] * 70, [1] * 154, 64, 2),  # few rows, more requests than a CTA has threads
    ([17000] + [30] * 20 + [9000, 5], [2] + [1] * 20 + [2, 2], 64, 2)])
def test_requests_in_parts_among_whole_ones(lengths, new, dim, group):
    p = Problem(lengths, new, 1, group, dim, 64, "f16", seed=sum(new), extra_width=230)
    out, lse = p.run()
    p.check(out, lse)
    again, lse2 = p.run(max_new=p.max_new + 3)
    p.check(again, lse2)


def test_a_long_chunk_beside_requests_of_one_token():
    """A step that mixes a prefill chunk with decoding requests, scratch memory given at its stated size."""
    new = [1] * 10 + [70] + [1] * 30
    lengths = [(r * 53) % 300 + 1 for r in range(10)] + [1400] + [(r * 31) % 200 + 1 for r in range(30)]
    for dim, heads, group in ((64, 2, 2), (256, 1, 2)):
        p = Problem(lengths, new, heads, group, dim, 16, "bf16", seed=dim)
        need = _workspace(sum(new), heads * group, heads, dim, len(new), 70, p.table.shape[1] * 16)
        space = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        p.check(*p.run(workspace=space[:need]))
        assert (space[need:] == 0x5A).all(), "written past the scratch memory"


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_queries_past_max_new_are_not_computed(dim):
    """A max_new below a request's queries: its rows from there on are not touched, and nobody else's are harmed."""
    lengths, new = [1500, 30, 1300], [40, 3, 33]
    p = Problem(lengths, new, 1, 2, dim, 64, "f16", seed=dim)
    want, want_lse = p.run(max_new=40)
    out, lse = torch.full_like(want, 7.0), torch.full_like(want_lse, 7.0)
    need = _workspace(sum(new), 2, 1, dim, 3, 25, p.table.shape[1] * 64)
    space = torch.full((need + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    p.run(max_new=25, out=out, out_lse=lse, workspace=space[:need])
    for first, count in ((0, 40), (40, 3), (43, 33)):
        got = min(count, 25)
        a, b = out[first:first + got].float(), want[first:first + got].float()
        assert ((a - b).abs() <= 2.0 ** -10 * b.abs() + 2.0 ** -10 * 6 * 0.35 * 2.72).all()
        assert (lse[first:first + got] - want_lse[first:first + got]).abs().max() <= 1e-4
        assert (out[first + got:first + count] == 7.0).all() and (lse[first + got:first + count] == 7.0).all()
    assert (space[need:] == 0x5A).all()


@pytest.mark.parametrize("dim,new", [(64, 2), (64, 70), (128, 70), (256, 70)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_scale_of_zero_keeps_what_is_not_finite(dim, new, dtype):
    """0 * NaN and 0 * inf are NaN: the row of such a query, and no other."""
    p = Problem([100], [new], 1, 1, dim, 16, dtype, seed=dim + new)
    clean, clean_lse = p.run(scale=0.0)
    p.check(clean, clean_lse, scale=0.0)
    p.q[0, 0, 5], p.q[1, 0, dim - 1] = float("nan"), float("-inf")
    out, lse = p.run(scale=0.0)
    assert torch.isnan(out[:2]).all() and torch.isnan(lse[:2]).all()
    assert torch.equal(out[2:], clean[2:]) and torch.equal(lse[2:], clean_lse[2:])
