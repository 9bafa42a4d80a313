"""The 4-bit cache's oracle, pinned by hand-worked cases and by brute force, and
the refusals of its calls that need no GPU."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import kv4 as ok


def test_scales_by_hand():
    assert ok.scale_of(0.0) == 0.0
    assert ok.scale_of(6.0) == 1.0
    assert ok.scale_of(6.0000005) == 1.0 + 2.0 ** -8     # the next number of 9 bits
    assert ok.scale_of(11.99) == 2.0                     # 1.99833 -> 512 / 256
    assert ok.scale_of(1.0) == 171 / 1024                # 0.16667 -> ceil(170.67) / 1024... of 9 bits: 342 / 2048
    assert ok.scale_of(3e38) == 10912.0
    assert ok.scale_of(1e-30) == 2.0 ** -23
    assert ok.scale_of(6 * 2.0 ** -23) == 2.0 ** -23
    assert ok.scale_of(65472.0) == 10912.0


def test_scale_is_the_smallest_of_its_grid():
    grid = sorted({Fraction(n, 2 ** 23) for n in range(512)} | {Fraction(n) * Fraction(2) ** e for n in range(256, 512) for e in range(-23, -10)})
    for amax in np.random.default_rng(1).lognormal(-10, 3, 200).astype(np.float32):
        need = Fraction(float(amax)) / 6
        if need <= grid[-1]:
            assert ok.scale_of(amax) == float(min(s for s in grid if s >= need))


def test_codes_are_nearest_with_ties_to_even():
    borders = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    for x, c in borders.items():
        assert ok.code_of(x, 1.0) == c and ok.code_of(-x, 1.0) == c | 8
    for x in np.linspace(-6, 6, 4001):
        c = ok.code_of(x, 1.0)
        got = ok.LEVELS[c & 7]
        assert all(abs(abs(x) - got) <= abs(abs(x) - level) for level in ok.LEVELS)
    assert ok.code_of(100.0, 1.0) == 7


def test_stored_values_are_exact_half_numbers_and_near():
    x = np.random.default_rng(2).standard_normal((5, 64)) * 10.0 ** np.random.default_rng(3).integers(-6, 4, (5, 1))
    s, c = ok.quantise(x)
    y = ok.values(s, c)
    assert np.array_equal(y.astype(np.float16).astype(np.float64), y)
    assert (np.abs(x - y) <= np.repeat(s, 32, -1) * (1 + 1e-12)).all()
    k, v = ok.values_of(ok.rows_of(x, -x), 64)
    assert np.array_equal(k, y) and np.array_equal(v, -y)


def test_groups_with_nan_or_infinity_are_nan():
    x = np.full((1, 64), 6.0)
    x[0, 3] = math.inf
    k, _ = ok.values_of(ok.rows_of(x, x), 64)
    assert np.isnan(k[0, :32]).all() and (k[0, 32:] == 6.0).all()


def test_pages_by_hand():
    # two pages of 4 held by request 0 (6 positions), none by request 1
    table = np.array([[7, 3, -1], [-1, -1, -1]], np.int32)
    free = np.array([9, 5, 2, 0], np.int32)
    s = ok.extend(np.array([6, 0]), np.array([3, 5]), table, free, 3, 4, 10)
    assert s["slots"].tolist() == [3 * 4 + 2, 3 * 4 + 3, 2 * 4, 5 * 4, 5 * 4 + 1, 5 * 4 + 2, 5 * 4 + 3, 9 * 4, -1, -1]
    assert s["positions"].tolist() == [6, 7, 8, 0, 1, 2, 3, 4, -1, -1]
    assert s["starts"].tolist() == [0, 3, 8] and s["lengths"].tolist() == [9, 5] and s["num_free"] == 0
    assert s["table"].tolist() == [[7, 3, 2], [5, 9, -1]]
    # one page fewer: request 1 no longer fits, and gets nothing
    s = ok.extend(np.array([6, 0]), np.array([3, 5]), table, free, 2, 4, 10)
    assert s["starts"].tolist() == [0, 3, 3] and s["lengths"].tolist() == [9, 0] and s["num_free"] == 1
    lengths, free2, n = ok.release(np.array([6, 0]), [True, False], table, free, 1, 4)
    assert lengths.tolist() == [0, 0] and free2.tolist() == [9, 7, 3, 0] and n == 3


def test_attention_by_hand():
    rows = {0: (np.array([1.0]), np.array([2.0])), 1: (np.array([0.0]), np.array([4.0]))}
    q = np.full((1, 1, 1), math.log(3.0))
    out, lse, _, _ = ok.attention(q, lambda r, h, p: rows[p], [2], [0, 1], 1, 1.0)
    assert abs(out[0, 0, 0] - (3 * 2 + 4) / 4) < 1e-12 and abs(lse[0, 0] - math.log(4.0)) < 1e-12
    out, lse, _, _ = ok.attention(q, lambda r, h, p: rows[p], [2], [0, 1], 1, 1.0, window=1)
    assert out[0, 0, 0] == 4.0
    out, lse, _, _ = ok.attention(q, lambda r, h, p: rows[p], [2], [0, 1], 1, 1.0, positions=np.array([[-1, 5, 0, 0]]))
    assert out[0, 0, 0] == 2.0 and abs(lse[0, 0] - math.log(6.0)) < 1e-12
    out, lse, _, _ = ok.attention(q, lambda r, h, p: rows[p], [0], [0, 1], 1, 1.0)
    assert out[0, 0, 0] == 0.0 and lse[0, 0] == -math.inf


# ---- refusals: argument errors are found before CUDA is touched

P = ctypes.c_void_p
FAKE = P(0x1000)  # never dereferenced: validation fails first
OTHER = P(0x2000)


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_lt_gb300 import build, load
    build.build()
    return load()


def test_row_bytes(lib):
    assert [lib.lt_kv4_row_bytes(d) for d in (64, 128, 256)] == [ok.row_bytes(d) for d in (64, 128, 256)] == [80, 144, 288]
    assert all(lib.lt_kv4_row_bytes(d) == 0 for d in (0, -64, 32, 96, 512))


def _release(lib, **kw):
    a = dict(lengths=FAKE, finished=FAKE, n=2, table=FAKE, width=4, free=FAKE, cap=8, num=FAKE, page=16, out=OTHER, onum=OTHER)
    a.update(kw)
    return lib.lt_page_release(a["lengths"], a["finished"], a["n"], a["table"], a["width"], a["free"], a["cap"], a["num"],
                               a["page"], a["out"], a["onum"], None)


def _extend(lib, **kw):
    a = dict(lengths=FAKE, new=FAKE, n=2, table=FAKE, width=4, free=FAKE, cap=8, num=FAKE, page=16, most=9, slots=OTHER,
             pos=OTHER, starts=OTHER, out=OTHER, onum=OTHER)
    a.update(kw)
    return lib.lt_page_extend(a["lengths"], a["new"], a["n"], a["table"], a["width"], a["free"], a["cap"], a["num"], a["page"],
                              a["most"], a["slots"], a["pos"], a["starts"], a["out"], a["onum"], None)


@pytest.mark.parametrize("bad", [dict(n=-1), dict(width=0), dict(cap=-1), dict(page=0), dict(page=48), dict(page=2048),
                                 dict(page=-16), dict(num=None), dict(onum=None), dict(onum=FAKE), dict(free=None),
                                 dict(lengths=None), dict(table=None), dict(out=None), dict(out=FAKE)])
def test_pages_refuse(lib, bad):
    assert _release(lib, **bad) == 1
    assert _extend(lib, **bad) == 1


@pytest.mark.parametrize("bad", [dict(finished=None)])
def test_release_refuses(lib, bad):
    assert _release(lib, **bad) == 1


@pytest.mark.parametrize("bad", [dict(new=None), dict(most=-1), dict(slots=None), dict(pos=None), dict(starts=None)])
def test_extend_refuses(lib, bad):
    assert _extend(lib, **bad) == 1


def _store(lib, **kw):
    a = dict(k=FAKE, v=FAKE, dtype=1, tokens=3, heads=2, dim=128, slots=FAKE, cache=FAKE, pages=4, page=16)
    a.update(kw)
    return lib.lt_kv4_store(a["k"], a["v"], a["dtype"], a["tokens"], a["heads"], a["dim"], 256, 128, 256, 128, a["slots"],
                            a["cache"], a["pages"], a["page"], None)


def _load(lib, **kw):
    a = dict(k=FAKE, v=FAKE, dtype=1, tokens=3, heads=2, dim=128, slots=FAKE, cache=FAKE, pages=4, page=16)
    a.update(kw)
    return lib.lt_kv4_load(a["cache"], a["pages"], a["page"], a["slots"], a["tokens"], a["heads"], a["dim"], a["k"], a["v"],
                           a["dtype"], None)


@pytest.mark.parametrize("bad,status", [(dict(k=None), 1), (dict(v=None), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1),
                                        (dict(tokens=-1), 1), (dict(heads=0), 1), (dict(dim=0), 1), (dict(dim=96), 2),
                                        (dict(dim=512), 2), (dict(slots=None), 1), (dict(cache=None), 1), (dict(pages=-1), 1),
                                        (dict(page=3), 1), (dict(cache=P(0x1008)), 1), (dict(k=P(0x1001)), 1)])
def test_store_and_load_refuse(lib, bad, status):
    assert _store(lib, **bad) == status
    assert _load(lib, **bad) == status


def test_store_and_load_of_nothing(lib):
    assert _store(lib, tokens=0, k=None, v=None, slots=None) == 0
    assert _load(lib, tokens=0, k=None, v=None, slots=None) == 0


def _attend(lib, **kw):
    a = dict(q=FAKE, dtype=1, tokens=3, qh=8, kh=2, dim=128, qt=1024, qs=128, cache=FAKE, pages=4, page=16, table=FAKE, width=4,
             lengths=FAKE, n=3, starts=None, new=1, pos=None, list_len=0, window=0, scale=0.1, out=FAKE, lse=None)
    a.update(kw)
    return lib.lt_kv4_attention(a["q"], a["dtype"], a["tokens"], a["qh"], a["kh"], a["dim"], a["qt"], a["qs"], a["cache"],
                                a["pages"], a["page"], a["table"], a["width"], a["lengths"], a["n"], a["starts"], a["new"],
                                a["pos"], a["list_len"], a["window"], a["scale"], a["out"], a["lse"], None, 0, None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(cache=None), 1), (dict(table=None), 1), (dict(lengths=None), 1),
    (dict(dtype=0), 1), (dict(dtype=3), 1), (dict(tokens=-1), 1), (dict(qh=7), 1), (dict(kh=0), 1), (dict(qh=0), 1),
    (dict(dim=0), 1), (dict(dim=96), 2), (dict(page=5), 1), (dict(page=2048), 1), (dict(pages=-1), 1), (dict(width=0), 1),
    (dict(n=-1), 1), (dict(n=2), 1), (dict(new=2), 1), (dict(new=0), 1), (dict(window=-1), 1), (dict(scale=math.nan), 1),
    (dict(scale=math.inf), 1), (dict(pos=FAKE), 1), (dict(list_len=4), 1), (dict(pos=FAKE, list_len=4, window=3), 1),
    (dict(list_len=-1), 1), (dict(qt=1020), 1), (dict(qs=4), 1), (dict(q=P(0x1008)), 1), (dict(out=P(0x1004)), 1),
    (dict(cache=P(0x1008)), 1), (dict(pages=1 << 31), 2), (dict(starts=FAKE, new=0), 1)])
def test_attention_refuses(lib, bad, status):
    assert _attend(lib, **bad) == status


def test_attention_of_nothing(lib):
    assert _attend(lib, tokens=0, n=0) == 0
    assert _attend(lib, tokens=0, n=3, starts=FAKE, new=4) == 0
    need = ctypes.c_int64(-1)
    assert lib.lt_kv4_workspace(0, 8, 2, 128, 0, 1, 0, 64, 0, ctypes.byref(need)) == 0 and need.value == 0
    assert lib.lt_kv4_workspace(4, 8, 2, 128, 4, 1, 0, 64, 0, None) == 1
    assert lib.lt_kv4_workspace(4, 8, 3, 128, 4, 1, 0, 64, 0, ctypes.byref(need)) == 1
    assert lib.lt_kv4_workspace(4, 8, 2, 128, 4, 1, 0, -64, 0, ctypes.byref(need)) == 1
    assert lib.lt_kv4_workspace(4, 8, 2, 128, 4, 1, 0, 64, -1, ctypes.byref(need)) == 1
    assert lib.lt_kv4_workspace(4, 8, 2, 80, 4, 1, 0, 64, 0, ctypes.byref(need)) == 2


def test_valid_calls_without_a_device_report_a_cuda_error(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the CUDA runtime does not fail here")
    assert _release(lib) == 3 and _extend(lib) == 3 and _store(lib) == 3 and _load(lib) == 3 and _attend(lib) == 3


def test_binding_refuses_cpu_tensors_and_bad_sizes():
    import sparse_attention_indexer_lt_gb300 as lt
    cache = torch.zeros(2, 1, 16, 144, dtype=torch.uint8)
    z = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        lt.kv4_store(torch.zeros(1, 1, 128), torch.zeros(1, 1, 128), cache, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(TypeError):
        lt.kv4_load(cache, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(TypeError):
        lt.kv4_attention(torch.zeros(1, 1, 128, dtype=torch.float16), cache, z[None], z)
    with pytest.raises(TypeError):
        lt.page_release(z, z.bool(), z[None], z, z, 16)
    with pytest.raises(TypeError):
        lt.page_extend(z, z, z[None], z, z, 16, 4)
    with pytest.raises(ValueError):
        lt.kv4_row_bytes(96)
    with pytest.raises(ValueError):
        lt.kv4_cache(2, 1, 24, 128, device="cpu")


def test_release_passes_over_cells_without_a_page():
    table = np.array([[7, -1, 3], [-1, -1, 4]], np.int32)
    free = np.array([9, 5, -7, -7, -7], np.int32)
    lengths, got, n = ok.release(np.array([12, 8]), [True, True], table, free, 2, 4)
    assert lengths.tolist() == [0, 0] and got.tolist() == [9, 5, 7, 3, -7] and n == 4
    # the next pages taken are pages
    s = ok.extend(np.array([0]), np.array([8]), np.full((1, 2), -1, np.int32), got, n, 4, 8)
    assert s["table"].tolist() == [[3, 7]] and (s["slots"] >= 0).all()
