"""The rotated append without a GPU: the oracle's rotation pinned, and every refusal."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import kv4 as ok

P = ctypes.c_void_p
FAKE = P(0x1000)  # never dereferenced: validation fails first
OTHER = P(0x2000)


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_lt_gb300 import build, load
    build.build()
    return load()


def test_rotation_by_hand():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    cos, sin = np.array([[0.0, 1.0]]), np.array([[1.0, 0.0]])
    # channels 0 and 2 make a quarter turn, 1 and 3 none, 4 to 7 do not turn
    assert ok.rotate(x, cos, sin).tolist() == [[[-3.0, 2.0, 1.0, 4.0, 5.0, 6.0, 7.0, 8.0]]]
    assert ok.rotate(x, cos, sin, True).tolist() == [[[-2.0, 1.0, 3.0, 4.0, 5.0, 6.0, 7.0, 8.0]]]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_the_complex_product_and_the_32_bit_one(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 3, 32)).astype(np.float32)
    angle = rng.uniform(0, 1000, (50, 12))
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    got = ok.rotate(x, cos, sin, interleaved)
    a, b = (x[..., 0:24:2], x[..., 1:24:2]) if interleaved else (x[..., :12], x[..., 12:24])
    z = (a.astype(np.float64) + 1j * b) * (cos.astype(np.float64) + 1j * sin)[:, None]
    ga, gb = (got[..., 0:24:2], got[..., 1:24:2]) if interleaved else (got[..., :12], got[..., 12:24])
    # three roundings of at most half a unit of numbers no larger than |a| + |b|
    assert np.abs(ga - z.real).max() <= 3 * 2.0 ** -24 * (np.abs(a) + np.abs(b)).max()
    assert np.abs(gb - z.imag).max() <= 3 * 2.0 ** -24 * (np.abs(a) + np.abs(b)).max()
    assert np.array_equal(got[..., 24:], x[..., 24:])
    c, s = cos[:, None], sin[:, None]
    assert np.array_equal(ga, a * c - b * s) and np.array_equal(gb, b * c + a * s)  # numpy's float32, unfused


def _append(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dtype=1, tokens=3, qh=4, kh=2, dim=128, qt=1024, qs=128, cos=FAKE, sin=FAKE, most=64, rotary=128,
             pairs=0, positions=FAKE, slots=FAKE, cache=FAKE, pages=4, page=16, out=OTHER, ot=512, os=128)
    a.update(kw)
    return lib.lt_kv4_append(a["q"], a["k"], a["v"], a["dtype"], a["tokens"], a["qh"], a["kh"], a["dim"], a["qt"], a["qs"], 256, 128,
                             256, 128, a["cos"], a["sin"], a["most"], a["rotary"], a["pairs"], a["positions"], a["slots"], a["cache"],
                             a["pages"], a["page"], a["out"], a["ot"], a["os"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(out=None), 1), (dict(cos=None), 1), (dict(sin=None), 1),
    (dict(positions=None), 1), (dict(slots=None), 1), (dict(cache=None), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1),
    (dict(tokens=-1), 1), (dict(qh=-1), 1), (dict(kh=0), 1), (dict(dim=0), 1), (dict(pages=-1), 1), (dict(page=24), 1),
    (dict(page=2048), 1), (dict(most=-1), 1), (dict(rotary=-16), 1), (dict(rotary=144), 1), (dict(cos=P(0x1008)), 1),
    (dict(sin=P(0x1004)), 1), (dict(cache=P(0x1008)), 1), (dict(q=P(0x1001)), 1), (dict(out=P(0x2001)), 1), (dict(k=P(0x1001)), 1),
    (dict(out=FAKE), 1), (dict(dim=96, rotary=32), 2), (dict(rotary=24), 2), (dict(rotary=0), 2), (dict(kh=20000), 2),
    (dict(qh=40000), 2)])
def test_append_refuses(lib, bad, status):
    assert _append(lib, **bad) == status


def test_append_of_nothing(lib):
    assert _append(lib, tokens=0, q=None, k=None, v=None, slots=None, positions=None, out=None) == 0
    assert _append(lib, most=0, cos=None, sin=None) == 0  # every position is outside empty tables


def test_a_valid_append_without_a_device_reports_a_cuda_error(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the CUDA runtime does not fail here")
    assert _append(lib) == 3
    assert _append(lib, q=None, qh=0, out=None) == 3
    assert _append(lib, out=FAKE, ot=1024, os=128) == 3  # in place


def test_binding_refuses_cpu_tensors():
    import sparse_attention_indexer_lt_gb300 as lt
    cache = torch.zeros(2, 1, 16, 144, dtype=torch.uint8)
    x = torch.zeros(1, 1, 128)
    with pytest.raises(TypeError):
        lt.kv4_append(x, x, x, cache, torch.zeros(1, dtype=torch.int64), torch.zeros(1, dtype=torch.int32), torch.zeros(4, 64),
                      torch.zeros(4, 64))
    assert math.isfinite(float(x.sum()))
