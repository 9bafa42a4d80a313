"""Caps, slopes and prefixes of the 4-bit cache's attention without a GPU: the oracle pinned, and the refusals."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import kv4 as ok

P = ctypes.c_void_p
FAKE = P(0x1000)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_lt_gb300 import build, load
    build.build()
    return load()


def one(q, rows, n, new=1, **kw):
    return ok.attention(np.full((new, 1, 1), q), lambda r, h, p: rows[p], [n], [0, new], 1, 1.0, **kw)[:2]


def test_oracle_by_hand():
    rows = [(np.array([0.0]), np.array([2.0])), (np.array([1.0]), np.array([4.0])), (np.array([1.0]), np.array([12.0]))]
    # a cap: logits 0 and 3 tanh(5 / 3) of two positions
    w = math.exp(3 * math.tanh(5 / 3))
    out, lse = one(5.0, rows, 2, softcap=3.0)
    assert abs(out[0, 0, 0] - (2 + 4 * w) / (1 + w)) < 1e-12 and abs(lse[0, 0] - math.log(1 + w)) < 1e-12
    # a slope of ln 2: the position before has half the weight, the one before that a quarter
    out, lse = one(0.0, rows, 3, slopes=[math.log(2.0)])
    assert abs(out[0, 0, 0] - (2 / 4 + 4 / 2 + 12) / 1.75) < 1e-12 and abs(lse[0, 0] - math.log(1.75)) < 1e-12
    # the first of three queries lies at position 0 and sees what the prefix shows it, by the distance ahead
    out, _ = one(0.0, rows, 3, new=3, prefix=[2])
    assert out[:, 0, 0].tolist() == [3.0, 3.0, 6.0]
    out, _ = one(0.0, rows, 3, new=3, prefix=[99], slopes=[math.log(2.0)])
    assert abs(out[0, 0, 0] - (2 + 4 / 2 + 12 / 4) / 1.75) < 1e-12
    assert one(0.0, rows, 3, new=3, prefix=[-5])[0][:, 0, 0].tolist() == [2.0, 3.0, 6.0]
    # a query before the first position sees the prefix alone
    out, lse = one(0.0, rows, 1, new=2, prefix=[1])
    assert out[:, 0, 0].tolist() == [2.0, 2.0]
    # a list: the distance of what it names
    out, _ = one(0.0, rows, 3, positions=np.array([[0, 2, -1]]), slopes=[math.log(2.0)])
    assert abs(out[0, 0, 0] - (2 / 4 + 12) / 1.25) < 1e-12


def _attend(lib, **kw):
    a = dict(tokens=3, pos=None, list_len=0, window=0, cap=0.0, slopes=None, prefix=None, q=FAKE)
    a.update(kw)
    return lib.lt_kv4_attention_ex(a["q"], 1, a["tokens"], 8, 2, 128, 1024, 128, FAKE, 4, 16, FAKE, 4, FAKE, 3, None, 1, a["pos"],
                                   a["list_len"], a["window"], 0.1, a["cap"], a["slopes"], a["prefix"], FAKE, None, None, 0, None)


@pytest.mark.parametrize("bad,status", [
    (dict(cap=-1.0), 1), (dict(cap=math.nan), 1), (dict(cap=math.inf), 1), (dict(cap=2.0 ** -11), 2), (dict(cap=2.0 ** 21), 2),
    (dict(prefix=FAKE, window=5), 1), (dict(prefix=FAKE, pos=FAKE, list_len=4), 1), (dict(slopes=P(0x1002)), 1),
    (dict(prefix=P(0x1001)), 1), (dict(cap=30.0, q=None), 1), (dict(cap=30.0, window=-1), 1)])
def test_refusals(lib, bad, status):
    assert _attend(lib, **bad) == status


def test_valid_calls_without_a_device_report_a_cuda_error(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the CUDA runtime does not fail here")
    for kw in (dict(cap=30.0), dict(slopes=FAKE), dict(prefix=FAKE), dict(cap=2.0 ** 20, slopes=FAKE, window=5),
               dict(cap=2.0 ** -10, slopes=FAKE, pos=FAKE, list_len=4)):
        assert _attend(lib, **kw) == 3
    assert _attend(lib, cap=30.0, tokens=3) == 3
