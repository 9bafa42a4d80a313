"""4-bit weights without a GPU: the oracle pinned, and every refusal."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv4 as ok
from oracle import w4 as ow

P = ctypes.c_void_p
FAKE = P(0x1000)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_lt_gb300 import build, load
    build.build()
    return load()


def test_weights_by_hand():
    w = np.zeros((2, 64))
    w[0, :4], w[0, 32] = [6.0, -3.0, 0.5, 1.2], 0.75
    w[1, 33] = -12.0
    codes, scales = ow.quantise(w)
    assert scales.tolist() == [[1.0, 0.125], [0.0, 2.0]]
    assert codes[0, :2].tolist() == [7 | (13 << 4), 1 | (2 << 4)] and codes[0, 16] == 7 and codes[1, 16] == 15 << 4
    got = ow.weights(codes, scales)
    assert got[0, :4].tolist() == [6.0, -3.0, 0.5, 1.0] and got[0, 32] == 0.75 and got[1, 33] == -12.0
    y, size = ow.linear(np.arange(64.0)[None], codes, scales, np.array([1.0, 2.0]))
    assert y.tolist() == [[1.0 + -3.0 + 1.0 + 3.0 + 24.0, 2.0 - 33 * 12.0]] and size.tolist() == [[3.0 + 1.0 + 3.0 + 24.0, 33 * 12.0]]


def test_a_weight_is_stored_as_a_key_is():
    w = np.random.default_rng(0).standard_normal((3, 128))
    codes, scales = ow.quantise(w)
    rows = ok.rows_of(w, w)
    assert np.array_equal(rows[:, :64], codes) and np.array_equal(rows[:, 128:136].copy().view(np.float16), scales)
    assert np.array_equal(ow.weights(codes, scales), ok.values_of(rows, 128)[0])


def _linear(lib, **kw):
    a = dict(x=FAKE, dtype=1, tokens=3, xs=128, codes=FAKE, scales=FAKE, n=5, k=128, bias=None, out=FAKE, os=5, ws=None, bytes=0)
    a.update(kw)
    return lib.lt_w4_linear(a["x"], a["dtype"], a["tokens"], a["xs"], a["codes"], a["scales"], a["n"], a["k"], a["bias"], a["out"],
                            a["os"], a["ws"], a["bytes"], None)


def _quantise(lib, **kw):
    a = dict(w=FAKE, dtype=1, n=5, k=128, stride=128, codes=FAKE, scales=FAKE)
    a.update(kw)
    return lib.lt_w4_quantise(a["w"], a["dtype"], a["n"], a["k"], a["stride"], a["codes"], a["scales"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), 1), (dict(codes=None), 1), (dict(scales=None), 1), (dict(out=None), 1), (dict(dtype=0), 1), (dict(dtype=3), 1),
    (dict(tokens=-1), 1), (dict(n=-1), 1), (dict(k=-32), 1), (dict(xs=100), 1), (dict(x=P(0x1008)), 1), (dict(codes=P(0x1008)), 1),
    (dict(scales=P(0x1002)), 1), (dict(out=P(0x1001)), 1), (dict(bias=P(0x1001)), 1), (dict(k=48), 2), (dict(k=0), 2),
    (dict(n=1 << 31), 2), (dict(k=1 << 31), 2), (dict(tokens=1 << 31), 2), (dict(n=1 << 30), 2), (dict(k=1 << 30), 2),
    (dict(tokens=524281), 2)])
def test_linear_refuses(lib, bad, status):
    assert _linear(lib, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(w=None), 1), (dict(codes=None), 1), (dict(scales=None), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(n=-1), 1),
    (dict(k=-32), 1), (dict(w=P(0x1001)), 1), (dict(codes=P(0x1004)), 1), (dict(scales=P(0x1004)), 1), (dict(k=48), 2), (dict(k=0), 2)])
def test_quantise_refuses(lib, bad, status):
    assert _quantise(lib, **bad) == status


def test_nothing_to_do(lib):
    assert _linear(lib, tokens=0, x=None, out=None) == 0 and _linear(lib, n=0, codes=None, scales=None, out=None) == 0
    assert _quantise(lib, n=0, w=None, codes=None, scales=None) == 0
    need = ctypes.c_int64(-1)
    assert lib.lt_w4_workspace(0, 5, 128, ctypes.byref(need)) == 0 and need.value == 0
    assert lib.lt_w4_workspace(3, 5, 128, None) == 1 and lib.lt_w4_workspace(-3, 5, 128, ctypes.byref(need)) == 1
    assert lib.lt_w4_workspace(3, 5, 100, ctypes.byref(need)) == 2


def test_valid_calls_without_a_device_report_a_cuda_error(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the CUDA runtime does not fail here")
    assert _linear(lib) == 3 and _quantise(lib) == 3


def test_binding_refuses_cpu_tensors():
    import sparse_attention_indexer_lt_gb300 as lt
    with pytest.raises(TypeError):
        lt.w4_quantise(torch.zeros(2, 64))
    with pytest.raises(TypeError):
        lt.w4_linear(torch.zeros(1, 64, dtype=torch.float16), torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.float16))
