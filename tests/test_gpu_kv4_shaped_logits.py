"""Single shaped logits: slopes of any finite size, and rows that do not go by their neighbours."""
import numpy as np
import pytest
import torch

from test_gpu_kv4 import EPS, Problem, num

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_lt_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=30.0), dict(window=50)])
def test_a_rows_bits_do_not_go_by_its_neighbours(dim, kw):
    """Heads of one kv head share warps: with many query rows one's result stays as it is whatever the other's slope."""
    p = Problem([700], [80], 1, 3, dim, 16, "f16", seed=dim + 80, spread=2.0)
    got = [p.run(slopes=torch.tensor([0.3, other, 0.01], device="cuda"), **kw) for other in (0.3, 0.0, 6.0, 1e6, -5.0)]
    for out, lse in got[1:]:
        for h in (0, 2):
            assert torch.equal(out[:, h], got[0][0][:, h]) and torch.equal(lse[:, h], got[0][1][:, h])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,listed", [(3, False), (80, False), (2, True)])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_slopes_of_any_finite_size(dim, new, listed, softcap):
    """From 1e30 on a query sees itself alone (with the other sign, the first position alone). Magnitudes above 2^95 count
    as that, whatever the distance."""
    n = 260
    slopes = [1e30, 3e38, float(np.finfo(np.float32).max), -1e30, -3e38, 0.0]
    pos = np.tile(np.arange(n - 2), (new, 1)) if listed else None  # (without the last query's own position)
    p = Problem([n], [new], 1, len(slopes), dim, 16, "f16", seed=4, positions=pos)
    out, lse = (num(x) for x in p.run(softcap=softcap, slopes=torch.tensor(slopes, device="cuda")))
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    q = num(p.q)
    for i in (0, new - 1):
        own = n - new + i
        seen = range(n - 2) if listed else range(own + 1)
        for h, slope in enumerate(slopes[:-1]):
            at = min(seen, key=lambda x: abs(own - x)) if slope > 0 else max(seen, key=lambda x: abs(own - x))
            k, v = p.rows_at(0, 0, at)
            s = float(k @ q[i, h]) * dim ** -0.5
            s = softcap * np.tanh(s / softcap) if softcap else s
            far = min(abs(slope), 2.0 ** 95) * abs(own - at)
            s += -far if slope > 0 else far
            reach = np.abs(k * q[i, h]).sum() * dim ** -0.5
            assert np.abs(out[i, h] - v).max() <= 2.0 ** -10 * np.abs(v).max()  # its weight is 1: the output's rounding, and the weight's
            assert abs(lse[i, h] - s) <= (dim + 8) * EPS * reach + 2.0 ** -20 * (1 + abs(s)) + 8 * EPS * max(softcap, 1.0)
