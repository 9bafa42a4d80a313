"""Single shaped logits: how far off a cap is, slopes of any finite size, and rows that do not go by their neighbours.

A query that sees one position has that position's logit as its lse, so that caps are seen through nothing else. In units of
eps = 2^-24: the claim, 8 of caps to 64 and 16 of the capped logit above, is what the steps of the hyperbolic tangent
may add. Besides, a logit s in units of log 2 carries 3 roundings (the scale's factor 2, their product), of which a cap
lets |s| / cosh(s / cap)^2 through, at most 0.45 caps; the cap in units of log 2 carries 2, the way back from them 2
and the sum's logarithm, 6 after and before the shift by it, some 4 of (|lse| + 12).
"""
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


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,group,listed", [(64, 8, False), (128, 32, False), (64, 80, False), (128, 80, False), (256, 80, False), (128, 16, True)])
@pytest.mark.parametrize("cap", [2.0 ** -10, 1.0, 30.0, 64.0, 65.0, 1000.0, 2.0 ** 20])
def test_capped_logits(cap, dim, group, listed, dtype):
    requests = 24
    p = Problem([1] * requests, [1] * requests, 1, group, dim, 16, dtype, seed=dim + group, positions=np.zeros((requests, 1)) if listed else None)
    p.cache[..., 0] = p.cache[..., 0] & 0xF0 | 2  # the first channel's code is 1
    p.q[:] = 0
    p.q[:, :, 0] = torch.linspace(-1.0, 1.0, requests * group).view(requests, group).to(p.q.dtype)
    k = np.array([p.rows_at(r, 0, 0)[0][0] for r in range(requests)])
    for reach in (0.6, 4.0, 40.0):  # caps: below them, around them, far past them
        scale = float(np.float32(reach * cap / k.max()))
        _, lse = p.run(scale=scale, softcap=cap)
        s = scale * num(p.q)[:, :, 0] * k[:, None]
        want = cap * np.tanh(s / cap)
        through = np.abs(s) / np.cosh(np.minimum(np.abs(s) / cap, 300.0)) ** 2
        claim = 8 * cap if cap <= 64 else 16 * np.abs(want)
        tol = EPS * (claim + 3 * through + 4 * (np.abs(want) + 12.0))
        err = np.abs(num(lse) - want)
        assert (err <= tol).all(), f"reach {reach}: worst {float((err / tol).max()):.3g} of its bound"


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
