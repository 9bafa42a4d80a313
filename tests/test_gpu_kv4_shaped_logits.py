"""Single shaped logits: rows that do not go by their neighbours."""
import pytest
import torch

from test_gpu_kv4 import Problem

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
