"""A failure while the launch of a product with 4-bit weights is planned."""
import subprocess
import sys
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_lt_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def test_a_failure_while_the_launch_is_planned_passes():
    """The first call of a process asks the device what fits; where that fails the call says so, and the next ones are right."""
    code = """
import torch
import sparse_attention_indexer_lt_gb300 as lt
codes, scales = lt.w4_quantise(torch.randn(256, 512, device="cuda"))
x = torch.randn(64, 512, device="cuda").half()
lt.load().lt_test_inject(1, 1)
try:
    lt.w4_linear(x, codes, scales)
    raise SystemExit("the failure is not reported")
except lt.LtError as e:
    assert "CUDA" in str(e), e
y = lt.w4_linear(x, codes, scales)
assert torch.equal(y[:2], lt.w4_linear(x, codes, scales)[:2]) and y.isfinite().all()
print("done")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=Path(__file__).resolve().parent.parent, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr
