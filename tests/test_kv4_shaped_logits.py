"""The error bounds of capped logits, from the steps that the kernels take."""
import re
from pathlib import Path

import numpy as np

SOURCE = Path(__file__).resolve().parent.parent / "sparse_attention_indexer_lt_gb300" / "csrc" / "lt_kv4_attention.cuh"
EPS = 2.0 ** -24


def test_the_polynomial_is_off_by_three_units():
    """tanh(x) / x for u = x^2 up to 1, every step a fused one in 32 bits."""
    body = SOURCE.read_text().split("constexpr float tanh_term(int i)")[1].split("}")[0]
    terms = np.array([float(x) for x in re.findall(r"(-?\d\.\d+)f", body)], np.float32)
    assert len(terms) == 7
    x = np.linspace(2.0 ** -12, 1.0, 1 << 20).astype(np.float32)
    u = x * x
    t = np.full_like(u, terms[6])
    for c in terms[5::-1]:
        t = (t.astype(np.float64) * u + float(c)).astype(np.float32)  # (the product is exact in 64 bits)
    true = np.tanh(x.astype(np.float64)) / x
    assert np.abs(t / true - 1.0).max() < 3 * EPS
    # a term that is off by 2^-20 shows
    assert np.abs((t + u * 2.0 ** -20) / true - 1.0).max() > 3 * EPS


def test_the_steps_by_exponential_and_reciprocal_add_up_to_eight_units():
    """cap - 2 cap r with r = 1 / (1 + e^2x): 2 units of the reciprocal, 1 of the sum, 4 of the exponential, relative; two roundings of
    the argument; and the last step's."""
    r = np.linspace(1e-5, 1.0 - 1e-5, 1 << 20)
    x = 0.5 * np.log(1.0 / r - 1.0)
    off = 2 * r * (2 + 1) + 2 * r * (1 - r) * 4 + 2 * np.abs(x) / np.cosh(x) ** 2 + np.abs(1 - 2 * r)
    assert 7.0 < off.max() < 8.0
