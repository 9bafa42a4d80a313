"""The 4-bit layer's operators as they are used together: projections, pages, rotated appends, attention, the output product."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from sparse_attention_indexer_lt_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "layer_step.py")
    spec = importlib.util.spec_from_file_location("layer_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("kw", [
    dict(), dict(dtype=torch.float16), dict(prompts=(1,), steps=2, hidden=32, kv_heads=1, group=1, rotary=64),
    dict(prompts=(300, 5, 129, 64), hidden=1056, kv_heads=4, group=2, head_dim=128, rotary=128, page_size=64),
    dict(prompts=(40, 200), hidden=512, kv_heads=1, group=8, head_dim=256, rotary=64, softcap=100.0, page_size=8)])
def test_layer(example, kw):
    """Queries, attention outputs and results are rounded to the 16-bit type on the way, each by half a unit: 2^-9 (bf16) or
    2^-12 (fp16) of an output's terms and those of the logits of up to four units' size; together within 2^-5 and 2^-8 of the
    outputs' size."""
    seen, held = example.run(**kw)
    torch.cuda.synchronize()
    assert example.check(seen, held) <= (2.0 ** -8 if kw.get("dtype") == torch.float16 else 2.0 ** -5)


def test_the_same_in_a_graph(example):
    """A decode step's calls captured and replayed give what the calls give."""
    import sparse_attention_indexer_lt_gb300 as lt
    seen, held = example.run(steps=1)
    x, y, step = seen[-1]
    h, d, group = held["kv_heads"], held["head_dim"], held["group"]

    def call():
        q, k, v = lt.w4_linear(x, *held["qkv"], bias=held["bias"]).view(x.shape[0], -1, d).split([h * group, h, h], 1)
        q = lt.kv4_append(q, k, v, held["cache"], step.slots, step.positions, held["cos"], held["sin"])
        a = lt.kv4_attention(q, held["cache"], held["table"], step.lengths, starts=step.starts, softcap=held["softcap"],
                             slopes=held["slopes"], prefix=held["prefix"])
        return lt.w4_linear(a.view(x.shape[0], -1), *held["out"])
    assert torch.equal(call(), y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    x.normal_()
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone()
    assert torch.equal(got, call()) and not torch.equal(got, y)
