"""The example's serving loop on the GPU: replayed from a graph it gives what it gives eagerly."""
import importlib.util
import os

import pytest

import tiled_tensor_core_03_gb300 as gr

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_serving_loop_example():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("serving_loop",
                                                  os.path.join(ROOT, "examples", "serving_loop.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    kw = dict(batch=3, prompt=300, steps=12, budget=100, window=64, recent=16, width=256, q_heads=8,
              kv_heads=2, dim=64, page=16)
    eager = example.serve(graph=False, **kw)
    replayed = example.serve(graph=True, **kw)
    assert gr.status() == gr.OK
    for x, y in zip(eager, replayed):
        assert torch.isfinite(x.float()).all() and torch.equal(x, y)
    assert eager[2].tolist() == [112, 112, 112]
