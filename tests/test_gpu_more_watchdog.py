"""Ragged and cross attention: a dropped producer arrival makes a bounded wait expire; the call reports a timeout, and the
next one on the same kept workspace is right.  No fault, trap or hang: the wait gives up after 20 ms."""
import numpy as np
import pytest

import tiled_tensor_core_03_gb300 as gr

from test_gpu_serving import _cache, _i32, _rand
from test_gpu_watchdog import _restore  # noqa: F401

pytestmark = pytest.mark.gpu


def _calls(kind):
    rng = np.random.default_rng(9)
    if kind.startswith("ragged"):
        d = 128 if kind.endswith("128") else 64
        cache, _ = _cache(rng, 100, 2, 64, d, garbage=False)
        import torch
        pages = torch.arange(100, dtype=torch.int32, device="cuda").view(2, 50)
        q, _ = _rand(rng, (71, 8, d), "bf16")
        lengths, starts = _i32([3200, 1000]), _i32([0, 70, 71])
        return lambda: gr.kv_cache_attention_ragged(q, cache, pages, lengths, starts)
    tokens = 1 if kind == "cross step" else 300
    q, _ = _rand(rng, (2, tokens, 4, 64), "fp16")
    k, _ = _rand(rng, (2, 900, 4, 64), "fp16")
    return lambda: gr.flash_attention_cross(q, k, k, _i32([900, 500]))


@pytest.mark.parametrize("kind", ["ragged 64", "ragged 128", "cross step", "cross"])
def test_dropped_arrival_times_out_and_recovers(kind):
    import torch
    call = _calls(kind)
    want = call()
    assert gr.status() == gr.OK
    gr.gemm_relu_debug_set(1, 20_000_000)
    call()
    assert gr.status() == gr.ERR_TIMEOUT
    assert gr.status() == gr.OK            # reading clears the word
    gr.gemm_relu_debug_set(0, 0)
    for _ in range(2):
        assert torch.equal(call(), want)
    assert gr.status() == gr.OK
