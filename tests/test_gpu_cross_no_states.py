"""flash_attention_cross on tensors without any states: 0 for every query, and numbers of states that are out of range are
reported as elsewhere."""
import pytest

import tiled_tensor_core_03_gb300 as gr

from test_gpu_serving import _cuda, _i32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 40])
@pytest.mark.parametrize("batch", [1, 3, 300])
def test_lengths_out_of_range_are_reported(batch, tokens):
    import torch
    q = torch.ones((batch, tokens, 4, 64), device="cuda", dtype=torch.float16)
    k = torch.ones((batch, 0, 2, 64), device="cuda", dtype=torch.float16)

    def call(lengths):
        out = torch.full_like(q, 7.0)
        gr.flash_attention_cross(q, k, k, lengths, out=out)
        assert (out == 0).all()
        return gr.status()
    assert call(None) == gr.OK
    assert call(_i32([0] * batch)) == gr.OK
    for bad in (1, -1, 1 << 30):
        assert call(_i32([0] * (batch - 1) + [bad])) == gr.ERR_PAGE
        assert gr.status() == gr.OK
