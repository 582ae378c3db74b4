"""The step form of flash_attention_cross is cut for as many blocks as the SMs' shared memory holds, not for more."""
import pytest

import tiled_tensor_core_03_gb300 as gr

from test_gpu_serving import _cuda  # noqa: F401

pytestmark = pytest.mark.gpu

# blocks an SM holds: their shared memory is two rings of stages and a row of sums for each of four warps
STAGES = {64: 4, 128: 3}


def _fit(d, rows, an_sm):
    rows = 8 if rows <= 8 else 16
    stages = 2 * STAGES[d] * 64 * d * 2
    join = 4 * rows * (d + 4) * 4 + 2 * 4 * rows * 4
    return an_sm // (stages + join + 2 * STAGES[d] * 8 + 16 + 1024 + 1024)   # aligned to 1 KB, and 1 KB reserved


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 8, 9, 16])
def test_parts_fit_the_gpu(d, group):
    import torch
    p = torch.cuda.get_device_properties(0)
    fit = _fit(d, group, 228 * 1024)
    assert fit == {64: 3 if group <= 8 else 2, 128: 1}[d]
    cut = 0
    for heads in (1, 2, 7, 32, 72, 104, 128, 152, 300):
        used = gr.flash_attention_cross_x16_workspace_bytes(1, 1, 30000, heads * group, heads, d)
        if used == 0:
            continue
        one = heads * (8 if group <= 8 else 16) * (d + 4) * 4
        parts, rest = divmod(used - gr.CROSS_COUNTER_BYTES, one)
        assert rest == 0 and parts > 1
        assert parts * heads <= fit * p.multi_processor_count, (heads, parts)
        cut += 1
    assert cut >= 4
