"""CPU-only: a block may store into another block's shared memory only once that block runs, so
every kernel that does so passes a barrier of its whole cluster before the first such store."""
import os
import re

import pytest

from tiled_tensor_core_03_gb300 import _build

FILES = ("gemm_relu_2sm.cuh", "gemm_relu_gemv.cuh", "gemm_relu_splitk.cuh", "kv_cache.cuh")


def _kernels(name):
    """The text of each __global__ function of a file, comments taken out."""
    with open(os.path.join(_build.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    starts = [m.start() for m in re.finditer(r"__global__", text)] + [len(text)]
    return [text[a:b] for a, b in zip(starts, starts[1:])]


def test_every_file_that_reaches_other_blocks_is_listed():
    found = {f for f in os.listdir(_build.CSRC) if f != "sm103.cuh"
             and any("mapa_shared(" in k for k in _kernels(f))}
    assert set(FILES) == found


@pytest.mark.parametrize("name", FILES)
def test_cluster_barrier_before_the_first_remote_store(name):
    remote = [k for k in _kernels(name) if "mapa_shared(" in k]
    assert remote
    for kernel in remote:
        waits = [kernel.find(w) for w in ("cluster_wait()", "cluster_sync()") if w in kernel]
        assert waits and min(waits) < kernel.find("mapa_shared(")
