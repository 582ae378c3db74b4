"""flash_attention_cross with more items than CTAs: the order by length, rounds back and forth, a short last round, items of
one tile and of no states between others.  Against the definition in 64 bits, tolerances as in test_gpu_serving.py."""
import numpy as np
import pytest

import tiled_tensor_core_03_gb300 as gr

from test_gpu_cross import _against, _cross
from test_gpu_serving import DTYPES, _cuda, _i32, _rand  # noqa: F401

pytestmark = pytest.mark.gpu


def _items(b, sq, hkv, group):
    tiles = -(-sq // (128 // group))
    return b * hkv * -(-tiles // 2)


def _heads(b, sq, group, rounds):
    """K/V heads with which the call takes `rounds` rounds and part of another."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    one = _items(b, sq, 1, group)
    hkv = -(-(rounds * sms + 1) // one)
    assert _items(b, sq, hkv, group) > rounds * sms
    return hkv


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("b,sq,group,d,rounds,lengths", [
    # ties, sequences without states, an odd number of tiles
    (9, 300, 1, 64, 1, [513, 0, 129, 513, 1, 384, 0, 128, 385]),
    (9, 300, 1, 128, 2, [0, 0, 300, 70, 300, 299, 128, 129, 5]),
    # groups that do not divide a tile: 42 and 18 queries a tile
    (7, 200, 3, 64, 1, [200, 128, 127, 0, 400, 200, 1]),
    (5, 90, 7, 128, 2, [257, 256, 0, 255, 129]),
    # all sequences alike, and none named
    (4, 257, 1, 64, 3, [100] * 4),
    (3, 130, 2, 128, 2, None),
    # more sequences than the order has room for
    (131, 40, 1, 64, 1, [(i * 37) % 190 for i in range(131)]),
    (129, 17, 2, 128, 2, [150 - i for i in range(129)]),
    (128, 20, 1, 64, 1, [(i * 53) % 140 for i in range(128)])])
def test_cross_in_rounds(b, sq, group, d, rounds, lengths, dtype):
    hkv = _heads(b, sq, group, rounds)
    skv = 400 if lengths is None else max(lengths) + 3
    _cross(np.random.default_rng(b + sq + d), b, sq, skv, hkv * group, hkv, d, lengths, dtype)


@pytest.mark.parametrize("d", [64, 128])
def test_cross_in_rounds_beside_padding_that_is_not_finite(d):
    """NaN and infinities behind each sequence's states, in calls of several rounds: a CTA that walks a second time has all
    its items again."""
    import torch
    b, sq, dtype = 6, 150, "bf16"
    lengths = [200, 0, 129, 384, 128, 1]
    hkv = _heads(b, sq, 1, 2)
    rng = np.random.default_rng(d)
    q, _ = _rand(rng, (b, sq, hkv, d), dtype)
    k, _ = _rand(rng, (b, 390, hkv, d), dtype)
    v, _ = _rand(rng, (b, 390, hkv, d), dtype)
    want = gr.flash_attention_cross(q, k, v, _i32(lengths))
    for i, n in enumerate(lengths):
        k[i, n:] = float("nan")
        v[i, n::2] = float("inf")
        v[i, n + 1::2] = float("nan")
    got = gr.flash_attention_cross(q, k, v, _i32(lengths))
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    _against(got, q, k, v, lengths, dtype)
