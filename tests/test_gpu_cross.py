"""flash_attention_cross on the GPU against the definition in 64 bits.  Tolerances as in
test_gpu_serving.py: roundings counted, half a step each; weights are rounded to the inputs' type."""
import numpy as np
import pytest

import tiled_tensor_core_03_gb300 as gr

from test_gpu_serving import DTYPES, _check, _cuda, _f64, _half_step, _i32, _rand  # noqa: F401

pytestmark = pytest.mark.gpu


def _against(out, q, k, v, lengths, dtype):
    import torch
    from gpu_attend import attend
    got = _f64(out)
    for i in range(q.shape[0]):
        n = k.shape[1] if lengths is None else lengths[i]
        see = torch.ones((q.shape[1], n), dtype=torch.bool, device="cuda")
        o, absv, size = attend(q[i], k[i, :n], v[i, :n], see)
        _check(got[i], o, absv, size, q.shape[3], dtype, _half_step(dtype))


def _cross(rng, b, sq, skv, hq, hkv, d, lengths, dtype, scale=2.0):
    import torch
    q, _ = _rand(rng, (b, sq, hq, d), dtype, scale)
    k, _ = _rand(rng, (b, skv, hkv, d), dtype)
    v, _ = _rand(rng, (b, skv, hkv, d), dtype)
    n = None if lengths is None else _i32(lengths)
    out = gr.flash_attention_cross(q, k, v, n)
    again = gr.flash_attention_cross(q, k, v, n)
    assert gr.status() == gr.OK
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    _against(out, q, k, v, lengths, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("b,sq,skv,hq,hkv,d,lengths", [
    (1, 1, 1, 1, 1, 64, None), (1, 1, 700, 4, 2, 128, None), (3, 1, 300, 8, 8, 64, [300, 0, 129]),
    (2, 130, 70, 2, 2, 64, [70, 1]), (1, 129, 513, 3, 1, 128, None), (2, 300, 128, 6, 2, 64, [127, 128]),
    (1, 5, 2000, 7, 1, 128, [1999]), (2, 33, 257, 8, 1, 64, [256, 257]), (1, 257, 40, 5, 5, 128, [0]),
    (4, 2, 1500, 16, 16, 64, [1500, 3, 640, 128]), (1, 600, 900, 7, 1, 64, [897]), (1, 9, 300, 128, 1, 64, None),
    (1, 3, 200, 100, 1, 128, None), (7, 1, 385, 10, 5, 64, [1, 2, 3, 385, 384, 0, 200])])
def test_cross(b, sq, skv, hq, hkv, d, lengths, dtype):
    _cross(np.random.default_rng(sq * 7 + skv + d + hq), b, sq, skv, hq, hkv, d, lengths, dtype)


def test_cross_few_rows_over_many_states():
    rng = np.random.default_rng(1)
    _cross(rng, 1, 1, 50000, 4, 4, 64, None, "fp16")
    _cross(rng, 2, 4, 30000, 8, 2, 128, [30000, 12345], "bf16")


def test_cross_large_scores():
    rng = np.random.default_rng(2)
    _cross(rng, 2, 200, 500, 4, 2, 128, [500, 333], "fp16", scale=16.0)
    _cross(rng, 1, 3, 900, 4, 2, 64, None, "bf16", scale=64.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sq", [1, 3, 200])
def test_cross_padding_is_not_seen(sq, dtype):
    """States behind a sequence's last hold NaN and infinities."""
    import torch
    rng = np.random.default_rng(3)
    lengths = [200, 0, 129, 384]
    q, _ = _rand(rng, (4, sq, 6, 64), dtype)
    k, _ = _rand(rng, (4, 384, 2, 64), dtype)
    v, _ = _rand(rng, (4, 384, 2, 64), dtype)
    want = gr.flash_attention_cross(q, k, v, _i32(lengths))
    for i, n in enumerate(lengths):
        k[i, n:] = float("nan")
        v[i, n::2] = float("inf")
        v[i, n + 1::2] = float("nan")
    got = gr.flash_attention_cross(q, k, v, _i32(lengths))
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    _against(got, q, k, v, lengths, dtype)


def test_cross_not_finite_among_the_states():
    """An infinity in V makes its element infinite for all rows of its sequence and head, a NaN in K all."""
    rng = np.random.default_rng(4)
    q, _ = _rand(rng, (2, 150, 4, 64), "fp16")
    k, _ = _rand(rng, (2, 300, 2, 64), "fp16")
    v, _ = _rand(rng, (2, 300, 2, 64), "fp16")
    clean = _f64(gr.flash_attention_cross(q, k, v, _i32([300, 290])))
    v[0, 100, 1, 5] = float("inf")
    k[1, 289, 0, 7] = float("nan")
    got = _f64(gr.flash_attention_cross(q, k, v, _i32([300, 290])))
    assert (got[0, :, 2:, 5] == np.inf).all() and np.isnan(got[1, :, :2]).all()
    got[0, :, 2:, 5], got[1, :, :2] = clean[0, :, 2:, 5], clean[1, :, :2]
    assert np.array_equal(got, clean)


def test_cross_lengths_out_of_range():
    rng = np.random.default_rng(5)
    q, _ = _rand(rng, (3, 2, 4, 64), "fp16")
    k, _ = _rand(rng, (3, 50, 2, 64), "fp16")
    out = _f64(gr.flash_attention_cross(q, k, k, _i32([51, 50, -1])))
    assert gr.status() == gr.ERR_PAGE
    assert (out[0] == 0).all() and (out[2] == 0).all() and (out[1] != 0).any()


def test_cross_strides_streams_and_graphs():
    """Slices of a fused projection of the states, heads before tokens; calls on two streams; captured and replayed."""
    import torch
    rng = np.random.default_rng(6)
    q, _ = _rand(rng, (2, 4, 33, 64), "bf16")
    q = q.transpose(1, 2)
    x, _ = _rand(rng, (2, 2000, 4, 64), "bf16")
    k, v = x.split([2, 2], dim=2)
    n = _i32([2000, 1111])
    want = gr.flash_attention_cross(q.contiguous(), k.contiguous(), v.contiguous(), n)
    assert torch.equal(gr.flash_attention_cross(q, k, v, n), want)
    side = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for s in side:
            got.append(gr.flash_attention_cross(q, k, v, n, stream=s))
            got.append(gr.flash_attention_cross(q[:, :1], k, v, n, stream=s))
    torch.cuda.synchronize()
    one = gr.flash_attention_cross(q[:, :1], k, v, n)
    assert all(torch.equal(y, one if y.shape[1] == 1 else want) for y in got)
    out = torch.zeros(2, 33, 4, 64, dtype=torch.bfloat16, device="cuda")
    out1 = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gr.flash_attention_cross(q, k, v, n, out=out)
        gr.flash_attention_cross(q[:, :1], k, v, n, out=out1)
    n.copy_(_i32([7, 2000]))
    for _ in range(3):
        out.zero_(), out1.zero_()
        graph.replay()
        assert torch.equal(out, gr.flash_attention_cross(q, k, v, n))
        assert torch.equal(out1, gr.flash_attention_cross(q[:, :1], k, v, n))


def test_cross_without_rows_or_states():
    import torch
    z = torch.zeros
    kw = dict(device="cuda", dtype=torch.float16)
    assert gr.flash_attention_cross(z(2, 0, 4, 64, **kw), z(2, 9, 4, 64, **kw), z(2, 9, 4, 64, **kw)).shape == (2, 0, 4, 64)
    out = gr.flash_attention_cross(z(2, 3, 4, 64, **kw) + 1, z(2, 0, 4, 64, **kw), z(2, 0, 4, 64, **kw))
    assert (out == 0).all()


@pytest.mark.parametrize("hq,d", [(3, 128), (7, 64), (100, 64)])
def test_cross_same_bits_whatever_ran_before(hq, d):
    """Groups that do not divide a tile's 128 rows, after calls that leave other values in shared memory."""
    import torch
    rng = np.random.default_rng(8)
    q, _ = _rand(rng, (1, 129, hq, d), "fp16", 2.0)
    k, _ = _rand(rng, (1, 513, 1, d), "fp16")
    want = gr.flash_attention_cross(q, k, k)
    for scale in (0.0, 1000.0, 30000.0):
        x = torch.full((4, 300, 8, d), scale, device="cuda", dtype=torch.float16)
        gr.flash_attention_cross(x, x, x)
        assert torch.equal(gr.flash_attention_cross(q, k, k).view(torch.int16), want.view(torch.int16))
