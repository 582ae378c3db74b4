"""rotary on the GPU against the definition in 64 bits."""
import math

import numpy as np
import pytest

import tiled_tensor_core_03_gb300 as gr

from test_gpu_serving import DTYPES, _cuda, _dt, _f64, _half_step, _rand  # noqa: F401

pytestmark = pytest.mark.gpu


def _reference(x, positions, freq, interleaved, amplitude, inverse):
    """x float64 [..., heads, d], positions [...], freq [half]: the result, and a bound on each element before its rounding
    (|x1| + |x2|) a."""
    half = len(freq)
    t = positions[..., None, None].astype(np.float64) * freq
    if inverse:
        t = -t
    c, s = amplitude * np.cos(t), amplitude * np.sin(t)
    one, two = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
                else (slice(0, half), slice(half, 2 * half)))
    y, size = x.copy(), np.zeros_like(x)
    a, b = x[..., one], x[..., two]
    y[..., one], y[..., two] = a * c - b * s, b * c + a * s
    size[..., one] = size[..., two] = abs(amplitude) * (np.abs(a) + np.abs(b))
    return y, size


def _check(got, x, positions, freq, interleaved, amplitude, inverse, dtype):
    want, size = _reference(x, positions, freq, interleaved, amplitude, inverse)
    # in 32 bits: the angle is off by 2^-26 turns and by 2^-51 of its turns (both of the 64-bit angles), sine and cosine by
    # 2 ulp (2^-22), the amplitude, its two products and the sum by 2^-24 each; the result is rounded once
    turns = np.abs(positions).max(initial=0) * np.abs(freq).max() / (2 * math.pi)
    rel = 2 * math.pi * (2.0 ** -26 + 2.0 ** -51 * turns) + 2.0 ** -22 + 4 * 2.0 ** -24
    least = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -134     # half of the smallest step
    bound = _half_step(dtype) * np.abs(want) + rel * (1 + _half_step(dtype)) * size + least
    err = np.abs(got - want)
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("b,t,hq,hkv,d,rot,interleaved,far,inverse", [
    (1, 1, 1, 1, 64, 64, False, 0, False), (2, 37, 4, 2, 128, 128, False, 5000, False),
    (3, 5, 7, 1, 64, 32, True, 100000, True), (1, 300, 8, 8, 128, 64, True, 70, False),
    (2, 9, 3, 3, 64, 20, False, 1000, False), (2, 9, 3, 3, 64, 20, True, 1000, True),
    (1, 700, 2, 1, 256, 256, False, 10 ** 6, False), (1, 3, 5, 2, 512, 512, True, 44, False),
    (2, 33, 1, 1, 8, 2, False, 9, False), (1, 21, 2, 2, 512, 510, False, 3, True), (1, 4, 40, 0, 80, 80, False, 1, False),
    (5, 1, 33, 5, 96, 48, False, 10 ** 9, False), (1, 1000, 3, 1, 72, 8, True, 12, False)])
def test_rotary(b, t, hq, hkv, d, rot, interleaved, far, inverse, dtype):
    import torch
    rng = np.random.default_rng(t + d + rot + far % 1000)
    q, q64 = _rand(rng, (b, t, hq, d), dtype)
    k, k64 = _rand(rng, (b, t, hkv, d), dtype) if hkv else (None, None)
    pos = rng.integers(0, far + 1, (b, t))
    freq = gr.rotary_frequencies(rot)
    amplitude = 1.0 if far < 100 else 1.2
    for p in (torch.from_numpy(pos).cuda(), torch.from_numpy(pos.astype(np.int32)).cuda()):
        y, z = gr.rotary(q, k, p, freq, interleaved, amplitude, inverse)
        a = float(np.float32(amplitude))
        _check(_f64(y), q64, pos, _f64(freq), interleaved, a, inverse, dtype)
        if hkv:
            _check(_f64(z), k64, pos, _f64(freq), interleaved, a, inverse, dtype)
        else:
            assert z is None
    # 32-bit frequencies are what they are
    y, _ = gr.rotary(q, k, p, freq.float(), interleaved, amplitude, inverse)
    _check(_f64(y), q64, pos, _f64(freq.float()), interleaved, a, inverse, dtype)


def test_rotary_positions_of_any_size():
    """Negative positions and ones past 2^31, where an angle in 32 bits has no meaning left."""
    import torch
    rng = np.random.default_rng(1)
    pos = np.array([[-1, -5000, 2 ** 31 + 7, 2 ** 33 + 12345, -(2 ** 35) - 3, 0, 2 ** 31 - 1]])
    q, q64 = _rand(rng, (1, 7, 2, 64), "fp16")
    freq = gr.rotary_frequencies(64)
    y, _ = gr.rotary(q, None, torch.from_numpy(pos).cuda(), freq)
    _check(_f64(y), q64, pos, _f64(freq), False, 1.0, False, "fp16")
    near = torch.from_numpy(pos[:, [0, 1, 5, 6]].astype(np.int32)).cuda()
    y, _ = gr.rotary(q[:, [0, 1, 5, 6]].contiguous(), None, near, freq)
    _check(_f64(y), q64[:, [0, 1, 5, 6]], pos[:, [0, 1, 5, 6]], _f64(freq), False, 1.0, False, "fp16")


def test_rotary_frequencies_of_any_size():
    """Above a radian a token, above a turn, negative, tiny, zero."""
    import torch
    rng = np.random.default_rng(2)
    freq = torch.tensor([0.0, 1.0, 1.999, 2.0, 6.5, 100.25, 3e5, 2.0 ** 30, -0.75, -33.0, 1e-9, 1e-19, 1e-30, 4.0, 8.0, -1e-3],
                        dtype=torch.float64, device="cuda")
    q, q64 = _rand(rng, (1, 40, 2, 32), "fp16")
    pos = np.arange(40)[None]
    y, _ = gr.rotary(q, None, torch.from_numpy(pos).cuda(), freq)
    _check(_f64(y), q64, pos, _f64(freq), False, 1.0, False, "fp16")


def test_rotary_frequencies_for_long_contexts():
    import torch
    f = gr.rotary_frequencies(64, base=500000.0)
    want = 500000.0 ** (-np.arange(32) / 32)
    assert np.allclose(_f64(f), want, rtol=1e-13)
    assert np.allclose(_f64(gr.rotary_frequencies(64, 500000.0, factor=8)), want / 8, rtol=1e-13)
    g = _f64(gr.rotary_frequencies(64, 500000.0, factor=8, context=8192, low=1, high=4))
    turns = 8192 * want / (2 * math.pi)
    assert np.allclose(g[turns >= 4], want[turns >= 4], rtol=1e-13)
    assert np.allclose(g[turns <= 1], want[turns <= 1] / 8, rtol=1e-13)
    between = (turns > 1) & (turns < 4)
    assert between.any() and (g[between] < want[between]).all() and (g[between] > want[between] / 8).all()
    assert f.dtype == torch.float64 and f.is_cuda


@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, True), (20, False)])
def test_rotary_in_place_and_strides(rot, interleaved):
    """In place on slices of a fused projection: v and the elements past rot keep their bits; packed rows, heads before
    tokens, an expanded input."""
    import torch
    rng = np.random.default_rng(3)
    x, _ = _rand(rng, (2, 50, 4 + 2 + 2, 128), "bf16")
    pos = torch.arange(100, device="cuda").view(2, 50)
    freq = gr.rotary_frequencies(rot)
    was = x.clone()
    q, k, v = x.split([4, 2, 2], dim=2)
    wq, wk = gr.rotary(q.contiguous(), k.contiguous(), pos, freq, interleaved)
    aq, ak = gr.rotary(q, k, pos, freq, interleaved)
    assert torch.equal(aq, wq) and torch.equal(ak, wk) and torch.equal(x, was)
    bq, bk = gr.rotary(q.reshape(100, 4, 128), k.reshape(100, 2, 128), pos.view(-1), freq, interleaved)
    assert torch.equal(bq.view_as(wq), wq) and torch.equal(bk.view_as(wk), wk)
    h = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(gr.rotary(h, None, pos, freq, interleaved)[0], wq)
    e = q[:, :, :1].expand(2, 50, 3, 128)
    assert torch.equal(gr.rotary(e, None, pos, freq, interleaved)[0][:, :, 2], wq[:, :, 0])
    to = torch.zeros_like(x)
    oq, ok = to[:, :, 2:6], to[:, :, 6:]
    r = gr.rotary(q, k, pos, freq, interleaved, out=(oq, ok))
    assert r[0] is oq and torch.equal(oq, wq) and torch.equal(ok, wk) and (to[:, :, :2] == 0).all()
    gr.rotary(q, k, pos, freq, interleaved, out=(q, k))
    assert torch.equal(q, wq) and torch.equal(k, wk) and torch.equal(v, was[:, :, 6:])
    assert torch.equal(q[..., rot:], was[:, :, :4, rot:])


def test_rotary_inverse_is_the_gradient():
    """The gradient of sum(g . rotary(x)) is the inverse rotation of g: against the formula's own (autograd on the 64-bit
    definition) and against differences."""
    import torch
    rng = np.random.default_rng(4)
    pos = torch.from_numpy(rng.integers(0, 3000, (2, 11))).cuda()
    for rot, interleaved, amplitude in ((64, False, 1.0), (32, True, 1.25), (20, False, 0.5)):
        freq = gr.rotary_frequencies(rot)
        x, x64 = _rand(rng, (2, 11, 3, 64), "fp16")
        g, g64 = _rand(rng, (2, 11, 3, 64), "fp16")
        dx, _ = gr.rotary(g, None, pos, freq, interleaved, amplitude, inverse=True)
        half = rot // 2
        leaf = x.double().requires_grad_()
        t = pos[..., None, None].double() * freq
        a, b = (leaf[..., 0:rot:2], leaf[..., 1:rot:2]) if interleaved else (leaf[..., :half], leaf[..., half:rot])
        c, s = amplitude * t.cos(), amplitude * t.sin()
        ya, yb = a * c - b * s, b * c + a * s
        y = torch.cat([torch.stack([ya, yb], -1).flatten(-2) if interleaved else torch.cat([ya, yb], -1),
                       leaf[..., rot:]], -1)
        y.backward(g.double())
        want = leaf.grad
        size = amplitude * 2 * g.double().abs().amax()
        assert float((dx.double() - want).abs().max()) <= float(_half_step("fp16") * want.abs().max() + 2.0 ** -20 * size)
        # differences: the map is linear, so a step of any length gives the derivative; outputs are rounded to fp16
        v, _ = _rand(rng, (2, 11, 3, 64), "fp16")
        step = [gr.rotary((x + e * v).contiguous(), None, pos, freq, interleaved, amplitude)[0].double()
                for e in (4.0, -4.0)]
        inputs = ((x + 4.0 * v).double() - (x - 4.0 * v).double())
        slope = ((step[0] - step[1]) * g.double()).sum()
        analytic = (dx.double() * inputs).sum()
        # 4224 roundings of outputs up to 2^6 (half a step 2^-6) and of dx, each with a random sign
        noise = 8 * math.sqrt(x.numel()) * 2.0 ** -6
        assert abs(float(slope - analytic)) <= noise * float(g.double().abs().mean() + 1), (float(slope), float(analytic))


def test_rotary_streams_and_graphs():
    import torch
    rng = np.random.default_rng(5)
    q, _ = _rand(rng, (64, 8, 128), "fp16")
    k, _ = _rand(rng, (64, 2, 128), "fp16")
    pos = torch.arange(64, device="cuda", dtype=torch.int32)
    freq = gr.rotary_frequencies(128)
    want = gr.rotary(q, k, pos, freq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gr.rotary(q, k, pos, freq, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = torch.zeros_like(q), torch.zeros_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gr.rotary(q, k, pos, freq, out=out)
    pos.add_(1000)
    graph.replay()
    want = gr.rotary(q, k, pos, freq)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_rotary_without_rows():
    import torch
    kw = dict(device="cuda", dtype=torch.float16)
    freq = gr.rotary_frequencies(64)
    q, k = gr.rotary(torch.zeros((0, 4, 64), **kw), torch.zeros((0, 2, 64), **kw),
                     torch.zeros(0, dtype=torch.int32, device="cuda"), freq)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    pos = torch.arange(3, device="cuda")
    x = torch.ones((3, 2, 64), **kw)
    q, k = gr.rotary(torch.zeros((3, 0, 64), **kw), x, pos, freq)
    assert q.shape == (3, 0, 64) and torch.equal(k, gr.rotary(x, None, pos, freq)[0])


def test_rotary_refusals():
    import torch
    x = torch.zeros((2, 3, 4, 64), dtype=torch.float16, device="cuda")
    pos = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    freq = gr.rotary_frequencies(64)
    for args in ((x, x.bfloat16(), pos, freq), (x, x[:, :2], pos, freq), (x, x[0], pos, freq), (x, x, pos[0], freq),
                 (x, x, pos.float(), freq), (x, x, pos, freq.half()), (x, x, pos, gr.rotary_frequencies(66)),
                 (x[..., 1:], None, pos, freq), (x.cpu(), x, pos, freq), (x, x, pos, freq.cpu()),
                 (x[0, 0], None, pos[0], freq), (torch.zeros((2, 3, 4, 65), dtype=torch.float16, device="cuda")[..., 1:],
                                                None, pos, freq)):
        with pytest.raises(ValueError):
            gr.rotary(*args)
    with pytest.raises(TypeError):
        gr.rotary(x.float(), None, pos, freq)
    for out in ((x[:, :2], None), (x.bfloat16(), None), (x[:1].expand(2, 3, 4, 64), None), (x, x),
                (x.transpose(1, 2).contiguous().transpose(1, 2)[..., :32], None)):
        with pytest.raises(ValueError):
            gr.rotary(x, None, pos, freq, out=out)
    square = torch.zeros((2, 4, 4, 64), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):    # begins where q does, with other strides
        gr.rotary(square, None, torch.zeros((2, 4), dtype=torch.int32, device="cuda"), freq,
                  out=(square.transpose(1, 2), None))
    for kw in (dict(rot=3), dict(rot=0), dict(rot=8, factor=0.5), dict(rot=8, base=0), dict(rot=8, low=4, high=4)):
        with pytest.raises(ValueError):
            gr.rotary_frequencies(**kw)
