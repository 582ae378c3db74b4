"""The serving operators on the GPU against the plain 64-bit implementations.

Tolerances count roundings (half a step each: fp16 2^-11, bf16 2^-8 relative to the value)
and the bounds of serving_reference.weight_error for what happens in 32 bits; what is
stored in 8 bits, and which tokens stay, has to be equal."""
import numpy as np
import pytest

import tiled_tensor_core_03_gb300 as gr

import serving_reference as ref

pytestmark = pytest.mark.gpu

DTYPES = ("fp16", "bf16")


@pytest.fixture(autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert gr.status() == gr.OK


def _dt(name):
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16}[name]


def _rand(rng, shape, dtype, scale=1.0):
    """A CUDA tensor and the same values in float64."""
    import torch
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(_dt(dtype))
    return t.cuda(), t.double().numpy()


def _f64(t):
    return t.double().cpu().numpy()


def _i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _half_step(dtype):
    import torch
    return torch.finfo(_dt(dtype)).eps / 2


def _check(got, want, absv, size, d, dtype, p_half):
    """|got - want| within the output's rounding, the weights' rounding to p_half, and 32 bits."""
    err = np.abs(got - want)
    # 2^-22 of sum w |v|: 32-bit sums of up to some thousands of terms
    bound = _half_step(dtype) * np.abs(want) + (p_half + ref.weight_error(size, d) + 2.0 ** -22) * absv \
        * (1 + _half_step(dtype)) + 2.0 ** -25
    assert np.isfinite(got).all()
    assert (err <= bound).all(), (float((err / bound).max()), np.argwhere(err > bound)[:5])


# ---------------------------------------------------------------- flash_attention_window


def _window(rng, b, sq, skv, hq, hkv, d, window, sinks, dtype, scale=1.0):
    q, q64 = _rand(rng, (b, sq, hq, d), dtype, scale)
    k, k64 = _rand(rng, (b, skv, hkv, d), dtype)
    v, v64 = _rand(rng, (b, skv, hkv, d), dtype)
    out = gr.flash_attention_window(q, k, v, window, sinks)
    again = gr.flash_attention_window(q, k, v, window, sinks)
    assert gr.status() == gr.OK
    got = _f64(out)
    for i in range(b):
        o, absv, _, size = ref.attend(q64[i], k64[i], v64[i], window, sinks)
        _check(got[i], o, absv, size, d, dtype, _half_step(dtype))
    import torch
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("b,sq,skv,hq,hkv,d,window,sinks", [
    (1, 1, 1, 1, 1, 64, 1, 0), (1, 1, 300, 4, 2, 128, 7, 2), (2, 130, 130, 2, 2, 64, 0, 0),
    (1, 129, 129, 3, 1, 128, 1, 0), (1, 300, 300, 3, 3, 64, 64, 4), (1, 257, 500, 6, 2, 128, 128, 1),
    (1, 128, 640, 5, 5, 64, 200, 130), (2, 100, 40, 4, 1, 64, 16, 3), (1, 513, 513, 1, 1, 128, 127, 300),
    (1, 400, 1000, 2, 1, 64, 129, 128), (1, 33, 2000, 8, 1, 128, 1999, 5), (1, 600, 600, 7, 1, 64, 255, 0)])
def test_window(b, sq, skv, hq, hkv, d, window, sinks, dtype):
    _window(np.random.default_rng(sq * 7 + skv + d + window), b, sq, skv, hq, hkv, d, window, sinks, dtype)


def test_window_large_scores():
    """Scores of tens of units: the running reference moves often and weights underflow."""
    _window(np.random.default_rng(5), 1, 500, 500, 2, 1, 128, 300, 4, "fp16", scale=6.0)


def test_window_without_window_is_causal_attention():
    import torch
    rng = np.random.default_rng(6)
    q, _ = _rand(rng, (2, 400, 3, 128), "fp16")
    k, _ = _rand(rng, (2, 400, 3, 128), "fp16")
    v, _ = _rand(rng, (2, 400, 3, 128), "fp16")
    a = gr.flash_attention_window(q, k, v, 0)
    b = gr.flash_attention(q, k, v, causal=True)
    # the same blocks in the same order: the same bits
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("batch,n_q,n_kv,group,kvh,d,window", [
    (1, 300, 32768, 1, 7, 128, 900),     # 16 MB of K and V a head: four heads together, then three
    (1, 900, 70000, 3, 3, 64, 0),        # five tiles of two heads; 18 MB a head
    (5, 700, 700, 3, 7, 64, 100),        # all heads together, several rounds of a grid
    (1, 300, 260000, 2, 3, 128, 5000),   # no two heads fit
])
def test_window_order_of_heads(batch, n_q, n_kv, group, kvh, d, window):
    """Heads whose work is interleaved give the bits that each gives alone."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(n_q)
    q = torch.randn(batch, n_q, kvh * group, d, device="cuda", dtype=torch.float16, generator=g)
    k, v = (torch.randn(batch, n_kv, kvh, d, device="cuda", dtype=torch.float16, generator=g)
            for _ in range(2))
    out = gr.flash_attention_window(q, k, v, window, 4)
    for b in range(batch):
        for h in range(kvh):
            alone = gr.flash_attention_window(q[b:b + 1, :, h * group:(h + 1) * group], k[b:b + 1, :, h:h + 1],
                                              v[b:b + 1, :, h:h + 1], window, 4)
            mine = out[b:b + 1, :, h * group:(h + 1) * group]
            assert torch.equal(mine.view(torch.int16), alone.view(torch.int16)), (b, h)


def test_window_strides_and_stream():
    """Slices of a fused projection, heads before tokens, an axis of one with an odd stride; on a
    side stream."""
    import torch
    rng = np.random.default_rng(7)
    x, x64 = _rand(rng, (2, 200, 4 + 2 + 2, 64), "bf16")
    q, k, v = x.split([4, 2, 2], dim=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = gr.flash_attention_window(q, k, v, 50, 3, stream=side)
    side.synchronize()
    dense = gr.flash_attention_window(q.contiguous(), k.contiguous(), v.contiguous(), 50, 3)
    assert torch.equal(out, dense)
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)
    vt = v.transpose(0, 2).contiguous().transpose(0, 2)
    assert torch.equal(gr.flash_attention_window(qt, k, vt, 50, 3), dense)
    one = q[:1].as_strided((1, 200, 4, 64), (3, *q.stride()[1:]))
    assert torch.equal(gr.flash_attention_window(one, k[:1], v[:1], 50, 3), dense[:1])
    for bad in (q[..., ::2], x[:, :, :, 1:].as_strided((2, 200, 4, 64), q.stride(), 1)):
        with pytest.raises(ValueError):
            gr.flash_attention_window(bad, k, v, 50, 3)
    with pytest.raises(gr.GemmReluError):
        gr.flash_attention_window(q, k[:, :, :1].expand(2, 200, 2, 64), v, 50, 3)
    with pytest.raises(ValueError):
        gr.flash_attention_window(q[:, :, :3], k, v, 50, 3)
    with pytest.raises(TypeError):
        gr.flash_attention_window(q.float(), k.float(), v.float(), 50, 3)


@pytest.mark.parametrize("dtype", DTYPES)
def test_window_not_finite_reaches_those_who_see_it(dtype):
    """A NaN or infinity in K or V of one token: rows that see it are not finite as the formula
    says, all others are as if it were 0."""
    import torch
    rng = np.random.default_rng(8)
    n, window, sinks, d = 300, 40, 2, 64
    q, q64 = _rand(rng, (1, n, 2, d), dtype)
    k, k64 = _rand(rng, (1, n, 1, d), dtype)
    v, v64 = _rand(rng, (1, n, 1, d), dtype)
    for at, where, value in ((150, "v", np.nan), (20, "v", np.inf), (299, "v", np.nan), (200, "k", np.nan),
                             (128, "k", -np.inf)):
        kk, vv, kk64, vv64 = k.clone(), v.clone(), k64.copy(), v64.copy()
        (vv if where == "v" else kk)[0, at, 0, 5] = value
        (vv64 if where == "v" else kk64)[0, at, 0, 5] = value
        got = _f64(gr.flash_attention_window(q, kk, vv, window, sinks))[0]
        o, absv, _, size = ref.attend(q64[0], kk64[0], vv64[0], window, sinks)
        sees = np.array([at <= p and (at > p - window or at < sinks) for p in range(n)])
        if where == "v":
            assert np.array_equal(np.isfinite(got), np.isfinite(o))
            assert not np.isfinite(got[sees, :, 5]).any() and np.isfinite(np.delete(got, 5, 2)).all()
        else:
            assert np.isfinite(got[~sees]).all()
            assert np.array_equal(np.isnan(got), np.isnan(o))
        rows = ~sees
        _check(got[rows], o[rows], absv[rows], size[rows], d, dtype, _half_step(dtype))


def test_window_empty():
    import torch
    x = torch.zeros((0, 5, 2, 64), dtype=torch.float16, device="cuda")
    assert gr.flash_attention_window(x, x, x, 3).shape == x.shape
    q = torch.ones((1, 5, 2, 64), dtype=torch.float16, device="cuda")
    assert (gr.flash_attention_window(q, q[:, :0], q[:, :0], 3) == 0).all()


def test_window_dropped_arrival_times_out_and_recovers():
    rng = np.random.default_rng(9)
    gr.gemm_relu_debug_set(1, 20_000_000)
    try:
        q, _ = _rand(rng, (1, 300, 2, 64), "fp16")
        gr.flash_attention_window(q, q, q, 100, 4)
        assert gr.status() == gr.ERR_TIMEOUT
    finally:
        gr.gemm_relu_debug_set(0, 0)
    _window(rng, 1, 300, 300, 2, 1, 64, 100, 4, "fp16")


# ---------------------------------------------------------------- the cache


def _cache(rng, num_pages, hkv, page, d, garbage=True):
    """A pool of random finite e4m3 values and power-of-two scales, or of random bytes (NaN among
    them); and the same as float64 arrays [k, v, k_scale, v_scale]."""
    import torch
    codes = rng.integers(0, 256, (2, num_pages, hkv, page, d)).astype(np.uint8)
    if not garbage:
        codes = np.where((codes & 0x7f) == 0x7f, codes - 1, codes).astype(np.uint8)
        codes = np.where((codes & 0x7f) > 0x60, codes & 0xdf, codes).astype(np.uint8)
    scales = 2.0 ** rng.integers(-9, -4, (2, num_pages, hkv))
    t = [torch.from_numpy(c).cuda().view(torch.float8_e4m3fn) for c in codes]
    s = [torch.from_numpy(x.astype(np.float32)).cuda() for x in scales]
    return gr.KVCache(*t, *s), [ref.e4m3_decode(codes[0]), ref.e4m3_decode(codes[1]), scales[0], scales[1]]


def _tables(rng, counts, num_pages, width=None):
    """Pages in no order; -1 past a sequence's last."""
    ids = rng.permutation(num_pages)[:sum(counts)]
    t = np.full((len(counts), width or max(max(counts), 1)), -1)
    at = 0
    for i, c in enumerate(counts):
        t[i, :c] = ids[at:at + c]
        at += c
    return t


def _same_cache(cache, want):
    for x, w in zip(cache, want):
        assert np.array_equal(_f64(x.float()), w, equal_nan=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page,d,hkv,lengths,counts", [
    (16, 64, 1, [1], [1]), (16, 128, 3, [40, 17, 16], [40, 1, 3]), (32, 64, 2, [33, 100, 64], [2, 70, 64]),
    (64, 128, 2, [64, 65, 63, 200], [1, 1, 1, 150]), (128, 128, 1, [128, 129, 300], [5, 129, 300]),
    (128, 64, 2, [50, 256], [50, 0])])
def test_append(page, d, hkv, lengths, counts, dtype):
    """Fresh pages, pages that grow with and without a larger scale, several pages at once; slots
    that are not written keep their bytes (the pool starts as random bytes)."""
    rng = np.random.default_rng(page + d + hkv)
    need = [-(-n // page) for n in lengths]
    cache, want = _cache(rng, sum(need) + 2, hkv, page, d)
    # what a page already holds is finite
    table = _tables(rng, need, sum(need) + 2)
    clean, clean64 = _cache(rng, sum(need) + 2, hkv, page, d, garbage=False)
    b, t = len(lengths), max(counts)
    for x, c, w, c64 in zip(cache, clean, want, clean64):
        for i in range(b):
            at = (lengths[i] - counts[i]) // page
            if lengths[i] - counts[i] > at * page and counts[i] > 0:
                x[int(table[i, at])] = c[int(table[i, at])]
                w[table[i, at]] = c64[table[i, at]]
    mag = rng.choice([0.1, 1.0, 300.0], (b, t, hkv, 1))
    import torch
    k, _ = _rand(rng, (b, t, hkv, d), dtype)
    k = (k.float() * torch.from_numpy(mag).float().cuda()).to(_dt(dtype))
    v, _ = _rand(rng, (b, t, hkv, d), dtype, 0.01)
    gr.kv_cache_append(cache, k, v, _i32(table), _i32(lengths), _i32(counts))
    assert gr.status() == gr.OK
    for i in range(b):
        for x, which in ((k, 0), (v, 1)):
            ref.append(want[which], want[which + 2], _f64(x)[i], table[i], page, lengths[i], counts[i])
    _same_cache(cache, want)
    # written again: the same
    gr.kv_cache_append(cache, k, v, _i32(table), _i32(lengths), _i32(counts))
    _same_cache(cache, want)


def test_append_numbers_at_the_edges():
    """NaN and infinities become NaN and leave the scale alone; zeros, subnormals, the largest
    finite values; strided input; no counts."""
    import torch
    rng = np.random.default_rng(3)
    cache, want = _cache(rng, 6, 2, 16, 64)
    x = torch.zeros((4, 16, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    x[0, :, 0] = torch.randn((16, 2, 64), device="cuda").bfloat16()
    x[0, 3, 0, 0, 7] = float("nan")
    x[0, 4, 0, 1, 8] = float("inf")
    x[0, 5, 0, 1, 9] = -float("inf")
    x[1] = 1e-39
    x[2] = 3e38
    x[3, :, 1] = float("nan")
    k, v = x[:, :, 0], x[:, :, 1]
    table = np.array([[5], [0], [3], [1]])
    gr.kv_cache_append(cache, k, v, _i32(table), _i32([16] * 4))
    for i in range(4):
        for t, which in ((k, 0), (v, 1)):
            ref.append(want[which], want[which + 2], _f64(t)[i], table[i], 16, 16, 16)
    _same_cache(cache, want)


@pytest.mark.parametrize("exponent", [-110, -60, -30, -20, 0, 20, 24, 30, 100])
def test_append_beside_a_far_scale(exponent):
    """New fp16 tokens of every magnitude in a page whose scale is far from theirs."""
    import torch
    rng = np.random.default_rng(exponent + 200)
    cache, want = _cache(rng, 1, 1, 16, 64, garbage=False)
    for which in (2, 3):
        want[which][0, 0] = 2.0 ** max(exponent, -100)
        cache[which][0, 0] = 2.0 ** max(exponent, -100)
    mag = torch.tensor([2.0 ** -24, 2.0 ** -14, 1e-3, 1.0, 60000.0], device="cuda")[:, None, None]
    k = (torch.randn((1, 5, 1, 64), device="cuda").clamp(-1, 1) * mag).half()
    gr.kv_cache_append(cache, k, k, _i32([[0]]), _i32([12]))
    for which in (0, 1):
        ref.append(want[which], want[which + 2], _f64(k)[0], [0], 16, 12, 5)
    _same_cache(cache, want)


def test_append_refuses_what_only_the_device_sees():
    """Pages outside the pool, bad lengths and counts: nothing is written for them, the others
    are, and the status says so."""
    rng = np.random.default_rng(4)
    cache, want = _cache(rng, 4, 1, 16, 64)
    k, _ = _rand(rng, (6, 4, 1, 64), "fp16")
    table = np.array([[4], [-1], [0], [1], [2], [3]])
    lengths, counts = [4, 4, 4, 17, 2, -1], [4, 4, 4, 4, 3, 0]
    gr.kv_cache_append(cache, k, k, _i32(table), _i32(lengths), _i32(counts))
    assert gr.status() == gr.ERR_PAGE
    for which in (0, 1):
        ref.append(want[which], want[which + 2], _f64(k)[2], table[2], 16, 4, 4)
    _same_cache(cache, want)
    gr.kv_cache_append(cache, k, k, _i32(table), _i32([4] * 6), _i32([5] * 6))
    assert gr.status() == gr.ERR_PAGE
    _same_cache(cache, want)


# ---------------------------------------------------------------- attention over the cache


def _attend(rng, page, d, hkv, group, tokens, lengths, window, sinks, dtype, weights=False, scale=2.0,
            width=None, slots=None):
    import torch
    need = [-(-n // page) for n in lengths]
    total = sum(need) + 1
    cache, c64 = _cache(rng, total, hkv, page, d, garbage=False)
    table = _tables(rng, need, total, width)
    # slots past a sequence's length hold NaN
    for i, n in enumerate(lengths):
        if n % page:
            pid = int(table[i, n // page])
            for t in cache[:2]:
                t.view(torch.uint8)[pid, :, n % page:] = 0x7f
    b = len(lengths)
    q, q64 = _rand(rng, (b, tokens, hkv * group, d), dtype, scale)
    w = torch.rand((b, hkv, table.shape[1] * page), device="cuda") if weights else None
    w0 = None if w is None else _f64(w)
    w1 = None if w is None else w.clone()
    out = gr.kv_cache_attention(q, cache, _i32(table), _i32(lengths), window, sinks, weights=w)
    again = gr.kv_cache_attention(q, cache, _i32(table), _i32(lengths), window, sinks, weights=w1)
    assert gr.status() == gr.OK
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    got = _f64(out)
    for i, n in enumerate(lengths):
        ids = table[i, :need[i]]
        k, v = ((x[ids] * s[ids][..., None, None]).transpose(0, 2, 1, 3).reshape(-1, hkv, d)[:n]
                for x, s in ((c64[0], c64[2]), (c64[1], c64[3])))
        o, absv, mass, size = ref.attend(q64[i], k, v, window, sinks)
        _check(got[i], o, absv, size, d, dtype, 2.0 ** -11)
        if weights:
            rel = ref.weight_error(size.max(initial=0), d) + 2.0 ** -20
            err = np.abs(_f64(w)[i, :, :n] - w0[i, :, :n] - mass)
            assert (err <= rel * mass + 2.0 ** -23 * (w0[i, :, :n] + mass)).all(), float(err.max())
            assert np.array_equal(_f64(w)[i, :, n:], w0[i, :, n:])
    if weights:
        assert torch.equal(w, w1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page,d,hkv,group,tokens,lengths,window,sinks", [
    (16, 64, 1, 1, 1, [1], 0, 0), (64, 128, 2, 4, 1, [1, 64, 65, 0, 200], 0, 0),
    (128, 128, 1, 8, 1, [1000, 3], 0, 0), (16, 128, 2, 3, 4, [50, 4, 3, 1], 0, 0),
    (32, 64, 3, 1, 7, [333, 31, 7], 40, 2), (16, 64, 2, 8, 3, [700], 100, 70),
    (64, 128, 1, 5, 1, [900, 20], 64, 4), (128, 64, 4, 2, 17, [300, 129], 1, 0),
    (32, 128, 1, 16, 2, [4097], 0, 0), (64, 64, 1, 1, 64, [100, 10], 30, 1)])
def test_cache_attention(page, d, hkv, group, tokens, lengths, window, sinks, dtype):
    rng = np.random.default_rng(page + d + tokens + sum(lengths))
    _attend(rng, page, d, hkv, group, tokens, lengths, window, sinks, dtype)


@pytest.mark.parametrize("page,d,hkv,group,tokens,lengths,window,sinks", [
    (16, 64, 1, 1, 1, [5], 0, 0), (64, 128, 2, 4, 1, [500, 64, 0, 1], 0, 0),
    (128, 128, 1, 3, 7, [300, 2], 50, 3), (32, 64, 2, 8, 3, [1000, 40], 200, 4)])
def test_cache_attention_weights(page, d, hkv, group, tokens, lengths, window, sinks):
    rng = np.random.default_rng(page + d + tokens + sum(lengths))
    _attend(rng, page, d, hkv, group, tokens, lengths, window, sinks, "fp16", weights=True)


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("page,d,hkv,group,tokens,lengths,window,sinks", [
    (64, 128, 1, 8, 17, [700, 64, 17, 9], 0, 0),     # 17 tiles of 8 rows: nine at a time, the last one empty
    (32, 64, 2, 8, 33, [500, 40], 100, 3),           # 17 tiles of 16
    (16, 128, 2, 3, 90, [400, 95, 0], 0, 0),         # 34 tiles in three passes of twelve
    (128, 128, 1, 4, 8, [6000], 0, 0)])              # four tiles, each cut into many parts
def test_cache_attention_many_row_tiles(page, d, hkv, group, tokens, lengths, window, sinks, weights):
    rng = np.random.default_rng(page + d + tokens + sum(lengths))
    _attend(rng, page, d, hkv, group, tokens, lengths, window, sinks, "bf16", weights=weights)


def test_cache_attention_many_sequences_and_large_scores():
    """More sequences than threads that count them, most of them empty or short, a table wider than
    any needs; scores of tens of units."""
    rng = np.random.default_rng(11)
    lengths = [int(x) for x in rng.integers(0, 40, 401)]
    _attend(rng, 16, 64, 1, 2, 1, lengths, 0, 0, "fp16", width=9)
    _attend(rng, 64, 128, 2, 2, 2, [400, 90], 0, 0, "bf16", scale=16.0)


def test_cache_attention_scales_far_apart():
    """Pages whose scales differ by 2^40: each output is within its bound (the largest weight times
    scale sets what the others are rounded against)."""
    import torch
    rng = np.random.default_rng(12)
    cache, c64 = _cache(rng, 4, 1, 64, 64, garbage=False)
    for s, s64 in ((cache[2], c64[2]), (cache[3], c64[3])):
        s[:, 0] = torch.tensor([2.0 ** -8, 2.0 ** -48, 2.0 ** -8, 2.0 ** -100], device="cuda")
        s64[:, 0] = [2.0 ** -8, 2.0 ** -48, 2.0 ** -8, 2.0 ** -100]
    q, q64 = _rand(rng, (1, 1, 4, 64), "bf16")
    for order in ([0, 1, 2, 3], [3, 1, 0, 2], [1, 3, 1, 1]):
        out = gr.kv_cache_attention(q, cache, _i32([order]), _i32([256]))
        k, v = ((x[order] * s[order][..., None, None]).transpose(0, 2, 1, 3).reshape(-1, 1, 64)
                for x, s in ((c64[0], c64[2]), (c64[1], c64[3])))
        o, absv, _, size = ref.attend(q64[0], k, v, 0, 0)
        _check(_f64(out)[0], o, absv, size, 64, "bf16", 2.0 ** -11)


def test_cache_attention_not_finite_reaches_those_who_see_it():
    """A NaN in V of a token that later rows see and earlier ones do not (and one that left the
    window): rows that see it are NaN in its element, the others are as without it."""
    import torch
    rng = np.random.default_rng(13)
    n, tokens, window, d = 200, 40, 50, 128
    cache, c64 = _cache(rng, 4, 1, 64, d, garbage=False)
    table = [[2, 0, 3, 1]]
    q, q64 = _rand(rng, (1, tokens, 2, d), "fp16")
    k, v = ((x[table[0]] * s[table[0]][..., None, None]).transpose(0, 2, 1, 3).reshape(-1, 1, d)[:n]
            for x, s in ((c64[0], c64[2]), (c64[1], c64[3])))
    clean = _f64(gr.kv_cache_attention(q, cache, _i32(table), _i32([n]), window))[0]
    for at in (180, 199, 125, 165):
        v2 = [t.clone() for t in cache]
        v2[1].view(torch.uint8)[table[0][at // 64], 0, at % 64, 77] = 0xff
        got = _f64(gr.kv_cache_attention(q, gr.KVCache(*v2), _i32(table), _i32([n]), window))[0]
        sees = np.array([at <= p and at > p - window for p in range(n - tokens, n)])
        assert np.isnan(got[sees, :, 77]).all()
        got[sees, :, 77] = clean[sees, :, 77]
        if sees.all():
            continue
        bad = np.isnan(got)
        assert not bad[~sees].any() and not bad.any()
        assert np.allclose(got, clean, rtol=2 ** -9, atol=1e-6)
    k2 = [t.clone() for t in cache]
    k2[0].view(torch.uint8)[table[0][2], 0, 52, 3] = 0x7f      # token 180
    got = _f64(gr.kv_cache_attention(q, gr.KVCache(*k2), _i32(table), _i32([n]), window))[0]
    assert np.isnan(got[20:]).all()
    assert np.array_equal(got[:20], clean[:20])


def test_cache_attention_refuses_what_only_the_device_sees():
    """A page outside the pool is skipped, a bad length is a sequence without tokens; the others
    are right and the status says so."""
    import torch
    rng = np.random.default_rng(14)
    cache, c64 = _cache(rng, 8, 2, 16, 64, garbage=False)
    q, q64 = _rand(rng, (4, 1, 4, 64), "fp16")
    table = np.array([[0, 1], [2, 99], [-7, 3], [4, 5]])
    w = torch.zeros((4, 2, 32), device="cuda")
    out = _f64(gr.kv_cache_attention(q, cache, _i32(table), _i32([33, 30, 30, 30]), weights=w))
    assert gr.status() == gr.ERR_PAGE
    assert (out[0] == 0).all()
    for i, ids, n in ((1, [2], 16), (2, [3], 14), (3, [4, 5], 30)):
        k, v = ((x[ids] * s[ids][..., None, None]).transpose(0, 2, 1, 3).reshape(-1, 2, 64)[:n]
                for x, s in ((c64[0], c64[2]), (c64[1], c64[3])))
        o, absv, _, size = ref.attend(q64[i], k, v, 0, 0)
        _check(out[i], o, absv, size, 64, "fp16", 2.0 ** -11)
    w = _f64(w)
    assert (w[0] == 0).all() and (w[1, :, 16:] == 0).all() and (w[2, :, :16] == 0).all()
    assert np.allclose(w[1:].sum(-1), 2, rtol=1e-5)
    out = _f64(gr.kv_cache_attention(q, cache, _i32(table), _i32([-1, 0, 0, 0])))
    assert gr.status() == gr.ERR_PAGE
    assert (out == 0).all()


def test_cache_attention_workspace_and_errors():
    import torch
    rng = np.random.default_rng(15)
    cache, _ = _cache(rng, 4, 2, 16, 64, garbage=False)
    q, _ = _rand(rng, (2, 1, 4, 64), "fp16")
    pages, lengths = _i32([[0, 1], [2, 3]]), _i32([20, 31])
    ws = gr.kv_cache_attention_workspace(q, cache)
    guard = torch.full((ws.numel() + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    guard[256:256 + gr.KV_COUNTER_BYTES] = 0
    out = torch.full_like(q, 7.0)
    got = gr.kv_cache_attention(q, cache, pages, lengths, out=out, workspace=guard[256:-256])
    assert got is out
    assert (guard[:256] == 0x5a).all() and (guard[-256:] == 0x5a).all()
    assert (guard[256:256 + gr.KV_COUNTER_BYTES] == 0).all()       # left as they were found
    assert torch.equal(out, gr.kv_cache_attention(q, cache, pages, lengths))
    with pytest.raises(gr.GemmReluError) as e:
        gr.kv_cache_attention(q, cache, pages, lengths, workspace=ws[:-256])
    assert e.value.code == gr.ERR_WORKSPACE
    for kw in (dict(window=-1), dict(sinks=-1), dict(weights=torch.zeros((2, 2, 31), device="cuda")),
               dict(out=out[:1])):
        with pytest.raises(ValueError):
            gr.kv_cache_attention(q, cache, pages, lengths, **kw)
    for bad in ((q[:, :, :3], pages, lengths), (q, pages.long(), lengths), (q, pages, lengths[:1])):
        with pytest.raises(ValueError):
            gr.kv_cache_attention(bad[0], cache, *bad[1:])
    with pytest.raises(TypeError):
        gr.kv_cache_attention(q.float(), cache, pages, lengths)
    assert gr.kv_cache_attention(q[:, :0], cache, pages, lengths).shape == (2, 0, 4, 64)


def test_cache_attention_dropped_arrival_times_out_and_recovers():
    rng = np.random.default_rng(16)
    cache, _ = _cache(rng, 4, 1, 64, 128, garbage=False)
    q, _ = _rand(rng, (1, 1, 4, 128), "fp16")
    args = (q, cache, _i32([[0, 1, 2, 3]]), _i32([250]))
    want = gr.kv_cache_attention(*args)
    gr.gemm_relu_debug_set(1, 20_000_000)
    try:
        # block 0 of this many has no unit of so short a sequence; take a batch that gives it one
        big = (q.expand(400, 1, 4, 128).contiguous(), cache, _i32([[0, 1, 2, 3]] * 400), _i32([250] * 400))
        gr.kv_cache_attention(*big)
        assert gr.status() == gr.ERR_TIMEOUT
    finally:
        gr.gemm_relu_debug_set(0, 0)
    import torch
    assert torch.equal(gr.kv_cache_attention(*args), want)


# ---------------------------------------------------------------- eviction


def _evict(rng, page, d, hkv, lengths, budget, sinks, recent, weights=None, same_pool=False,
           garbage=False):
    import torch
    need = [-(-n // page) for n in lengths]
    keep = [-(-min(n, budget) // page) for n in lengths]
    total = sum(need) + sum(keep) + 1
    cache, c64 = _cache(rng, total, hkv, page, d, garbage=garbage)
    to, t64 = (cache, c64) if same_pool else _cache(rng, total, hkv, page, d)
    both = _tables(rng, need + keep, total)
    table = both[:len(need), :max(max(need), 1)]
    to_table = both[len(need):, :-(-budget // page)]
    if to_table.shape[1] * page < budget:
        to_table = np.pad(to_table, ((0, 0), (0, -(-budget // page) - to_table.shape[1])), constant_values=-1)
    width = table.shape[1] * page
    b = len(lengths)
    if weights is None:
        weights = np.exp(2 * rng.standard_normal((b, hkv, width)))
        weights[rng.random(weights.shape) < 0.2] = 0
    w = torch.from_numpy(weights[..., :width].astype(np.float32)).cuda()
    before = [x.copy() for x in c64]
    n2, w2, kept = gr.kv_cache_evict(cache, w, _i32(table), _i32(lengths), budget, sinks, recent, to,
                                     _i32(to_table))
    assert gr.status() == gr.OK
    assert n2.cpu().tolist() == [min(n, budget) for n in lengths]
    w64 = _f64(w)
    for i, n in enumerate(lengths):
        m = min(n, budget)
        for h in range(hkv):
            want = ref.keep(w64[i, h], n, budget, sinks, recent)
            assert kept[i, h, :m].cpu().tolist() == want and (kept[i, h, m:] == -1).all()
            assert np.array_equal(_f64(w2)[i, h, :m], w64[i, h, want], equal_nan=True)
            assert (w2[i, h, m:] == 0).all()
            at = np.array(want, dtype=int)
            for which in (0, 1):
                x = np.zeros((keep[i] * page, d))
                ids = table[i, at // page]
                x[:m] = before[which][ids, h, at % page] * before[which + 2][ids, h][:, None]
                for j in range(keep[i]):
                    part = x[j * page:(j + 1) * page]
                    s = ref.scale_for(ref.finite_amax(part))
                    t64[which][to_table[i, j], h] = ref.e4m3_round(part / s)
                    t64[which + 2][to_table[i, j], h] = s
    _same_cache(to, t64)
    if not same_pool:
        _same_cache(cache, before)


@pytest.mark.parametrize("page,d,hkv,lengths,budget,sinks,recent", [
    (16, 64, 1, [1], 1, 0, 0), (16, 64, 2, [40, 17, 16, 0], 17, 1, 3), (32, 128, 3, [100, 33, 5], 32, 0, 0),
    (64, 128, 2, [300, 64], 100, 4, 96), (128, 64, 1, [1000, 999], 500, 0, 500),
    (64, 64, 1, [5000], 1111, 7, 300), (16, 128, 2, [2500], 2499, 10, 20), (128, 128, 1, [700], 3, 1, 1)])
def test_evict(page, d, hkv, lengths, budget, sinks, recent):
    _evict(np.random.default_rng(page + d + budget), page, d, hkv, lengths, budget, sinks, recent)


@pytest.mark.parametrize("n,budget", [(5000, 700), (20000, 12345), (70000, 1000), (140000, 100000)])
def test_evict_long(n, budget):
    """Clusters of 1 to 8 blocks a head, and more tokens than their registers hold; ties at
    the border."""
    rng = np.random.default_rng(n)
    w = np.round(np.exp(rng.standard_normal((2, 1, n + 128))) * 50) / 50
    _evict(rng, 128, 64, 1, [n, n // 3], budget, 4, budget // 4, weights=w)


def test_evict_keeps_nan():
    """Any bytes, NaN codes among them: NaN stays NaN and counts for no scale."""
    _evict(np.random.default_rng(25), 64, 128, 2, [300, 70], 100, 4, 10, garbage=True)


def test_evict_scales_far_apart():
    """Tokens of pages whose scales differ by up to 2^40 in one new page."""
    import torch
    rng = np.random.default_rng(26)
    cache, c64 = _cache(rng, 4, 1, 16, 64, garbage=False)
    to, _ = _cache(rng, 1, 1, 16, 64)
    for which in (2, 3):
        c64[which][:, 0] = [2.0 ** -8, 2.0 ** -20, 2.0 ** -28, 2.0 ** -48]
        cache[which][:, 0] = torch.tensor(c64[which][:, 0], dtype=torch.float32, device="cuda")
    for kept in ([0, 17, 33, 50], [17, 33, 34, 49], [48, 49, 62, 63]):
        w = torch.zeros((1, 1, 64), device="cuda")
        w[0, 0, kept] = 1.0
        gr.kv_cache_evict(cache, w, _i32([[0, 1, 2, 3]]), _i32([64]), 4, 0, 0, to, _i32([[0]]))
        for which in (0, 1):
            x = np.zeros((16, 64))
            at = np.array(kept)
            x[:4] = c64[which][at // 16, 0, at % 16] * c64[which + 2][at // 16, 0][:, None]
            s = ref.scale_for(ref.finite_amax(x))
            assert _f64(to[which + 2])[0, 0] == s
            assert np.array_equal(_f64(to[which].float())[0, 0], ref.e4m3_round(x / s))


def test_evict_within_one_pool():
    _evict(np.random.default_rng(21), 32, 64, 2, [200, 90], 64, 2, 10, same_pool=True)


def test_evict_ties_and_odd_weights():
    """All equal, all zero, -0 and 0, NaN, infinities, negative weights, neighbours in the last bit."""
    rng = np.random.default_rng(22)
    w = np.zeros((6, 1, 320))
    w[1] = 3.5
    w[2] = rng.choice([0.0, -0.0, 1.0], 320)
    w[3] = rng.choice([np.nan, -np.inf, np.inf, -1.0, 2.0], 320)
    w[4] = 1 + rng.integers(0, 3, 320) * 2.0 ** -23
    w[5] = -np.abs(rng.standard_normal(320)).astype(np.float32)
    _evict(rng, 32, 64, 1, [300, 320, 310, 299, 320, 300], 150, 3, 20, weights=w)


def test_evict_refuses_what_only_the_device_sees():
    import torch
    rng = np.random.default_rng(23)
    cache, _ = _cache(rng, 8, 1, 16, 64, garbage=False)
    to, t64 = _cache(rng, 2, 1, 16, 64)
    w = torch.rand((3, 1, 32), device="cuda")
    n, _, kept = gr.kv_cache_evict(cache, w, _i32([[0, 1], [2, 3], [4, 80]]), _i32([33, 30, 10]), 8, 1, 1, to,
                                   _i32([[0], [2], [1]]))
    assert gr.status() == gr.ERR_PAGE
    assert n.cpu().tolist() == [0, 8, 8] and (kept[0] == -1).all()
    assert np.array_equal(_f64(to[0].float())[0], t64[0][0], equal_nan=True)   # nothing for it
    for bad in (dict(budget=0), dict(budget=40), dict(sinks=5, recent=5), dict(weights=w[:, :, :31]),
                dict(weights=w.double())):
        a = dict(budget=8, sinks=1, recent=1, weights=w)
        a.update(bad)
        with pytest.raises(ValueError):
            gr.kv_cache_evict(cache, a["weights"], _i32([[0, 1]] * 3), _i32([3] * 3), a["budget"], a["sinks"],
                              a["recent"], to, _i32([[0]] * 3))


def test_pages_past_four_gib():
    """Pages whose bytes start past 2^32 in the pool: written, read and moved like any other."""
    import torch
    rng = np.random.default_rng(27)
    num, hkv, page, d = 66000, 4, 128, 128            # 4.3 GB each of K and V
    cache = gr.KVCache.empty(num, hkv, d, page)
    far = num - 1 - np.arange(6)
    assert int(far.min()) * hkv * page * d > 2 ** 32
    n = 300
    k, k64 = _rand(rng, (1, n, hkv, d), "bf16")
    v, v64 = _rand(rng, (1, n, hkv, d), "bf16")
    q, q64 = _rand(rng, (1, 2, 2 * hkv, d), "bf16")
    pages, lengths = _i32([far[:3]]), _i32([n])
    gr.kv_cache_append(cache, k, v, pages, lengths)
    w = torch.zeros((1, hkv, 3 * page), device="cuda")
    out = gr.kv_cache_attention(q, cache, pages, lengths, weights=w)
    held = []
    for x, which in ((k64, 0), (v64, 1)):
        c, s = np.zeros((3, hkv, page, d)), np.ones((3, hkv))
        ref.append(c, s, x[0], [0, 1, 2], page, n, n)
        assert np.array_equal(_f64(cache[which][pages[0].long()].float())[:2], c[:2])
        assert np.array_equal(_f64(cache[which + 2][pages[0].long()]), s)
        held.append((c * s[..., None, None]).transpose(0, 2, 1, 3).reshape(-1, hkv, d)[:n])
    o, absv, _, size = ref.attend(q64[0], held[0], held[1], 0, 0)
    _check(_f64(out)[0], o, absv, size, d, "bf16", 2.0 ** -11)
    n2, _, kept = gr.kv_cache_evict(cache, w, pages, lengths, 200, 2, 20, cache, _i32([far[3:5]]))
    assert n2.item() == 200
    again = gr.kv_cache_attention(q, cache, _i32([far[3:5]]), n2)
    for h in range(hkv):
        at = kept[0, h].cpu().numpy()
        # the kept tokens' values are stored as they were, or rounded again under another scale
        got = _f64(cache[0][far[3], h].float()) * float(cache[2][far[3], h])
        assert np.allclose(got, held[0][at[:128], h], rtol=2.0 ** -4, atol=2.0 ** -9)
    assert torch.isfinite(again).all()


# ---------------------------------------------------------------- together


def test_together_in_a_graph():
    """A prompt, its cache, an eviction by the last queries' weights and ten decode steps captured
    in one graph each, replayed: the same as the eager calls."""
    import torch
    rng = np.random.default_rng(31)
    b, n, hq, hkv, d, page = 2, 150, 4, 2, 64, 16

    def serve(graph):
        r = np.random.default_rng(32)
        x, _ = _rand(r, (b, n, hq + 2 * hkv, d), "bf16")
        q, k, v = x.split([hq, hkv, hkv], dim=2)
        steps, _ = _rand(r, (10, b, 1, hq + 2 * hkv, d), "bf16")
        cache = gr.KVCache.empty(60, hkv, d, page)
        for t in cache:
            t.view(torch.uint8).zero_()
        pages = _i32(np.arange(2 * 10).reshape(2, 10))
        lengths = _i32([n, n - 30])
        w = torch.zeros((b, hkv, 10 * page), device="cuda")
        outs = [gr.flash_attention_window(q, k, v, 64, 4)]
        gr.kv_cache_append(cache, k, v, pages, lengths, _i32([n, n - 30]))
        outs.append(gr.kv_cache_attention(q[:, -8:], cache, pages, lengths, weights=w))
        to_pages = _i32(20 + np.arange(2 * 6).reshape(2, 6))
        lengths, w, _ = gr.kv_cache_evict(cache, w, pages, lengths, 64, 4, 16, cache, to_pages)
        step_in = torch.empty_like(steps[0])
        o = torch.empty((b, 1, hq, d), dtype=torch.bfloat16, device="cuda")

        def step():
            lengths.add_(1)
            sq, sk, sv = step_in.split([hq, hkv, hkv], dim=2)
            gr.kv_cache_append(cache, sk, sv, to_pages, lengths)
            gr.kv_cache_attention(sq, cache, to_pages, lengths, window=40, sinks=2, weights=w, out=o)

        if graph:
            saved = lengths.clone(), w.clone(), [t.clone() for t in cache]
            step_in.copy_(steps[0])
            step()                                  # warm up, then take its changes back
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            lengths.copy_(saved[0])
            w.copy_(saved[1])
            for t, s in zip(cache, saved[2]):
                t.copy_(s)
        for s in steps:
            step_in.copy_(s)
            g.replay() if graph else step()
            outs.append(o.clone())
        return outs + [w, lengths] + [t.float() for t in cache]

    for x, y in zip(serve(False), serve(True)):
        assert torch.equal(x, y)
        assert torch.isfinite(x).all()
