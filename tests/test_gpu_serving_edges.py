"""The serving operators where it is easy to go wrong: values that are not finite or very large
beside keys that a row does not see, scales far apart, freed pages, status and streams.  References
and tolerances as in test_gpu_serving.py."""
import numpy as np
import pytest

import tiled_tensor_core_03_gb300 as gr

import serving_reference as ref
from test_gpu_serving import DTYPES, _cache, _check, _cuda, _dt, _f64, _half_step, _i32, _rand, _tables  # noqa: F401

pytestmark = pytest.mark.gpu

# ---------------------------------------------------------------- flash_attention_window


def _sees(n, at, window, sinks):
    return np.array([at <= p and (window == 0 or at > p - window or at < sinks) for p in range(n)])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sinks", [2, 64, 130])
def test_window_not_finite_beside_rows_that_left_sinks_behind(sinks, d, dtype):
    """Rows whose window has left some of the sinks behind (positions from window to window + sinks)
    beside a V that is not finite, in a key they do not see and in a sink: every element that it
    does not reach is as the formula says, also in the rows that see it."""
    rng = np.random.default_rng(sinks + d)
    n, window = 300, 40
    q, q64 = _rand(rng, (1, n, 2, d), dtype)
    k, k64 = _rand(rng, (1, n, 1, d), dtype)
    v, v64 = _rand(rng, (1, n, 1, d), dtype)
    for at, value in ((window + min(sinks, 80) + 1, np.nan), (120, np.inf), (1, np.inf), (299, -np.inf)):
        vv, vv64 = v.clone(), v64.copy()
        vv[0, at, 0, 5] = value
        vv64[0, at, 0, 5] = value
        got = _f64(gr.flash_attention_window(q, k, vv, window, sinks))[0]
        o, absv, _, size = ref.attend(q64[0], k64[0], vv64[0], window, sinks)
        sees = _sees(n, at, window, sinks)
        assert not np.isfinite(got[sees][..., 5]).any()
        _check(got[~sees], o[~sees], absv[~sees], size[~sees], d, dtype, _half_step(dtype))
        got, o, absv = (np.delete(x, 5, 2) for x in (got, o, absv))
        _check(got, o, absv, size, d, dtype, _half_step(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
def test_window_first_score_minus_infinity(dtype):
    """A key whose score is -infinity has weight 0, also where it is the first that a row sees and
    a V that the row does not see is not finite."""
    rng = np.random.default_rng(41)
    n, d = 200, 64
    q, q64 = _rand(rng, (1, n, 1, d), dtype)
    k, k64 = _rand(rng, (1, n, 1, d), dtype)
    v, v64 = _rand(rng, (1, n, 1, d), dtype)
    q, q64 = q.abs(), np.abs(q64)
    k[0, :2, 0, 5], k64[0, :2, 0, 5] = -np.inf, -np.inf
    v[0, 199, 0, 7], v64[0, 199, 0, 7] = np.nan, np.nan
    for window, sinks in ((0, 0), (50, 2)):
        got = _f64(gr.flash_attention_window(q, k, v, window, sinks))[0, 2:199]
        with np.errstate(invalid="ignore"):
            o, absv, _, _ = ref.attend(q64[0], k64[0], v64[0], window, sinks)
        size = ref.attend(q64[0], np.where(np.isinf(k64[0]), 0, k64[0]), v64[0], window, sinks)[3]
        _check(got, o[2:199], absv[2:199], size[2:199], d, dtype, _half_step(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,window,sinks,everywhere", [(3000, 0, 0, False), (3000, 700, 4, False), (700, 300, 70, True)])
def test_window_not_finite_holds_nobody_up(n, window, sinks, everywhere, dtype):
    """An infinity in V of the first token, which every row sees, or one in every fifth token: no wait
    inside the kernel gets long (their limit is 20 ms here), and every row is written."""
    import torch
    rng = np.random.default_rng(42)
    d, hq = 128, 4
    q, _ = _rand(rng, (1, n, hq, d), dtype)
    k, _ = _rand(rng, (1, n, 1, d), dtype)
    v, _ = _rand(rng, (1, n, 1, d), dtype)
    at = torch.arange(0, n, 5, device="cuda") if everywhere else torch.zeros(1, dtype=torch.long, device="cuda")
    clean = v.clone()
    clean[0, at, 0, 9] = 0
    dirty = clean.clone()
    dirty[0, at, 0, 9] = float("inf")
    gr.gemm_relu_debug_set(0, 20_000_000)
    try:
        want = gr.flash_attention_window(q, k, clean, window, sinks)
        got = gr.flash_attention_window(q, k, dirty, window, sinks)
        assert gr.status() == gr.OK
    finally:
        gr.gemm_relu_debug_set(0, 0)
    keep = [c for c in range(d) if c != 9]
    assert torch.equal(got[..., keep], want[..., keep])
    sees = torch.from_numpy(np.any([_sees(n, int(a), window, sinks) for a in at.cpu()], axis=0)).cuda()
    assert not torch.isfinite(got[0, sees][..., 9]).any()
    assert torch.equal(got[0, ~sees], want[0, ~sees])


def test_window_not_finite_in_many_heads_and_sequences():
    """Garbage of every kind past the prompts of a padded batch, more items than CTAs: what comes before
    the padding is as if the padding were 0."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(43)
    b, n, hq, hkv, d = 4, 1500, 12, 6, 64
    q, k, v = (torch.randn(b, n, h, d, device="cuda", dtype=torch.bfloat16, generator=g) for h in (hq, hkv, hkv))
    lengths = [1500, 1401, 77, 900]
    k0, v0 = k.clone(), v.clone()
    for i, m in enumerate(lengths):
        k0[i, m:], v0[i, m:] = 0, 0
        bytes_ = torch.randint(-2 ** 15, 2 ** 15, k[i, m:].shape, device="cuda", generator=g).short()
        k[i, m:], v[i, m:] = bytes_.view(torch.bfloat16), bytes_.flip(0).view(torch.bfloat16)
        v[i, m:, :, ::3] = float("nan")
    for window, sinks in ((0, 0), (200, 3)):
        got = gr.flash_attention_window(q, k, v, window, sinks)
        want = gr.flash_attention_window(q, k0, v0, window, sinks)
        for i, m in enumerate(lengths):
            assert torch.equal(got[i, :m], want[i, :m])


@pytest.mark.parametrize("n,window,sinks,scale", [(600, 0, 0, 0.1), (600, 0, 0, 2.0), (900, 300, 130, 0.1)])
@pytest.mark.parametrize("size_of_v", [1e37, 1e30, 1e-30])
def test_window_very_large_and_small_values(n, window, sinks, scale, size_of_v):
    """Sums of finite bf16 V would leave fp32 before they are divided: the mean does not."""
    import torch
    rng = np.random.default_rng(44)
    d = 64
    q, q64 = _rand(rng, (1, n, 2, d), "bf16", scale)
    k, k64 = _rand(rng, (1, n, 1, d), "bf16")
    v = torch.from_numpy(rng.uniform(0.5, 4.0, (1, n, 1, d)) * size_of_v).to(torch.bfloat16)
    got = _f64(gr.flash_attention_window(q, k, v.cuda(), window, sinks))[0] / size_of_v
    o, absv, _, size = ref.attend(q64[0], k64[0], v.double().numpy()[0] / size_of_v, window, sinks)
    _check(got, o, absv, size, d, "bf16", _half_step("bf16"))


@pytest.mark.parametrize("dtype,scale", [("fp16", 3e3), ("fp16", 3e4), ("bf16", 3e3), ("bf16", 1e6), ("bf16", 1e9)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 5)])
def test_window_huge_scores(window, sinks, dtype, scale):
    """Finite scores of any size: where one key's score is far above all others its V is the result."""
    rng = np.random.default_rng(45)
    n, d = 400, 64
    q, q64 = _rand(rng, (1, n, 2, d), dtype, scale / 4)      # (fp16: within 65504)
    k, k64 = _rand(rng, (1, n, 1, d), dtype, scale / 4)
    v, v64 = _rand(rng, (1, n, 1, d), dtype)
    got = _f64(gr.flash_attention_window(q, k, v, window, sinks))[0]
    assert np.isfinite(got).all()
    clear = 0
    for i in range(n):
        see = np.flatnonzero(ref.seen(i, n, window, sinks))
        for h in range(2):
            x = k64[0, see, 0] @ q64[0, i, h] / 8
            order = np.argsort(x)
            # 2^-15 of the largest terms: far above what 32-bit scores may be off by
            gap = x[order[-1]] - x[order[-2]] if len(see) > 1 else np.inf
            if gap > 100 + 2.0 ** -15 * (np.abs(k64[0, see, 0]) @ np.abs(q64[0, i, h])).max() / 8:
                clear += 1
                # the weight and the result are each rounded once
                want, half = v64[0, see[order[-1]], 0], _half_step(dtype)
                assert (np.abs(got[i, h] - want) <= ((1 + half) ** 2 - 1) * np.abs(want)).all(), (i, h)
    assert clear > n


def test_window_waits_that_run_out_beside_values_that_are_not_finite():
    """A CTA that never gets its data gives up while others go over their items again: the call ends with
    a timeout, the next one is right."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(46)
    q, k, v = (torch.randn(2, 900, h, 64, device="cuda", dtype=torch.bfloat16, generator=g) for h in (8, 4, 4))
    want = gr.flash_attention_window(q, k, v, 100, 4)
    dirty = v.clone()
    dirty[:, 7::50] = float("nan")
    for limit in (20_000_000, 1_000_000):
        gr.gemm_relu_debug_set(1, limit)
        try:
            gr.flash_attention_window(q, k, dirty, 100, 4)
            assert gr.status() == gr.ERR_TIMEOUT
        finally:
            gr.gemm_relu_debug_set(0, 0)
        assert torch.equal(gr.flash_attention_window(q, k, v, 100, 4), want)
        assert gr.status() == gr.OK

# ---------------------------------------------------------------- attention over the cache


def _cache_check(out, q64, c64, ids, n, d, dtype, window=0, sinks=0):
    """As _check, without its absolute term: values of every size count."""
    hkv = c64[0].shape[1]
    k, v = ((x[ids] * s[ids][..., None, None]).transpose(0, 2, 1, 3).reshape(-1, hkv, d)[:n]
            for x, s in ((c64[0], c64[2]), (c64[1], c64[3])))
    o, absv, _, size = ref.attend(q64, k, v, window, sinks)
    top = 2.0 ** np.floor(np.log2(np.maximum(absv.max(), 2.0 ** -120)))     # so that 2^-25 counts for nothing
    rows = absv.max(-1, keepdims=True)
    rows = 2.0 ** np.floor(np.log2(np.where(rows > 0, rows, top)))
    _check(out / rows, o / rows, absv / rows, size, d, dtype, 2.0 ** -11)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 5, 12])
@pytest.mark.parametrize("exponent", [-20, -33, -40, -90])
def test_cache_attention_small_scale_with_all_the_weight(exponent, group, d):
    """A page with a tiny V scale holds nearly all the weight beside one whose V scale is larger by
    2^20 to 2^90, read before or after it or both: the result has the bits of the small page."""
    import torch
    rng = np.random.default_rng(51)
    cache, c64 = _cache(rng, 3, 1, 64, d, garbage=False)
    for h, s in ((0, 1.0), (1, 2.0 ** exponent), (2, 1.0)):
        for which, x in ((2, 2.0 ** -3), (3, s)):
            cache[which][h, 0] = x
            c64[which][h, 0] = x
        # every score of pages 0 and 2 lies some 100 nats below page 1's
        values = torch.from_numpy(np.abs(c64[0][h]) % 8 + 8).to(torch.float8_e4m3fn) if h == 1 else \
            torch.from_numpy(-(np.abs(c64[0][h]) % 8) - 8).to(torch.float8_e4m3fn)
        cache[0][h] = values.cuda()
        c64[0][h] = values.double().numpy()
    q = _rand(rng, (1, 1, group, d), "bf16")[0].abs() + 3
    q64 = _f64(q)
    # 64 units of 64 tokens go to 16 blocks: each warp reads pages of both scales
    for order in ([0, 1] * 32, [1, 2] * 32, [0, 2, 0, 1] * 16, [0] * 63 + [1], [1] + [2] * 63):
        out = gr.kv_cache_attention(q, cache, _i32([order]), _i32([64 * len(order)]))
        _cache_check(_f64(out)[0], q64[0], c64, order, 64 * len(order), d, "bf16")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page,d,hkv,group,tokens,lengths", [
    (64, 128, 2, 4, 1, [3000, 200]), (16, 64, 1, 8, 3, [1500, 40]), (128, 64, 2, 1, 1, [5000]),
    (32, 128, 1, 16, 2, [900, 4000])])
def test_cache_attention_scales_of_every_size(page, d, hkv, group, tokens, lengths, dtype):
    """V scales between 2^-70 and 2^7 (2^-4 for fp16 outputs) in every order, scores of tens of nats, so that
    any page may carry the result; sequences cut into several parts."""
    import torch
    rng = np.random.default_rng(page + d + group)
    need = [-(-n // page) for n in lengths]
    cache, c64 = _cache(rng, sum(need), hkv, page, d, garbage=False)
    s = 2.0 ** rng.integers(-70 if dtype == "bf16" else -4, 8, (sum(need), hkv))
    cache[3].copy_(torch.from_numpy(s.astype(np.float32)))
    c64[3][...] = s
    table = _tables(rng, need, sum(need))
    for scale in (0.05, 10.0, 200.0):
        q, q64 = _rand(rng, (len(lengths), tokens, hkv * group, d), dtype, scale)
        out = _f64(gr.kv_cache_attention(q, cache, _i32(table), _i32(lengths)))
        for i, n in enumerate(lengths):
            _cache_check(out[i], q64[i], c64, table[i, :need[i]], n, d, dtype)


def test_cache_attention_zero_pages():
    """Pages of zeros carry the least scale there is; they count in the softmax and add nothing."""
    rng = np.random.default_rng(53)
    cache, c64 = _cache(rng, 6, 1, 16, 64, garbage=False)
    for i in (0, 2, 3):
        cache[1][i] = 0
        cache[3][i] = 2.0 ** -100
        c64[1][i], c64[3][i] = 0, 2.0 ** -100
    q, q64 = _rand(rng, (1, 1, 4, 64), "bf16")
    for order in ([0, 1, 2, 3, 4, 5] * 40, [1, 0, 4, 2] * 60, [0, 2, 3] * 50, [5, 0] * 100):
        out = gr.kv_cache_attention(q, cache, _i32([order]), _i32([16 * len(order) - 3]))
        _cache_check(_f64(out)[0], q64[0], c64, order, 16 * len(order) - 3, 64, "bf16")


@pytest.mark.parametrize("scale", [2.0 ** 10, 2.0 ** 30])
def test_cache_attention_huge_scores_and_small_scales(scale):
    """Scores up to 2^40 (one token takes all the weight) and V scales around 2^-60."""
    import torch
    rng = np.random.default_rng(54)
    cache, c64 = _cache(rng, 40, 1, 64, 64, garbage=False)
    for which, e in ((2, 2), (3, -60)):
        s = 2.0 ** (e + rng.integers(-2, 3, (40, 1)))
        c64[which][...] = s
        cache[which].copy_(torch.from_numpy(s.astype(np.float32)))
    q, q64 = _rand(rng, (1, 1, 3, 64), "bf16", scale)
    order = list(range(40))
    out = gr.kv_cache_attention(q, cache, _i32([order]), _i32([2550]))
    k = (c64[0] * c64[2][..., None, None]).transpose(0, 2, 1, 3).reshape(-1, 64)[:2550]
    v = (c64[1] * c64[3][..., None, None]).transpose(0, 2, 1, 3).reshape(-1, 64)[:2550]
    for h in range(3):
        x = np.sort(k @ q64[0, 0, h])
        assert (x[-1] - x[-2]) / 8 > 100
        want = v[np.argmax(k @ q64[0, 0, h])]
        assert np.array_equal(_f64(out)[0, 0, h], want)


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("page,tokens,n,window,sinks", [
    (16, 1, 300, 100, 0), (16, 3, 300, 100, 20), (32, 1, 1000, 400, 4), (16, 1, 70, 1, 1), (32, 2, 500, 33, 65)])
def test_cache_attention_freed_pages(page, tokens, n, window, sinks, weights):
    """Pages of which no query sees a token are never asked for: a sequence may have given them up."""
    import torch
    rng = np.random.default_rng(page + n + window)
    need, d, hkv = -(-n // page), 64, 2
    cache, c64 = _cache(rng, need, hkv, page, d, garbage=False)
    table = _tables(rng, [need], need)
    low = n - tokens - window + 1            # the first token that the first query's window holds
    freed = [i for i in range(need) if (i + 1) * page <= low and i * page >= sinks]
    assert freed
    given = table.copy()
    given[0, freed] = rng.choice([-1, need, 2 ** 31 - 1], len(freed))
    q, q64 = _rand(rng, (1, tokens, 2 * hkv, d), "fp16")
    w = torch.zeros((1, hkv, need * page), device="cuda") if weights else None
    out = _f64(gr.kv_cache_attention(q, cache, _i32(given), _i32([n]), window, sinks, weights=w))
    assert gr.status() == gr.OK
    k, v = ((x[table[0]] * s[table[0]][..., None, None]).transpose(0, 2, 1, 3).reshape(-1, hkv, d)[:n]
            for x, s in ((c64[0], c64[2]), (c64[1], c64[3])))
    o, absv, mass, size = ref.attend(q64[0], k, v, window, sinks)
    _check(out[0], o, absv, size, d, "fp16", 2.0 ** -11)
    if weights:
        rel = ref.weight_error(size.max(), d) + 2.0 ** -20
        assert (np.abs(_f64(w)[0, :, :n] - mass) <= rel * mass).all()

# ---------------------------------------------------------------- status and streams


@pytest.mark.parametrize("page_first", [True, False])
def test_status_a_timeout_outranks_a_bad_page(page_first):
    """A bad page leaves the other outputs right, a timeout leaves a call's outputs unspecified: with
    both since the last look, the status is the timeout, whichever came first."""
    rng = np.random.default_rng(61)
    cache, _ = _cache(rng, 2, 1, 16, 64)
    x, _ = _rand(rng, (1, 4, 1, 64), "fp16")
    q, _ = _rand(rng, (1, 300, 2, 64), "fp16")

    def bad_page():
        gr.kv_cache_append(cache, x, x, _i32([[7]]), _i32([4]))

    def timeout():
        gr.gemm_relu_debug_set(1, 20_000_000)
        try:
            gr.flash_attention_window(q, q, q, 100, 4)
        finally:
            gr.gemm_relu_debug_set(0, 0)
    for step in (bad_page, timeout) if page_first else (timeout, bad_page):
        step()
    assert gr.status() == gr.ERR_TIMEOUT
    assert gr.status() == gr.OK
    bad_page()
    assert gr.status() == gr.ERR_PAGE


def _stream_id(handle):
    import ctypes
    out = ctypes.c_uint64()
    assert gr.lib().gemm_relu_stream_id(ctypes.c_void_p(handle), ctypes.byref(out)) == gr.OK
    return out.value


PER_THREAD = 2      # cudaStreamPerThread


def test_stream_ids_tell_streams_with_one_handle_apart():
    import ctypes
    import threading
    import torch
    handles = [0] + [torch.cuda.Stream().cuda_stream for _ in range(3)]
    ids = [_stream_id(h) for h in handles]
    assert len(set(ids)) == len(set(handles)) and ids == [_stream_id(h) for h in handles]
    assert gr.lib().gemm_relu_stream_id(None, None) == gr.ERR_INVALID_ARG
    seen = []
    for _ in range(20):        # created and destroyed: the handle may come back, the id does not
        s = ctypes.c_void_p()
        torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(s))
        seen.append(_stream_id(s.value))
        torch.cuda.cudart().cudaStreamDestroy(s.value)
    assert len(set(seen)) == 20 and not set(seen) & set(ids)
    mine = []

    def look():
        torch.cuda.set_device(0)
        mine.append(_stream_id(PER_THREAD))
    for _ in range(2):
        t = threading.Thread(target=look)
        t.start()
        t.join()
    look()
    assert len(set(mine)) == 3


def test_cache_attention_on_streams_of_one_handle():
    """Two threads, each on its own cudaStreamPerThread, whose calls overlap on the GPU: each has a
    workspace of its own.  Then more streams than workspaces are kept."""
    import ctypes
    import threading
    import torch
    rng = np.random.default_rng(62)
    cache, _ = _cache(rng, 400, 2, 64, 128, garbage=False)
    work, want = [], []
    for n in (9000, 25000):
        q, _ = _rand(rng, (1, 1, 8, 128), "bf16")
        pages = _i32(np.arange(-(-n // 64))[None])
        args = (q, cache, pages, _i32([n]))
        want.append(gr.kv_cache_attention(*args))
        work.append((args, [torch.empty_like(q) for _ in range(200)]))
    torch.cuda.synchronize()
    start = threading.Barrier(2)
    failed = []

    def go(args, outs):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.ExternalStream(PER_THREAD)
            start.wait(60)
            for out in outs:
                gr.kv_cache_attention(*args, out=out, stream=stream)
            stream.synchronize()
        except Exception as e:      # shown by the test, not by the thread
            failed.append(e)
    threads = [threading.Thread(target=go, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for (_, outs), x in zip(work, want):
        assert all(torch.equal(o, x) for o in outs)
    args, _ = work[0]
    handles = [ctypes.c_void_p() for _ in range(70)]
    for h in handles:
        assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(h))) == 0
        s = torch.cuda.ExternalStream(h.value)
        o = gr.kv_cache_attention(*args, stream=s)
        s.synchronize()
        assert torch.equal(o, want[0])
    for h in handles:
        torch.cuda.cudart().cudaStreamDestroy(h.value)


def test_no_memory_is_torchs_error():
    """Scores of 2^20 tokens and 2^17 rows for the weights would take 512 GiB."""
    import torch
    cache = gr.KVCache.empty(1, 1, 64, 128)
    q = torch.zeros((1, 2048, 64, 64), dtype=torch.float16, device="cuda")
    pages = torch.zeros((1, 8192), dtype=torch.int32, device="cuda")
    weights = torch.zeros((1, 1, 2 ** 20), device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        gr.kv_cache_attention(q, cache, pages, _i32([1]), weights=weights)
    assert not weights.any()
