"""CPU-only: the serving operators' number format and references against independent
statements, the host logic of the library (argument checks, the work lists of the attention
kernels), and the refusals of the torch front end.  Nothing here launches a kernel."""
import ctypes

import numpy as np
import pytest

import tiled_tensor_core_03_gb300 as gr
from tiled_tensor_core_03_gb300 import _build

import serving_reference as ref


@pytest.fixture(scope="module")
def lib():
    if _build.needs_build():
        _build.build()
    return gr.lib()


# ---------------------------------------------------------------- the reference


def test_reference_e4m3_matches_torch():
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(ref.VALUES, want, equal_nan=True)
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.uniform(-448, 448, 4000), rng.standard_normal(4000) * 2.0 ** -8,
                        (ref.VALUES[:126] + ref.VALUES[1:127]) / 2])   # every tie
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(ref.e4m3_round(x), want)
    assert np.isnan(ref.e4m3_round(np.array([np.nan, np.inf, -np.inf]))).all()


@pytest.mark.parametrize("amax,want", [(448.0, 1.0), (448.5, 2.0), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                                       (1.76, 2.0 ** -7), (0.0, 2.0 ** -100), (1e-40, 2.0 ** -100)])
def test_reference_scale(amax, want):
    assert ref.scale_for(amax) == want


def test_reference_attention_closed_forms():
    rng = np.random.default_rng(2)
    v = rng.standard_normal((9, 2, 4))
    o = ref.attend(np.zeros((3, 4, 4)), rng.standard_normal((9, 2, 4)), v, 2, 1)[0]
    for i in range(3):          # equal scores: the mean of what is seen
        p = 6 + i
        assert np.allclose(o[i, 1], v[[0, p - 1, p], 0].mean(0))
        assert np.allclose(o[i, 2], v[[0, p - 1, p], 1].mean(0))
    assert (ref.attend(np.zeros((3, 2, 4)), v[:1], v[:1], 0, 0)[0][:2] == 0).all()


def test_reference_keep():
    w = np.array([0.0, 5, 1, 5, np.nan, 2, 1, 0, 0, 9])
    assert ref.keep(w, 10, 5, 1, 1) == [0, 1, 3, 5, 9]
    assert ref.keep(w, 10, 4, 1, 1) == [0, 1, 3, 9]
    assert ref.keep(w, 8, 4, 1, 1) == [0, 1, 3, 7]
    assert ref.keep(w, 10, 7, 1, 1) == [0, 1, 2, 3, 5, 6, 9]    # equal ones: the earlier
    assert ref.keep(w, 4, 5, 1, 1) == [0, 1, 2, 3]


# ---------------------------------------------------------------- work lists


def _blocks(lib, first, last, window, sinks):
    out = (ctypes.c_int * 3)()
    assert lib.flash_attention_window_debug_blocks(first, last, window, sinks, out) == gr.OK
    s, low, high = out
    return list(range(s)) + list(range(low, high))


def test_window_block_list(lib):
    """Exactly the blocks of 128 keys that some row of a tile sees, each once, in order."""
    rng = np.random.default_rng(3)
    for _ in range(300):
        first = int(rng.integers(-200, 1500))
        last = first + int(rng.integers(0, 128))
        window = int(rng.choice([0, 1, 2, 100, 127, 128, 129, 400, 3000]))
        sinks = int(rng.choice([0, 1, 4, 128, 129, 300, 5000]))
        want = set()
        for p in range(first, last + 1):
            if p >= 0:
                want |= set((np.flatnonzero(ref.seen(p, p + 1, window, sinks)) // 128).tolist())
        assert _blocks(lib, first, last, window, sinks) == sorted(want), (first, last, window, sinks)


def _units(lib, n, tokens, window, sinks):
    out = (ctypes.c_int * 3)()
    assert lib.kv_cache_debug_span(n, tokens, window, sinks, out) == gr.OK
    s, low, units = out
    return [u if u < s else low + u - s for u in range(units)]


def test_cache_units(lib):
    """The 64-token units of a sequence hold every token that some row sees, none past the
    length, each once, in order; at most two units more than the tokens need."""
    rng = np.random.default_rng(4)
    for _ in range(400):
        n, tokens = int(rng.integers(0, 1200)), int(rng.integers(1, 70))
        window = int(rng.choice([0, 1, 5, 63, 64, 65, 500, 5000]))
        sinks = int(rng.choice([0, 1, 4, 64, 65, 200, 5000]))
        got = _units(lib, n, tokens, window, sinks)
        assert got == sorted(set(got)) and all(64 * u < n for u in got)
        want = set()
        for p in range(max(0, n - tokens), n):
            want |= set((np.flatnonzero(ref.seen(p, n, window, sinks)) // 64).tolist())
        assert want <= set(got), (n, tokens, window, sinks)
        assert len(got) <= len(want) + 2


def test_cache_ranges(lib):
    """Blocks' ranges of units cover all of them once, differ by at most one, and the
    owner of every unit is the block whose range holds it."""
    for total in (1, 2, 7, 63, 64, 303, 304, 305, 5000):
        for grid in (1, 2, 64, 304):
            at = 0
            sizes = []
            for c in range(grid):
                lo = lib.kv_cache_debug_range(c, total, grid, 0)
                hi = lib.kv_cache_debug_range(c + 1, total, grid, 0)
                assert lo == at and hi >= lo
                for x in range(lo, hi):
                    assert lib.kv_cache_debug_range(x, total, grid, 1) == c
                sizes.append(hi - lo)
                at = hi
            assert at == total and max(sizes) - min(sizes) <= 1


# ---------------------------------------------------------------- refusals of the C ABI

P = 0x1000   # an aligned address that is never read: every call below ends before the device


def _pool(**kw):
    f = dict(k=P, v=P, k_scale=P, v_scale=P, num_pages=4, kv_heads=2, page=64, head_dim=128)
    f.update(kw)
    return gr.KVCachePool(**f)


def _strides(*s):
    return (ctypes.c_int64 * 3)(*s)


S = _strides(2048, 256, 128)
BAD_POOLS = [dict(k=None), dict(v=P + 8), dict(k_scale=None), dict(num_pages=0), dict(kv_heads=0),
             dict(page=48), dict(page=256), dict(head_dim=96), dict(num_pages=1 << 31)]
BAD_STRIDES = [None, _strides(2048, 256, -128), _strides(2048, 252, 128)]


def _append(lib, pool=None, k=P, v=P, dtype=0, batch=2, tokens=8, ks=S, vs=S, pages=P, max_pages=4,
            lengths=P, counts=None):
    return gr.kv_cache_append_x16(pool or _pool(), k, v, dtype, batch, tokens, ks, vs,
                                   pages, max_pages, lengths, counts, None)


def test_append_refusals(lib):
    for kw in BAD_POOLS:
        assert _append(lib, pool=_pool(**kw)) == gr.ERR_INVALID_ARG, kw
    for s in BAD_STRIDES:
        assert _append(lib, ks=s) == _append(lib, vs=s) == gr.ERR_INVALID_ARG
    for kw in (dict(k=None), dict(v=P + 2), dict(dtype=2), dict(batch=-1), dict(tokens=-1),
               dict(pages=None), dict(max_pages=0), dict(max_pages=1 << 30), dict(lengths=None),
               dict(lengths=P + 1), dict(counts=P + 2), dict(batch=70000)):
        assert _append(lib, **kw) == gr.ERR_INVALID_ARG, kw
    assert lib.kv_cache_append_x16(None, P, P, 0, 1, 1, S, S, P, 4, P, None, None) == gr.ERR_INVALID_ARG
    assert _append(lib, batch=0, k=None) == gr.OK
    assert _append(lib, tokens=0, pages=None) == gr.OK


def _attention(lib, pool=None, q=P, dtype=0, batch=2, tokens=1, q_heads=8, qs=S, out=P, pages=P,
               max_pages=4, lengths=P, window=0, sinks=0, weights=None, width=0, ws=P, ws_bytes=1 << 40):
    return gr.kv_cache_attention_x16(pool or _pool(), q, dtype, batch, tokens, q_heads,
                                      qs, out, pages, max_pages, lengths, window, sinks, weights, width,
                                      ws, ws_bytes, None)


def test_attention_refusals(lib):
    for kw in BAD_POOLS:
        assert _attention(lib, pool=_pool(**kw)) == gr.ERR_INVALID_ARG, kw
    for s in BAD_STRIDES:
        assert _attention(lib, qs=s) == gr.ERR_INVALID_ARG
    for kw in (dict(q=None), dict(out=None), dict(out=P + 8), dict(dtype=-1), dict(q_heads=7),
               dict(q_heads=0), dict(window=-1), dict(sinks=-1), dict(weights=P, width=255),
               dict(weights=P + 1, width=256), dict(pages=P + 1), dict(batch=65536),
               dict(tokens=65536), dict(tokens=60000, q_heads=65534)):
        assert _attention(lib, **kw) == gr.ERR_INVALID_ARG, kw
    assert _attention(lib, batch=0, q=None) == gr.OK
    assert _attention(lib, tokens=0, q=None) == gr.OK
    assert lib.kv_cache_attention_x16_workspace_bytes(1, 1, 7, 2, 128, 0) == 0
    assert lib.kv_cache_attention_x16_workspace_bytes(1, 1, 8, 2, 96, 0) == 0


def _evict(lib, pool=None, to=None, weights=P, width=256, pages=P, max_pages=4, lengths=P, batch=2,
           budget=100, sinks=4, recent=20, to_pages=P, to_max=2, to_lengths=P, to_weights=P, kept=P):
    return gr.kv_cache_evict_e4m3(pool or _pool(), weights, width, pages, max_pages,
                                   lengths, batch, budget, sinks, recent, to or _pool(),
                                   to_pages, to_max, to_lengths, to_weights, kept, None)


def test_evict_refusals(lib):
    for kw in BAD_POOLS:
        assert _evict(lib, pool=_pool(**kw)) == gr.ERR_INVALID_ARG, kw
        assert _evict(lib, to=_pool(**kw)) == gr.ERR_INVALID_ARG, kw
    for kw in (dict(to=_pool(page=32)), dict(to=_pool(kv_heads=4)), dict(to=_pool(head_dim=64)),
               dict(budget=0), dict(budget=129), dict(sinks=-1), dict(recent=-1), dict(sinks=81),
               dict(width=255), dict(weights=None), dict(kept=None), dict(to_lengths=None),
               dict(to_weights=P + 2), dict(to_pages=None), dict(pages=None), dict(lengths=None)):
        assert _evict(lib, **kw) == gr.ERR_INVALID_ARG, kw
    assert _evict(lib, batch=0, weights=None) == gr.OK


def _window(lib, q=P, k=P, v=P, o=P, dtype=0, batch=1, n_q=8, n_kv=8, hq=4, hkv=2, d=64, qs=S, ks=S,
            vs=S, window=4, sinks=1):
    return gr.flash_attention_window_x16(q, k, v, o, dtype, batch, n_q, n_kv, hq, hkv, d, qs, ks, vs,
                                          window, sinks, None)


def test_window_refusals(lib):
    for s in BAD_STRIDES + [_strides(2048, 0, 128)]:
        assert _window(lib, qs=s) == _window(lib, ks=s) == _window(lib, vs=s) == gr.ERR_INVALID_ARG
    for kw in (dict(q=None), dict(k=P + 8), dict(v=None), dict(o=None), dict(o=P + 8), dict(dtype=3),
               dict(batch=-1), dict(batch=65536), dict(n_q=-1), dict(n_kv=-1), dict(hq=5), dict(hkv=0),
               dict(d=32), dict(window=-1), dict(sinks=-2)):
        assert _window(lib, **kw) == gr.ERR_INVALID_ARG, kw
    for kw in (dict(batch=0), dict(n_q=0), dict(hq=0)):
        assert _window(lib, q=None, o=None, **kw) == gr.OK


# ---------------------------------------------------------------- refusals of the torch front end


def test_front_end_wants_cuda_tensors(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros((1, 8, 2, 64), dtype=torch.float16)
    i = torch.zeros((1, 4), dtype=torch.int32)
    cache = gr.KVCache.empty(4, 2, 64, page=16, device="cpu")
    with pytest.raises(ValueError):
        gr.flash_attention_window(x, x, x, 4)
    with pytest.raises(ValueError):
        gr.kv_cache_append(cache, x, x, i, i[:, 0])
    with pytest.raises(ValueError):
        gr.kv_cache_attention(x, cache, i, i[:, 0])
    with pytest.raises(ValueError):
        gr.kv_cache_evict(cache, torch.zeros((1, 2, 64)), i, i[:, 0], 8, 0, 0, cache, i)
    for bad in (dict(head_dim=96), dict(head_dim=64, page=24)):
        with pytest.raises(ValueError):
            gr.KVCache.empty(4, 2, device="cpu", **bad)
