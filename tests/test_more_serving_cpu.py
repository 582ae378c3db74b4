"""CPU-only: argument checks of rotary_x16, flash_attention_cross_x16 and kv_cache_attention_ragged_x16, and the
refusals of their torch front end.  Nothing here launches a kernel."""
import ctypes
import math

import pytest

import tiled_tensor_core_03_gb300 as gr

from test_serving_cpu import BAD_POOLS, BAD_STRIDES, P, S, _pool, _strides, lib  # noqa: F401


# ---------------------------------------------------------------- the C ABI


def _cross(lib, q=P, k=P, v=P, o=P, dtype=0, batch=1, n_q=8, n_kv=8, hq=4, hkv=2, d=64, qs=S, ks=S, vs=S, lengths=P):
    return gr.flash_attention_cross_x16(q, k, v, o, dtype, batch, n_q, n_kv, hq, hkv, d, qs, ks, vs, lengths, None, 0,
                                        None)


def test_cross_refusals(lib):
    for s in BAD_STRIDES + [_strides(2048, 0, 128)]:
        assert _cross(lib, qs=s) == _cross(lib, ks=s) == _cross(lib, vs=s) == gr.ERR_INVALID_ARG
    for kw in (dict(q=None), dict(k=P + 8), dict(v=None), dict(o=None), dict(o=P + 8), dict(dtype=3),
               dict(batch=-1), dict(batch=65536), dict(n_q=-1), dict(n_kv=-1), dict(hq=5), dict(hkv=0),
               dict(d=32), dict(lengths=P + 2), dict(hq=258), dict(hq=129, hkv=1), dict(n_kv=1 << 31)):
        assert _cross(lib, **kw) == gr.ERR_INVALID_ARG, kw
    for kw in (dict(batch=0), dict(n_q=0), dict(hq=0)):
        assert _cross(lib, q=None, o=None, **kw) == gr.OK
    for sizes in ((0, 1, 8, 4, 2, 64), (1, 1, 8, 5, 2, 64), (1, 1, 8, 4, 2, 96), (1, 1, 8, 4, 0, 64)):
        assert gr.flash_attention_cross_x16_workspace_bytes(*sizes) == 0


def _ragged(lib, pool=None, q=P, dtype=0, rows=9, q_heads=8, qs=(2048, 128), out=P, batch=3, starts=P, pages=P,
            max_pages=4, lengths=P, window=0, sinks=0, ws=P, ws_bytes=1 << 40):
    strides = None if qs is None else (ctypes.c_int64 * 2)(*qs)
    return gr.kv_cache_attention_ragged_x16(pool or _pool(), q, dtype, rows, q_heads, strides, out, batch, starts,
                                            pages, max_pages, lengths, window, sinks, ws, ws_bytes, None)


def test_ragged_refusals(lib):
    for kw in BAD_POOLS:
        assert _ragged(lib, pool=_pool(**kw)) == gr.ERR_INVALID_ARG, kw
    for kw in (dict(q=None), dict(q=P + 8), dict(out=None), dict(out=P + 8), dict(dtype=-1), dict(q_heads=7),
               dict(q_heads=0), dict(window=-1), dict(sinks=-1), dict(pages=None), dict(pages=P + 1), dict(starts=None),
               dict(starts=P + 2), dict(lengths=None), dict(lengths=P + 1), dict(qs=None), dict(qs=(2044, 128)),
               dict(qs=(2048, -128)), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(batch=-1), dict(batch=16385),
               dict(max_pages=0), dict(max_pages=1 << 30), dict(rows=1 << 24, q_heads=128),
               dict(rows=1 << 24, q_heads=64, max_pages=1 << 20, pool=_pool(page=128))):
        assert _ragged(lib, **kw) == gr.ERR_INVALID_ARG, kw
    assert lib.kv_cache_attention_ragged_x16(None, P, 0, 1, 8, (ctypes.c_int64 * 2)(1024, 128), P, 1, P, P, 4, P, 0, 0,
                                             P, 1 << 40, None) == gr.ERR_INVALID_ARG
    assert _ragged(lib, batch=0, q=None) == gr.OK
    assert _ragged(lib, rows=0, q=None, starts=None) == gr.OK
    assert gr.kv_cache_attention_ragged_x16_workspace_bytes(96) == 0


def _tensor(x=P, y=P, heads=2, xs=(2048, 256, 128), ys=(2048, 256, 128)):
    return gr.RotaryTensor(x, y, heads, (ctypes.c_int64 * 3)(*xs), (ctypes.c_int64 * 3)(*ys))


def _rotary(lib, q=None, k=None, dtype=0, batch=2, tokens=8, head_dim=128, rot=128, positions=P, pos_type=0, freq=P,
            freq_type=1, amplitude=1.0):
    return gr.rotary_x16(q or _tensor(), k or _tensor(heads=1), dtype, batch, tokens, head_dim, rot, False, positions,
                         pos_type, freq, freq_type, amplitude)


def test_rotary_refusals(lib):
    for bad in (dict(x=None), dict(x=P + 8), dict(y=None), dict(y=P + 2), dict(heads=-1), dict(heads=65536),
                dict(xs=(2048, 252, 128)), dict(xs=(2048, 256, -128)), dict(ys=(2044, 256, 128))):
        assert _rotary(lib, q=_tensor(**bad)) == _rotary(lib, k=_tensor(**bad)) == gr.ERR_INVALID_ARG, bad
    for kw in (dict(dtype=2), dict(batch=-1), dict(tokens=-1), dict(batch=1 << 16, tokens=1 << 15), dict(head_dim=4),
               dict(head_dim=130), dict(head_dim=520), dict(rot=0), dict(rot=3), dict(rot=130), dict(positions=None),
               dict(positions=P + 2), dict(positions=P + 4, pos_type=1), dict(pos_type=2), dict(freq=None),
               dict(freq=P + 4), dict(freq_type=2), dict(amplitude=math.nan), dict(amplitude=math.inf),
               dict(q=_tensor(heads=40000), k=_tensor(heads=40000))):
        assert _rotary(lib, **kw) == gr.ERR_INVALID_ARG, kw
    assert _rotary(lib, batch=0, positions=None) == gr.OK
    assert _rotary(lib, q=_tensor(heads=0, x=None), k=_tensor(heads=0, y=None), freq=None) == gr.OK
    assert lib.rotary_x16(None, None, 0, 1, 1, 128, 128, 0, P, 0, P, 1, 1.0, 0, None) == gr.ERR_INVALID_ARG


# ---------------------------------------------------------------- the torch front end


def test_front_end_wants_cuda_tensors(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros((1, 8, 2, 64), dtype=torch.float16)
    i = torch.zeros((1, 4), dtype=torch.int32)
    cache = gr.KVCache.empty(4, 2, 64, page=16, device="cpu")
    with pytest.raises(ValueError):
        gr.flash_attention_cross(x, x, x)
    with pytest.raises(ValueError):
        gr.kv_cache_attention_ragged(x[0], cache, i, i[:, 0], i[0, :2])
    with pytest.raises(ValueError):
        gr.kv_cache_attention_ragged_workspace(cache)
    with pytest.raises(ValueError):
        gr.rotary(x, x, torch.zeros((1, 8), dtype=torch.int32), gr.rotary_frequencies(64, device="cpu"))
    with pytest.raises(TypeError):
        gr.rotary(None, None, None, None)


def test_frequencies(lib):
    pytest.importorskip("torch")
    f = gr.rotary_frequencies(8, base=16.0, device="cpu")
    assert f.tolist() == [1.0, 0.5, 0.25, 0.125]
    assert gr.rotary_frequencies(8, base=16.0, factor=4, device="cpu").tolist() == [0.25, 0.125, 0.0625, 0.03125]
    # 8 pi tokens: 4, 2, 1 and 1/2 turns; between 1 and 4 turns the share that is kept is (turns - 1) / 3
    g = gr.rotary_frequencies(8, base=16.0, factor=4, context=8 * math.pi, low=1, high=4, device="cpu").tolist()
    assert g == pytest.approx([1.0, 0.5 * (1 / 3 + 2 / 3 / 4), 0.0625, 0.03125])
    for kw in (dict(rot=3), dict(rot=0), dict(rot=8, factor=0.5), dict(rot=8, base=0), dict(rot=8, low=4, high=4)):
        with pytest.raises(ValueError):
            gr.rotary_frequencies(device="cpu", **kw)
