"""Rotary positions, append, ragged attention and cross attention together, as a serving step calls them: every result
against the definition in 64 bits, from what the call was given.  Tolerances as in test_gpu_serving.py."""
import importlib.util
import os

import numpy as np
import pytest

import tiled_tensor_core_03_gb300 as gr

from test_gpu_rotary import _check as _check_rotary
from test_gpu_serving import DTYPES, _check, _cuda, _dt, _f64, _half_step, _i32  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page,d,window,sinks", [(32, 64, 0, 0), (16, 128, 50, 4)])
def test_steps_of_chunks_and_single_tokens(page, d, window, sinks, dtype):
    import torch
    from gpu_attend import attend, seen
    hq, hkv, n, states = 6, 2, 4, [90, 0, 200, 129]
    g = torch.Generator(device="cuda").manual_seed(page + d)
    most = -(-400 // page)
    cache = gr.KVCache.empty(n * most, hkv, d, page)
    for t in cache[:2]:
        t.view(torch.uint8).fill_(0x7f)          # whatever is there before: NaN
    pages = torch.randperm(n * most, device="cuda", generator=g).to(torch.int32).view(n, most)
    inv_freq = gr.rotary_frequencies(d // 2, factor=4, context=256)
    sk, sv = torch.randn((n, 200, 2 * hkv, d), device="cuda", generator=g).to(_dt(dtype)).split([hkv, hkv], dim=2)
    had = np.zeros(n, dtype=int)
    for counts in ([130, 1, 64, 3], [1, 100, 1, 0], [70, 1, 0, 200], [1, 1, 1, 1]):
        had += counts
        starts = np.concatenate([[0], np.cumsum(counts)])
        rows = int(starts[-1])
        pos = np.concatenate([np.arange(a - c, a) for a, c in zip(had, counts)])
        x = torch.randn((rows, hq + 2 * hkv, d), device="cuda", generator=g).to(_dt(dtype))
        q, k, v = x.split([hq, hkv, hkv], dim=1)
        q64, k64 = _f64(q), _f64(k)
        gr.rotary(q, k, torch.from_numpy(pos).cuda(), inv_freq, interleaved=True, amplitude=1.125, out=(q, k))
        _check_rotary(_f64(q), q64, pos, _f64(inv_freq), True, 1.125, False, dtype)
        _check_rotary(_f64(k), k64, pos, _f64(inv_freq), True, 1.125, False, dtype)

        at = torch.from_numpy(starts[:-1, None] + np.arange(max(counts))).cuda().clamp(max=rows - 1)
        gr.kv_cache_append(cache, k[at], v[at], pages, _i32(had), _i32(counts))
        o = gr.kv_cache_attention_ragged(q, cache, pages, _i32(had), _i32(starts), window, sinks)
        y = gr.flash_attention_cross(q[at], sk, sv, _i32(states))
        assert gr.status() == gr.OK
        for i in range(n):
            ids = pages[i, :-(-int(had[i]) // page)].long()
            kk, vv = ((t[ids].double() * s[ids].double()[..., None, None]).transpose(1, 2).flatten(0, 1)[:had[i]]
                      for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
            r = slice(int(starts[i]), int(starts[i + 1]))
            w, absv, size = attend(q[r], kk, vv, seen(counts[i], int(had[i]), window, sinks))
            _check(_f64(o)[r], w, absv, size, d, dtype, 2.0 ** -11)
            # the stored values stand for what was appended: e4m3's half step 2^-4, and 2^-10 of the page's scale
            new = slice(int(had[i]) - counts[i], int(had[i]))
            for held, given, s in ((kk, k, cache.k_scale), (vv, v, cache.v_scale)):
                step = s[ids].double().repeat_interleave(page, 0)[new][..., None]
                off = (held[new] - given[r].double()).abs()
                assert bool((off <= 2.0 ** -4 * given[r].double().abs() + 2.0 ** -10 * step).all())
            see = torch.ones((at.shape[1], states[i]), dtype=torch.bool, device="cuda")
            w, absv, size = attend(q[at][i], sk[i, :states[i]], sv[i, :states[i]], see)
            _check(_f64(y)[i], w, absv, size, d, dtype, _half_step(dtype))


def test_a_step_captured_and_replayed():
    """Rotary in place, append, ragged and cross attention in one graph, replayed on new contents: as called eagerly."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    hq, hkv, d, page, n = 8, 2, 128, 64, 3
    cache = gr.KVCache.empty(12, hkv, d, page)
    pages = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    freq = gr.rotary_frequencies(d)
    lengths, starts = _i32([100, 7, 30]), _i32([0, 40, 41, 60])
    counts = starts[1:] - starts[:-1]
    x = torch.randn((60, hq + 2 * hkv, d), device="cuda", generator=g).half()
    s = torch.randn((n, 300, 2 * hkv, d), device="cuda", generator=g).half()
    sk, sv = s.split([hkv, hkv], dim=2)
    state_lengths = _i32([300, 17, 120])
    rows = (starts[:-1, None] + torch.arange(40, device="cuda")).clamp(max=59)
    pos = torch.zeros(60, dtype=torch.int64, device="cuda")
    # the first rows of the longest: some tokens are there before
    gr.kv_cache_append(cache, x[:60, hq:hq + hkv][None].expand(3, 60, hkv, d), x[:60, hq + hkv:][None].expand(3, 60, hkv, d),
                       pages, _i32([60, 6, 11]), _i32([60, 6, 11]))

    def step(y):
        q, k, v = y.split([hq, hkv, hkv], dim=1)
        gr.rotary(q, k, pos, freq, out=(q, k))
        gr.kv_cache_append(cache, k[rows], v[rows], pages, lengths, counts)
        return gr.kv_cache_attention_ragged(q, cache, pages, lengths, starts), gr.flash_attention_cross(
            q[rows][:, :1], sk, sv, state_lengths)

    def set_up(seed):
        h = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(x.shape, device="cuda", generator=h))
        pos.copy_(torch.randint(0, 5000, (60,), device="cuda", generator=h))
        for t, held in zip(cache, before):
            t.copy_(held)
    before = [t.clone() for t in cache]
    set_up(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x.clone())
    torch.cuda.current_stream().wait_stream(side)
    z = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z.copy_(x)
        captured = step(z)
    for seed in (4, 5, 6):
        set_up(seed)
        want = [t.clone() for t in step(x.clone())]
        held = [t.clone() for t in cache]
        set_up(seed)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cache, held))


def test_chunked_prompts_example():
    torch = pytest.importorskip("torch")
    spec = importlib.util.spec_from_file_location("chunked_prompts", os.path.join(ROOT, "examples", "chunked_prompts.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    kw = dict(prompts=(150, 9, 70), states=(40, 1, 99), steps=5)
    for budget in (32, 300):
        answers, taken = example.serve(budget=budget, **kw)
        assert answers.shape == (3, 5, 256) and bool(torch.isfinite(answers.float()).all())
        again, _ = example.serve(budget=budget, **kw)
        assert torch.equal(answers, again)
    assert taken == 5
