"""kv_cache_attention_ragged where a CTA goes through many items, of one tile and of two: against the definition in 64 bits,
with NaN of V in blocks that are masked in part.  Tolerances as in test_gpu_serving.py."""
import numpy as np
import pytest

import tiled_tensor_core_03_gb300 as gr

from test_gpu_ragged import SENTINEL, _held, _starts
from test_gpu_serving import DTYPES, _cache, _check, _cuda, _f64, _i32, _rand, _tables  # noqa: F401

pytestmark = pytest.mark.gpu


def _sequences(rng, group, hkv, sms):
    """(length, query tokens): chunks of two tiles and more, each with single tokens and chunks of one tile behind it, until
    there are three items a CTA and more."""
    two = 128 // group + 1                                  # tokens whose rows need a second tile
    out, items = [], 0
    while items * hkv < 3 * sms:
        t = int(rng.integers(two, 5 * two))
        out.append((t + int(rng.integers(0, 400)), t))
        for _ in range(int(rng.integers(1, 9))):            # one tile: some of them one token
            t = 1 if rng.random() < 0.6 else int(rng.integers(1, max(2, two)))
            out.append((t + int(rng.integers(0, 300)), t))
        items = sum(-(-t * group // 256) for _, t in out)
    return out


def _segments(rng, page, d, hkv, group, window, sinks, dtype):
    import torch
    from gpu_attend import attend, seen
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    seqs = _sequences(rng, group, hkv, sms)
    need = [-(-n // page) for n, _ in seqs]
    cache, c64 = _cache(rng, sum(need), hkv, page, d, garbage=False)
    table = _tables(rng, need, sum(need))
    bad = []                                                # (sequence, token, head, element)
    for i, (n, t) in enumerate(seqs):
        if n % page:                                        # slots past the length
            for x in cache[:2]:
                x.view(torch.uint8)[int(table[i, n // page]), :, n % page:] = 0x7f
        if rng.random() < 0.5:                              # a token that some of the chunk's rows see, if it is one of two
            j, h, c = n - 1 - int(rng.integers(0, t)), int(rng.integers(0, hkv)), int(rng.integers(0, d))
            cache[1].view(torch.uint8)[int(table[i, j // page]), h, j % page, c] = 0xff
            c64[1][int(table[i, j // page]), h, j % page, c] = 0.0
            bad.append((i, j, h, c))
    starts = _starts(seqs)
    q, _ = _rand(rng, (starts[-1] + 3, hkv * group, d), dtype, 2.0)
    args = (q, cache, _i32(table), _i32([n for n, _ in seqs]), _i32(starts), window, sinks)
    out = gr.kv_cache_attention_ragged(*args, out=torch.full_like(q, SENTINEL))
    again = gr.kv_cache_attention_ragged(*args, out=torch.full_like(q, SENTINEL))
    assert gr.status() == gr.OK
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    got = _f64(out)
    assert (got[starts[-1]:] == SENTINEL).all()
    for i, (n, t) in enumerate(seqs):
        ids, r = table[i, :need[i]], slice(starts[i], starts[i + 1])
        see = seen(t, n, window, sinks)
        o, absv, size = attend(q[r], _held(c64, 0, ids, n), _held(c64, 1, ids, n), see)
        mine = got[r]
        for j, h, c in [x[1:] for x in bad if x[0] == i]:
            rows, heads = see[:, j].cpu().numpy(), slice(h * group, (h + 1) * group)
            assert np.isnan(mine[rows, heads, c]).all(), (i, j, h, c)
            mine[rows, heads, c] = o[rows, heads, c]
        _check(mine, o, absv, size, d, dtype, 2.0 ** -11)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page,d,hkv,group,window,sinks", [
    (16, 128, 1, 4, 0, 0), (128, 128, 2, 1, 0, 0), (64, 128, 1, 5, 100, 3), (128, 128, 1, 2, 130, 140),
    (16, 64, 2, 4, 0, 0), (128, 64, 1, 3, 70, 2)])
def test_ragged_many_segments(page, d, hkv, group, window, sinks, dtype):
    _segments(np.random.default_rng(page + d + group), page, d, hkv, group, window, sinks, dtype)


@pytest.mark.parametrize("d", [64, 128])
def test_ragged_nan_of_a_second_tile_before_single_tokens(d):
    """The last rows of an item of two tiles see a NaN that its first rows do not; single tokens follow it in every
    CTA's range.  What the flag of that item says must reach its second tile."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(30)
    seqs = ([(64, 64)] + [(2, 1)] * 9) * sms                # 256 rows, then nine items of four
    page, group = 16, 4
    need = [-(-n // page) for n, _ in seqs]
    cache, _ = _cache(rng, sum(need), 1, page, d, garbage=False)
    table = _tables(rng, need, sum(need))
    starts = _starts(seqs)
    q, _ = _rand(rng, (starts[-1], group, d), "bf16")
    args = (_i32(table), _i32([n for n, _ in seqs]), _i32(starts))
    clean = _f64(gr.kv_cache_attention_ragged(q, cache, *args))
    sees = np.zeros(starts[-1], dtype=bool)
    for i, (n, t) in enumerate(seqs):
        if t == 64:                                         # token 60: rows 240 to 255, of the second tile
            cache.v.view(torch.uint8)[int(table[i, 60 // page]), 0, 60 % page, 7] = 0x7f
            sees[starts[i] + 60:starts[i] + 64] = True
    for _ in range(20):
        got = _f64(gr.kv_cache_attention_ragged(q, cache, *args))
        assert np.isnan(got[sees, :, 7]).all()
        got[sees, :, 7] = clean[sees, :, 7]
        assert np.array_equal(got, clean)
