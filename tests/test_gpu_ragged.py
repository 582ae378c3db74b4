"""kv_cache_attention_ragged on the GPU against the definition in 64 bits.  Tolerances as in
test_gpu_serving.py: roundings counted, half a step each; weights are rounded to fp16."""
import numpy as np
import pytest

import tiled_tensor_core_03_gb300 as gr

from test_gpu_serving import DTYPES, _cache, _check, _cuda, _dt, _f64, _i32, _rand, _tables  # noqa: F401

pytestmark = pytest.mark.gpu

SENTINEL = -77.0


def _held(c64, which, ids, n):
    """K or V of a sequence's pages as a float64 CUDA tensor [n, hkv, d]."""
    import torch
    x, s = c64[which], c64[which + 2]
    y = (x[ids] * s[ids][..., None, None]).transpose(0, 2, 1, 3)
    return torch.from_numpy(y.reshape(-1, *y.shape[2:])[:n].copy()).cuda()


def _starts(seqs, lead=0):
    return [lead] + [lead + int(x) for x in np.cumsum([t for _, t in seqs])]


def _ragged(rng, page, d, hkv, group, seqs, window, sinks, dtype, scale=2.0, lead=0, tail=0, width=None,
            change=None):
    """seqs: (length, query tokens) of each sequence; rows before the first and behind the last stay."""
    import torch
    from gpu_attend import attend, seen
    need = [-(-n // page) for n, _ in seqs]
    total = sum(need) + 1
    cache, c64 = _cache(rng, total, hkv, page, d, garbage=False)
    if change:
        change(cache, c64)
    table = _tables(rng, need, total, width)
    for i, (n, _) in enumerate(seqs):   # slots past a sequence's length hold NaN
        if n % page:
            pid = int(table[i, n // page])
            for t in cache[:2]:
                t.view(torch.uint8)[pid, :, n % page:] = 0x7f
    starts = _starts(seqs, lead)
    rows = starts[-1] + tail
    q, q64 = _rand(rng, (rows, hkv * group, d), dtype, scale)
    out = torch.full_like(q, SENTINEL)
    args = (q, cache, _i32(table), _i32([n for n, _ in seqs]), _i32(starts), window, sinks)
    assert gr.kv_cache_attention_ragged(*args, out=out) is out
    again = gr.kv_cache_attention_ragged(*args, out=torch.full_like(q, SENTINEL))
    assert gr.status() == gr.OK
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    got = _f64(out)
    assert (got[:lead] == SENTINEL).all() and (got[starts[-1]:] == SENTINEL).all()
    for i, (n, t) in enumerate(seqs):
        ids = table[i, :need[i]]
        r = slice(starts[i], starts[i + 1])
        see = seen(t, n, window, sinks)
        o, absv, size = attend(q.double()[r], _held(c64, 0, ids, n), _held(c64, 1, ids, n), see)
        _check(got[r], o, absv, size, d, dtype, 2.0 ** -11)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page,d,hkv,group,seqs,window,sinks", [
    (64, 128, 1, 1, [(1, 1)], 0, 0),
    (16, 64, 1, 1, [(5, 3)], 0, 0),
    (64, 128, 2, 4, [(200, 70)], 0, 0),
    (128, 128, 2, 4, [(300, 1), (129, 129), (128, 40), (0, 0), (77, 0), (513, 200)], 0, 0),
    (32, 64, 3, 3, [(1000, 333), (31, 7), (2, 2)], 0, 0),
    (16, 128, 1, 7, [(600, 91), (40, 40)], 100, 3),
    (16, 64, 2, 8, [(700, 300), (1, 1), (260, 2)], 40, 0),
    (64, 128, 1, 5, [(900, 500)], 1, 0),
    (64, 64, 1, 1, [(1500, 700)], 300, 140),
    (32, 128, 2, 1, [(257, 257), (128, 128), (256, 256)], 0, 0),
    (128, 64, 1, 16, [(1024, 64), (90, 33)], 129, 128),
    (64, 128, 1, 40, [(300, 17)], 0, 0),
    (64, 64, 1, 130, [(40, 5)], 0, 0),
])
def test_ragged(page, d, hkv, group, seqs, window, sinks, dtype):
    rng = np.random.default_rng(page + d + sum(n + 3 * t for n, t in seqs))
    _ragged(rng, page, d, hkv, group, seqs, window, sinks, dtype)


def test_ragged_rows_of_no_sequence_are_left_alone():
    rng = np.random.default_rng(1)
    _ragged(rng, 64, 128, 2, 4, [(100, 30), (50, 0), (70, 1)], 0, 0, "fp16", lead=5, tail=9)
    _ragged(rng, 16, 64, 1, 1, [(10, 0)], 0, 0, "bf16", lead=0, tail=4)


def test_ragged_more_queries_than_tokens():
    """Rows at negative positions see nothing and become 0; so does a sequence without tokens."""
    rng = np.random.default_rng(2)
    _ragged(rng, 64, 128, 2, 2, [(3, 10), (0, 6), (130, 400)], 0, 0, "fp16")
    _ragged(rng, 16, 64, 1, 3, [(0, 200), (5, 300)], 8, 2, "bf16")


@pytest.mark.parametrize("d,group", [(128, 4), (64, 1)])
def test_ragged_cut_into_many_parts(d, group):
    """Few rows over a long cache: each item is cut into parts of many blocks, which are joined."""
    rng = np.random.default_rng(3)
    _ragged(rng, 64, d, 1, group, [(30000, 40)], 0, 0, "fp16")
    _ragged(rng, 128, d, 2, group, [(9000, 100), (5000, 1), (20000, 3)], 0, 0, "bf16", scale=4.0)
    _ragged(rng, 32, d, 1, group, [(7000, 600)], 0, 0, "fp16", scale=8.0)


def test_ragged_many_sequences():
    """More sequences than a warp's lanes, most of them empty or of one token; long chunks among them."""
    rng = np.random.default_rng(4)
    seqs = [(int(n), int(min(n, rng.integers(0, 4)))) for n in rng.integers(0, 60, 500)]
    seqs[77], seqs[300] = (1500, 1500), (900, 5)
    _ragged(rng, 16, 64, 1, 2, seqs, 0, 0, "fp16", width=120)


def test_ragged_equals_the_padded_call():
    """The same tokens through kv_cache_attention, up to the roundings of both."""
    import torch
    rng = np.random.default_rng(5)
    cache, _ = _cache(rng, 40, 2, 64, 128, garbage=False)
    table = _tables(rng, [10, 10, 10], 40)
    q, _ = _rand(rng, (3, 6, 8, 128), "fp16", 2.0)
    lengths = _i32([640, 600, 577])
    a = gr.kv_cache_attention(q, cache, _i32(table), lengths, 100, 4)
    b = gr.kv_cache_attention_ragged(q.view(18, 8, 128), cache, _i32(table), lengths, _i32([0, 6, 12, 18]), 100, 4)
    a, b = a.view(18, 8, 128).float(), b.float()
    # each is within the weights' rounding (2^-11 of sum w |v|) and its own (2^-11) of the formula's value
    size = float(cache.v_scale.max()) * 448
    assert float((a - b).abs().max()) <= 4 * 2.0 ** -11 * size
    assert float((a - b).norm() / a.norm()) < 2.0 ** -10
    assert torch.isfinite(b).all()


def test_ragged_large_scores():
    rng = np.random.default_rng(6)
    _ragged(rng, 64, 128, 1, 4, [(700, 90)], 0, 0, "fp16", scale=16.0)
    _ragged(rng, 64, 64, 2, 2, [(700, 300), (40, 1)], 200, 4, "bf16", scale=64.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("power", [10, 14, 20, 30, 60])
def test_ragged_finite_scores_of_any_size(power, dtype):
    """Scores that are whole multiples of 2^power: the weights of equal largest ones are equal, whatever the
    scores' size and the pages' V scales are.  (fp16 queries reach 2^15.)"""
    import torch
    d, n, page = 64, 256, 64
    if dtype == "fp16" and power > 20:
        pytest.skip("beyond fp16 times the K scales used here")
    cache = gr.KVCache.empty(4, 1, d, page)
    k = torch.zeros((4, 1, page, d), device="cuda")
    k[..., 0] = torch.tensor([0.0, 1.0, 0.0, 1.0], device="cuda")[:, None, None]   # pages 1 and 3 score
    cache.k.copy_(k.to(torch.float8_e4m3fn))
    g = torch.Generator(device="cuda").manual_seed(power)
    v = torch.randn((4, 1, page, d), device="cuda", generator=g).to(torch.float8_e4m3fn)
    cache.v.copy_(v)
    cache.k_scale.fill_(2.0 ** (power - 4))
    vs = torch.tensor([1.0, 0.5, 4.0, 8.0], device="cuda")
    cache.v_scale.copy_(vs[:, None])
    q = torch.zeros((3, 1, d), dtype=_dt(dtype), device="cuda")
    q[:, 0, 0] = 16 * 8.0   # / sqrt(64)
    out = gr.kv_cache_attention_ragged(q, cache, _i32([[0, 1, 2, 3]]), _i32([n]), _i32([0, 3])).double()
    held = v.double() * vs[:, None, None, None].double()
    seen = torch.cat([held[1, 0], held[3, 0]])     # all others weigh exp(-2^power) = 0
    for i in range(3):
        s = seen[:len(seen) - 2 + i]
        want, size = s.mean(0), s.abs().mean(0)
        half = torch.finfo(_dt(dtype)).eps / 2
        assert bool(((out[i, 0] - want).abs() <= half * want.abs() + (2.0 ** -11 + 2.0 ** -18) * size).all())


def test_ragged_scales_far_apart():
    """Pages whose scales differ by 2^40 and more: what each weight counts, in the sum of weights and in the sum
    with V, is rounded against the largest, and nothing is lost."""
    import torch

    def change(cache, c64):
        n = cache.k.shape[0]
        far = [2.0 ** -8, 2.0 ** -48, 2.0 ** -8, 2.0 ** -100]
        for s, s64 in ((cache[2], c64[2]), (cache[3], c64[3])):
            for i in range(n):
                s64[i] = far[(i * 7) % 4]
            s.copy_(torch.from_numpy(s64.astype(np.float32)))
    for seed in range(3):
        rng = np.random.default_rng(20 + seed)
        _ragged(rng, 64, 64, 1, 4, [(256, 70)], 0, 0, "bf16", change=change)
        _ragged(rng, 16, 128, 2, 2, [(300, 40), (77, 2)], 50, 3, "fp16", change=change)


def test_ragged_queries_of_any_size():
    """bf16 rows around 2^100 and 2^-100, zeros among them, beside pages of zeros."""
    import torch
    from gpu_attend import attend, seen
    rng = np.random.default_rng(8)
    cache, c64 = _cache(rng, 5, 1, 64, 64, garbage=False)
    cache.k_scale[2], c64[2][2] = 2.0 ** -100, 2.0 ** -100
    cache.v_scale[2], c64[3][2] = 2.0 ** -100, 2.0 ** -100
    q, _ = _rand(rng, (80, 2, 64), "bf16")
    q[10:20] *= 2.0 ** -90
    q[20:30] = 0
    q[30:40] *= 2.0 ** -126
    out = gr.kv_cache_attention_ragged(q, cache, _i32([[2, 0, 1, 3]]), _i32([200]), _i32([0, 80]))
    o, absv, size = attend(q.double(), _held(c64, 0, [2, 0, 1, 3], 200), _held(c64, 1, [2, 0, 1, 3], 200),
                           seen(80, 200, 0, 0))
    _check(_f64(out), o, absv, size, 64, "bf16", 2.0 ** -11)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 50])
def test_ragged_not_finite_reaches_those_who_see_it(window, d):
    """A NaN in V reaches exactly its element of the rows that see it; one in K all of them."""
    import torch
    rng = np.random.default_rng(13)
    n, t = 400, 160
    cache, _ = _cache(rng, 7, 1, 64, d, garbage=False)
    table = [[2, 0, 3, 1, 6, 5, 4]]
    q, _ = _rand(rng, (t, 2, d), "fp16")
    args = (_i32(table), _i32([n]), _i32([0, t]), window)
    clean = _f64(gr.kv_cache_attention_ragged(q, cache, *args))
    for at in (0, 245, 380, 399, 300, 256):
        other = [x.clone() for x in cache]
        other[1].view(torch.uint8)[table[0][at // 64], 0, at % 64, 37] = 0xff
        got = _f64(gr.kv_cache_attention_ragged(q, gr.KVCache(*other), *args))
        sees = np.array([at <= p and (window == 0 or at > p - window) for p in range(n - t, n)])
        assert np.isnan(got[sees, :, 37]).all(), at
        got[sees, :, 37] = clean[sees, :, 37]
        # (the value that it took the place of is gone from that element alone)
        assert np.array_equal(got, clean), at
        other = [x.clone() for x in cache]
        other[0].view(torch.uint8)[table[0][at // 64], 0, at % 64, 3] = 0x7f
        got = _f64(gr.kv_cache_attention_ragged(q, gr.KVCache(*other), *args))
        assert np.isnan(got[sees]).all() and np.array_equal(got[~sees], clean[~sees]), at


def test_ragged_not_finite_in_cut_items():
    """The same where parts of an item are joined, and in every token."""
    import torch
    rng = np.random.default_rng(14)
    cache, _ = _cache(rng, 160, 1, 64, 128, garbage=False)
    q, _ = _rand(rng, (20, 4, 128), "bf16")
    table = torch.arange(160, dtype=torch.int32, device="cuda")[None]
    args = (table, _i32([10000]), _i32([0, 20]))
    clean = _f64(gr.kv_cache_attention_ragged(q, cache, *args))
    cache.v.view(torch.uint8)[9999 // 64, 0, 9999 % 64, 5] = 0x7f
    got = _f64(gr.kv_cache_attention_ragged(q, cache, *args))
    assert np.isnan(got[19, :, 5]).all() and not np.isnan(got[:19]).any()
    assert np.array_equal(got[:19], clean[:19])
    cache.v.view(torch.uint8)[:, :, :, 5] = 0x7f
    got = _f64(gr.kv_cache_attention_ragged(q, cache, *args))
    assert np.isnan(got[..., 5]).all() and not np.isnan(np.delete(got, 5, 2)).any()


def test_ragged_refuses_what_only_the_device_sees():
    """A page outside the pool is skipped, a bad length is a sequence without tokens, bad starts a sequence without
    rows; the others are right and the status says so."""
    import torch
    from gpu_attend import attend
    rng = np.random.default_rng(15)
    cache, c64 = _cache(rng, 8, 2, 16, 64, garbage=False)
    cache.v.view(torch.uint8)[6] = 0x7f
    q, _ = _rand(rng, (8, 4, 64), "fp16")
    table = np.array([[0, 1], [2, 99], [-7, 3], [4, 5]])

    def call(lengths, starts):
        out = torch.full_like(q, SENTINEL)
        gr.kv_cache_attention_ragged(q, cache, _i32(table), _i32(lengths), _i32(starts), out=out)
        assert gr.status() == gr.ERR_PAGE
        assert gr.status() == gr.OK
        return _f64(out)
    out = call([33, 30, 30, 30], [0, 2, 4, 6, 8])
    assert (out[:2] == 0).all()
    for i, ids, there in ((1, [2, 0], range(16)), (2, [0, 3], range(16, 30)), (3, [4, 5], range(30))):
        see = torch.zeros((2, 30), dtype=torch.bool, device="cuda")
        for r in range(2):
            see[r, [j for j in there if j <= 28 + r]] = True
        rows = slice(2 * i, 2 * i + 2)
        o, absv, size = attend(q.double()[rows], _held(c64, 0, ids, 30), _held(c64, 1, ids, 30), see)
        _check(out[rows], o, absv, size, 64, "fp16", 2.0 ** -11)
    good = [30, 16, 16, 30]
    table = np.array([[0, 1], [2, 3], [3, 2], [4, 5]])
    for starts, skipped in (([0, 2, 1, 6, 8], [1]), ([0, 2, 4, 9, 8], [2, 3]), ([-1, 2, 4, 6, 8], [0]),
                            ([0, 2, 4, 6, 1 << 30], [3])):
        out = call(good, starts)
        for i in range(4):
            lo, hi = max(0, starts[i]), min(8, starts[i + 1])
            if i not in skipped:
                assert np.isfinite(out[lo:hi]).all() and (out[lo:hi] != SENTINEL).all()
    out = call(good, [0, 2, 4, 6, 9])
    assert (out[6:] == SENTINEL).all()


def test_ragged_pages_given_up_are_not_read():
    """Pages that no query's window reaches may be named by anything."""
    import torch
    rng = np.random.default_rng(16)
    for page in (16, 64, 128):
        need = -(-1000 // page)
        cache, _ = _cache(rng, need + 1, 1, page, 64, garbage=False)
        table = _tables(rng, [need], need + 1)
        q, _ = _rand(rng, (30, 2, 64), "fp16")
        args = (_i32([1000]), _i32([0, 30]), 200, 5)
        want = gr.kv_cache_attention_ragged(q, cache, _i32(table), *args)
        low = 1000 - 30 - 200 + 1          # first token in the first row's window
        table[0, 1 if page >= 5 else 0:low // page] = 1 << 30
        got = gr.kv_cache_attention_ragged(q, cache, _i32(table), *args)
        assert gr.status() == gr.OK
        assert torch.equal(got, want)


def test_ragged_strides():
    """Queries as a slice of a fused projection, heads before rows, one head for all."""
    import torch
    rng = np.random.default_rng(17)
    cache, _ = _cache(rng, 10, 2, 64, 64, garbage=False)
    rest = (cache, _i32([[3, 1, 4, 5, 2]]), _i32([300]), _i32([0, 50]))
    x, _ = _rand(rng, (50, 12, 64), "bf16")
    same = [(x[:, 2:10], None), (x.transpose(0, 1).contiguous().transpose(0, 1)[:, 4:12], None),
            (x[:, :1].expand(50, 8, 64), None), (x[:1, :8].expand(50, 8, 64), None)]
    for q, _ in same:
        got = gr.kv_cache_attention_ragged(q, *rest)
        assert torch.equal(got, gr.kv_cache_attention_ragged(q.contiguous(), *rest))


def test_ragged_streams_graphs_and_workspaces():
    """Calls on two streams at once, a call captured and replayed on new contents, a workspace of one's own and
    of larger calls."""
    import torch
    rng = np.random.default_rng(18)
    cache, _ = _cache(rng, 200, 2, 64, 128, garbage=False)
    table = torch.arange(200, dtype=torch.int32, device="cuda").view(2, 100)
    lengths, starts = _i32([6400, 5000]), _i32([0, 60, 61])
    q, _ = _rand(rng, (61, 8, 128), "fp16")
    want = gr.kv_cache_attention_ragged(q, cache, table, lengths, starts)
    side = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s in side:
            got.append(gr.kv_cache_attention_ragged(q, cache, table, lengths, starts, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
    ws = gr.kv_cache_attention_ragged_workspace(cache)
    small = gr.kv_cache_attention_ragged(q[:3], cache, table, lengths, _i32([0, 1, 3]), workspace=ws)
    assert torch.equal(gr.kv_cache_attention_ragged(q, cache, table, lengths, starts, workspace=ws), want)
    assert torch.equal(gr.kv_cache_attention_ragged(q[:3], cache, table, lengths, _i32([0, 1, 3]), workspace=ws),
                       small)
    out = torch.zeros_like(q)
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gr.kv_cache_attention_ragged(q, cache, table, lengths, starts, out=out)
    out2 = torch.zeros_like(q)
    with torch.cuda.graph(graph2):
        gr.kv_cache_attention_ragged(q, cache, table, lengths, starts, out=out2)
    for _ in range(3):
        graph.replay()
        with torch.cuda.stream(side[0]):
            graph2.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out2, want)
        out.zero_(), out2.zero_()
    q2, _ = _rand(rng, (61, 8, 128), "fp16")
    q.copy_(q2)
    lengths.copy_(_i32([3000, 6400]))
    starts.copy_(_i32([0, 1, 61]))
    graph.replay()
    assert torch.equal(out, gr.kv_cache_attention_ragged(q, cache, table, lengths, starts))


def test_ragged_pages_past_four_gib():
    """Page numbers whose bytes lie past 2^32."""
    import torch
    page, hkv, d = 128, 8, 128
    n = (1 << 32) // (page * hkv * d) + 40
    values = [torch.zeros((n, hkv, page, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones((n, hkv), device="cuda") for _ in range(2)]
    cache = gr.KVCache(*(x.view(torch.float8_e4m3fn) for x in values), *scales)
    g = torch.Generator(device="cuda").manual_seed(1)
    small = [torch.randint(0, 120, (3, hkv, page, d), dtype=torch.uint8, device="cuda", generator=g)
             for _ in range(2)]
    for x, y in zip(values, small):
        x[n - 3:] = y
    near = gr.KVCache(*(y.view(torch.float8_e4m3fn) for y in small), *(s[:3].contiguous() for s in scales))
    q = torch.randn((70, 16, d), device="cuda", generator=g).half() * 0.05
    rest = (_i32([300]), _i32([0, 70]))
    far = gr.kv_cache_attention_ragged(q, cache, _i32([[n - 1, n - 3, n - 2]]), *rest)
    assert torch.equal(far, gr.kv_cache_attention_ragged(q, near, _i32([[2, 0, 1]]), *rest))
