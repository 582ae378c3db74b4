"""Serving operators around attention: what is measured, and their plain forms.

Four operators that a serving loop runs next to each other:

  window  attention of a prompt with a sliding window and first tokens that stay visible
  append  new tokens' K and V written into a paged 8-bit cache, one scale per page and head
  cache   attention of one or a few new tokens over that cache, optionally with each token's
          attention weight added to an accumulator
  evict   the cache cut down to a budget of tokens by accumulated weight

`run` computes them with elementary torch operations in 32 bits, or, where `own` is true, with
this repository's kernels.  Sizes are generic ones of 8 to 32 heads of 64 or 128, and the 4096
tokens by 32 heads by 128 of this repository's attention benchmark.
"""
import random
from collections import namedtuple

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
MIN_SCALE = 2.0 ** -100

Cache = namedtuple("Cache", "k v k_scale v_scale")


# ---------------------------------------------------------------------------------- cases


def listed():
    return [
        # a short ragged prompt of a small model: latency
        dict(name="window short ragged", op="window", b=1, sq=203, skv=203, hq=8, hkv=2, d=64,
             window=64, sinks=4, dtype="fp16", fused=False),
        # the attention benchmark's shape with shared heads and a 1024-token window
        dict(name="window prompt 4x4096", op="window", b=4, sq=4096, skv=4096, hq=32, hkv=8,
             d=128, window=1024, sinks=4, dtype="bf16", fused=True),
        # a long document, wide window
        dict(name="window long 16384", op="window", b=1, sq=16384, skv=16384, hq=32, hkv=8,
             d=128, window=4096, sinks=64, dtype="fp16", fused=False),
        # a decode step's new tokens, one a sequence
        dict(name="append step b64", op="append", b=64, tokens=1, before=4000, hkv=8, d=128,
             page=64, dtype="bf16"),
        # four ragged prompts written after prefill
        dict(name="append prompts 4x4096", op="append", b=4, tokens=4096, before=0, hkv=8, d=128,
             page=64, dtype="fp16"),
        # one user's decode step: latency
        dict(name="decode b1 1000", op="cache", b=1, tokens=1, longest=1000, hq=32, hkv=8, d=128,
             page=64, window=0, sinks=0, weights=False, dtype="fp16"),
        # a decode step of an ordinary batch, ragged lengths
        dict(name="decode b32 4096", op="cache", b=32, tokens=1, longest=4096, hq=32, hkv=8,
             d=128, page=64, window=0, sinks=0, weights=False, dtype="bf16"),
        # long contexts: the cache is all that is read
        dict(name="decode b64 32768", op="cache", b=64, tokens=1, longest=32768, hq=32, hkv=8,
             d=128, page=64, window=0, sinks=0, weights=False, dtype="fp16"),
        # four drafted tokens at once, window and sinks, small pages, unshared heads of 64
        dict(name="draft4 window b16", op="cache", b=16, tokens=4, longest=8192, hq=16, hkv=16,
             d=64, page=16, window=2000, sinks=4, weights=False, dtype="fp16"),
        # a step that also collects the weights an eviction goes by
        dict(name="decode weights b8 16384", op="cache", b=8, tokens=1, longest=16384, hq=32,
             hkv=8, d=128, page=128, window=0, sinks=0, weights=True, dtype="bf16"),
        # one sequence cut to a quarter: latency
        dict(name="evict b1 2000", op="evict", b=1, longest=2000, hkv=8, d=128, page=64,
             budget=512, sinks=4, recent=128),
        # a batch of long sequences cut to 4096 tokens
        dict(name="evict b16 16384", op="evict", b=16, longest=16384, hkv=8, d=128, page=64,
             budget=4096, sinks=4, recent=1024),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["window", "append", "cache", "cache", "evict"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["fp16", "bf16"])
    sinks = rng.choice([0, 1, 4, 64])
    if op == "window":
        sq = _log(rng, 1, 8192)
        b = rng.randint(1, max(1, min(4, 8192 // sq)))
        skv = sq + rng.choice([0, 0, _log(rng, 1, 4096)])
        return dict(op=op, b=b, sq=sq, skv=skv, hq=hkv * min(group, 4), hkv=hkv, d=d,
                    window=_log(rng, 1, min(4096, skv)), sinks=sinks, dtype=dtype,
                    fused=rng.random() < 0.5 and skv == sq)
    if op == "append":
        tokens = _log(rng, 1, 4096)
        return dict(op=op, b=rng.randint(1, max(1, min(64, 16384 // tokens))), tokens=tokens,
                    before=rng.choice([0, _log(rng, 1, 2000)]), hkv=hkv, d=d, page=page,
                    dtype=dtype)
    longest = _log(rng, 8, 32768)
    b = rng.randint(1, max(1, min(64, 400000 // longest)))
    if op == "cache":
        return dict(op=op, b=b, tokens=min(longest, rng.choice([1, 1, 1, 2, 4, 7])),
                    longest=longest, hq=hkv * group, hkv=hkv, d=d, page=page,
                    window=rng.choice([0, 0, _log(rng, 16, 8192)]), sinks=sinks,
                    weights=rng.random() < 0.3, dtype=dtype)
    budget = _log(rng, 4, longest)
    sinks = min(sinks, budget // 2)
    return dict(op=op, b=min(b, 16), longest=longest, hkv=hkv, d=d, page=page, budget=budget,
                sinks=sinks, recent=rng.randint(0, budget - sinks))


def _lengths(case):
    """Ragged lengths of the sequences: the first has the longest, the others 40% of it up."""
    rng = random.Random(case["b"] * 1000003 + case["longest"])
    least = max(case.get("tokens", 1), int(0.4 * case["longest"]))
    return [case["longest"]] + [rng.randint(least, case["longest"]) for _ in range(case["b"] - 1)]


def _append_lengths(case):
    """(length before, tokens added) of each sequence."""
    rng = random.Random(case["b"] * 1000003 + case["tokens"])
    n = case["tokens"]
    return [(rng.randint(0, case["before"]), n if i == 0 else rng.randint(max(1, n // 2), n))
            for i in range(case["b"])]


def _pages_of(tokens, page):
    return -(-tokens // page)


def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "window":
        off, w, s = case["skv"] - case["sq"], case["window"], case["sinks"]
        # query at p sees min(p + 1, w) keys of the window and the sinks left of it
        seen = sum(min(p + 1, w) + min(s, max(0, p + 1 - w))
                   for p in range(off, off + case["sq"]))
        return {"flops": 4.0 * d * case["hq"] * case["b"] * seen,
                "bytes": 2.0 * d * case["b"] * (2 * case["sq"] * case["hq"]
                                                + 2 * case["skv"] * hkv)}
    if case["op"] == "append":
        n = sum(t for _, t in _append_lengths(case))
        return {"flops": 4.0 * n * hkv * d, "bytes": 2.0 * n * hkv * d * (2 + 1)}
    if case["op"] == "cache":
        w, s, t = case["window"], case["sinks"], case["tokens"]
        seen = read = 0
        for n in _lengths(case):
            for p in range(n - t, n):
                seen += p + 1 if w == 0 else min(p + 1, w) + min(s, max(0, p + 1 - w))
            read += n if w == 0 else min(n, w + t - 1) + min(s, max(0, n - (w + t - 1)))
        return {"flops": 4.0 * d * case["hq"] * seen,
                "bytes": read * hkv * (2.0 * d + 8 * case["weights"])
                + 4.0 * d * case["hq"] * t * case["b"]}
    n = sum(_lengths(case))
    kept = sum(min(m, case["budget"]) for m in _lengths(case))
    return {"flops": 4.0 * n * hkv, "bytes": 4.0 * n * hkv + kept * hkv * (4.0 * d + 8)}


# ---------------------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _pool(num_pages, case, g):
    """A pool of pages as traffic leaves it: e4m3 values of N(0, 110^2) cut at 448, scales around
    2^-7 (values around 0.9).  One page more than num_pages is a spare that no sequence owns."""
    shape = (num_pages + 1, case["hkv"], case["page"], case["d"])

    def values():
        x = torch.randn(shape, device="cuda", dtype=torch.float16, generator=g)
        return x.mul_(110).clamp_(-448, 448).to(E4M3)

    def scales():
        e = torch.randint(-8, -5, shape[:2], device="cuda", generator=g)
        return torch.pow(2.0, e.float())

    return Cache(values(), values(), scales(), scales())


def _tables(counts, width, g):
    """Each sequence's pages, drawn from the pool in no order; -1 past its last one."""
    total = sum(counts)
    ids = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    table = torch.full((len(counts), width), -1, device="cuda", dtype=torch.int32)
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = ids[at:at + c]
        at += c
    return table


def _int32(values):
    return torch.tensor(values, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    d, hkv = case["d"], case["hkv"]
    dt = DTYPES.get(case.get("dtype"))

    def rand(*shape):
        return torch.randn(shape, device="cuda", dtype=torch.float32, generator=g).to(dt)

    if case["op"] == "window":
        hq = case["hq"]
        if case["fused"]:   # slices of one projection's output
            x = rand(case["b"], case["sq"], hq + 2 * hkv, d)
            c["q"], c["k_new"], c["v_new"] = x.split([hq, hkv, hkv], dim=2)
        else:
            c["q"] = rand(case["b"], case["sq"], hq, d)
            c["k_new"] = rand(case["b"], case["skv"], hkv, d)
            c["v_new"] = rand(case["b"], case["skv"], hkv, d)
        return c
    page = case["page"]
    if case["op"] == "append":
        had = _append_lengths(case)
        counts = [_pages_of(a + n, page) for a, n in had]
        c["cache"] = _pool(sum(counts), case, g)
        c["pages"] = _tables(counts, max(counts), g)
        # a few channels of K are much larger than the others
        c["k_new"] = (rand(case["b"], case["tokens"], hkv, d)
                      * (1 + 7 * (torch.arange(d, device="cuda") % 32 == 5))).to(dt)
        c["v_new"] = rand(case["b"], case["tokens"], hkv, d)
        c["lengths"] = _int32([a + n for a, n in had])
        c["counts"] = _int32([n for _, n in had])
        return c
    lengths = _lengths(case)
    counts = [_pages_of(n, page) for n in lengths]
    c["cache"] = _pool(sum(counts), case, g)
    c["pages"] = _tables(counts, max(counts), g)
    c["lengths"] = _int32(lengths)
    width = max(counts) * page
    if case["op"] == "cache":
        c["q"] = rand(case["b"], case["tokens"], case["hq"], d) * 2
        c["w"] = (torch.rand((case["b"], hkv, width), device="cuda", generator=g)
                  if case["weights"] else None)
        return c
    # accumulated weights: a heavy tail, and a tenth of the tokens that nothing looked at
    w = torch.exp(2 * torch.randn((case["b"], hkv, width), device="cuda", generator=g))
    c["w"] = torch.where(torch.rand(w.shape, device="cuda", generator=g) < 0.1, 0.0, w)
    keep = [_pages_of(min(n, case["budget"]), page) for n in lengths]
    c["to"] = _pool(sum(keep), case, g)
    c["to_pages"] = _tables(keep, _pages_of(case["budget"], page), g)
    return c


# ---------------------------------------------------------------------------------- plain forms


def _softmax(x, seen):
    """softmax over the last axis of the entries that are seen; 0 in a row that sees none."""
    x = torch.where(seen, x, float("-inf"))
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
    s = e.sum(-1, keepdim=True)
    return e / torch.where(s == 0, 1.0, s)


def _plain_window(c):
    """Queries in blocks of B >= window positions: block i sees keys of the block before it and of
    its own, and the sinks left of its window."""
    q, k, v = (c[n].float() for n in ("q", "k_new", "v_new"))
    b, sq, hq, d = q.shape
    skv, hkv = k.shape[1], k.shape[2]
    w, sinks, off, dev = c["window"], min(c["sinks"], skv), skv - sq, q.device
    B = max(w, 64)
    nb = -(-sq // B)
    pad = torch.nn.functional.pad
    # [b, hkv, nb, group * B, d]
    qb = pad(q, (0, 0, 0, 0, 0, nb * B - sq)).view(b, nb, B, hkv, hq // hkv, d)
    qb = qb.permute(0, 3, 1, 4, 2, 5).reshape(b, hkv, nb, -1, d)
    # key position p stands at p + B; block i takes positions off + iB - B to off + iB + B
    kb, vb = (pad(x, (0, 0, 0, 0, B, nb * B - sq)).permute(0, 2, 1, 3)[:, :, off:]
              .unfold(2, 2 * B, B) for x in (k, v))          # [b, hkv, nb, d, 2B]
    ks, vs = (x[:, :sinks].permute(0, 2, 1, 3).unsqueeze(2) for x in (k, v))  # [b, hkv, 1, S, d]
    x = torch.cat([qb @ ks.transpose(-1, -2), qb @ kb], -1) * d ** -0.5
    p = off + torch.arange(nb * B, device=dev).view(nb, B, 1)
    js = torch.arange(sinks, device=dev).view(1, 1, -1).expand(nb, B, sinks)
    jw = (off + torch.arange(nb, device=dev).view(nb, 1, 1) * B - B
          + torch.arange(2 * B, device=dev).view(1, 1, -1)).expand(nb, B, 2 * B)
    seen = torch.cat([js <= p - w, (jw <= p) & (jw > p - w) & (jw >= 0)], -1)
    x = _softmax(x, seen.repeat(1, hq // hkv, 1))
    o = x[..., :sinks] @ vs + x[..., sinks:] @ vb.transpose(-1, -2)
    o = o.view(b, hkv, nb, hq // hkv, B, d).permute(0, 2, 4, 1, 3, 5)
    return o.reshape(b, nb * B, hq, d)[:, :sq].to(c["q"].dtype)


def _scale_for(amax):
    """The smallest power of two s >= 2^-100 with amax <= 448 s."""
    m, e = torch.frexp(amax)                     # amax = m 2^e, 448 = 0.875 * 2^9
    s = torch.ldexp(torch.ones_like(amax), e - torch.where(m <= 0.875, 9, 8))
    return torch.where(amax == 0, MIN_SCALE, s.clamp(min=MIN_SCALE))


def _quantise(x, scale):
    return torch.where(torch.isfinite(x), x, float("nan")).div(scale).to(E4M3)


def _finite_amax(x):
    return torch.where(torch.isfinite(x), x.abs(), 0.0).amax((-1, -2))


def _plain_append(c):
    cache, page, dev = c["cache"], c["page"], c["pages"].device
    b, tokens = c["k_new"].shape[:2]
    spare = cache.k.shape[0] - 1
    end = c["lengths"].long()
    start = end - c["counts"].long()
    # every page that the new tokens can touch: [b, n]
    at = (start // page)[:, None] + torch.arange(_pages_of(tokens, page) + 1, device=dev)
    touched = at * page < end[:, None]
    ids = c["pages"].long().gather(1, at.clamp(max=c["pages"].shape[1] - 1))
    ids = torch.where(touched, ids, spare)
    pos = at[:, :, None] * page + torch.arange(page, device=dev)          # [b, n, page]
    new = ((pos >= start[:, None, None]) & (pos < end[:, None, None]))[:, :, None, :, None]
    old = (pos < start[:, None, None])[:, :, None, :, None]
    src = (pos - start[:, None, None]).clamp(0, tokens - 1)
    for x, held, scales in ((c["k_new"], cache.k, cache.k_scale),
                            (c["v_new"], cache.v, cache.v_scale)):
        y = x[torch.arange(b, device=dev)[:, None, None], src].float().permute(0, 1, 3, 2, 4)
        was = held[ids].float()                                           # [b, n, hkv, page, d]
        s_old = torch.where(at * page < start[:, None], 1.0, 0.0)[:, :, None] * scales[ids]
        s = torch.maximum(_scale_for(_finite_amax(torch.where(new, y, 0.0))), s_old)
        grown = (was * (s_old / s)[..., None, None]).to(E4M3).float()
        out = torch.where(new, _quantise(y, s[..., None, None]).float(),
                          torch.where(old, grown, was))
        held[ids] = out.to(E4M3)
        scales[ids] = s
    return tuple(x[:-1] for x in cache)


def _held(cache, which, pages):
    """K or V of each sequence's pages in 32 bits, in order: [b, hkv, tokens, d]."""
    values, scales = (cache.k, cache.k_scale) if which == "k" else (cache.v, cache.v_scale)
    ids = pages.long().clamp(min=0)
    x = values[ids].float() * scales[ids][..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_cache(c):
    q = c["q"].float()
    b, t, hq, d = q.shape
    hkv = c["hkv"]
    k = _held(c["cache"], "k", c["pages"])
    n = c["lengths"].long().view(b, 1, 1, 1, 1)
    p = n - t + torch.arange(t, device=q.device).view(1, 1, 1, t, 1)
    j = torch.arange(k.shape[2], device=q.device)
    seen = j <= p
    if c["window"]:
        seen = seen & ((j > p - c["window"]) | (j < c["sinks"]))
    qg = q.view(b, t, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)           # [b, hkv, group, t, d]
    x = (qg.flatten(2, 3) @ k.transpose(-1, -2)).view(b, hkv, hq // hkv, t, -1) * d ** -0.5
    del k
    x = _softmax(x, seen)
    v = _held(c["cache"], "v", c["pages"])
    v = torch.where((j < n[:, 0, 0])[..., None], v, 0.0)                  # slots not written yet
    o = (x.flatten(2, 3) @ v).view(b, hkv, hq // hkv, t, d).permute(0, 3, 1, 2, 4)
    o = o.reshape(b, t, hq, d).to(c["q"].dtype)
    if c["w"] is None:
        return o
    c["w"] += x.sum((2, 3))
    return o, c["w"]


def _plain_evict(c):
    cache, to, page, budget = c["cache"], c["to"], c["page"], c["budget"]
    w, dev = c["w"], c["w"].device
    b, hkv, width = w.shape
    n = c["lengths"].long().view(b, 1, 1)
    j = torch.arange(width, device=dev)
    key = torch.where(torch.isnan(w), float("-inf"), w)
    key = torch.where((j < c["sinks"]) | (j >= n - c["recent"]), float("inf"), key)
    # a token that is there goes before one that is not, then the heavier one, then the first
    by_key = torch.sort(key, dim=-1, descending=True, stable=True).indices
    order = by_key.gather(-1, torch.sort((by_key >= n).int(), dim=-1, stable=True).indices)
    slots = to.k.shape[2] * c["to_pages"].shape[1]
    rank = torch.arange(slots, device=dev)
    m = torch.clamp(n, max=budget)
    kept = torch.where(rank < m, torch.nn.functional.pad(order, (0, max(0, slots - width)))
                       [..., :slots], width).sort(-1).values              # [b, hkv, slots]
    live = rank < m
    src = kept.clamp(max=width - 1)
    ids = c["pages"].long()[torch.arange(b, device=dev)[:, None, None], src // page].clamp(min=0)
    heads = torch.arange(hkv, device=dev)[None, :, None]
    # pages of the new cache that hold tokens; the others' writes go to the spare page
    used = torch.arange(c["to_pages"].shape[1], device=dev) * page < m[:, :, 0]
    to_ids = torch.where(used, c["to_pages"].long(), to.k.shape[0] - 1)   # [b, n]
    for held, scales, out, out_scales in ((cache.k, cache.k_scale, to.k, to.k_scale),
                                          (cache.v, cache.v_scale, to.v, to.v_scale)):
        x = held[ids, heads, src % page].float() * scales[ids, heads][..., None]
        x = torch.where(live[..., None], x, 0.0).view(b, hkv, -1, page, x.shape[-1])
        x = x.transpose(1, 2)                                             # [b, n, hkv, page, d]
        s = _scale_for(_finite_amax(x))
        out[to_ids] = _quantise(x, s[..., None, None])
        out_scales[to_ids] = s
    new_w = torch.where(live, w.gather(-1, src), 0.0)
    kept = torch.where(live, kept, -1)[..., :budget].to(torch.int32)
    return (m.view(b).to(torch.int32), new_w, kept) + tuple(x[:-1] for x in to)


def _own(c):
    import tiled_tensor_core_03_gb300 as gr
    if c["op"] == "window":
        return gr.flash_attention_window(c["q"], c["k_new"], c["v_new"], c["window"], c["sinks"])
    if c["op"] == "append":
        gr.kv_cache_append(c["cache"], c["k_new"], c["v_new"], c["pages"], c["lengths"],
                           c["counts"])
        return tuple(x[:-1] for x in c["cache"])
    if c["op"] == "cache":
        o = gr.kv_cache_attention(c["q"], c["cache"], c["pages"], c["lengths"],
                                  window=c["window"], sinks=c["sinks"], weights=c["w"])
        return o if c["w"] is None else (o, c["w"])
    lengths, w, kept = gr.kv_cache_evict(c["cache"], c["w"], c["pages"], c["lengths"],
                                         c["budget"], c["sinks"], c["recent"], c["to"],
                                         c["to_pages"])
    return (lengths, w, kept) + tuple(x[:-1] for x in c["to"])


def run(state):
    if own:
        return _own(state)
    return {"window": _plain_window, "append": _plain_append, "cache": _plain_cache,
            "evict": _plain_evict}[state["op"]](state)


# ---------------------------------------------------------------------------------- 64 bits


def exact(case, seed):
    """The definitions in 64 bits, one sequence (and a run of queries) at a time."""
    return {"window": _exact_window, "append": _exact_append, "cache": _exact_cache,
            "evict": _exact_evict}[case["op"]](prepare(case, seed))


def _exact_attend(q, k, v, p, window, sinks):
    """q [t, hq, d], k and v [n, hkv, d] whose first key has position 0 (or the positions `at`);
    returns o [t, hq, d] and the weights of each K/V head's tokens [hkv, n]."""
    k, at = k if isinstance(k, tuple) else (k, torch.arange(k.shape[0], device=k.device))
    group = q.shape[1] // k.shape[1]
    see = at[None, :] <= p[:, None]
    if window:
        see &= (at[None, :] > p[:, None] - window) | (at[None, :] < sinks)
    o = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    w = torch.zeros((k.shape[1], k.shape[0]), dtype=torch.float64, device=q.device)
    for h in range(q.shape[1]):
        x = q[:, h].double() @ k[:, h // group].double().T / q.shape[2] ** 0.5
        a = torch.exp(x.masked_fill(~see, float("-inf"))
                      - x.masked_fill(~see, float("-inf")).max(1, keepdim=True).values)
        a = (a / a.sum(1, keepdim=True)).masked_fill(~see, 0.0)
        o[:, h] = a @ v[:, h // group].double()
        w[h // group] += a.sum(0)
    return o, w


def _exact_window(c):
    q, k, v = c["q"], c["k_new"], c["v_new"]
    off = k.shape[1] - q.shape[1]
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    for i in range(q.shape[0]):
        for t in range(0, q.shape[1], 1024):
            rows = slice(t, min(t + 1024, q.shape[1]))
            p = off + torch.arange(rows.start, rows.stop, device=q.device)
            lo = max(0, int(p[0]) - c["window"] + 1)
            s = min(c["sinks"], lo)
            at = torch.cat([torch.arange(s, device=q.device),
                            torch.arange(lo, int(p[-1]) + 1, device=q.device)])
            out[i, rows] = _exact_attend(q[i, rows], (k[i, at], at), v[i, at], p, c["window"],
                                         c["sinks"])[0]
    return out


def _power_of_two(amax):
    """The scale of a block by trial: doubled from the least one until 448 times it holds amax."""
    s = torch.full_like(amax, MIN_SCALE, dtype=torch.float64)
    for step in (128, 64, 32, 16, 8, 4, 2, 1):
        t = s * 2.0 ** step
        s = torch.where(448 * t / 2 < amax, t, s)
    return s


def _exact_append(c):
    cache, page = c["cache"], c["page"]
    out = [x.double() for x in cache]
    for i, (had, new) in enumerate(_append_lengths(c)):
        for at in range(had // page, _pages_of(had + new, page)):
            lo, hi = max(had, at * page), min(had + new, (at + 1) * page)
            pid = int(c["pages"][i, at])
            for n, x in ((0, c["k_new"]), (1, c["v_new"])):
                y = x[i, lo - had:hi - had].double().transpose(0, 1)      # [hkv, tokens, d]
                s = _power_of_two(y.abs().amax((1, 2)))
                if lo > at * page:
                    was = out[n + 2][pid].clone()
                    s = torch.maximum(s, was)
                    out[n][pid][:, :lo - at * page] *= (was / s)[:, None, None]
                out[n][pid][:, lo - at * page:hi - at * page] = y / s[:, None, None]
                out[n + 2][pid] = s
    return tuple(x[:-1] for x in out)


def _exact_cache(c):
    q, page = c["q"], c["page"]
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    w = None if c["w"] is None else c["w"].double()
    for i, n in enumerate(_lengths(c)):
        ids = c["pages"][i, :_pages_of(n, page)].long()
        k, v = ((x[ids].float() * s[ids][..., None, None]).transpose(1, 2).flatten(0, 1)[:n]
                for x, s in ((c["cache"].k, c["cache"].k_scale),
                             (c["cache"].v, c["cache"].v_scale)))
        p = torch.arange(n - q.shape[1], n, device=q.device)
        out[i], a = _exact_attend(q[i], k, v, p, c["window"], c["sinks"])
        if w is not None:
            w[i, :, :n] += a
    return out if w is None else (out, w)


def _exact_evict(c):
    cache, to, page, budget = c["cache"], c["to"], c["page"], c["budget"]
    out = [x.double() for x in to]
    slots = page * c["to_pages"].shape[1]
    lengths, (b, hkv, _) = _lengths(c), c["w"].shape
    new_w = torch.zeros((b, hkv, slots), dtype=torch.float64, device=c["w"].device)
    for i, n in enumerate(lengths):
        m = min(n, budget)
        for h in range(hkv):
            w = c["w"][i, h, :n].double()
            if n > budget:
                free = torch.arange(c["sinks"], n - c["recent"], device=w.device)
                # heaviest first; equal weights keep their order
                heavy = free[torch.argsort(-w[free], stable=True)[:budget - c["sinks"]
                                                                  - c["recent"]]]
                keep = torch.cat([torch.arange(c["sinks"], device=w.device), heavy,
                                  torch.arange(n - c["recent"], n, device=w.device)]).sort().values
            else:
                keep = torch.arange(n, device=w.device)
            new_w[i, h, :m] = w[keep]
            ids = c["pages"][i].long()[keep // page]
            dst = c["to_pages"][i, :_pages_of(m, page)].long()
            for k, (x, s) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
                y = torch.zeros((len(dst) * page, x.shape[-1]), dtype=torch.float64,
                                device=w.device)
                y[:m] = x[ids, h, keep % page].double() * s[ids, h].double()[:, None]
                y = y.view(len(dst), page, -1)
                s = _power_of_two(y.abs().amax((1, 2)))
                out[k][dst, h] = y / s[:, None, None]
                out[k + 2][dst, h] = s
    return (None, new_w, None) + tuple(x[:-1] for x in out)
