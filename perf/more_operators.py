"""Serving operators next to the paged cache: what is measured, and their plain forms.

Three operators that a serving loop runs between its projections:

  rotary  rotary positions of new queries and keys (halves or interleaved pairs, all or part of
          a head, frequencies scaled for long contexts, and the inverse rotation)
  ragged  attention of a batch of chunks over the paged 8-bit cache: each sequence brings as many
          new tokens as it has, packed row after row
  cross   attention to an encoder's states, whose number differs from sequence to sequence

`run` computes them with elementary torch operations in 32 bits (angles in 64), or, where `own` is
true, with this repository's kernels.  Sizes are generic ones of 4 to 32 heads of 64 or 128.
"""
import math
import random
from collections import namedtuple

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn

Cache = namedtuple("Cache", "k v k_scale v_scale")


# ---------------------------------------------------------------------------------- cases


def listed():
    return [
        # a decode step's tokens, one a sequence: latency
        dict(name="rotary step b64", op="rotary", b=64, tokens=1, far=8000, hq=32, hkv=8, d=128,
             rot=128, interleaved=False, scaling=1.0, inverse=False, fused=True, dtype="fp16"),
        # prompts of a batch, slices of a fused projection, context stretched four times
        dict(name="rotary prompts 4x4096", op="rotary", b=4, tokens=4096, far=0, hq=32, hkv=8,
             d=128, rot=128, interleaved=False, scaling=4.0, inverse=False, fused=True,
             dtype="bf16"),
        # the gradient's way back, half of each head, pairs side by side, far positions
        dict(name="rotary back 3x5001 part", op="rotary", b=3, tokens=5001, far=1000000, hq=16,
             hkv=16, d=64, rot=32, interleaved=True, scaling=1.0, inverse=True, fused=False,
             dtype="fp16"),
        # a few drafted tokens a sequence: latency
        dict(name="ragged drafts b4", op="ragged", b=4, most=5, longest=700, hq=32, hkv=8, d=128,
             page=64, window=0, sinks=0, dtype="fp16"),
        # one prompt's next chunk in the middle of a context
        dict(name="ragged chunk 1x512", op="ragged", b=1, most=512, longest=4096, hq=32, hkv=8,
             d=128, page=64, window=0, sinks=0, dtype="bf16"),
        # a step that mixes chunks of prompts with tokens of running answers
        dict(name="ragged mixed b16", op="ragged", b=16, most=1000, longest=8000, hq=32, hkv=8,
             d=128, page=32, window=0, sinks=0, dtype="fp16"),
        # sliding window and sinks, small pages, unshared heads of 64
        dict(name="ragged window b6", op="ragged", b=6, most=2000, longest=12000, hq=16, hkv=16,
             d=64, page=16, window=1024, sinks=4, dtype="bf16"),
        # a long document's last chunk: nearly all of the flops are here
        dict(name="ragged long 2048 in 32768", op="ragged", b=1, most=2048, longest=32768, hq=32,
             hkv=8, d=128, page=128, window=0, sinks=0, dtype="bf16"),
        # one token of an answer over an encoder's states: latency, then the states' stream
        dict(name="cross step b2", op="cross", b=2, tokens=1, states=700, hq=8, hkv=8, d=64,
             dtype="fp16"),
        dict(name="cross step b48", op="cross", b=48, tokens=1, states=1500, hq=16, hkv=16, d=64,
             dtype="bf16"),
        # an answer's tokens at once, ragged states
        dict(name="cross 8x448", op="cross", b=8, tokens=448, states=1500, hq=16, hkv=16, d=64,
             dtype="fp16"),
        # long answers over long inputs, shared heads
        dict(name="cross 2x4096 on 8192", op="cross", b=2, tokens=4096, states=8192, hq=32, hkv=8,
             d=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rotary", "ragged", "ragged", "cross"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "rotary":
        tokens = _log(rng, 1, 16384)
        return dict(op=op, b=rng.randint(1, max(1, min(64, 16384 // tokens))), tokens=tokens,
                    far=_log(rng, 1, 1000000), hq=hkv * min(group, 4), hkv=hkv, d=d,
                    rot=rng.choice([d, d, d // 2, d // 4, 20]), interleaved=rng.random() < 0.5,
                    scaling=rng.choice([1.0, 4.0, 16.0]), inverse=rng.random() < 0.3,
                    fused=rng.random() < 0.5, dtype=dtype)
    if op == "ragged":
        longest = _log(rng, 1, 32768)
        # (sequences) x (heads) x (chunk) x (context) up to that of the longest listed one
        fit = 2 ** 31 // (hkv * group * longest)
        most = min(longest, _log(rng, 1, 4096), fit)
        fit //= most
        return dict(op=op, b=rng.randint(1, max(1, min(64, fit, 400000 // longest))), most=most,
                    longest=longest, hq=hkv * group, hkv=hkv, d=d,
                    page=rng.choice([16, 32, 64, 128]),
                    window=rng.choice([0, 0, _log(rng, 16, 8192)]),
                    sinks=rng.choice([0, 1, 4, 64]), dtype=dtype)
    tokens, states = _log(rng, 1, 4096), _log(rng, 1, 8192)
    group = min(group, 4)
    fit = 2 ** 31 // (hkv * group * tokens * states)
    return dict(op=op, b=rng.randint(1, max(1, min(64, fit))), tokens=tokens, states=states,
                hq=hkv * group, hkv=hkv, d=d, dtype=dtype)


def _chunks(case):
    """(length, new tokens among them) of each sequence.  The first has the longest context and
    the largest chunk; a third of the others bring one token, the rest a part of a chunk."""
    rng = random.Random(case["b"] * 1000003 + case["longest"])
    out = [(case["longest"], case["most"])]
    for _ in range(case["b"] - 1):
        n = rng.randint(max(1, int(0.2 * case["longest"])), case["longest"])
        t = 1 if rng.random() < 1 / 3 else rng.randint(max(1, case["most"] // 4), case["most"])
        out.append((n, min(n, t)))
    return out


def _states(case):
    """Number of states of each sequence: the first has all, the others 40% of them up."""
    rng = random.Random(case["b"] * 1000003 + case["states"])
    n = case["states"]
    return [n] + [rng.randint(max(1, int(0.4 * n)), n) for _ in range(case["b"] - 1)]


def _pages_of(tokens, page):
    return -(-tokens // page)


def work(case):
    d, hkv, hq = case["d"], case["hkv"], case["hq"]
    if case["op"] == "rotary":
        rows = case["b"] * case["tokens"]
        return {"bytes": rows * (4.0 * (hq + hkv) * d + 4), "flops": 3.0 * rows * (hq + hkv)
                * case["rot"]}
    if case["op"] == "ragged":
        w, s = case["window"], case["sinks"]
        seen = read = rows = 0
        for n, t in _chunks(case):
            rows += t
            if w == 0:
                seen += t * (n - t) + t * (t + 1) // 2
                read += n
            else:
                seen += sum(min(p + 1, w) + min(s, max(0, p + 1 - w)) for p in range(n - t, n))
                read += min(n, w + t - 1) + min(s, max(0, n - (w + t - 1)))
        return {"flops": 4.0 * d * hq * seen, "bytes": read * hkv * 2.0 * d + 4.0 * d * hq * rows}
    n = sum(_states(case))
    return {"flops": 4.0 * d * hq * case["tokens"] * n,
            "bytes": 4.0 * d * (hq * case["b"] * case["tokens"] + hkv * n)}


# ---------------------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _frequencies(case):
    """Radians a token of each pair, in 64 bits.  Stretched contexts: pairs that turn less than once
    within 4096 tokens are slowed down by the factor, those above 32 turns are left alone."""
    i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
    f = 10000.0 ** (-2 * i / case["rot"])
    if case["scaling"] != 1.0:
        keep = ((4096 * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        f = f * (keep + (1 - keep) / case["scaling"])
    return f


def _pool(num_pages, case, g):
    """A pool of pages as traffic leaves it: e4m3 values of N(0, 110^2) cut at 448, scales around
    2^-7 (values around 0.9)."""
    shape = (num_pages, case["hkv"], case["page"], case["d"])

    def values():
        x = torch.randn(shape, device="cuda", dtype=torch.float16, generator=g)
        return x.mul_(110).clamp_(-448, 448).to(E4M3)

    def scales():
        e = torch.randint(-8, -5, shape[:2], device="cuda", generator=g)
        return torch.pow(2.0, e.float())

    return Cache(values(), values(), scales(), scales())


def _tables(counts, width, g):
    """Each sequence's pages, drawn from the pool in no order; -1 past its last one."""
    ids = torch.randperm(sum(counts), device="cuda", generator=g).to(torch.int32)
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
    d, hq, hkv, dt = case["d"], case["hq"], case["hkv"], DTYPES[case["dtype"]]

    def rand(*shape):
        return torch.randn(shape, device="cuda", dtype=torch.float32, generator=g).to(dt)

    if case["op"] == "rotary":
        b, t = case["b"], case["tokens"]
        if case["fused"]:   # slices of one projection's output
            c["q"], c["k"], _ = rand(b, t, hq + 2 * hkv, d).split([hq, hkv, hkv], dim=2)
        else:
            c["q"], c["k"] = rand(b, t, hq, d), rand(b, t, hkv, d)
        first = torch.randint(0, case["far"] + 1, (b, 1), device="cuda", generator=g)
        c["positions"] = (first + torch.arange(t, device="cuda")).to(torch.int32)
        c["inv_freq"] = _frequencies(case)
        c["amplitude"] = 1.0 if case["scaling"] == 1.0 else 0.1 * math.log(case["scaling"]) + 1
        return c
    if case["op"] == "ragged":
        page, had = case["page"], _chunks(case)
        counts = [_pages_of(n, page) for n, _ in had]
        c["cache"] = _pool(sum(counts), case, g)
        c["pages"] = _tables(counts, max(counts), g)
        c["lengths"] = _int32([n for n, _ in had])
        starts = [0]
        for _, t in had:
            starts.append(starts[-1] + t)
        c["starts"] = _int32(starts)
        c["q"] = rand(starts[-1], hq, d) * 2
        return c
    c["q"] = rand(case["b"], case["tokens"], hq, d) * 2
    x = rand(case["b"], case["states"], 2 * hkv, d)      # one projection of the states
    c["k"], c["v"] = x.split([hkv, hkv], dim=2)
    c["lengths"] = _int32(_states(case))
    return c


# ---------------------------------------------------------------------------------- plain forms


def _plain_rotary(c):
    angle = c["positions"].double()[..., None, None] * c["inv_freq"]       # [b, t, 1, rot / 2]
    cos = (angle.cos() * c["amplitude"]).float()
    sin = (angle.sin() * (-c["amplitude"] if c["inverse"] else c["amplitude"])).float()

    def turned(x):
        y, rest = x[..., :c["rot"]].float(), x[..., c["rot"]:]
        a, b = (y[..., 0::2], y[..., 1::2]) if c["interleaved"] else y.chunk(2, -1)
        a, b = a * cos - b * sin, b * cos + a * sin
        y = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
        return torch.cat([y.to(x.dtype), rest], -1)

    return turned(c["q"]), turned(c["k"])


def _softmax(x, seen):
    """softmax over the last axis of the entries that are seen; 0 in a row that sees none."""
    x = torch.where(seen, x, float("-inf"))
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
    s = e.sum(-1, keepdim=True)
    return e / torch.where(s == 0, 1.0, s)


def _held(cache, which, pages):
    """K or V of each sequence's pages in 32 bits, in order: [b, hkv, tokens, d]."""
    values, scales = (cache.k, cache.k_scale) if which == "k" else (cache.v, cache.v_scale)
    ids = pages.long().clamp(min=0)
    x = values[ids].float() * scales[ids][..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_ragged(c):
    q, dev = c["q"].float(), c["q"].device
    rows, hq, d = q.shape
    hkv, b, t = c["hkv"], c["b"], c["most"]
    starts, n = c["starts"].long(), c["lengths"].long()
    count = starts[1:] - starts[:-1]
    i = torch.arange(t, device=dev)
    at = (starts[:-1, None] + i).clamp(max=rows - 1)                      # [b, t]
    qg = q[at].view(b, t, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    k = _held(c["cache"], "k", c["pages"])
    j = torch.arange(k.shape[2], device=dev)
    p = ((n - count)[:, None] + i)[:, None, None, :, None]                # [b, 1, 1, t, 1]
    seen = (j <= p) & (j < n[:, None, None, None, None])
    if c["window"]:
        seen = seen & ((j > p - c["window"]) | (j < c["sinks"]))
    x = (qg @ k.transpose(-1, -2)).view(b, hkv, hq // hkv, t, -1) * d ** -0.5
    del k
    x = _softmax(x, seen)
    v = _held(c["cache"], "v", c["pages"])
    v = torch.where((j < n[:, None])[:, None, :, None], v, 0.0)           # slots not written yet
    o = (x.flatten(2, 3) @ v).view(b, hkv, hq // hkv, t, d).permute(0, 3, 1, 2, 4)
    r = torch.arange(rows, device=dev)
    seq = torch.searchsorted(starts[1:].contiguous(), r, right=True)
    return o.reshape(b, t, hq, d)[seq, r - starts[seq]].to(c["q"].dtype)


def _plain_cross(c):
    q, k, v = (c[n].float() for n in ("q", "k", "v"))
    b, t, hq, d = q.shape
    hkv, group = c["hkv"], hq // c["hkv"]
    seen = torch.arange(k.shape[1], device=q.device) < c["lengths"].long()[:, None, None, None]
    qg = q.view(b, t, hkv, group, d).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [b, hkv, group t, d]
    x = _softmax((qg @ k.permute(0, 2, 3, 1)) * d ** -0.5, seen)
    o = (x @ v.permute(0, 2, 1, 3)).view(b, hkv, group, t, d).permute(0, 3, 1, 2, 4)
    return o.reshape(b, t, hq, d).to(c["q"].dtype)


def _own(c):
    import tiled_tensor_core_03_gb300 as gr
    if c["op"] == "rotary":
        return gr.rotary(c["q"], c["k"], c["positions"], c["inv_freq"],
                         interleaved=c["interleaved"], amplitude=c["amplitude"],
                         inverse=c["inverse"])
    if c["op"] == "ragged":
        return gr.kv_cache_attention_ragged(c["q"], c["cache"], c["pages"], c["lengths"],
                                            c["starts"], window=c["window"], sinks=c["sinks"])
    return gr.flash_attention_cross(c["q"], c["k"], c["v"], c["lengths"])


def run(state):
    if own:
        return _own(state)
    return {"rotary": _plain_rotary, "ragged": _plain_ragged, "cross": _plain_cross}[
        state["op"]](state)


# ---------------------------------------------------------------------------------- 64 bits


def exact(case, seed):
    """The definitions in 64 bits, one sequence and head at a time."""
    if work(case)["flops"] > 8e12:
        return None
    return {"rotary": _exact_rotary, "ragged": _exact_ragged, "cross": _exact_cross}[case["op"]](
        prepare(case, seed))


def _exact_rotary(c):
    """Each pair as a complex number, multiplied by amplitude e^(+-i angle)."""
    sign = -1.0 if c["inverse"] else 1.0
    angle = sign * c["positions"].double()[:, :, None, None] * c["inv_freq"]
    turn = torch.polar(torch.full_like(angle, c["amplitude"]), angle)
    half, out = c["rot"] // 2, []
    for x in (c["q"], c["k"]):
        y = x.double().clone()
        re, im = ((slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["interleaved"]
                  else (slice(0, half), slice(half, c["rot"])))
        z = torch.complex(y[..., re].contiguous(), y[..., im].contiguous()) * turn
        y[..., re], y[..., im] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_attend(q, k, v, see):
    """q [t, d], k and v [n, d], see [t, n] or None (all)."""
    x = q.double() @ k.double().T / q.shape[1] ** 0.5
    if see is not None:
        x = x.masked_fill(~see, float("-inf"))
    return torch.softmax(x, -1) @ v.double()


def _exact_ragged(c):
    q, out = c["q"], torch.empty(c["q"].shape, dtype=torch.float64, device=c["q"].device)
    group, at = c["hq"] // c["hkv"], 0
    for i, (n, t) in enumerate(_chunks(c)):
        ids = c["pages"][i, :_pages_of(n, c["page"])].long()
        k, v = ((x[ids].double() * s[ids].double()[..., None, None]).transpose(1, 2)
                .flatten(0, 1)[:n] for x, s in ((c["cache"].k, c["cache"].k_scale),
                                                (c["cache"].v, c["cache"].v_scale)))
        j = torch.arange(n, device=q.device)
        for lo in range(0, t, 1024):
            rows = torch.arange(lo, min(t, lo + 1024), device=q.device)
            p = (n - t + rows)[:, None]
            see = j <= p
            if c["window"]:
                see &= (j > p - c["window"]) | (j < c["sinks"])
            for h in range(c["hq"]):
                out[at + rows, h] = _exact_attend(q[at + rows, h], k[:, h // group],
                                                  v[:, h // group], see)
        at += t
    return out


def _exact_cross(c):
    q, out = c["q"], torch.empty(c["q"].shape, dtype=torch.float64, device=c["q"].device)
    group = c["hq"] // c["hkv"]
    for i, n in enumerate(_states(c)):
        for h in range(c["hq"]):
            out[i, :, h] = _exact_attend(q[i, :, h], c["k"][i, :n, h // group],
                                         c["v"][i, :n, h // group], None)
    return out
