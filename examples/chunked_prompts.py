"""Prompts in chunks and running answers in the same steps, with an encoder's states beside them.

    python examples/chunked_prompts.py [--requests 6] [--budget 256] [--steps 24]

One decoder layer with random weights: self-attention with rotary positions over the paged 8-bit cache, then
cross attention to each request's encoder states.  Every step has room for `budget` tokens: a
request that is answering brings one, and what is left goes to the next chunks of prompts.  A step:

  1. one projection of all rows; q and k turned to their positions, in place (rotary);
  2. k and v into the requests' pages (kv_cache_append);
  3. attention of every row over its request's pages (kv_cache_attention_ragged);
  4. attention of the requests' last rows to their encoder states (flash_attention_cross), and the next
     token of those whose prompt is done.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tiled_tensor_core_03_gb300 as gr  # noqa: E402


class Layer:
    def __init__(self, width, q_heads, kv_heads, dim, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.split, self.dim = [q_heads, kv_heads, kv_heads], dim

        def weight(a, b):
            return (torch.randn(a, b, device="cuda", generator=g) / a ** 0.5).to(dtype)
        self.qkv, self.out = weight(width, sum(self.split) * dim), weight(q_heads * dim, width)
        self.q, self.kv = weight(width, q_heads * dim), weight(width, 2 * kv_heads * dim)
        self.join = weight(q_heads * dim, width)

    def project(self, x):
        """[rows, width] -> q, k, v as slices of one tensor (no copies)."""
        return (x @ self.qkv).view(x.shape[0], -1, self.dim).split(self.split, dim=1)

    def states(self, x):
        """K and V of encoder states [requests, states, width], as slices of one tensor."""
        return (x @ self.kv).view(*x.shape[:2], -1, self.dim).split(self.split[1:], dim=2)


def serve(prompts=(500, 37, 260, 801, 64, 130), states=(300, 150, 75, 280, 10, 222), budget=256, steps=24, page=32,
          q_heads=8, kv_heads=2, dim=64, width=256, dtype=torch.bfloat16, seed=0):
    """Returns the rows after the layer of every request's last prompt token and of its answer's tokens,
    and the steps that it took."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    layer = Layer(width, q_heads, kv_heads, dim, dtype, seed)
    n = len(prompts)
    tokens = [torch.randn(p, width, device="cuda", generator=g).to(dtype) for p in prompts]
    encoded = torch.randn(n, max(states), width, device="cuda", generator=g).to(dtype)
    sk, sv = layer.states(encoded)
    state_lengths = torch.tensor(states, dtype=torch.int32, device="cuda")
    most = -(-(max(prompts) + steps) // page)
    cache = gr.KVCache.empty(n * most, kv_heads, dim, page)
    pages = torch.randperm(n * most, device="cuda", generator=g).to(torch.int32).view(n, most)
    inv_freq = gr.rotary_frequencies(dim, factor=4.0, context=4096)
    workspace = gr.kv_cache_attention_ragged_workspace(cache)
    had, answers, taken = [0] * n, [[] for _ in range(n)], 0
    while any(len(a) < steps for a in answers):
        # what each request brings: the tokens of an answer first
        counts, left = [0] * n, budget
        for i in sorted(range(n), key=lambda i: had[i] < prompts[i]):
            if len(answers[i]) < steps:
                counts[i] = min(left, len(tokens[i]))
                left -= counts[i]
        ends = torch.tensor(counts).cumsum(0).tolist()
        starts = torch.tensor([0] + ends, dtype=torch.int32, device="cuda")
        had = [a + c for a, c in zip(had, counts)]
        lengths = torch.tensor(had, dtype=torch.int32, device="cuda")
        x = torch.cat([t[:c] for t, c in zip(tokens, counts)])
        positions = torch.cat([torch.arange(a - c, a, device="cuda") for a, c in zip(had, counts)])
        # 1. and 2.
        q, k, v = layer.project(x)
        gr.rotary(q, k, positions, inv_freq, out=(q, k))
        rows = (starts[:-1, None] + torch.arange(max(counts), device="cuda")).clamp(max=len(x) - 1)
        gr.kv_cache_append(cache, k[rows], v[rows], pages, lengths, torch.tensor(counts, dtype=torch.int32, device="cuda"))
        # 3.
        o = gr.kv_cache_attention_ragged(q, cache, pages, lengths, starts, workspace=workspace)
        x = x + o.flatten(1) @ layer.out
        # 4.
        last = x[(starts[1:] - 1).clamp(min=0)]
        y = gr.flash_attention_cross((last @ layer.q).view(n, 1, q_heads, dim), sk, sv, state_lengths)
        y = last + y.flatten(1) @ layer.join
        y = y / y.float().norm(dim=-1, keepdim=True).to(dtype) * width ** 0.5
        for i, c in enumerate(counts):
            tokens[i] = tokens[i][c:]
            if c and had[i] >= prompts[i]:
                answers[i].append(y[i])
                tokens[i] = y[i:i + 1]
        taken += 1
    if gr.status() != gr.OK:
        raise RuntimeError("a device-side check failed")
    return torch.stack([torch.stack(a) for a in answers]), taken


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("requests", 6), ("budget", 256), ("steps", 24)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    g = torch.Generator().manual_seed(2)
    kw = dict(prompts=torch.randint(1, 1000, (a.requests,), generator=g).tolist(),
              states=torch.randint(1, 400, (a.requests,), generator=g).tolist(), budget=a.budget, steps=a.steps)
    serve(**kw)                                  # first use: libraries, allocator
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    answers, taken = serve(**kw)
    stop.record()
    stop.synchronize()
    print(f"prompts of {kw['prompts']} tokens and {a.steps} tokens each in {taken} steps of up to {a.budget} tokens: "
          f"{start.elapsed_time(stop):.1f} ms in all, answers finite: {bool(torch.isfinite(answers).all())}")


if __name__ == "__main__":
    main()
