"""The serving operators together, as a model's attention layer uses them to answer.

    python examples/serving_loop.py [--prompt 2000] [--steps 64] [--batch 4] [--budget 512]

One attention layer with shared K/V heads, random weights:

  1. the prompts: projections, windowed attention with sinks, K and V into the paged 8-bit cache;
  2. the last queries look over the whole cache once and leave their attention weights;
  3. the cache is cut down to `budget` tokens a head by those weights, the old pages are free;
  4. a loop of single tokens: append, attend (and go on adding weights), captured in a CUDA graph.

Every step's result feeds the next one through the output projection.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tiled_tensor_core_03_gb300 as gr  # noqa: E402


class Layer:
    """x -> x + attention(x): one fused q, k, v projection and an output projection."""

    def __init__(self, width, q_heads, kv_heads, dim, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.split = [q_heads, kv_heads, kv_heads]
        self.heads, self.dim = q_heads, dim

        def weight(a, b):
            return (torch.randn(a, b, device="cuda", generator=g) / a ** 0.5).to(dtype)
        self.qkv = weight(width, (q_heads + 2 * kv_heads) * dim)
        self.out = weight(q_heads * dim, width)

    def project(self, x):
        """[batch, tokens, width] -> q, k, v as slices of one tensor (no copies)."""
        y = (x @ self.qkv).view(*x.shape[:2], sum(self.split), self.dim)
        return y.split(self.split, dim=2)

    def join(self, x, o):
        return x + o.flatten(2) @ self.out


def serve(batch=4, prompt=2000, steps=64, budget=512, window=256, sinks=4, recent=64, page=64,
          q_heads=16, kv_heads=4, dim=128, dtype=torch.bfloat16, width=1024, seed=0, graph=True):
    """Returns (prompt output, the steps' outputs, lengths, the tokens kept by the eviction)."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    layer = Layer(width, q_heads, kv_heads, dim, dtype, seed)
    lengths = torch.tensor([max(1, prompt - 100 * i) for i in range(batch)], dtype=torch.int32,
                           device="cuda")
    prompt_pages = -(-prompt // page)
    kept_pages = -(-(budget + steps) // page)
    cache = gr.KVCache.empty(batch * (prompt_pages + kept_pages), kv_heads, dim, page)

    # 1. the prompts, padded on the right: padding comes after what a query sees
    x = torch.randn(batch, prompt, width, device="cuda", generator=g).to(dtype)
    q, k, v = layer.project(x)
    o = gr.flash_attention_window(q, k, v, window, sinks)
    pages = torch.arange(batch * prompt_pages, dtype=torch.int32, device="cuda").view(batch, -1)
    gr.kv_cache_append(cache, k, v, pages, lengths, counts=lengths)
    first = layer.join(x, o)

    # 2. the last 8 queries of each prompt leave their weights
    weights = torch.zeros(batch, kv_heads, prompt_pages * page, device="cuda")
    last = lengths.long()[:, None] - 8 + torch.arange(8, device="cuda")
    tail = q[torch.arange(batch, device="cuda")[:, None], last.clamp(min=0)].contiguous()
    gr.kv_cache_attention(tail, cache, pages, lengths, weights=weights)

    # 3. cut down; the table is wide enough for the steps to come
    to_pages = (batch * prompt_pages
                + torch.arange(batch * kept_pages, dtype=torch.int32, device="cuda")).view(batch, -1)
    lengths, weights, kept = gr.kv_cache_evict(cache, weights, pages, lengths, budget, sinks,
                                               recent, cache, to_pages)

    # 4. single tokens; every tensor of a step stays where it is, so a graph can replay it
    token = first[torch.arange(batch, device="cuda"), last[:, -1].clamp(min=0)][:, None].contiguous()
    workspace = gr.kv_cache_attention_workspace(layer.project(token)[0].contiguous(), cache, weights)

    def step():
        lengths.add_(1)
        q1, k1, v1 = layer.project(token)
        gr.kv_cache_append(cache, k1, v1, to_pages, lengths)
        o1 = gr.kv_cache_attention(q1, cache, to_pages, lengths, weights=weights,
                                   workspace=workspace)
        y = layer.join(token, o1)
        token.copy_(y / y.float().norm(dim=-1, keepdim=True).to(dtype) * width ** 0.5)

    replay = step
    if graph:
        held = [t.clone() for t in (token, lengths, weights, *cache)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()                                   # what torch sets up on first use
        torch.cuda.current_stream().wait_stream(side)
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        for t, h in zip((token, lengths, weights, *cache), held):
            t.copy_(h)
        replay = captured.replay
    outputs = []
    for _ in range(steps):
        replay()
        outputs.append(token.clone())
    if gr.status() != gr.OK:
        raise RuntimeError("a device-side check failed")
    return first, torch.stack(outputs), lengths, kept


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("batch", 4), ("prompt", 2000), ("steps", 64), ("budget", 512)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    serve(a.batch, a.prompt, a.steps, a.budget)      # first use: libraries, allocator
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    _, outputs, lengths, kept = serve(a.batch, a.prompt, a.steps, a.budget)
    stop.record()
    stop.synchronize()
    print(f"{a.batch} prompts of up to {a.prompt} tokens cut to {kept.shape[2]} a head, "
          f"{a.steps} steps: lengths {lengths.tolist()}, {start.elapsed_time(stop):.1f} ms in all, "
          f"outputs finite: {bool(torch.isfinite(outputs).all())}")


if __name__ == "__main__":
    main()
