"""Operators of a serving loop: torch front end of include/kv_cache.h (a paged K/V cache
held in 8 bits), of flash_attention_window and flash_attention_cross in include/flash_attention.h
and of include/rotary.h (rotary positions).

The cache is a tuple (k, v, k_scale, v_scale): e4m3 values
[num_pages, kv_heads, page, head_dim] and fp32 scales [num_pages, kv_heads].
Tensors are checked and marshalled by the extension _serving (csrc/serving_binding.cpp); all
arithmetic runs in the library's kernels.  Calls are asynchronous on `stream` (default:
torch's current stream) and allocate their outputs and workspaces on it.
"""
import ctypes
import math
from typing import NamedTuple

import torch

from . import GemmReluError, lib

try:
    from . import _serving
except ImportError as e:
    raise ImportError("the extension _serving is missing or does not fit this torch; build it "
                      "with `python -c 'import __graft_entry__ as g; g.build()'`") from e

_HEAD_DIMS = (64, 128)
_PAGES = (16, 32, 64, 128)

_serving.bind(GemmReluError, torch.OutOfMemoryError, *(
    ctypes.cast(getattr(lib(), name), ctypes.c_void_p).value
    for name in ("flash_attention_window_x16", "kv_cache_append_x16", "kv_cache_attention_x16",
                 "kv_cache_attention_x16_workspace_bytes", "kv_cache_evict_e4m3",
                 "gemm_relu_stream_capturing", "gemm_relu_stream_id", "flash_attention_cross_x16",
                 "kv_cache_attention_ragged_x16", "kv_cache_attention_ragged_x16_workspace_bytes",
                 "rotary_x16", "flash_attention_cross_x16_workspace_bytes")))


class KVCache(NamedTuple):
    """The pool: value of a token's element = k (or v) * its page's and head's scale."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    @classmethod
    def empty(cls, num_pages, kv_heads, head_dim, page=64, device="cuda"):
        """A pool of pages of `page` (16, 32, 64 or 128) tokens; nothing needs initialising."""
        if head_dim not in _HEAD_DIMS or page not in _PAGES:
            raise ValueError(f"head_dim must be one of {_HEAD_DIMS}, page one of {_PAGES}")
        values = [torch.empty((num_pages, kv_heads, page, head_dim), dtype=torch.float8_e4m3fn,
                              device=device) for _ in range(2)]
        scales = [torch.ones((num_pages, kv_heads), dtype=torch.float32, device=device)
                  for _ in range(2)]
        return cls(*values, *scales)


def flash_attention_window(q, k, v, window, sinks=0, out=None, stream=None):
    """softmax(q k^T / sqrt(d)) v of a prompt with a sliding window: q [batch, q_seq, q_heads, d],
    k and v [batch, kv_seq, kv_heads, d], fp16 or bf16, d = 64 or 128; query head h reads K/V
    head h // (q_heads // kv_heads).  Strides between heads are positive multiples of 8 elements:
    an expanded axis (stride 0) is refused with GemmReluError.

    Query i stands at p = i + kv_seq - q_seq and sees the keys j <= p; with a window > 0
    only those with j > p - window or j < sinks.  A query that sees nothing gets 0."""
    if stream is not None:
        with torch.cuda.stream(stream):   # what is allocated belongs to it
            return _serving.window(q, k, v, window, sinks, out)
    return _serving.window(q, k, v, window, sinks, out)


def flash_attention_cross_workspace(q, k):
    """A device workspace for flash_attention_cross calls of these sizes (uint8 tensor, its counters
    zeroed on the current stream); for calls that follow one another."""
    return _serving.cross_workspace(q, k)


def flash_attention_cross(q, k, v, lengths=None, out=None, workspace=None, stream=None):
    """softmax(q k^T / sqrt(d)) v over an encoder's states: q [batch, q_seq, q_heads, d], k and v
    [batch, kv_seq, kv_heads, d], fp16 or bf16, d = 64 or 128; query head h reads K/V head
    h // (q_heads // kv_heads).  Strides as for flash_attention_window.

    Every query of sequence b sees the states j < lengths[b] (int32 [batch]; default: all kv_seq).
    Where there are none it gets 0.  What stands behind them, NaN among it, is not seen; with more than 16
    query rows a K/V head, padding that is not finite takes two to three times as long as finite.

    A call of few query rows and heads needs a workspace: without one it uses one that is kept per
    stream, or its own where it is being captured."""
    if stream is not None:
        with torch.cuda.stream(stream):   # what is allocated belongs to it
            return _serving.cross(q, k, v, lengths, out, workspace)
    return _serving.cross(q, k, v, lengths, out, workspace)


def rotary_frequencies(rot, base=10000.0, factor=1.0, context=None, low=1.0, high=32.0, device="cuda"):
    """Radians a token of each of rot / 2 pairs, for rotary(): float64 [rot / 2], base^(-2 i / rot).

    With a factor > 1 (a context stretched by it): without `context` every frequency is divided by it.
    With `context`, the tokens that the model was trained on, a pair that makes at most `low` turns within
    them is divided by it, one that makes at least `high` is left alone, and in between the two are mixed in
    proportion to its turns."""
    if rot < 2 or rot % 2 or not base > 0 or not factor >= 1 or not low < high:
        raise ValueError("need an even rot >= 2, base > 0, factor >= 1 and low < high")
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    f = float(base) ** (-2 * i / rot)
    if factor == 1:
        return f
    if context is None:
        return f / factor
    keep = ((context * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
    return f * (keep + (1 - keep) / factor)


def rotary(q, k, positions, inv_freq, interleaved=False, amplitude=1.0, inverse=False, out=None,
           stream=None):
    """Rotary positions: q [batch, tokens, q_heads, d] and k [batch, tokens, kv_heads, d] (or both
    [rows, heads, d]; k may be None), fp16 or bf16, d a multiple of 8 up to 512, turned by
    t = positions * inv_freq.  Returns (q, k).

    positions int32 or int64 [batch, tokens] (or [rows]); inv_freq float32 or float64 [rot / 2], as
    rotary_frequencies makes them.  The first rot elements of a head turn in pairs (p, p + rot / 2), or
    `interleaved` (2p, 2p + 1), and are multiplied by `amplitude`; the others are copied.  With `inverse`
    they turn back: rotary(dq, dk, ..., inverse=True) is the gradient with respect to the inputs.  A rot that is
    no multiple of 16 takes about three times as long.

    Heads are contiguous and start on 16-byte boundaries; other strides are free.  `out`: a tuple of
    tensors for the results, which may be q and k themselves; other overlaps are not checked."""
    if stream is not None:
        with torch.cuda.stream(stream):   # what is allocated belongs to it
            return _serving.rotary(q, k, positions, inv_freq, interleaved, amplitude, inverse, out)
    return _serving.rotary(q, k, positions, inv_freq, interleaved, amplitude, inverse, out)


def kv_cache_append(cache, k, v, pages, lengths, counts=None, stream=None):
    """Write new tokens' k and v (fp16 or bf16 [batch, tokens, kv_heads, head_dim], strides
    between heads any multiples of 8, 0 among them) into their sequences' pages.

    pages int32 [batch, max_pages]; lengths int32 [batch] INCLUDES the new tokens;
    counts int32 [batch] says how many of the `tokens` rows are new ones (default: all):
    row i becomes token lengths - counts + i."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _serving.append(cache, k, v, pages, lengths, counts)
    return _serving.append(cache, k, v, pages, lengths, counts)


def kv_cache_attention_workspace(q, cache, weights=None):
    """A device workspace for kv_cache_attention calls of these sizes (uint8 tensor, its
    counters zeroed on the current stream); for calls that follow one another."""
    return _serving.workspace(q, cache, weights)


def kv_cache_attention(q, cache, pages, lengths, window=0, sinks=0, weights=None, out=None,
                       workspace=None, stream=None):
    """softmax(q K^T / sqrt(head_dim)) V of the last tokens of every sequence over the cache:
    q fp16 or bf16 [batch, tokens, q_heads, head_dim] (strides between heads any
    multiples of 8), query head h reading K/V head h // (q_heads // kv_heads).

    lengths int32 [batch] includes these tokens; token i sees the tokens t <= p = length -
    tokens + i, with a window > 0 only those with t > p - window or t < sinks (pages that
    no query sees a token of may have been given up: their numbers are not read).  With
    `weights` (fp32 [batch, kv_heads, at least max_pages * page]) each token's softmax
    weights, summed over the query tokens and heads of its group, are added to it.

    Without a `workspace` the call uses one that is kept per stream (up to 64 MB, for up to 64
    streams), or its own where it needs more or is being captured."""
    if stream is not None:
        with torch.cuda.stream(stream):   # what is allocated belongs to it
            return _serving.attention(cache, q, pages, lengths, window, sinks, weights, out,
                                      workspace)
    return _serving.attention(cache, q, pages, lengths, window, sinks, weights, out, workspace)


def kv_cache_attention_ragged_workspace(cache):
    """A device workspace for kv_cache_attention_ragged calls of any sizes on this cache (uint8 tensor,
    its counters zeroed on the current stream); for calls that follow one another."""
    return _serving.ragged_workspace(cache[0])


def kv_cache_attention_ragged(q, cache, pages, lengths, starts, window=0, sinks=0, out=None,
                              workspace=None, stream=None):
    """kv_cache_attention for sequences that bring different numbers of tokens, as when chunks of prompts,
    drafts and single tokens share a step: q fp16 or bf16 [rows, q_heads, head_dim], strides any
    multiples of 8.

    starts int32 [batch + 1], ascending: sequence b's query tokens are the rows starts[b] ..
    starts[b + 1] - 1, the last of its lengths[b] tokens (pages int32 [batch, max_pages]), all of which
    have been appended.  What a token sees is kv_cache_attention's.  Rows that belong to no sequence
    are not written.  Without a `workspace` the call uses one that is kept per stream (about 40 MB), or
    its own where it is being captured."""
    if stream is not None:
        with torch.cuda.stream(stream):   # what is allocated belongs to it
            return _serving.ragged(cache, q, pages, lengths, starts, window, sinks, out, workspace)
    return _serving.ragged(cache, q, pages, lengths, starts, window, sinks, out, workspace)


def kv_cache_evict(cache, weights, pages, lengths, budget, sinks, recent, to, to_pages,
                   stream=None):
    """Keep `budget` tokens of every sequence and head: the first `sinks`, the last
    `recent` and the heaviest others by `weights` (fp32 [batch, kv_heads, at least
    max_pages * page]; ties go to the earlier token), moved in order into the pages
    to_pages (int32 [batch, to_max_pages]) of the pool `to` (may be `cache`; pages that
    no sequence uses).

    Returns (lengths int32 [batch], weights fp32 [batch, kv_heads, to_max_pages * page],
    kept int32 [batch, kv_heads, budget]: former positions, -1 past the length)."""
    if stream is not None:
        with torch.cuda.stream(stream):   # what is allocated belongs to it
            return _serving.evict(cache, weights, pages, lengths, budget, sinks, recent, to,
                                  to_pages)
    return _serving.evict(cache, weights, pages, lengths, budget, sinks, recent, to, to_pages)
