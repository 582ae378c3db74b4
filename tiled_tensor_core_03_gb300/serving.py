"""Operators of a serving loop: torch front end of include/kv_cache.h (a paged K/V cache
held in 8 bits) and of flash_attention_window in include/flash_attention.h.

The cache is a tuple (k, v, k_scale, v_scale): e4m3 values
[num_pages, kv_heads, page, head_dim] and fp32 scales [num_pages, kv_heads].
The functions check and marshal tensors; all arithmetic runs in the library's
kernels.  Calls are asynchronous on `stream` (default: torch's current stream)
and allocate their outputs and workspaces on it.
"""
import ctypes
from typing import NamedTuple

import torch

from . import OK, F16, BF16, KV_COUNTER_BYTES, GemmReluError, lib

_DTYPES = {torch.float16: F16, torch.bfloat16: BF16}
_VALUES = (torch.float8_e4m3fn, torch.uint8)
_HEAD_DIMS = (64, 128)
_PAGES = (16, 32, 64, 128)


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


class Pool(ctypes.Structure):
    """kv_cache_pool of the C ABI."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("kv_heads", ctypes.c_int64), ("page", ctypes.c_int64),
                ("head_dim", ctypes.c_int64)]


Strides = ctypes.c_int64 * 3


# The checks below run before every launch of a few microseconds, so each asks a
# tensor as few questions as it can.

def _device(t):
    """The current device's number, which t (and every other tensor) must be on."""
    d = t.get_device()
    if d < 0 or d != torch.cuda.current_device():
        raise ValueError("tensors must be on the current CUDA device")
    return d


def _pool(cache, d):
    """(Pool, shape) of a cache on device d."""
    k, v, ks, vs = cache
    shape = k.shape
    if len(shape) != 4 or v.shape != shape or k.dtype not in _VALUES or v.dtype != k.dtype \
            or not k.is_contiguous() or not v.is_contiguous():
        raise ValueError("cache k and v must be contiguous e4m3 tensors of one shape "
                         "[num_pages, kv_heads, page, head_dim]")
    pages, heads, page, dim = shape
    if dim not in _HEAD_DIMS or page not in _PAGES:
        raise ValueError(f"head_dim must be one of {_HEAD_DIMS}, page one of {_PAGES}: "
                         f"got {tuple(shape)}")
    shape2 = ks.shape
    if shape2 != (pages, heads) or vs.shape != shape2 or ks.dtype is not torch.float32 \
            or vs.dtype is not torch.float32 or not ks.is_contiguous() or not vs.is_contiguous():
        raise ValueError("cache scales must be contiguous float32 [num_pages, kv_heads]")
    if not d == k.get_device() == v.get_device() == ks.get_device() == vs.get_device():
        raise ValueError(f"the cache must be on cuda:{d}")
    return Pool(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), pages, heads, page,
                dim), shape


def _ints(t, shape, name, d):
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous() or t.get_device() != d:
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} "
                         f"on cuda:{d}")
    return t.data_ptr()


def _table(pages, batch, name, d):
    """(pointer, max_pages) of a page table."""
    if pages.dim() != 2:
        raise ValueError(f"{name} must be int32 [batch, max_pages]")
    width = pages.shape[1]
    return _ints(pages, (batch, width), name, d), width


def _strides(t, name):
    """(pointer, {batch, token, head} strides) of a 16-bit [batch, tokens, heads, head_dim]
    tensor whose heads start on 16-byte boundaries."""
    p = t.data_ptr()
    a, b, c, e = t.stride()
    if e != 1 or (a | b | c | p >> 1) & 7:
        # an axis of one element is never stepped over
        a, b, c = (0 if n == 1 else x for n, x in zip(t.shape, (a, b, c)))
        if e != 1 or (a | b | c | p >> 1) & 7:
            raise ValueError(f"{name}: heads must be contiguous and start on 16-byte boundaries "
                             f"(strides {t.stride()}, address {p:#x})")
    return p, Strides(a, b, c)


def _current(d):
    return torch._C._cuda_getCurrentRawStream(d)   # current_stream().cuda_stream, directly


def flash_attention_window(q, k, v, window, sinks=0, out=None, stream=None):
    """softmax(q k^T / sqrt(d)) v of a prompt with a sliding window: q [batch, q_seq, q_heads, d],
    k and v [batch, kv_seq, kv_heads, d], fp16 or bf16, any strides between heads, d = 64 or
    128; query head h reads K/V head h // (q_heads // kv_heads).

    Query i stands at p = i + kv_seq - q_seq and sees the keys j <= p; with a window > 0
    only those with j > p - window or j < sinks.  A query that sees nothing gets 0."""
    d = _device(q)
    dtype = _DTYPES.get(q.dtype)
    if dtype is None or k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must all be float16 or all bfloat16")
    shape, kv_shape = q.shape, k.shape
    if len(shape) != 4 or len(kv_shape) != 4 or v.shape != kv_shape or k.get_device() != d \
            or v.get_device() != d:
        raise ValueError("q must be [batch, q_seq, q_heads, d], k and v [batch, kv_seq, "
                         "kv_heads, d], all on one device")
    batch, q_seq, q_heads, dim = shape
    _, kv_seq, kv_heads, _ = kv_shape
    if kv_shape[0] != batch or kv_shape[3] != dim or dim not in _HEAD_DIMS or kv_heads == 0 \
            or q_heads % kv_heads:
        raise ValueError(f"shapes {tuple(shape)} and {tuple(kv_shape)} do not go together")
    if window < 0 or sinks < 0:
        raise ValueError("window and sinks must not be negative")
    if out is not None and (out.shape != shape or out.dtype != q.dtype or out.get_device() != d
                            or not out.is_contiguous()):
        raise ValueError("out must be a contiguous tensor like q")
    if stream is not None:
        with torch.cuda.stream(stream):   # what is allocated belongs to it
            return flash_attention_window(q, k, v, window, sinks, out)
    if out is None:
        out = q.new_empty(shape)
    if q.numel() == 0:
        return out
    qp, qs = _strides(q, "q")
    kp, ks = _strides(k, "k")
    vp, vs = _strides(v, "v")
    rc = lib().flash_attention_window_x16(qp, kp, vp, out.data_ptr(), dtype, batch, q_seq, kv_seq,
                                          q_heads, kv_heads, dim, qs, ks, vs, window, sinks,
                                          _current(d))
    if rc != OK:
        raise GemmReluError(rc, "flash_attention_window_x16")
    return out


def kv_cache_append(cache, k, v, pages, lengths, counts=None, stream=None):
    """Write new tokens' k and v (fp16 or bf16 [batch, tokens, kv_heads, head_dim], any
    strides between heads) into their sequences' pages.

    pages int32 [batch, max_pages]; lengths int32 [batch] INCLUDES the new tokens;
    counts int32 [batch] says how many of the `tokens` rows are new ones (default: all):
    row i becomes token lengths - counts + i."""
    d = _device(k)
    dtype = _DTYPES.get(k.dtype)
    if dtype is None or v.dtype != k.dtype:
        raise TypeError("k and v must both be float16 or both bfloat16")
    shape = k.shape
    if len(shape) != 4 or v.shape != shape or v.get_device() != d:
        raise ValueError("k and v must have the same shape [batch, tokens, kv_heads, head_dim]")
    pool, held = _pool(cache, d)
    batch, tokens, heads, dim = shape
    if heads != held[1] or dim != held[3]:
        raise ValueError(f"k has {heads} heads of {dim}, the cache {held[1]} of {held[3]}")
    table, width = _table(pages, batch, "pages", d)
    lens = _ints(lengths, (batch,), "lengths", d)
    new = None if counts is None else _ints(counts, (batch,), "counts", d)
    if batch == 0 or tokens == 0:
        return
    kp, ks = _strides(k, "k")
    vp, vs = _strides(v, "v")
    rc = lib().kv_cache_append_x16(ctypes.byref(pool), kp, vp, dtype, batch, tokens, ks, vs, table,
                                   width, lens, new,
                                   _current(d) if stream is None else stream.cuda_stream)
    if rc != OK:
        raise GemmReluError(rc, "kv_cache_append_x16")


def kv_cache_attention_workspace(q, cache, weights=None):
    """A device workspace for kv_cache_attention calls of these sizes (uint8 tensor, its
    counters zeroed on the current stream); for calls that follow one another."""
    batch, tokens, heads, dim = q.shape
    n = lib().kv_cache_attention_x16_workspace_bytes(
        batch, tokens, heads, cache[0].shape[1], dim, 0 if weights is None else weights.shape[2])
    w = torch.empty(max(n, KV_COUNTER_BYTES), dtype=torch.uint8, device=q.device)
    w[:KV_COUNTER_BYTES].zero_()
    return w


# Workspaces of calls that bring none and collect no weights (a few MB whose size depends
# on head_dim alone), one per device, stream and head_dim: calls on a stream follow one
# another.  Calls being captured get their own, since their graph may run anywhere.
_workspaces = {}


def _workspace(q, cache, weights, s):
    if weights is not None or torch.cuda.is_current_stream_capturing():
        return kv_cache_attention_workspace(q, cache, weights)
    key = (q.get_device(), s, q.shape[3])
    w = _workspaces.get(key)
    if w is None:
        w = _workspaces[key] = kv_cache_attention_workspace(q, cache)
    return w


def kv_cache_attention(q, cache, pages, lengths, window=0, sinks=0, weights=None, out=None,
                       workspace=None, stream=None):
    """softmax(q K^T / sqrt(head_dim)) V of the last tokens of every sequence over the cache:
    q fp16 or bf16 [batch, tokens, q_heads, head_dim] (any strides between heads), query
    head h reading K/V head h // (q_heads // kv_heads).

    lengths int32 [batch] includes these tokens; token i sees the tokens t <= p = length -
    tokens + i, with a window > 0 only those with t > p - window or t < sinks.  With
    `weights` (fp32 [batch, kv_heads, at least max_pages * page]) each token's softmax
    weights, summed over the query tokens and heads of its group, are added to it."""
    d = _device(q)
    dtype = _DTYPES.get(q.dtype)
    if dtype is None:
        raise TypeError("q must be float16 or bfloat16")
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be [batch, tokens, q_heads, head_dim]")
    pool, held = _pool(cache, d)
    batch, tokens, heads, dim = shape
    if dim != held[3] or heads % held[1] or heads == 0:
        raise ValueError(f"q has {heads} heads of {dim}, the cache {held[1]} of {held[3]}")
    if window < 0 or sinks < 0:
        raise ValueError("window and sinks must not be negative")
    table, max_pages = _table(pages, batch, "pages", d)
    lens = _ints(lengths, (batch,), "lengths", d)
    width, wp = 0, None
    if weights is not None:
        if weights.dtype != torch.float32 or weights.dim() != 3 or not weights.is_contiguous() \
                or weights.shape[:2] != (batch, held[1]) or weights.get_device() != d \
                or weights.shape[2] < max_pages * held[2]:
            raise ValueError("weights must be contiguous float32 [batch, kv_heads, at least "
                             f"{max_pages * held[2]}] on cuda:{d}")
        width, wp = weights.shape[2], weights.data_ptr()
    if out is not None and (out.shape != shape or out.dtype != q.dtype or out.get_device() != d
                            or not out.is_contiguous()):
        raise ValueError("out must be a contiguous tensor like q")
    if stream is not None:
        with torch.cuda.stream(stream):   # what is allocated belongs to it
            return kv_cache_attention(q, cache, pages, lengths, window, sinks, weights, out,
                                      workspace)
    if out is None:
        out = q.new_empty(shape)
    if batch == 0 or tokens == 0:
        return out
    qp, qs = _strides(q, "q")
    s = _current(d)
    w = _workspace(q, cache, weights, s) if workspace is None else workspace
    rc = lib().kv_cache_attention_x16(ctypes.byref(pool), qp, dtype, batch, tokens, heads, qs,
                                      out.data_ptr(), table, max_pages, lens, window, sinks, wp,
                                      width, w.data_ptr(), w.nbytes, s)
    if rc != OK:
        raise GemmReluError(rc, "kv_cache_attention_x16")
    return out


def kv_cache_evict(cache, weights, pages, lengths, budget, sinks, recent, to, to_pages,
                   stream=None):
    """Keep `budget` tokens of every sequence and head: the first `sinks`, the last
    `recent` and the heaviest others by `weights` (fp32 [batch, kv_heads, at least
    max_pages * page]; ties go to the earlier token), moved in order into the pages
    to_pages (int32 [batch, to_max_pages]) of the pool `to` (may be `cache`; pages that
    no sequence uses).

    Returns (lengths int32 [batch], weights fp32 [batch, kv_heads, to_max_pages * page],
    kept int32 [batch, kv_heads, budget]: former positions, -1 past the length)."""
    d = _device(weights)
    pool, held = _pool(cache, d)
    dest, to_held = _pool(to, d)
    if held[1:] != to_held[1:]:
        raise ValueError("both pools must have the same kv_heads, page and head_dim")
    if weights.dim() != 3 or weights.dtype != torch.float32 or not weights.is_contiguous() \
            or weights.shape[1] != held[1]:
        raise ValueError("weights must be contiguous float32 [batch, kv_heads, tokens]")
    batch, heads, width = weights.shape
    page = held[2]
    table, max_pages = _table(pages, batch, "pages", d)
    to_table, to_max = _table(to_pages, batch, "to_pages", d)
    lens = _ints(lengths, (batch,), "lengths", d)
    if width < max_pages * page:
        raise ValueError(f"weights has room for {width} tokens, the page table for "
                         f"{max_pages * page}")
    if budget < 1 or sinks < 0 or recent < 0 or sinks + recent > budget:
        raise ValueError("need budget >= 1, sinks and recent >= 0, sinks + recent <= budget")
    if to_max * page < budget:
        raise ValueError(f"to_pages has room for {to_max * page} tokens, the budget is {budget}")

    if stream is not None:
        with torch.cuda.stream(stream):   # what is allocated belongs to it
            return kv_cache_evict(cache, weights, pages, lengths, budget, sinks, recent, to,
                                  to_pages)
    new_lengths = lengths.new_empty(batch)
    new_weights = weights.new_empty((batch, heads, to_max * page))
    kept = lengths.new_empty((batch, heads, budget))
    if batch == 0:
        return new_lengths, new_weights, kept
    rc = lib().kv_cache_evict_e4m3(
        ctypes.byref(pool), weights.data_ptr(), width, table, max_pages, lens, batch, budget,
        sinks, recent, ctypes.byref(dest), to_table, to_max, new_lengths.data_ptr(),
        new_weights.data_ptr(), kept.data_ptr(), _current(d))
    if rc != OK:
        raise GemmReluError(rc, "kv_cache_evict_e4m3")
    return new_lengths, new_weights, kept
