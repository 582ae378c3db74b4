// kv_cache.cuh -- the paged 8-bit K/V cache: its number format, the kernel
// that writes new tokens, and the two of an eviction (which tokens stay;
// their move into new pages).
//
// A page and head hold e4m3 values v with one scale s: a token's element is
// v * s.  s is the smallest power of two with amax <= 448 s, so v = x / s is an
// exact shift of exponents followed by one rounding to e4m3 (3 mantissa bits:
// relative error at most 2^-4 for normal values, 2^-10 s below 2^-6 s).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "gemm_relu_kernels.cuh"

namespace gemmrelu {
namespace kvc {

constexpr unsigned kStatusPage = 8;   // == GEMMRELU_ERR_PAGE

__device__ __forceinline__ void record_page_error() { atomicCAS(&g_status, 0u, kStatusPage); }

// ---------------------------------------------------------------- the number format

constexpr float kMinScale = 7.888609052210118e-31f;   // 2^-100

// The smallest power of two s >= 2^-100 with amax <= 448 s, for finite amax >= 0.
// amax = f * 2^E with f in [1, 2), 448 = 1.75 * 2^8: s = 2^(E-8) up to
// f = 1.75, else 2^(E-7).
__device__ __forceinline__ float scale_for(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 127 - ((b & 0x7fffffu) <= 0x600000u ? 8 : 7);
    return e <= -100 ? kMinScale : __uint_as_float((uint32_t)(e + 127) << 23);
}

// 1 / s for a power of two s in [2^-100, 2^121].
__device__ __forceinline__ float inverse_scale(float s) {
    return __uint_as_float((254u << 23) - __float_as_uint(s));
}

// Two fp32 values to e4m3, low byte = a: round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Two e4m3 values to fp16 (exact), low half = low byte.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
    const uint32_t h = e4m3x2_to_half2(two);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

template <bool kBf16>
__device__ __forceinline__ float2 pair_to_float2(uint32_t x) {
    if constexpr (kBf16) {
        return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    } else {
        return __half22float2(*reinterpret_cast<const __half2 *>(&x));
    }
}

// |x| where x is finite, else 0: what counts for a block's scale.
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.0f;
}

// x, or NaN in the place of an infinity (which e4m3 lacks).
__device__ __forceinline__ float storable(float x) {
    return fabsf(x) < INFINITY ? x : __uint_as_float(0x7fffffffu);
}

// Largest of the block's non-negative values; `slots` has one word per warp.
// The barrier inside also orders earlier reads of the block before later writes.
__device__ __forceinline__ float block_max(float x, uint32_t *slots) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(x));
    if ((threadIdx.x & 31) == 0)
        slots[threadIdx.x >> 5] = m;
    __syncthreads();
    uint32_t r = 0;
    for (unsigned w = 0; w < blockDim.x / 32; ++w)
        r = max(r, slots[w]);
    return __uint_as_float(r);
}

// The pool as the kernels see it.
struct Pool {
    uint8_t *values[2];   // K, V
    float *scales[2];
    int64_t num_pages;
    int kv_heads;
    int page, page_shift;
};

// ---------------------------------------------------------------- append

struct AppendParams {
    Pool pool;
    const uint16_t *x[2];            // K, V: [batch][tokens][kv_heads][D]
    int64_t stride[2][3];            // sequence, token, head
    const int32_t *pages, *lengths, *counts;
    int64_t max_pages;
    int batch, tokens, touched;      // touched: most pages that one sequence's new tokens reach
};

constexpr int kAppendThreads = 256;

// One block per (sequence, touched page, head, K or V): the new tokens' elements stay in
// registers (kVec vectors of 8 a thread) between the block's maximum and
// the rounding, so they are read once.
template <int D, int kVec, bool kBf16>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p) {
    __shared__ uint32_t slots[kAppendThreads / 32];
    pdl_launch_dependents();
    pdl_wait_primary();
    int64_t i = blockIdx.x;
    const int kv = (int)(i & 1);
    i >>= 1;
    const int h = (int)(i % p.pool.kv_heads);
    i /= p.pool.kv_heads;
    const int nth = (int)(i % p.touched);
    const int b = (int)(i / p.touched);

    const int end = p.lengths[b];
    const int count = p.counts ? p.counts[b] : p.tokens;
    if (count < 0 || count > p.tokens || end < count ||
        (int64_t)end > p.max_pages * p.pool.page) {
        if (threadIdx.x == 0)
            record_page_error();
        return;
    }
    const int start = end - count;
    const int at = (start >> p.pool.page_shift) + nth;   // index in the page table's row
    const int64_t first = (int64_t)at << p.pool.page_shift;
    if (count == 0 || first >= end)
        return;
    const int lo = start > first ? (int)(start - first) : 0;                       // new slots
    const int hi = end - first < p.pool.page ? (int)(end - first) : p.pool.page;   // [lo, hi)
    const int64_t id = p.pages[b * p.max_pages + at];
    if (id < 0 || id >= p.pool.num_pages) {
        if (threadIdx.x == 0)
            record_page_error();
        return;
    }

    constexpr int kPerToken = D / 8;
    const uint16_t *src = p.x[kv] + b * p.stride[kv][0] + h * p.stride[kv][2];
    uint4 x[kVec];
    float amax = 0.0f;
#pragma unroll
    for (int n = 0; n < kVec; ++n) {
        const int v = threadIdx.x + n * kAppendThreads, slot = v / kPerToken;
        x[n] = make_uint4(0, 0, 0, 0);
        if (slot >= lo && slot < hi)
            x[n] = *reinterpret_cast<const uint4 *>(src + (first + slot - start) * p.stride[kv][1] +
                                                    8 * (v % kPerToken));
    }
#pragma unroll
    for (int n = 0; n < kVec; ++n) {
        const uint32_t w[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = pair_to_float2<kBf16>(w[e]);
            amax = fmaxf(amax, fmaxf(finite_abs(f.x), finite_abs(f.y)));
        }
    }
    float *scale_at = p.pool.scales[kv] + id * p.pool.kv_heads + h;
    const float held = lo > 0 ? *scale_at : 0.0f;   // 0: a fresh page
    amax = block_max(amax, slots);
    const float scale = fmaxf(held, scale_for(amax));
    const float inv = inverse_scale(scale);
    if (threadIdx.x == 0 && scale != held)
        *scale_at = scale;
    uint8_t *dst = p.pool.values[kv] + (id * p.pool.kv_heads + h) * p.pool.page * D;
#pragma unroll
    for (int n = 0; n < kVec; ++n) {
        const int v = threadIdx.x + n * kAppendThreads, slot = v / kPerToken;
        if (slot >= lo && slot < hi) {
            const uint32_t w[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
            uint32_t q[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = pair_to_float2<kBf16>(w[e]);
                q[e] = to_e4m3x2(storable(f.x) * inv, storable(f.y) * inv);
            }
            *reinterpret_cast<uint2 *>(dst + 8 * v) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
        } else if (slot < lo && scale != held) {
            // an older token of a page whose scale grew
            uint2 old = *reinterpret_cast<const uint2 *>(dst + 8 * v);
            const float ratio = held * inv;
            uint32_t o[2] = {old.x, old.y};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 f = e4m3x2_to_float2(o[e] & 0xffffu), g = e4m3x2_to_float2(o[e] >> 16);
                o[e] = to_e4m3x2(f.x * ratio, f.y * ratio) | to_e4m3x2(g.x * ratio, g.y * ratio) << 16;
            }
            *reinterpret_cast<uint2 *>(dst + 8 * v) = make_uint2(o[0], o[1]);
        }
    }
}

// ---------------------------------------------------------------- evict

struct EvictParams {
    Pool from, to;
    const float *weights;
    int64_t width;                     // row length of weights
    const int32_t *pages, *lengths, *to_pages;
    int64_t max_pages, to_max_pages;
    int batch, budget, sinks, recent;
    int32_t *to_lengths;
    float *to_weights;
    int32_t *kept;
};

// A sequence's length, or 0 where it is out of range.
__device__ __forceinline__ int checked_length(const int32_t *lengths, int b, int64_t most) {
    const int n = lengths[b];
    if (n < 0 || n > most) {
        record_page_error();
        return 0;
    }
    return n;
}

// Weights as unsigned keys in ascending order: NaN lowest (with -infinity),
// -0 equal to +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    w = w == w ? w + 0.0f : -INFINITY;
    const uint32_t b = __float_as_uint(w);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

constexpr int kSelectThreads = 1024;

// One block per (sequence, head): which tokens stay.  Between the sinks and the
// recent tokens the k heaviest are those above the k-th largest key and the
// first few equal to it; the k-th largest key is found 8 bits at a time
// from the top with a histogram of the keys that share the bits found so far.
__global__ void __launch_bounds__(kSelectThreads) kv_evict_select_kernel(const EvictParams p) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t found[2];
    __shared__ uint32_t above[32], equal[32];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int h = blockIdx.x % p.from.kv_heads, b = blockIdx.x / p.from.kv_heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = checked_length(p.lengths, b, p.max_pages * p.from.page);
    const int m = n < p.budget ? n : p.budget;
    const float *w = p.weights + (int64_t)blockIdx.x * p.width;
    int32_t *kept = p.kept + (int64_t)blockIdx.x * p.budget;
    if (h == 0 && tid == 0)
        p.to_lengths[b] = m;
    for (int i = m + tid; i < p.budget; i += kSelectThreads)
        kept[i] = -1;
    if (n <= p.budget) {
        for (int i = tid; i < n; i += kSelectThreads)
            kept[i] = i;
        return;
    }
    const int lo = p.sinks, hi = n - p.recent;
    uint32_t need = (uint32_t)(p.budget - p.sinks - p.recent);   // of the keys that still match
    uint32_t prefix = 0, mask = 0;
    if (need > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kSelectThreads)
                hist[i] = 0;
            __syncthreads();
            for (int i = lo + tid; i < hi; i += kSelectThreads) {
                const uint32_t key = weight_key(w[i]);
                if ((key & mask) == prefix)
                    atomicAdd(&hist[(key >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (tid == 0) {
                uint32_t left = need;
                int bin = 255;
                while (hist[bin] < left)
                    left -= hist[bin--];
                found[0] = (uint32_t)bin;
                found[1] = left;
            }
            __syncthreads();
            prefix |= found[0] << shift;
            mask |= 255u << shift;
            need = found[1];
        }
    } else {
        prefix = 0xffffffffu;   // no weight has this key
    }
    // write the survivors in order; `need` = how many of the keys equal to prefix stay
    uint32_t out = 0, ties = 0;   // survivors and equal keys before this stretch of tokens
    for (int base = 0; base < n; base += kSelectThreads) {
        const int i = base + tid;
        bool sure = false, tie = false;
        if (i < n) {
            sure = i < lo || i >= hi;
            if (!sure) {
                const uint32_t key = weight_key(w[i]);
                sure = key > prefix;
                tie = key == prefix;
            }
        }
        const uint32_t below = (1u << lane) - 1;
        const uint32_t bs = __ballot_sync(0xffffffffu, sure), bt = __ballot_sync(0xffffffffu, tie);
        if (lane == 0) {
            above[warp] = __popc(bs);
            equal[warp] = __popc(bt);
        }
        __syncthreads();
        uint32_t s = 0, t = 0, all_s = 0, all_t = 0;
        for (int k = 0; k < kSelectThreads / 32; ++k) {
            s += k < warp ? above[k] : 0u;
            t += k < warp ? equal[k] : 0u;
            all_s += above[k];
            all_t += equal[k];
        }
        const uint32_t kept_ties = ties < need ? ties : need;
        const uint32_t tie_rank = ties + t + __popc(bt & below);
        const uint32_t at = out + s + __popc(bs & below) + (tie_rank < need ? tie_rank : need) - kept_ties;
        if (sure || (tie && tie_rank < need))
            kept[at] = i;
        ties += all_t;
        out += all_s + (ties < need ? ties : need) - kept_ties;
        __syncthreads();
    }
}

constexpr int kMoveThreads = 256;

// One block per (sequence, new page, head): gathers the page's kept tokens, K
// then V, 16 elements a thread and vector, and stores them under a
// scale of their own.  The bytes stay in registers between the maximum and the
// rounding.
template <int D, int kVec>
__global__ void __launch_bounds__(kMoveThreads) kv_evict_move_kernel(const EvictParams p) {
    __shared__ uint32_t slots[2][kMoveThreads / 32];
    pdl_launch_dependents();
    pdl_wait_primary();
    int64_t i = blockIdx.x;
    const int h = (int)(i % p.from.kv_heads);
    i /= p.from.kv_heads;
    const int at = (int)(i % p.to_max_pages);
    const int b = (int)(i / p.to_max_pages);
    const int page = p.from.page;
    const int64_t bh = (int64_t)b * p.from.kv_heads + h;
    const int m = p.to_lengths[b];   // written by the selection
    const int64_t first = (int64_t)at * page;
    const int32_t *kept = p.kept + bh * p.budget;
    float *to_w = p.to_weights + bh * p.to_max_pages * page;
    for (int s = threadIdx.x; s < page; s += kMoveThreads)
        to_w[first + s] = first + s < m ? p.weights[bh * p.width + kept[first + s]] : 0.0f;
    if (first >= m)
        return;
    const int64_t id = p.to_pages[b * p.to_max_pages + at];
    if (id < 0 || id >= p.to.num_pages) {
        if (threadIdx.x == 0)
            record_page_error();
        return;
    }
    constexpr int kPerToken = D / 16;
    uint4 x[2][kVec];
    float s[2][kVec];
#pragma unroll
    for (int n = 0; n < kVec; ++n) {
        const int v = threadIdx.x + n * kMoveThreads, slot = v / kPerToken;
        x[0][n] = x[1][n] = make_uint4(0, 0, 0, 0);
        s[0][n] = s[1][n] = 0.0f;
        if (slot < page && first + slot < m) {
            const int t = kept[first + slot];
            const int64_t from = p.pages[b * p.max_pages + (t >> p.from.page_shift)];
            if (from < 0 || from >= p.from.num_pages) {
                record_page_error();
            } else {
                const int64_t block = from * p.from.kv_heads + h;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    x[kv][n] = *reinterpret_cast<const uint4 *>(
                        p.from.values[kv] + (block * page + (t & (page - 1))) * D + 16 * (v % kPerToken));
                    s[kv][n] = p.from.scales[kv][block];
                }
            }
        }
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        float amax = 0.0f;
#pragma unroll
        for (int n = 0; n < kVec; ++n) {
            const uint32_t w[4] = {x[kv][n].x, x[kv][n].y, x[kv][n].z, x[kv][n].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = e4m3x2_to_float2(w[e] & 0xffffu), g = e4m3x2_to_float2(w[e] >> 16);
                amax = fmaxf(amax, fmaxf(fmaxf(finite_abs(f.x), finite_abs(f.y)),
                                         fmaxf(finite_abs(g.x), finite_abs(g.y))) * s[kv][n]);
            }
        }
        amax = block_max(amax, slots[kv]);
        const float scale = scale_for(amax), inv = inverse_scale(scale);
        const int64_t block = id * p.to.kv_heads + h;
        if (threadIdx.x == 0)
            p.to.scales[kv][block] = scale;
        uint8_t *dst = p.to.values[kv] + block * page * D;
#pragma unroll
        for (int n = 0; n < kVec; ++n) {
            const int v = threadIdx.x + n * kMoveThreads;
            if (v / kPerToken >= page)
                break;
            const float ratio = s[kv][n] * inv;
            uint32_t w[4] = {x[kv][n].x, x[kv][n].y, x[kv][n].z, x[kv][n].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = e4m3x2_to_float2(w[e] & 0xffffu), g = e4m3x2_to_float2(w[e] >> 16);
                w[e] = to_e4m3x2(f.x * ratio, f.y * ratio) | to_e4m3x2(g.x * ratio, g.y * ratio) << 16;
            }
            *reinterpret_cast<uint4 *>(dst + 16 * v) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

}  // namespace kvc
}  // namespace gemmrelu
