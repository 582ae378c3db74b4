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

// (a timeout that is there already stays)
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

// Elementwise larger of two pairs of magnitudes; a NaN gives way to the other.
template <bool kBf16>
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (kBf16)
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two fp16 values to e4m3, low byte first: round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t half2_to_e4m3x2(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}

// Two fp32 values to an fp16 pair, low half = a.
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Four e4m3 values times `ratio`, rounded to e4m3 again.
__device__ __forceinline__ uint32_t rescaled(uint32_t four, float ratio) {
    const float2 f = e4m3x2_to_float2(four & 0xffffu), g = e4m3x2_to_float2(four >> 16);
    return to_e4m3x2(f.x * ratio, f.y * ratio) | to_e4m3x2(g.x * ratio, g.y * ratio) << 16;
}

// The same for a power of two in [2^-14, 2^15] and results of at most 448: fp16 holds the
// products exactly, but for bits below 2^-24, far below e4m3's smallest half step of 2^-10.
__device__ __forceinline__ uint32_t rescaled_exact(uint32_t four, uint32_t ratio2) {
    uint32_t a = e4m3x2_to_half2(four & 0xffffu), b = e4m3x2_to_half2(four >> 16);
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(a) : "r"(ratio2));
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(b) : "r"(ratio2));
    return half2_to_e4m3x2(a) | half2_to_e4m3x2(b) << 16;
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
// the rounding, so they are read once.  A prompt is bound by HBM and, near it, by the issue of
// conversions (69% of issue slots, the ALU pipe full): 4 prompts of up to 4096 tokens, 8 heads of 128,
// fp16, 82.7 MB in 16.5 us, 5.0 TB/s.  Hence maxima on packed pairs (21.7 -> 19.0 us), the
// page number read behind the tokens (-> 17.9) and fp16 scaled and rounded as it is (-> 16.5).
// One token for each of 64 sequences takes 4.2 us, launch and three dependent reads.
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
    const int64_t id = p.pages[b * p.max_pages + at];   // (used once the tokens are on their way)

    constexpr int kPerToken = D / 8;
    const uint16_t *src = p.x[kv] + b * p.stride[kv][0] + h * p.stride[kv][2];
    uint4 x[kVec];
#pragma unroll
    for (int n = 0; n < kVec; ++n) {
        const int v = threadIdx.x + n * kAppendThreads, slot = v / kPerToken;
        x[n] = make_uint4(0, 0, 0, 0);
        if (slot >= lo && slot < hi)
            x[n] = *reinterpret_cast<const uint4 *>(src + (first + slot - start) * p.stride[kv][1] +
                                                    8 * (v % kPerToken));
    }
    if (id < 0 || id >= p.pool.num_pages) {
        if (threadIdx.x == 0)
            record_page_error();
        return;
    }
    float *scale_at = p.pool.scales[kv] + id * p.pool.kv_heads + h;
    const float held = lo > 0 ? *scale_at : 0.0f;   // 0: a fresh page
    uint32_t top = 0;
#pragma unroll
    for (int n = 0; n < kVec; ++n) {
        top = larger2<kBf16>(top, larger2<kBf16>(x[n].x & 0x7fff7fffu, x[n].y & 0x7fff7fffu));
        top = larger2<kBf16>(top, larger2<kBf16>(x[n].z & 0x7fff7fffu, x[n].w & 0x7fff7fffu));
    }
    const float2 tops = pair_to_float2<kBf16>(top);
    float amax = block_max(fmaxf(tops.x, tops.y), slots);
    const bool infinite = amax == INFINITY;   // seldom: look again, and store them as NaN
    if (infinite) {
        amax = 0.0f;
#pragma unroll
        for (int n = 0; n < kVec; ++n) {
            const uint32_t w[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = pair_to_float2<kBf16>(w[e]);
                amax = fmaxf(amax, fmaxf(finite_abs(f.x), finite_abs(f.y)));
            }
        }
        __syncthreads();
        amax = block_max(amax, slots);
    }
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
            if (!kBf16 && !infinite && inv <= 32768.0f && inv >= 0x1p-14f) {
                // fp16 all the way: 1 / scale is a normal number, and what fp16 rounds off a product lies
                // below 2^-24, far below e4m3's smallest half step of 2^-10
                const uint32_t inv2 = half2_of(inv, inv);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t y = w[e];
                    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(y) : "r"(inv2));
                    q[e] = half2_to_e4m3x2(y);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 f = pair_to_float2<kBf16>(w[e]);
                    if (infinite)
                        f = make_float2(storable(f.x), storable(f.y));
                    q[e] = to_e4m3x2(f.x * inv, f.y * inv);
                }
            }
            *reinterpret_cast<uint2 *>(dst + 8 * v) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
        } else if (slot < lo && scale != held) {
            // an older token of a page whose scale grew
            const uint2 old = *reinterpret_cast<const uint2 *>(dst + 8 * v);
            const float ratio = held * inv;
            *reinterpret_cast<uint2 *>(dst + 8 * v) = make_uint2(rescaled(old.x, ratio), rescaled(old.y, ratio));
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
    int cluster;                       // blocks per (sequence, head) of the selection
    int items;                         // (sequence, new page, head) items of the move
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

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kMaxSelectCluster = 8;
constexpr int kShortList = 512;   // keys that one warp finishes alone

// Which tokens stay, a cluster of 1 to 8 blocks per (sequence, head), each with a stretch of
// the tokens.  Sinks and recent tokens have the largest key there is, so the survivors are
// the `budget` largest keys: those above the k-th largest, k = budget, and the first few equal
// to it.  The keys are read once into registers
// (kKeys a thread; what does not fit is read again from L2), and the k-th largest is built
// two bits at a time from the top: of three candidates the largest that k keys reach.
// What bounds it is the rounds' latency and, with many keys, their compares, so once 512
// keys or fewer share the bits found one warp takes those and finishes alone (not across a
// cluster: 8 sequences of up to 32768 tokens took 73.6 us that way and 65.8 this way, one took
// 32.4 and 39.7).
// Measured for one sequence of 2000 tokens and for 16 of up to 16384, 8 heads: with the move
// 10.3 and 72 us, of which this is about 5 and 22.  Counting takes the same time whatever the
// weights are; a histogram of digits had its atomics collide, since weights share exponents (23 and
// 51 us); 1024 threads with 16 keys each took 13 and 29 us, most of it in 17 rounds of barriers.
template <int kKeys>
__global__ void __launch_bounds__(kSelectThreads, 1) kv_evict_select_kernel(const EvictParams p) {
    __shared__ uint2 warp_count[2][kSelectWarps];
    __shared__ int block_count[2][kMaxSelectCluster][3];
    __shared__ int slot_sure[kKeys * kSelectWarps], slot_tie[kKeys * kSelectWarps];
    __shared__ uint32_t list[kShortList];
    __shared__ int shared[4];   // list length, k-th key, keys above it; totals
    const int cluster = p.cluster, rank = cluster > 1 ? (int)cluster_ctarank() : 0;
    if (cluster > 1)
        cluster_arrive_relaxed();   // this block runs: the others may store into its shared memory
    pdl_launch_dependents();
    pdl_wait_primary();
    const int64_t bh = blockIdx.x / cluster;
    const int h = (int)(bh % p.from.kv_heads), b = (int)(bh / p.from.kv_heads);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t below = (1u << lane) - 1;
    const int n = checked_length(p.lengths, b, p.max_pages * p.from.page);
    const int m = n < p.budget ? n : p.budget;
    const float *w = p.weights + bh * p.width;
    int32_t *kept = p.kept + bh * p.budget;
    if (h == 0 && rank == 0 && tid == 0)
        p.to_lengths[b] = m;
    for (int i = m + rank * kSelectThreads + tid; i < p.budget; i += cluster * kSelectThreads)
        kept[i] = -1;
    if (n <= p.budget) {
        for (int i = rank * kSelectThreads + tid; i < n; i += cluster * kSelectThreads)
            kept[i] = i;
        if (cluster > 1)
            cluster_wait();
        return;   // all blocks of the cluster
    }
    const int lo = p.sinks, hi = n - p.recent;   // the tokens that compete for the rest
    const int stretch = (n + cluster - 1) / cluster;
    const int t0 = min(rank * stretch, n), t1 = min(t0 + stretch, n);
    constexpr int kGroup = kKeys * kSelectThreads;
    // token t0 + s * threads + tid is slot s of this thread; past the stretch 0, below every key
    auto key_of_weight = [&](int i, float x) {
        return i >= t1 ? 0u : i < lo || i >= hi ? 0xffffffffu : weight_key(x);
    };
    auto key_at = [&](int i) { return key_of_weight(i, i < t1 ? w[i] : 0.0f); };
    uint32_t key[kKeys];
    auto load = [&](int g0) {
        float x[kKeys];
#pragma unroll
        for (int s = 0; s < kKeys; ++s) {
            const int i = g0 + s * kSelectThreads + tid;
            x[s] = i < t1 ? w[i] : 0.0f;
        }
#pragma unroll
        for (int s = 0; s < kKeys; ++s)
            key[s] = key_of_weight(g0 + s * kSelectThreads + tid, x[s]);
    };
    load(t0);
    if (cluster > 1)
        cluster_wait();   // the others have started (behind the loads: no time of its own)

    int turn = 0;
    // how many of all keys reach three thresholds
    auto count = [&](uint32_t c1, uint32_t c2, uint32_t c3, int (&got)[3]) {
        int x[3] = {0, 0, 0};
#pragma unroll
        for (int s = 0; s < kKeys; ++s) {
            x[0] += key[s] >= c1;
            x[1] += key[s] >= c2;
            x[2] += key[s] >= c3;
        }
        if (stretch <= kGroup) {
            // a block's counts stay below 2^16: two in one word
            const uint32_t two = __reduce_add_sync(0xffffffffu, (uint32_t)x[0] | (uint32_t)x[1] << 16);
            const uint32_t one = __reduce_add_sync(0xffffffffu, (uint32_t)x[2]);
            if (lane == 0)
                warp_count[turn][warp] = make_uint2(two, one);
            __syncthreads();
            uint32_t sum_two = 0, sum_one = 0;
#pragma unroll
            for (int i = 0; i < kSelectWarps; ++i) {
                const uint2 c = warp_count[turn][i];
                sum_two += c.x;
                sum_one += c.y;
            }
            got[0] = (int)(sum_two & 0xffffu);
            got[1] = (int)(sum_two >> 16);
            got[2] = (int)sum_one;
        } else {
            for (int i = t0 + kGroup + tid; i < t1; i += kSelectThreads) {
                const uint32_t k = key_at(i);
                x[0] += k >= c1;
                x[1] += k >= c2;
                x[2] += k >= c3;
            }
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                x[i] = __reduce_add_sync(0xffffffffu, x[i]);
                if (lane == 0)
                    warp_count[turn][warp] = make_uint2((uint32_t)x[i], 0u);
                __syncthreads();
                got[i] = 0;
                for (int k = 0; k < kSelectWarps; ++k)
                    got[i] += (int)warp_count[turn][k].x;
                __syncthreads();
            }
        }
        if (cluster > 1) {
            if (warp == 0 && lane < cluster) {
                const uint32_t at = mapa_shared(smem_addr(&block_count[turn][rank][0]), (uint32_t)lane);
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    st_cluster_f32(at + 4 * i, __int_as_float(got[i]));
            }
            cluster_sync();
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                got[i] = 0;
                for (int c = 0; c < cluster; ++c)
                    got[i] += block_count[turn][c][i];
            }
        }
        turn ^= 1;
    };

    const int need = p.budget;
    uint32_t kth = 0;
    int ties_kept;
    {
        // `above` keys exceed all those that share the bits found, which `reach` - above do
        int above = 0, reach = n, shift = 30;
        for (; shift >= 0; shift -= 2) {
            int got[3];
            count(kth | 1u << shift, kth | 2u << shift, kth | 3u << shift, got);
            const int digit = got[2] >= need ? 3 : got[1] >= need ? 2 : got[0] >= need ? 1 : 0;
            above = digit == 3 ? above : got[digit];
            reach = digit == 0 ? reach : got[digit - 1];
            kth |= (uint32_t)digit << shift;
            if (cluster == 1 && stretch <= kGroup && reach - above <= kShortList)
                break;
        }
        if (shift >= 2) {   // (cluster is 1) the keys that share the bits, in no order
            if (tid == 0)
                shared[0] = 0;
            __syncthreads();
            const uint32_t mask = ~0u << shift;
            int mine_too = 0;
#pragma unroll
            for (int s = 0; s < kKeys; ++s)
                mine_too += __popc(__ballot_sync(0xffffffffu, (key[s] & mask) == kth && key[s] != 0));
            int at = 0;
            if (lane == 0 && mine_too > 0)
                at = atomicAdd(&shared[0], mine_too);
            at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
            for (int s = 0; s < kKeys; ++s) {
                const bool in = (key[s] & mask) == kth && key[s] != 0;
                const uint32_t who = __ballot_sync(0xffffffffu, in);
                if (in)
                    list[at + __popc(who & below)] = key[s];
                at += __popc(who);
            }
            __syncthreads();
            if (warp == 0) {
                uint32_t mine[kShortList / 32];
                const int length = shared[0];
#pragma unroll
                for (int s = 0; s < kShortList / 32; ++s)
                    mine[s] = s * 32 + lane < length ? list[s * 32 + lane] : 0u;
                const int want = need - above;
                int over = 0;
                for (shift -= 2; shift >= 0; shift -= 2) {
                    int x[3] = {0, 0, 0};
#pragma unroll
                    for (int s = 0; s < kShortList / 32; ++s) {
                        x[0] += mine[s] >= (kth | 1u << shift);
                        x[1] += mine[s] >= (kth | 2u << shift);
                        x[2] += mine[s] >= (kth | 3u << shift);
                    }
                    const uint32_t two = __reduce_add_sync(0xffffffffu, (uint32_t)x[0] | (uint32_t)x[1] << 16);
                    x[0] = (int)(two & 0xffffu);
                    x[1] = (int)(two >> 16);
                    x[2] = (int)__reduce_add_sync(0xffffffffu, (uint32_t)x[2]);
                    const int digit = x[2] >= want ? 3 : x[1] >= want ? 2 : x[0] >= want ? 1 : 0;
                    over = digit == 3 ? over : x[digit];
                    kth |= (uint32_t)digit << shift;
                }
                if (lane == 0) {
                    shared[1] = (int)kth;
                    shared[2] = above + over;
                }
            }
            __syncthreads();
            kth = (uint32_t)shared[1];
            above = shared[2];
        }
        ties_kept = need - above;
    }

    // survivors and equal keys of the blocks before
    int out = 0, ties = 0;
    if (cluster > 1) {
        int sure = 0, tie = 0;
        auto look = [&](uint32_t k) {
            sure += k > kth;
            tie += k == kth;
        };
#pragma unroll
        for (int s = 0; s < kKeys; ++s)
            look(key[s]);
        for (int i = t0 + kGroup + tid; i < t1; i += kSelectThreads)
            look(key_at(i));
        sure = __reduce_add_sync(0xffffffffu, sure);
        tie = __reduce_add_sync(0xffffffffu, tie);
        if (lane == 0)
            warp_count[turn][warp] = make_uint2((uint32_t)sure, (uint32_t)tie);
        __syncthreads();
        sure = tie = 0;
        for (int i = 0; i < kSelectWarps; ++i) {
            sure += (int)warp_count[turn][i].x;
            tie += (int)warp_count[turn][i].y;
        }
        if (warp == 0 && lane < cluster) {
            const uint32_t at = mapa_shared(smem_addr(&block_count[turn][rank][0]), (uint32_t)lane);
            st_cluster_f32(at, __int_as_float(sure));
            st_cluster_f32(at + 4, __int_as_float(tie));
        }
        cluster_sync();   // the last access to another block's memory
        for (int c = 0; c < rank; ++c) {
            out += block_count[turn][c][0];
            ties += block_count[turn][c][1];
        }
        out += min(ties, ties_kept);
    }
    // write this block's survivors in order, kGroup tokens at a time
    for (int g0 = t0; g0 < t1; g0 += kGroup) {
        if (g0 > t0)
            load(g0);
        auto sure_of = [&](int s) { return __ballot_sync(0xffffffffu, key[s] > kth); };
        auto tie_of = [&](int s) { return __ballot_sync(0xffffffffu, key[s] == kth); };
#pragma unroll
        for (int s = 0; s < kKeys; ++s) {
            const uint32_t sure = sure_of(s), tie = tie_of(s);
            if (lane == 0) {
                slot_sure[s * kSelectWarps + warp] = __popc(sure);
                slot_tie[s * kSelectWarps + warp] = __popc(tie);
            }
        }
        __syncthreads();
        if (warp < 2) {   // exclusive sums in token order, one warp each
            int *slot = warp == 0 ? slot_sure : slot_tie;
            constexpr int kEach = kKeys * kSelectWarps / 32;
            int a[kEach], sum = 0;
#pragma unroll
            for (int s = 0; s < kEach; ++s) {
                a[s] = slot[lane * kEach + s];
                sum += a[s];
            }
            int run = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, run, o);
                run += lane >= o ? x : 0;
            }
            int at = run - sum;
#pragma unroll
            for (int s = 0; s < kEach; ++s) {
                slot[lane * kEach + s] = at;
                at += a[s];
            }
            if (lane == 31)
                shared[2 + warp] = run;
        }
        __syncthreads();
        const int kept_before = min(ties, ties_kept);
#pragma unroll
        for (int s = 0; s < kKeys; ++s) {
            const uint32_t sure = sure_of(s), tie = tie_of(s);
            const int rank_tie = ties + slot_tie[s * kSelectWarps + warp] + __popc(tie & below);
            const int at = out + slot_sure[s * kSelectWarps + warp] + __popc(sure & below) +
                           min(rank_tie, ties_kept) - kept_before;
            const bool stays = (sure >> lane & 1u) || ((tie >> lane & 1u) && rank_tie < ties_kept);
            if (stays)
                kept[at] = g0 + s * kSelectThreads + tid;
        }
        const int more_sure = shared[2], more_ties = shared[3];
        ties += more_ties;
        out += more_sure + min(ties, ties_kept) - kept_before;
        __syncthreads();
    }
}

constexpr int kMoveThreads = 256;

// Largest magnitude of 16 e4m3 values as a code (0 .. 0x7e), or 0x7f where there is a NaN: e4m3
// magnitudes ascend with their codes, so two 16-bit lanes compare four bytes at a time.
__device__ __forceinline__ uint32_t largest_code(const uint4 &x) {
    const uint32_t hi = __vimax3_u16x2(__vmaxu2(x.x & 0x7f007f00u, x.y & 0x7f007f00u), x.z & 0x7f007f00u,
                                       x.w & 0x7f007f00u);
    const uint32_t lo = __vimax3_u16x2(__vmaxu2(x.x & 0x007f007fu, x.y & 0x007f007fu), x.z & 0x007f007fu,
                                       x.w & 0x007f007fu);
    const uint32_t m = __vmaxu2(hi >> 8, lo);
    return max(m >> 16, m & 0xffffu);
}

// The same with NaN out of the way.
__device__ __forceinline__ float largest_finite(const uint4 &x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        top = larger2<false>(top, e4m3x2_to_half2(w[e] & 0x7f7fu));
        top = larger2<false>(top, e4m3x2_to_half2(w[e] >> 16 & 0x7f7fu));
    }
    const float2 f = pair_to_float2<false>(top);
    return fmaxf(f.x, f.y);
}

// Gathers the kept tokens of (sequence, new page, head) items, 16 elements a thread and
// vector of K and of V, and stores them under scales of their own.  The bytes stay
// in registers between the maximum and the rounding.  A token's bytes are three dependent reads
// away (its position, its page, itself), so a block walks over items and reads the next
// item's positions and pages while this one's bytes are under way.  Bound by HBM on rows of D
// bytes and by issue (60% of the slots): 16 sequences cut from up to 16384 to 4096 tokens, 8
// heads of 128, 134 MB read and 134 written in about 50 us; an item per block and fp32
// arithmetic took 70.
template <int D, int kVec>
__global__ void __launch_bounds__(kMoveThreads, kVec == 4 ? 2 : 4) kv_evict_move_kernel(const EvictParams p) {
    __shared__ uint2 tops[2][kMoveThreads / 32];
    pdl_launch_dependents();
    pdl_wait_primary();
    constexpr int kPerToken = D / 16;
    const int page = p.from.page, shift = p.from.page_shift, heads = p.from.kv_heads;
    const int to_max = (int)p.to_max_pages, items = p.items;   // heads fastest, then pages, then sequences
    // the item in hand, and what a step over gridDim.x items adds, without divisions in the loop
    int h = blockIdx.x % heads, at = blockIdx.x / heads % to_max, b = blockIdx.x / heads / to_max;
    const int step_h = gridDim.x % heads, step_at = gridDim.x / heads % to_max, step_b = gridDim.x / heads / to_max;

    struct Item {
        int h, b, at, m, to;     // m: the sequence's new length; to: the new page, -1 for none
        int from[kVec];          // source page of each vector, -1: none
        int t[kVec];             // and its token
        float w;
    };
    auto look = [&]() {
        Item x;
        x.h = h;
        x.at = at;
        x.b = b;
        const int64_t bh = (int64_t)b * heads + h;
        const int first = at << shift;
        // written by the selection: -1 past the new length
        const int32_t *kept = p.kept + bh * p.budget + first;
        const int left = min(p.budget - first, page);
        const int mine = (int)threadIdx.x < left ? kept[threadIdx.x] : -1;
#pragma unroll
        for (int n = 0; n < kVec; ++n) {
            const int slot = (threadIdx.x + n * kMoveThreads) / kPerToken;
            x.t[n] = slot < left ? kept[slot] : -1;
        }
        x.m = p.to_lengths[b];
        x.to = p.to_pages[(int64_t)b * to_max + at];
        const int32_t *pages = p.pages + b * p.max_pages;
#pragma unroll
        for (int n = 0; n < kVec; ++n)
            x.from[n] = x.t[n] >= 0 ? pages[x.t[n] >> shift] : -1;
        x.w = mine >= 0 ? p.weights[bh * p.width + mine] : 0.0f;
        // on to the block's next item
        h += step_h;
        at += step_at;
        b += step_b;
        if (h >= heads) {
            h -= heads;
            ++at;
        }
        if (at >= to_max) {
            at -= to_max;
            ++b;
        }
        return x;
    };

    int turn = 0;
    int item = blockIdx.x;
    if (item >= items)
        return;
    Item next = look();
    for (; item < items; item += gridDim.x) {
        const Item x = next;
        const int first = x.at << shift;
        const bool there = first < x.m, good = there && x.to >= 0 && x.to < p.to.num_pages;
        uint4 v[2][kVec];
        float s[2][kVec];
#pragma unroll
        for (int n = 0; n < kVec; ++n) {
            v[0][n] = v[1][n] = make_uint4(0, 0, 0, 0);
            s[0][n] = s[1][n] = 0.0f;
            if (!good || x.t[n] < 0)
                continue;
            if (x.from[n] < 0 || x.from[n] >= p.from.num_pages) {
                record_page_error();
                continue;
            }
            const int64_t block = (int64_t)x.from[n] * heads + x.h;
            const int64_t from = (block * page + (x.t[n] & (page - 1))) * D + 16 * ((threadIdx.x + n * kMoveThreads) % kPerToken);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                v[kv][n] = *reinterpret_cast<const uint4 *>(p.from.values[kv] + from);
                s[kv][n] = p.from.scales[kv][block];
            }
        }
        if (item + (int)gridDim.x < items)
            next = look();
        if ((int)threadIdx.x < page)
            p.to_weights[(((int64_t)x.b * heads + x.h) * to_max << shift) + first + threadIdx.x] = x.w;
        if (there && !good && threadIdx.x == 0)
            record_page_error();
        if (!good)
            continue;
        uint32_t top[2];
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            float amax = 0.0f;
#pragma unroll
            for (int n = 0; n < kVec; ++n) {
                const uint32_t code = largest_code(v[kv][n]);
                float f = e4m3x2_to_float2(code).x;
                if (code == 0x7fu)   // a NaN: look again
                    f = largest_finite(v[kv][n]);
                amax = fmaxf(amax, f * s[kv][n]);
            }
            top[kv] = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
        }
        // the words alternate between items: one barrier each
        if ((threadIdx.x & 31) == 0)
            tops[turn][threadIdx.x >> 5] = make_uint2(top[0], top[1]);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kMoveThreads / 32; ++w) {
            top[0] = max(top[0], tops[turn][w].x);
            top[1] = max(top[1], tops[turn][w].y);
        }
        turn ^= 1;
        const int64_t block = (int64_t)x.to * heads + x.h;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const float scale = scale_for(__uint_as_float(top[kv])), inv = inverse_scale(scale);
            if (threadIdx.x == 0)
                p.to.scales[kv][block] = scale;
            uint8_t *dst = p.to.values[kv] + block * page * D;
#pragma unroll
            for (int n = 0; n < kVec; ++n) {
                const int i = threadIdx.x + n * kMoveThreads;
                if (i / kPerToken >= page)
                    break;
                const float ratio = s[kv][n] * inv;
                uint32_t w[4] = {v[kv][n].x, v[kv][n].y, v[kv][n].z, v[kv][n].w};
                // a power of two that fp16 holds (or 0: nothing there); 1 where a page's scale
                // stays, which the bytes pass as they are
                const uint32_t r = __float_as_uint(ratio);
                if (__all_sync(__activemask(), ratio == 1.0f)) {
                } else if ((r & 0x7fffffu) == 0 && ratio <= 32768.0f && (ratio >= 0x1p-14f || r == 0)) {
                    const uint32_t ratio2 = half2_of(ratio, ratio);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = rescaled_exact(w[e], ratio2);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = rescaled(w[e], ratio);
                }
                *reinterpret_cast<uint4 *>(dst + 16 * i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

}  // namespace kvc
}  // namespace gemmrelu
