// rotary.cuh -- rotary positions: pairs of a head's elements turned by position * frequency,
//
//   y1 = a (x1 cos t - x2 sin t),  y2 = a (x2 cos t + x1 sin t).
//
// The angle is kept in turns, as a 64-bit fraction: a frequency f radians a token is the integer
// f / (2 pi) * 2^64 mod 2^64, and its product with a position, wrapped at 64 bits, is the angle's
// fraction of a turn for any position (an fp32 product of the two loses all of it from 2^24 on).
//
// Bound: every element is read and written once.  So a block takes a few rows and works their cosines and sines out into shared
// memory once for all heads (sincospi of the fraction's top 32 bits as fp32: the angle is off by 2^-23 at most), and its
// threads go over the heads 16 bytes at a time.  A thread has one head under way: four took registers and with them
// occupancy (60 us against 57).  4 x 4096 tokens, 32 + 8 heads of 128, bf16: 57 us, 5.9 TB/s; 3 x 5001 tokens, half of 16 + 16
// heads of 64 turned in pairs side by side: 26 us, 4.7 TB/s (22 where one call after the other writes the same 61 MB, which then
// stay in L2); 64 single tokens: 2.8 us on the GPU.  Where rot is no multiple of 16, pairs go one at a time in accesses of 2
// bytes: the same tokens with rot 24 58 us and 20 72 (32: 22); 4 x 4096, heads of 128, 24 127, 20 146, 120 173 (96: 57).
#pragma once

#include "kv_attention.cuh"

namespace gemmrelu {
namespace rot {

using kvc::pair_to_float2;

constexpr int kRotThreads = 256;
constexpr int kMostTrig = 256;         // angles of a block

struct RotaryParams {
    const uint16_t *x[2];              // q, k
    uint16_t *y[2];
    int64_t xs[2][3], ys[2][3];        // sequence, token, head
    int heads0, heads;                 // q's, both
    int64_t rows;                      // batch * tokens
    int tokens, head_dim, half;        // half: rot / 2
    const void *positions, *inv_freq;
    bool pos64, freq64;
    bool copy;                         // elements past rot have to be written
    int turned, items;                 // work items of a head: those that turn pairs, all
    int rows_block, lanes;             // rows of a block, head lanes of a row
    float amplitude, sine;             // sine: the amplitude, negative for the inverse
};

// f radians as a fraction of a turn, in 2^-64: |f| = m 2^(e - 52) times 1 / (2 pi), whose product with m is
// taken in full.  (On integers: the GPU's fp64 rate is 1/64 of its fp32 rate.)
__device__ __forceinline__ uint64_t turns_of(double f) {
    const uint64_t bits = (uint64_t)__double_as_longlong(f);
    const int e = (int)(bits >> 52 & 0x7ff) - 1023;
    if (e < -66 || e > 31)
        return 0;
    const uint64_t m = (bits & 0xfffffffffffffull) | 1ull << 52;
    constexpr uint64_t kInvTwoPi = 0xa2f9836e4e441529ull;   // 1 / (2 pi) * 2^66, 2 / pi's first 64 bits
    const uint64_t hi = __umul64hi(m << 11, kInvTwoPi), lo = (m << 11) * kInvTwoPi;   // |f| / (2 pi) * 2^(129 - e)
    // hi : lo * 2^(e - 65), modulo 2^64
    const int s = e - 1;                                    // hi * 2^s is in units of 2^-64 turns
    uint64_t t;
    if (s <= 0)
        t = s > -64 ? hi >> -s : 0;
    else
        t = hi << s | lo >> (64 - s);
    return bits >> 63 ? 0 - t : t;
}

// Pairs x (elements of the pairs' first halves) and z (second halves), two of each, by (cos, sin).
template <bool kBf16>
__device__ __forceinline__ void turn_two(uint32_t &x, uint32_t &z, float4 cs) {
    const float2 a = pair_to_float2<kBf16>(x), b = pair_to_float2<kBf16>(z);
    x = kvc::pack_out<kBf16>(a.x * cs.x - b.x * cs.y, a.y * cs.z - b.y * cs.w);
    z = kvc::pack_out<kBf16>(b.x * cs.x + a.x * cs.y, b.y * cs.z + a.y * cs.w);
}

// One pair that lies side by side.
template <bool kBf16>
__device__ __forceinline__ void turn_one(uint32_t &x, float2 cs) {
    const float2 a = pair_to_float2<kBf16>(x);
    x = kvc::pack_out<kBf16>(a.x * cs.x - a.y * cs.y, a.y * cs.x + a.x * cs.y);
}

// A block: rows_block rows.  Its angles' cosines and sines are computed once, about one a thread, and
// stay in shared memory; each thread then keeps one item of one row (8 pairs: two vectors of 8 elements,
// one pair where the halves are not vectors, or two vectors that are copied) over every lanes-th head.
template <bool kBf16, bool kInterleaved, bool kVector>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryParams p) {
    __shared__ __align__(16) float2 trig[kMostTrig];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int64_t row0 = (int64_t)blockIdx.x * p.rows_block;
    for (int i = threadIdx.x; i < p.rows_block * p.half; i += kRotThreads) {
        const int r = i / p.half, f = i - r * p.half;
        float2 cs = make_float2(0.0f, 0.0f);
        if (row0 + r < p.rows) {
            const double freq = p.freq64 ? static_cast<const double *>(p.inv_freq)[f]
                                         : (double)static_cast<const float *>(p.inv_freq)[f];
            const int64_t pos = p.pos64 ? static_cast<const int64_t *>(p.positions)[row0 + r]
                                        : static_cast<const int32_t *>(p.positions)[row0 + r];
            const uint64_t turn = (uint64_t)pos * turns_of(freq);
            // the upper 32 bits, rounded, as a signed number of half turns in [-1, 1]
            const float half_turns = (float)(int32_t)((turn + 0x80000000ull) >> 32) * 4.656612873077393e-10f;
            sincospif(half_turns, &cs.y, &cs.x);
            cs.x *= p.amplitude;
            cs.y *= p.sine;
        }
        trig[i] = cs;
    }
    __syncthreads();
    const int item = threadIdx.x % p.items, rest = threadIdx.x / p.items;
    const int r = rest / p.lanes, lane = rest - r * p.lanes;
    const int64_t row = row0 + r;
    if (r >= p.rows_block || row >= p.rows)
        return;
    const int64_t b = row / p.tokens, token = row - b * p.tokens;
    const uint16_t *q_src = p.x[0] + b * p.xs[0][0] + token * p.xs[0][1];
    const uint16_t *k_src = p.x[1] + b * p.xs[1][0] + token * p.xs[1][1];
    uint16_t *q_dst = p.y[0] + b * p.ys[0][0] + token * p.ys[0][1];
    uint16_t *k_dst = p.y[1] + b * p.ys[1][0] + token * p.ys[1][1];
    auto src = [&](int h) {
        return h < p.heads0 ? q_src + h * p.xs[0][2] : k_src + (h - p.heads0) * p.xs[1][2];
    };
    auto dst = [&](int h) {
        return h < p.heads0 ? q_dst + h * p.ys[0][2] : k_dst + (h - p.heads0) * p.ys[1][2];
    };
    const float2 *cs = trig + r * p.half;
    const bool turns = item < p.turned;
    // what is copied: the vectors from `copied` on, two an item (the last one twice where their number is odd)
    const int copied = (2 * p.half + 7) / 8 * 8, copy0 = copied + 16 * (item - p.turned), copy1 = min(copy0 + 8, p.head_dim - 8);
    if constexpr (kVector) {
        constexpr int kPairs = 8;
        // pairs of this item: 8 item .. 8 item + 7
        const int x_at = !turns ? copy0 : kInterleaved ? 16 * item : 8 * item;
        const int z_at = !turns ? copy1 : kInterleaved ? x_at + 8 : p.half + 8 * item;
        float4 c[kPairs / 2];
#pragma unroll
        for (int i = 0; i < kPairs / 2; ++i)
            c[i] = turns ? *reinterpret_cast<const float4 *>(cs + 8 * item + 2 * i) : make_float4(1, 0, 1, 0);
#pragma unroll 1
        for (int h = lane; h < p.heads; h += p.lanes) {
            const uint16_t *s = src(h);
            uint16_t *d = dst(h);
            uint4 x = __ldcs(reinterpret_cast<const uint4 *>(s + x_at)), z = __ldcs(reinterpret_cast<const uint4 *>(s + z_at));
            if (turns) {
                if constexpr (kInterleaved) {
                    turn_one<kBf16>(x.x, make_float2(c[0].x, c[0].y));
                    turn_one<kBf16>(x.y, make_float2(c[0].z, c[0].w));
                    turn_one<kBf16>(x.z, make_float2(c[1].x, c[1].y));
                    turn_one<kBf16>(x.w, make_float2(c[1].z, c[1].w));
                    turn_one<kBf16>(z.x, make_float2(c[2].x, c[2].y));
                    turn_one<kBf16>(z.y, make_float2(c[2].z, c[2].w));
                    turn_one<kBf16>(z.z, make_float2(c[3].x, c[3].y));
                    turn_one<kBf16>(z.w, make_float2(c[3].z, c[3].w));
                } else {
                    turn_two<kBf16>(x.x, z.x, c[0]);
                    turn_two<kBf16>(x.y, z.y, c[1]);
                    turn_two<kBf16>(x.z, z.z, c[2]);
                    turn_two<kBf16>(x.w, z.w, c[3]);
                }
            }
            *reinterpret_cast<uint4 *>(d + x_at) = x;
            *reinterpret_cast<uint4 *>(d + z_at) = z;
        }
    } else if (!turns) {
        for (int h = lane; h < p.heads; h += p.lanes) {
            const uint16_t *s = src(h);
            uint16_t *d = dst(h);
            const uint4 x = *reinterpret_cast<const uint4 *>(s + copy0), z = *reinterpret_cast<const uint4 *>(s + copy1);
            *reinterpret_cast<uint4 *>(d + copy0) = x;
            *reinterpret_cast<uint4 *>(d + copy1) = z;
        }
    } else {
        // one pair of elements; the first item also copies what is left up to a vector's boundary
        const int x_at = kInterleaved ? 2 * item : item, z_at = kInterleaved ? x_at + 1 : item + p.half;
        const float2 c = cs[item];
        for (int h = lane; h < p.heads; h += p.lanes) {
            const uint16_t *s = src(h);
            uint16_t *d = dst(h);
            uint32_t x = s[x_at] | (uint32_t)s[z_at] << 16;
            turn_one<kBf16>(x, c);
            d[x_at] = (uint16_t)x;
            d[z_at] = (uint16_t)(x >> 16);
            if (p.copy && item == 0)
                for (int i = 2 * p.half; i < copied; ++i)
                    d[i] = s[i];
        }
    }
}

}  // namespace rot
}  // namespace gemmrelu
