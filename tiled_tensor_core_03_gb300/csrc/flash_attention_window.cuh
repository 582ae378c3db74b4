// flash_attention_window.cuh -- attention forward of a prompt with a sliding window and
// first tokens that stay visible:
//
//   O[i] = sum_j softmax_j(q_i . k_j / sqrt(d)) v_j  over the keys j that query i sees:
//   j <= p, and with a window W > 0 also j > p - W or j < sinks,  p = i + n_kv - n_q,
//
// for fp16 or bf16 [batch][seq][heads][d] tensors with strides, query head h reading K/V
// head h / group.  A query that sees nothing gets 0.
//
// The pipeline is flash_attention.cuh's: two 128-row tiles a CTA, ping-ponged between the
// tensor cores (tcgen05.mma, S = Q K^T and O += P V in TMEM, P read from TMEM) and one
// softmax thread per row, K/V blocks of 128 keys through a 2-stage TMA ring.  What differs:
//
//  - The CTA's two tiles are neighbours in the order (query tile, head of the group), so
//    with a shared K/V head they are two heads at the same queries and every block that
//    is loaded serves both.
//  - Blocks are a list: those with a sink that some query's window has left behind, then
//    those from the first query's window to the last query's position.  All else is
//    never loaded, so the work is proportional to the window.  Where the two tiles are
//    at different queries the list is the union, and each tile skips the blocks that it does
//    not see.
//  - A CTA stays and walks over work items, and every hand-off is counted across them: the
//    next item's Q, K and V arrive and its first scores are computed while this one's last
//    softmax and its output are still under way.  With a CTA per item, a window of 8
//    blocks spent a quarter of its time starting and ending.
//  - Of a block whose window part is past only the sinks are left; up to 32 of them
//    are computed as a block of 32 keys instead of 128.
//  - Scores are masked only in blocks where some row does not see some key: the
//    diagonal's, the window's low end, the sinks'.
//  - A key that a row does not see has weight 0, and 0 times a NaN or an infinity in its V
//    would still be NaN.  A CTA that finds a row with finite weights but without a finite result
//    (an element of some V is not finite) therefore walks over its items a second time.  There, in
//    the blocks that some row sees in part, such elements of V become 0 in shared memory and are
//    added by hand to the rows that see them.  That costs about what the first walk did and 3 us for
//    each of those few blocks (0.1 ms where all of V is not finite), whatever the rows' lengths are,
//    so that no wait inside the pipeline gets long: 4 x 4096 tokens, window 1024, one infinity in V 555 us.
//
// Bound: the tensor cores' 4 d flops a pair; blocks are 128 keys wide, so a window of W keys
// costs up to W + 255 keys and the sinks one block.  A tile's turn is a chain, S, softmax, P V, next
// S over the same TMEM columns: about 3300 cycles a block with two tiles in turn, for 2048 cycles
// of products (window 1024: tensor pipe active in 52% of the cycles).  Measured, 32 query heads on 8 of
// 128: 16384 tokens, window 4096, 685 to 702 us (the power limit moves it), 1.39 to 1.42 PFLOP/s of visible
// pairs, 0.71 to 0.73 of the measured burst of 1951.5 TFLOP/s; 4 x 4096 tokens, window 1024, 223 us,
// 1.08 PFLOP/s (9.3 blocks an item for 8 of keys, and 2500 cycles for an item's output); a prompt of 203
// tokens 6.9 us, launch and latency.
// Not kept: 2^x by range reduction and a polynomial for a share of the pairs (a quarter: 262 -> 306 us;
// exponentials are not the bound on this GPU), two threads a row on 16 softmax warps (326 us and more:
// registers), separate K and V rings (272 us), 192 or 168 registers for the softmax (285 us).
#pragma once

#include <cuda_bf16.h>

#include "flash_attention.cuh"

namespace gemmrelu {
namespace attn {

constexpr unsigned kStatusLength = 8;   // == GEMMRELU_ERR_PAGE

// n / d for 0 <= n < 2^31 by a product (Granlund and Montgomery, Division by Invariant Integers using
// Multiplication, 1994): with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1 it is
// (hi(m n) + n) >> l.  A work item needs four, and the compiler's long division delayed the next
// item's scores: 4 x 4096 tokens, 32 heads on 8 of 128, window 128 114 us, now 107.
struct Divisor {
    uint32_t m;
    int l;
    static Divisor of(uint32_t d) {
        Divisor v{0, 0};
        while (v.l < 31 && (1u << v.l) < d)
            ++v.l;
        v.m = (uint32_t)(((((uint64_t)1 << v.l) - d) << 32) / d) + 1;
        return v;
    }
    __host__ __device__ int quotient(int n) const {
#ifdef __CUDA_ARCH__
        return (int)((__umulhi(m, (uint32_t)n) + (uint32_t)n) >> l);
#else
        return (int)(((uint32_t)((uint64_t)m * (uint32_t)n >> 32) + (uint32_t)n) >> l);
#endif
    }
};

struct WindowParams {
    const uint16_t *v;
    int64_t vs[3];                 // sequence, token, head
    uint16_t *o;                   // [batch][n_q][q_heads][d]
    int n_q, n_kv, q_heads, group;
    int q_tiles, items;            // items = q_tiles * group: tiles of one K/V head
    int kv_heads, batch;
    int pairs, window, sinks;
    int chunk, chunk_items;        // K/V heads of all sequences whose items mix, and their items
    Divisor by_chunk, by_last, by_chunk_items, by_kv_heads, by_group;   // (last: the rest of heads)
    const int32_t *states;         // cross attention: keys of each sequence (or nullptr: n_kv)
    int tile_tokens;               //                  queries of a tile, each with all heads of the group
    float scale;                   // log2(e) / sqrt(d)
    float shift;                   // bf16: what a row's reference stands above its largest score
    int drop_arrive;
    uint64_t wait_limit_ns;
};

// D fp32, A and B both fp16 (0) or both bf16 (1).
__host__ __device__ constexpr uint32_t with_type(uint32_t idesc, bool bf16) {
    return idesc | (bf16 ? (1u << 7) | (1u << 10) : 0u);
}

// The blocks of 128 keys that some row of a tile sees: [0, sinks) and [low, high).
struct Blocks {
    int sinks, low, high;
    __host__ __device__ bool has(int blk) const { return blk < sinks || (blk >= low && blk < high); }
    __host__ __device__ int count() const { return sinks + high - low; }
};

// Rows at positions first .. last (first may be negative, last < n_kv).
__host__ __device__ inline Blocks blocks_seen(int first, int last, int window, int sinks) {
    Blocks b{0, 0, 0};
    if (last < 0)
        return b;
    b.high = last / BN + 1;
    if (window > 0 && first >= window) {
        const int low = first - window + 1;
        const int head = sinks < low ? sinks : low;
        b.low = low / BN;
        b.sinks = (head + BN - 1) / BN;
        if (b.sinks > b.low)
            b.sinks = b.low;
    }
    return b;
}

template <bool kBf16>
__device__ __forceinline__ float to_float(uint32_t x16) {
    if constexpr (kBf16)
        return __uint_as_float(x16 << 16);
    else
        return __half2float(__ushort_as_half((unsigned short)x16));
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
    if constexpr (kBf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        return pack_half2(a, b);
    }
}

// The halves of a pair that are an infinity or a NaN (all exponent bits set): 0x8000 in their place.
template <bool kBf16>
__device__ __forceinline__ uint32_t not_finite(uint32_t pair) {
    return kBf16 ? ((pair & 0x7f807f80u) + 0x00800080u) & 0x80008000u
                 : ((pair & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
}

template <bool kBf16>
__device__ __forceinline__ uint32_t finite_part(uint32_t pair) {
    return pair & ~((not_finite<kBf16>(pair) >> 15) * 0xffffu);
}

// One key of a block per thread: whether its V row (in global memory; nullptr past the last key) has
// elements that are not finite.  Those become 0 in the block's copy in shared memory, whose
// row `r` of 64 elements a sub-tile starts at `smem_row`.
template <int HD, bool kBf16>
__device__ __noinline__ bool clean_row(const uint16_t *row, uint32_t smem_row, int r) {
    uint32_t bad = 0;
    if (row != nullptr)
#pragma unroll 4
        for (int c = 0; c < HD / 8; ++c) {
            const uint4 x = *reinterpret_cast<const uint4 *>(row + 8 * c);
            bad |= not_finite<kBf16>(x.x) | not_finite<kBf16>(x.y) | not_finite<kBf16>(x.z) | not_finite<kBf16>(x.w);
        }
    if (bad)
#pragma unroll 1
        for (int c = 0; c < HD / 8; ++c) {
            const uint32_t at = smem_row + (c >> 3) * kSub + ((uint32_t)((c & 7) ^ (r & 7)) << 4);
            const uint4 x = ld_shared_v4(at);
            st_shared_v4(at, finite_part<kBf16>(x.x), finite_part<kBf16>(x.y), finite_part<kBf16>(x.z),
                         finite_part<kBf16>(x.w));
        }
    return bad != 0;
}

// Add what clean_row took out of a block to the warp's 32 rows of O in TMEM: `keys` has a bit for each of the
// block's keys with such elements, `v` points at the first one's row.  Their sum (an infinity, or a NaN)
// takes the place of what weights above 0 would give.
template <int HD, bool kBf16>
__device__ __noinline__ void add_not_finite(const WindowParams &p, const uint16_t *v, const uint32_t *keys, int key0,
                                            int pos, uint32_t o_addr) {
#pragma unroll 1
    for (int c0 = 0; c0 < HD; c0 += 32) {
        uint32_t o[32];
        tmem_ld_x32_sync(o_addr + c0, o);
#pragma unroll 1
        for (int w = 0; w < BN / 32; ++w) {
#pragma unroll 1
            for (uint32_t left = keys[w]; left; left &= left - 1) {
                const int i = 32 * w + __ffs(left) - 1, key = key0 + i;
                if (key > pos || (p.window > 0 && key <= pos - p.window && key >= p.sinks))
                    continue;
                const uint4 *row = reinterpret_cast<const uint4 *>(v + i * p.vs[1] + c0);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint4 y = row[c];
                    const uint32_t x[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t bad = not_finite<kBf16>(x[e]);
                        uint32_t &lo = o[8 * c + 2 * e], &hi = o[8 * c + 2 * e + 1];
                        if (bad & 0x8000u)
                            lo = __float_as_uint(__uint_as_float(lo) + to_float<kBf16>(x[e] & 0xffffu));
                        if (bad & 0x80000000u)
                            hi = __float_as_uint(__uint_as_float(hi) + to_float<kBf16>(x[e] >> 16));
                    }
                }
            }
            __syncwarp();
        }
        tmem_st_x32(o_addr + c0, o);
    }
    tmem_st_wait();
}

// Shared memory of flash_attention.cuh with more barriers: q_full, q_empty, k_full[kKV],
// v_full[kKV], kv_empty[kKV], s_full[2], p_full[2], o_full[2], o_empty[2], v_clean[2], drain.
template <int HD>
struct WindowCfg : Cfg<HD> {
    static constexpr uint32_t kNumBars = 2 + 3 * kKV + 10 + 1;
    static constexpr uint32_t kOffMisc = Cfg<HD>::kOffBar + kNumBars * 8;
    static constexpr uint32_t kOffKeys = kOffMisc + 16;   // [kTiles][2][BN / 32]: keys with V that is not finite
    static constexpr uint32_t kSmemBytes = kOffKeys + kTiles * 2 * (BN / 32) * 4 + 1024;
    static constexpr int kNarrow = 32;   // keys of a block with few sinks only
    static constexpr uint32_t kIdescNarrow = make_idesc_f16_f32(BM, kNarrow, 0, 0);
};

// Three warpgroups: two of softmax, one with the producer's and the issuer's warp.  384 threads
// launch with 168 registers; the third warpgroup keeps 72 and the others take 216 each, which
// holds a row's 128 scores and the loop around them: 2 * 216 + 72 = 3 * 168.
constexpr int kWindowThreads = 384;
constexpr float kHugeLog2 = 16777216.0f;   // 2^24: scores from here on are rounded before they are referred
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 216, kOtherRegs = 72;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "registers given back cover those taken");

// One thread of the (converged) warp, chosen by the hardware.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
    return r != 0;
}

// wait_bounded_eager by a whole warp, with one answer.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                          volatile uint32_t *abort_flag, unsigned where) {
    return __all_sync(0xffffffffu, wait_bounded_eager(bar, parity, limit_ns, abort_flag, where));
}

// The lowest n of 32 bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t keys_below(int n) {
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1;
}

// The entries of a block list that a tile takes part in: [0, head) and [from, to).
struct Turns {
    int head, from, to;
    __device__ __forceinline__ bool has(int j) const { return j < head || (j >= from && j < to); }
    __device__ __forceinline__ int count() const { return head + to - from; }
};

// A work item: two neighbouring tiles of one K/V head, and the list of the blocks that either
// sees: entries 0 .. sinks - 1 are the first blocks, the others follow from block low.
struct WindowItem {
    int kvh, batch;
    int tile0, tile1, head0, head1;
    bool two;
    int sinks, low, nb;
    int narrow;              // the entry with no more than 32 sinks and nothing else, or -1
    Turns t0, t1;
    __device__ __forceinline__ int block(int j) const { return j < sinks ? j : low + (j - sinks); }
};

// The items of this CTA, one a round.  Within a chunk of heads their cost falls, so that with
// rounds dealt out forwards and backwards in turn every CTA gets about the same sum.  (kCross: their cost falls over all
// of them, and the CTAs that a last, short round leaves out are those with the most before it.)
template <bool kCross>
struct WindowWalk {
    int base, total;
    bool back;
    __device__ __forceinline__ WindowWalk(const WindowParams &p)
        : base(0), total(p.pairs * p.kv_heads * p.batch), back(false) {}
    __device__ __forceinline__ bool more() const { return (kCross ? index() : base + (int)blockIdx.x) < total; }
    __device__ __forceinline__ int index() const {
        if (kCross)
            return base + (back ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
        return back ? min(base + (int)gridDim.x, total) - 1 - (int)blockIdx.x : base + (int)blockIdx.x;
    }
    __device__ __forceinline__ void next() {
        base += gridDim.x;
        back = !back;
    }
};

// Keys of a sequence in cross attention: none where the number is out of range.
__device__ __forceinline__ int states_of(const WindowParams &p, int batch) {
    if (p.states == nullptr)
        return p.n_kv;
    const int n = p.states[batch];
    if (n < 0 || n > p.n_kv) {
        atomicCAS(&g_status, 0u, kStatusLength);
        return 0;
    }
    return n;
}

template <int HD, bool kCross>
__device__ __forceinline__ WindowItem window_item(const WindowParams &p, int index, const uint8_t *order) {
    WindowItem w;
    // the last queries see the most keys: they go first
    const int chunk = p.by_chunk_items.quotient(index), first = chunk * p.chunk;
    const int heads = min(p.chunk, p.kv_heads * p.batch - first);
    index -= chunk * p.chunk_items;
    const int rank = (heads == p.chunk ? p.by_chunk : p.by_last).quotient(index);
    const int pair = p.pairs - 1 - rank, off = p.n_kv - p.n_q, item = 2 * pair;
    index = first + index - rank * heads;
    w.batch = p.by_kv_heads.quotient(index);
    w.kvh = index - w.batch * p.kv_heads;
    w.two = item + 1 < p.items;
    if constexpr (kCross) {   // every row sees every key that there is
        if (order != nullptr)
            w.batch = order[w.batch];
        w.tile0 = item;
        w.tile1 = item + 1;
        w.head0 = w.head1 = w.kvh * p.group;
        w.sinks = w.low = 0;
        w.nb = (states_of(p, w.batch) + BN - 1) / BN;
        w.narrow = -1;
        w.t0 = Turns{0, 0, w.nb};
        w.t1 = Turns{0, 0, w.two ? w.nb : 0};
        return w;
    }
    w.tile0 = p.by_group.quotient(item);
    const int g = item - w.tile0 * p.group;
    w.head0 = w.kvh * p.group + g;
    const bool same = g + 1 < p.group;   // the second tile: the next head, or the next queries
    w.tile1 = same ? w.tile0 : w.tile0 + 1;
    w.head1 = same ? w.head0 + 1 : w.kvh * p.group;
    auto seen_by = [&](int tile) {
        return blocks_seen(tile * BM + off, min(tile * BM + BM, p.n_q) - 1 + off, p.window, p.sinks);
    };
    const Blocks b0 = seen_by(w.tile0), b1 = !w.two ? Blocks{0, 0, 0} : same ? b0 : seen_by(w.tile1);
    Blocks all = b0;
    if (b1.count() > 0) {
        if (b0.count() == 0) {
            all = b1;
        } else {
            all.low = min(b0.low, b1.low);
            all.high = max(b0.high, b1.high);
            all.sinks = min(max(b0.sinks, b1.sinks), all.low);
        }
    }
    auto turns_of = [&](const Blocks &b) {
        if (b.count() == 0)
            return Turns{0, 0, 0};
        // (a tile's first blocks may reach into the part from `low` on)
        const int head = b.sinks <= all.sinks ? b.sinks : all.sinks + max(0, b.sinks - all.low);
        return Turns{head, all.sinks + b.low - all.low, all.sinks + b.high - all.low};
    };
    w.sinks = all.sinks;
    w.low = all.low;
    w.nb = all.count();
    w.t0 = turns_of(b0);
    w.t1 = turns_of(b1);
    const int last = p.sinks / BN, left = p.sinks - last * BN;
    w.narrow = left > 0 && left <= WindowCfg<HD>::kNarrow && last < all.sinks ? last : -1;
    return w;
}

// kCross: cross attention.  Queries see all keys of their sequence (states_of), and a tile's rows are
// tile_tokens queries with all heads of one K/V head's group.  Up to kMostOrdered sequences go by their number of keys,
// the longest first, so that a CTA whose first item is long gets a short one in the next round (448 queries, 16 heads of 64:
// 8 sequences of up to 1500 keys 33.4 us, 36.6 in the batch's order; 6 of up to 3000 38.2, and 52.0 where the heads' last
// queries all went first, and the CTAs with the least before it got nothing of the last round).
// Weights are rounded to the inputs' type, as in the windowed form: the second product takes both operands in one type (against
// 64 bits, bf16 0.0023 of the result, 0.0017 with weights in 32 bits; fp16 0.00029 and 0.00021).
constexpr int kMostOrdered = 128;

template <int HD, bool kBf16, bool kCross = false>
__global__ void __launch_bounds__(kWindowThreads, 1)
    flash_attention_window_kernel(const __grid_constant__ CUtensorMap tmQ,
                                  const __grid_constant__ CUtensorMap tmK,
                                  const __grid_constant__ CUtensorMap tmV,
                                  const __grid_constant__ WindowParams p) {
    using G = WindowCfg<HD>;
    constexpr uint32_t kIdescS = with_type(G::kIdescS, kBf16);
    constexpr uint32_t kIdescO = with_type(G::kIdescO, kBf16);
    constexpr uint32_t kIdescNarrow = with_type(G::kIdescNarrow, kBf16);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);

    const uint32_t bar0 = base + G::kOffBar;
    const uint32_t q_full = bar0, q_empty = bar0 + 8u;
    auto k_full = [&](uint32_t s) { return bar0 + 8u * (2 + s); };
    auto v_full = [&](uint32_t s) { return bar0 + 8u * (2 + kKV + s); };
    auto kv_empty = [&](uint32_t s) { return bar0 + 8u * (2 + 2 * kKV + s); };
    auto s_full = [&](uint32_t t) { return bar0 + 8u * (2 + 3 * kKV + t); };
    auto p_full = [&](uint32_t t) { return bar0 + 8u * (4 + 3 * kKV + t); };
    auto o_full = [&](uint32_t t) { return bar0 + 8u * (6 + 3 * kKV + t); };
    auto o_empty = [&](uint32_t t) { return bar0 + 8u * (8 + 3 * kKV + t); };
    auto v_clean = [&](uint32_t t) { return bar0 + 8u * (10 + 3 * kKV + t); };
    const uint32_t drain_bar = bar0 + 8u * (12 + 3 * kKV);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + G::kOffMisc);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + G::kOffMisc + 4);
    volatile uint32_t *redo_flag = reinterpret_cast<volatile uint32_t *>(gbase + G::kOffMisc + 8);

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);   // uniform
    const int lane = threadIdx.x & 31;
    const int off = p.n_kv - p.n_q;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1u);
        mbar_init(q_empty, 1u);
        for (uint32_t s = 0; s < (uint32_t)kKV; ++s) {
            mbar_init(k_full(s), 1u);
            mbar_init(v_full(s), 1u);
            mbar_init(kv_empty(s), 1u);
        }
        for (uint32_t t = 0; t < (uint32_t)kTiles; ++t) {
            mbar_init(s_full(t), 1u);
            mbar_init(p_full(t), 4u);
            mbar_init(o_full(t), 1u);
            mbar_init(o_empty(t), 4u);
            mbar_init(v_clean(t), 4u);
        }
        mbar_init(drain_bar, 1u);
        *abort_flag = 0u;
        *redo_flag = 0u;
        fence_mbar_init();
        pdl_launch_dependents();
    }
    if (warp == kProducerWarp && lane == 0) {
        tma_prefetch_map(&tmQ);
        tma_prefetch_map(&tmK);
        tma_prefetch_map(&tmV);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_addr(tmem_slot), G::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
    pdl_wait_primary();  // the previous grid of the stream has completed
    const uint8_t *order = nullptr;
    if constexpr (kCross) {
        // Rows of a tile that no copy writes (a group that does not divide 128): what they hold must not decide for the warp
        // how the other rows' weights are rounded.
        const int used = p.tile_tokens * p.group;
        for (int i = threadIdx.x; i < kTiles * G::kDSub * (BM - used) * 8; i += kWindowThreads)
            st_shared_v4(base + G::kOffQ + i / ((BM - used) * 8) * kSub + used * 128 + i % ((BM - used) * 8) * 16, 0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        tc_fence_before_sync();
        __syncthreads();
        tc_fence_after_sync();
        __shared__ uint8_t by_length[kMostOrdered];
        if (p.states != nullptr && p.batch <= kMostOrdered && p.pairs * p.kv_heads * p.batch > (int)gridDim.x) {
            if ((int)threadIdx.x < p.batch) {
                const int mine = states_of(p, threadIdx.x);
                int rank = 0;
                for (int i = 0; i < p.batch; ++i) {
                    const int n = states_of(p, i);
                    rank += n > mine || (n == mine && i < (int)threadIdx.x);
                }
                by_length[rank] = (uint8_t)threadIdx.x;
            }
            __syncthreads();
            order = by_length;
        }
    }

    // The end of a walk over the items, for every warp: whether a second one follows.
    auto once_more = [&](int pass) {
        __syncwarp();
        tc_fence_before_sync();
        named_bar_sync(1, kWindowThreads);
        tc_fence_after_sync();
        if (pass != 0 || *redo_flag == 0u)
            return false;
        const bool go = *abort_flag == 0u;
        named_bar_sync(1, kWindowThreads);   // all have read it before a wait of the second walk may set it
        return go;
    };

    if (warp >= kProducerWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        // ============================================================ TMA producer
        if (warp == kProducerWarp) {
            uint32_t queries = 0, blocks = 0;   // Q loads and K/V blocks issued
            bool ok = !(p.drop_arrive && blockIdx.x == 0);
            for (int pass = 0;; ++pass) {
                for (WindowWalk<kCross> walk(p); lane == 0 && ok && walk.more(); walk.next()) {
                    const WindowItem w = window_item<HD, kCross>(p, walk.index(), order);
                    if (w.nb == 0)
                        continue;
                    ok = wait_bounded_eager(q_empty, (queries & 1u) ^ 1u, p.wait_limit_ns, abort_flag,
                                            kSiteProducerEmpty);
                    if (!ok)
                        break;
                    const uint32_t q_bytes = kCross ? (uint32_t)(p.tile_tokens * p.group) * HD * 2u : G::kQBytes;
                    const int q_step = kCross ? p.tile_tokens : BM;
                    mbar_arrive_expect_tx(q_full, (w.two ? 2u : 1u) * q_bytes);
                    for (int t = 0; t < (w.two ? 2 : 1); ++t)
#pragma unroll
                        for (int d = 0; d < G::kDSub; ++d)
                            tma_load_4d(&tmQ, base + G::kOffQ + t * G::kQBytes + d * kSub, q_full,
                                        64 * d, t ? w.head1 : w.head0, (t ? w.tile1 : w.tile0) * q_step, w.batch);
                    ++queries;
                    for (int j = 0; j < w.nb; ++j) {
                        const uint32_t st = blocks % kKV, ph = blocks / kKV & 1u;
                        ok = wait_bounded_eager(kv_empty(st), ph ^ 1u, p.wait_limit_ns, abort_flag,
                                                kSiteProducerEmpty);
                        if (!ok)
                            break;
                        const int key = w.block(j) * BN;
                        mbar_arrive_expect_tx(k_full(st), G::kKBytes);
#pragma unroll
                        for (int d = 0; d < G::kDSub; ++d)
                            tma_load_4d(&tmK, base + G::kOffK + st * G::kKBytes + d * kSub, k_full(st),
                                        64 * d, w.kvh, key, w.batch);
                        mbar_arrive_expect_tx(v_full(st), G::kVBytes);
#pragma unroll
                        for (int d = 0; d < G::kDSub; ++d)
                            tma_load_4d(&tmV, base + G::kOffV + st * G::kVBytes + d * kSub, v_full(st),
                                        64 * d, w.kvh, key, w.batch);
                        ++blocks;
                    }
                }
                // every copy issued must have landed before the CTA may exit
                if (queries > 0)   // (lane 0)
                    wait_drain(q_full, (queries - 1) & 1u, p.wait_limit_ns, abort_flag);
                for (uint32_t i = blocks > (uint32_t)kKV ? blocks - kKV : 0u; i < blocks; ++i) {
                    wait_drain(k_full(i % kKV), i / kKV & 1u, p.wait_limit_ns, abort_flag);
                    wait_drain(v_full(i % kKV), i / kKV & 1u, p.wait_limit_ns, abort_flag);
                }
                if (!once_more(pass))
                    break;
            }
        }
        // ============================================================ MMA issuer
        if (warp == kMmaWarp) {
            // One elected thread issues, but the whole warp walks along: control flow and operands
            // are then uniform, and the MMAs' descriptors stay in uniform registers.  In a
            // branch of one lane each of them was moved there instruction by instruction, and
            // issuing bound the kernel (16384 tokens, window 4096, 32 heads of 128: 1077 us
            // against 781 us).  An item's list is worked out during the item before it, and a
            // load that the first tile has waited for is not waited for again (136 cycles).
            const bool leader = elect_one();
            const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
            const uint64_t q_desc = make_sdesc_sw128(base + G::kOffQ, 16, 1024);
            const uint64_t k_desc = make_sdesc_sw128(base + G::kOffK, 16, 1024);
            const uint64_t v_desc = make_sdesc_sw128(base + G::kOffV, kSub, 1024);
            bool ok = true;
            uint32_t queries = 0;                 // items with blocks so far
            uint32_t blocks = 0;                  // K/V blocks before the one in hand
            uint32_t turns0 = 0, turns1 = 0;      // P V products of each tile so far
            uint32_t outs0 = 0, outs1 = 0;        // items of each tile with an output so far
            // S_t = Q_t K^T of block number i
            auto score = [&](const uint32_t t, uint32_t i, bool narrow, bool waited) -> bool {
                const uint32_t st = i % kKV;
                if (!waited && !wait_warp(k_full(st), i / kKV & 1u, p.wait_limit_ns, abort_flag, kSiteMmaFull))
                    return false;
                tc_fence_after_sync();
                const uint64_t qd = q_desc + t * (G::kQBytes >> 4), kd = k_desc + st * (G::kKBytes >> 4);
                const uint32_t idesc = narrow ? kIdescNarrow : kIdescS;
#pragma unroll
                for (int kk = 0; kk < HD / UKA; ++kk) {
                    const uint32_t o = (kk / 4) * (kSub >> 4) + (kk % 4) * 2;
                    if (leader)
                        umma_f16(tmem + G::kTmemS + t * BN, qd + o, kd + o, idesc, kk > 0 ? 1u : 0u);
                }
                if (leader)
                    umma_commit(s_full(t));
                return true;
            };
            // O_t += P_t V of block number i, P_t from TMEM (over S_t); O_t starts afresh with
            // an item's first block, and is complete with its last
            auto pv = [&](const uint32_t t, uint32_t i, bool narrow, bool waited, bool fresh, bool complete,
                          uint32_t &turns, uint32_t &outs) -> bool {
                const uint32_t st = i % kKV;
                if ((!waited && !wait_warp(v_full(st), i / kKV & 1u, p.wait_limit_ns, abort_flag, kSiteMmaFull)) ||
                    (fresh && !wait_warp(o_empty(t), (outs & 1u) ^ 1u, p.wait_limit_ns, abort_flag,
                                                  kSiteMmaAccEmpty)) ||
                    !wait_warp(p_full(t), turns & 1u, p.wait_limit_ns, abort_flag, kSiteMmaAccEmpty))
                    return false;
                tc_fence_after_sync();
                const uint64_t vd = v_desc + st * (G::kVBytes >> 4);
                const uint32_t d_o = tmem + G::kTmemO + t * HD, a_p = tmem + G::kTmemS + t * BN;
                if (leader)
                    umma_f16_ts(d_o, a_p, vd, kIdescO, fresh ? 0u : 1u);
#pragma unroll
                for (int kk = 1; kk < G::kNarrow / UKA; ++kk)
                    if (leader)
                        umma_f16_ts(d_o, a_p + kk * (UKA / 2), vd + kk * ((UKA * 128) >> 4), kIdescO, 1u);
                if (!narrow) {
#pragma unroll
                    for (int kk = G::kNarrow / UKA; kk < BN / UKA; ++kk)
                        if (leader)
                            umma_f16_ts(d_o, a_p + kk * (UKA / 2), vd + kk * ((UKA * 128) >> 4), kIdescO, 1u);
                }
                ++turns;
                if (complete) {
                    if (leader)
                        umma_commit(o_full(t));
                    ++outs;
                }
                return true;
            };
            for (int pass = 0;; ++pass) {
                WindowWalk<kCross> walk(p);
                WindowItem w{};
                if (walk.more())
                    w = window_item<HD, kCross>(p, walk.index(), order);
                while (ok && walk.more()) {
                    const int nb = w.nb, narrow = w.narrow;
                    const Turns t0 = w.t0, t1 = w.t1;
                    if (nb > 0) {
                        ok = wait_warp(q_full, queries & 1u, p.wait_limit_ns, abort_flag, kSiteMmaFull);
                        ++queries;
                        if (ok && t0.has(0))
                            ok = score(0, blocks, narrow == 0, false);
                        if (ok && t1.has(0))
                            ok = score(1, blocks, narrow == 0, t0.has(0));
                        if (ok && nb == 1 && leader)
                            umma_commit(q_empty);
                    }
                    walk.next();
                    if (walk.more())
                        w = window_item<HD, kCross>(p, walk.index(), order);
                    bool fresh0 = true, fresh1 = true;
                    for (int j = 0; ok && j < nb; ++j, ++blocks) {
                        const bool here = j == narrow, there = j + 1 == narrow, more = j + 1 < nb;
                        if (t0.has(j)) {
                            ok = pv(0, blocks, here, false, fresh0, j + 1 == t0.to, turns0, outs0);
                            fresh0 = false;
                        }
                        if (ok && more && t0.has(j + 1))
                            ok = score(0, blocks + 1, there, false);
                        if (ok && t1.has(j)) {
                            ok = pv(1, blocks, here, t0.has(j), fresh1, j + 1 == t1.to, turns1, outs1);
                            fresh1 = false;
                        }
                        if (!ok)
                            break;
                        if (leader)
                            umma_commit(kv_empty(blocks % kKV));
                        if (more && t1.has(j + 1))
                            ok = score(1, blocks + 1, there, t0.has(j + 1));
                        if (ok && j + 2 == nb && leader)
                            umma_commit(q_empty);   // the item's last scores
                    }
                }
                // all MMAs of this thread complete before TMEM can be released
                if (leader)
                    umma_commit(drain_bar);
                wait_drain(drain_bar, pass & 1u, p.wait_limit_ns, abort_flag);
                if (!once_more(pass))
                    break;
            }
        }
        // the other two warps complete the warpgroup
        for (int pass = 0; warp > kMmaWarp; ++pass)
            if (!once_more(pass))
                break;
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ============================================================ softmax / output
        const int t = warp >> 2;                        // tile
        const int q = warp & 3;                         // TMEM lanes 32q .. 32q+31
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        const uint32_t s_addr = tmem_base + lane_base + G::kTmemS + t * BN;
        const uint32_t o_addr = tmem_base + lane_base + G::kTmemO + t * HD;
        uint32_t turns = 0, outputs = 0;
        uint32_t blocks = 0;                            // K/V blocks before the item in hand
        bool alive = true;
        // the second walk over the items (see above)
        uint32_t *keys = reinterpret_cast<uint32_t *>(gbase + G::kOffKeys) + t * 2 * (BN / 32);
        uint32_t redo = 0, cleaned = 0;
        auto reached = [&](uint32_t bar, uint32_t phase) {
            return __all_sync(0xffffffffu, wait_bounded(bar, phase & 1u, p.wait_limit_ns, abort_flag, kSiteEpiAccFull));
        };
        // (compiled once for each walk: the second one's code between the turns cost the first 2.7%)
        auto walk_items = [&](auto again) __attribute__((always_inline)) {
            constexpr bool kAgain = decltype(again)::value;
            for (WindowWalk<kCross> walk(p); alive && walk.more(); walk.next()) {
                const WindowItem w = window_item<HD, kCross>(p, walk.index(), order);
                const uint32_t block0 = blocks;
                blocks += w.nb;
                if (t == 1 && !w.two)
                    continue;
                const int tile = t ? w.tile1 : w.tile0;
                int head = t ? w.head1 : w.head0;
                const Turns mine = t ? w.t1 : w.t0;
                int qi = tile * BM + 32 * q + lane;             // query index
                int pos = qi + off;
                int first = tile * BM + off, last = min(tile * BM + BM, p.n_q) - 1 + off;
                if constexpr (kCross) {
                    const int r = 32 * q + lane, nth = p.by_group.quotient(r);
                    head += r - nth * p.group;
                    qi = nth < p.tile_tokens ? tile * p.tile_tokens + nth : p.n_q;
                    pos = first = last = states_of(p, w.batch) - 1;
                }
                // some row of a tile does not see some key of the block
                auto masked_for = [&](int first, int last, int key0) {
                    return key0 + BN - 1 > first ||
                           (p.window > 0 && key0 <= last - p.window && key0 + BN > p.sinks);
                };
                const int tile_b = t ? w.tile0 : w.tile1;       // the item's other tile
                const Turns other = t ? w.t0 : w.t1;
                const uint16_t *v_head = p.v + w.batch * p.vs[0] + w.kvh * p.vs[2];
                // the first key of a block whose elements that are not finite are still to be added
                int taken = -1;
                auto add_taken = [&]() {
                    if (taken >= 0)
                        add_not_finite<HD, kBf16>(p, v_head + taken * p.vs[1],
                                                  keys + ((turns - 1u) & 1u) * (BN / 32), taken, pos, o_addr);
                    taken = -1;
                };
                float m = -INFINITY, l = 0.0f;
                uint32_t done = 0;
                // one block of kKeys keys: scores from TMEM, P as 16-bit pairs over them
                auto softmax = [&](auto keys, int key0, bool masked) {
                    constexpr int kKeys = decltype(keys)::value;
                    uint32_t v[kKeys];
#pragma unroll
                    for (int c0 = 0; c0 < kKeys; c0 += 32)
                        tmem_ld_x32(s_addr + c0, *reinterpret_cast<uint32_t(*)[32]>(&v[c0]));
#pragma unroll
                    for (int c0 = 0; c0 < kKeys; c0 += 32)
                        tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&v[c0]));
                    if (masked) {
                        // a bit per key, 32 at a time: seen up to `hi`, above `lo` or below `head` (three
                        // compares a key instead: 262 us for 241 at window 1024)
                        const int hi = pos - key0;
                        const int lo = p.window > 0 ? hi - p.window : -1;
                        const int head = p.sinks - key0;
#pragma unroll
                        for (int c0 = 0; c0 < kKeys; c0 += 32) {
                            const uint32_t seen = keys_below(hi + 1 - c0) & (~keys_below(lo + 1 - c0) | keys_below(head - c0));
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[c0 + i] = seen & (1u << i) ? v[c0 + i] : __float_as_uint(-INFINITY);
                        }
                    }
                    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
                    for (int i = 0; i < kKeys; i += 2) {
                        mx0 = fmaxf(mx0, __uint_as_float(v[i]));
                        mx1 = fmaxf(mx1, __uint_as_float(v[i + 1]));
                    }
                    // scale > 0; with bf16 a sum of weights stays below 1, so that O, which is a sum with
                    // weights until it is divided, stays within the largest V and fp32
                    const float m_blk = __fadd_rn(__fmul_rn(fmaxf(mx0, mx1), p.scale), kBf16 ? p.shift : 0.0f);
                    // move the reference only when the maximum grew by more than kRescaleLog2;
                    // -infinity until the row has seen a key
                    const bool move = m_blk > m + kRescaleLog2;
                    const float m_new = move ? m_blk : m;
                    const float alpha = move ? fast_exp2(m - m_new) : 1.0f;   // 0 at the first block
                    const float m_ref = m_new == -INFINITY ? 0.0f : m_new;
                    // The products below take score * scale unrounded, the reference is rounded: from 2^24 on
                    // their difference at a row's largest key would be half a unit and more, at 2^31 an overflow.
                    float sc = p.scale;
                    if (__any_sync(0xffffffffu, fabsf(m_ref) >= kHugeLog2)) {
#pragma unroll
                        for (int i = 0; i < kKeys; ++i)
                            v[i] = __float_as_uint(__fmul_rn(__uint_as_float(v[i]), p.scale));
                        sc = 1.0f;
                    }
                    const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-m_ref, -m_ref);
                    float2 sa = make_float2(0.0f, 0.0f), sb = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int c0 = 0; c0 < kKeys; c0 += 32) {
                        uint32_t ph[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float2 x01 = __ffma2_rn(
                                make_float2(__uint_as_float(v[c0 + i]), __uint_as_float(v[c0 + i + 1])), sc2, nm2);
                            const float2 x23 = __ffma2_rn(
                                make_float2(__uint_as_float(v[c0 + i + 2]), __uint_as_float(v[c0 + i + 3])), sc2, nm2);
                            const float2 e01 = make_float2(fast_exp2(x01.x), fast_exp2(x01.y));
                            const float2 e23 = make_float2(fast_exp2(x23.x), fast_exp2(x23.y));
                            sa = __fadd2_rn(sa, e01);
                            sb = __fadd2_rn(sb, e23);
                            ph[i / 2] = pack_pair<kBf16>(e01.x, e01.y);
                            ph[i / 2 + 1] = pack_pair<kBf16>(e23.x, e23.y);
                        }
                        tmem_st_x16(s_addr + c0 / 2, ph);
                    }
                    l = l * alpha + ((sa.x + sa.y) + (sb.x + sb.y));
                    m = m_new;
                    // rescale this warp's output rows when any of their references moved
                    // (the previous P V of this tile completed before S_j was written)
                    if (done > 0 && __any_sync(0xffffffffu, move)) {
#pragma unroll 1
                        for (int c0 = 0; c0 < HD; c0 += 32) {
                            uint32_t o[32];
                            tmem_ld_x32_sync(o_addr + c0, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            tmem_st_x32(o_addr + c0, o);
                        }
                    }
                    tmem_st_wait();
                };
                for (int j = 0; j < w.nb; ++j) {
                    if (!mine.has(j))
                        continue;
                    const bool ok = wait_bounded_eager(s_full((uint32_t)t), turns & 1u, p.wait_limit_ns,
                                                       abort_flag, kSiteEpiAccFull);
                    if (!__all_sync(0xffffffffu, ok)) {
                        alive = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const int key0 = w.block(j) * BN;
                    if constexpr (kAgain) {
                        add_taken();   // (the P V before this turn is done)
                        // where every row of both tiles sees every key the products do it all
                        const int first_b = kCross ? first : tile_b * BM + off;
                        const int last_b = kCross ? last : min(tile_b * BM + BM, p.n_q) - 1 + off;
                        if (masked_for(first, last, key0) || (other.has(j) && masked_for(first_b, last_b, key0))) {
                            const uint32_t i = block0 + j, st = i % kKV;
                            alive = reached(v_full(st), i / kKV);
                            if (!alive)
                                break;
                            const int r = 32 * q + lane, key = key0 + r;
                            const bool bad = clean_row<HD, kBf16>(key < p.n_kv ? v_head + key * p.vs[1] : nullptr,
                                                                  base + G::kOffV + st * G::kVBytes + r * 128, r);
                            fence_proxy_async_smem();
                            uint32_t *words = keys + (turns & 1u) * (BN / 32);
                            const uint32_t word = __ballot_sync(0xffffffffu, bad);
                            if (lane == 0) {
                                words[q] = word;
                                mbar_arrive(v_clean((uint32_t)t));
                            }
                            __syncwarp();
                            // (bounded, unlike a named barrier: another warp of the tile may have given up)
                            alive = reached(v_clean((uint32_t)t), cleaned++);
                            if (!alive)
                                break;
                            if (words[0] | words[1] | words[2] | words[3])
                                taken = key0;
                        }
                    }
                    const bool masked = masked_for(first, last, key0);
                    if (j == w.narrow)
                        softmax(std::integral_constant<int, G::kNarrow>{}, key0, true);
                    else
                        softmax(std::integral_constant<int, BN>{}, key0, masked);
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(p_full((uint32_t)t));
                    ++turns;
                    ++done;
                }
                if (!alive)
                    break;
                // the tile's last P V, then O / l rounded once
                if (done > 0) {
                    const bool ok = wait_bounded_eager(o_full((uint32_t)t), outputs & 1u, p.wait_limit_ns,
                                                       abort_flag, kSiteEpiAccFull);
                    if (!__all_sync(0xffffffffu, ok)) {
                        alive = false;
                        break;
                    }
                    ++outputs;
                    tc_fence_after_sync();
                    if constexpr (kAgain)
                        add_taken();
                }
                const float inv_l = l == 0.0f ? 0.0f : 1.0f / l;
                uint16_t *dst = p.o + (((int64_t)w.batch * p.n_q + qi) * p.q_heads + head) * HD;
                bool fine = true;
#pragma unroll 1
                for (int c0 = 0; c0 < HD; c0 += 32) {
                    uint32_t o[32];
                    uint32_t h[16];
                    if (done > 0) {
                        tmem_ld_x32_sync(o_addr + c0, o);
                        if (c0 + 32 == HD) {   // O_t may be written again
                            tc_fence_before_sync();
                            __syncwarp();
                            if (lane == 0)
                                mbar_arrive(o_empty((uint32_t)t));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float x = done > 0 ? __uint_as_float(o[2 * i]) * inv_l : 0.0f;
                        const float y = done > 0 ? __uint_as_float(o[2 * i + 1]) * inv_l : 0.0f;
                        fine = fine && fabsf(x) < INFINITY && fabsf(y) < INFINITY;
                        h[i] = pack_pair<kBf16>(x, y);
                    }
                    if (qi < p.n_q) {
                        uint4 *d4 = reinterpret_cast<uint4 *>(dst + c0);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            d4[i] = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
                    }
                }
                redo |= !fine && l == l && qi < p.n_q;   // (a NaN among its weights: the row is NaN)
            }
        };
        walk_items(std::false_type{});
        if (redo != 0u)
            *redo_flag = 1u;
        if (once_more(0)) {
            walk_items(std::true_type{});
            once_more(1);
        }
    }

    // ---------------------------------------------------------------- teardown
    if (warp == kMmaWarp)
        tmem_dealloc(tmem_base, G::kTmemCols);
}

}  // namespace attn
}  // namespace gemmrelu
