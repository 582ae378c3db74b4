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
//  - Scores are masked only in blocks where some row does not see some key: the
//    diagonal's, the window's low end, the sinks'.
//  - A key that a row does not see has weight 0, and 0 times a NaN or an infinity in its V
//    would still be NaN.  A row whose result is not finite (never, with finite inputs) is
//    therefore computed again from its visible keys alone, a warp per row.
//
// Bound: the tensor cores' 4 d flops a visible pair and, on the other pipe, one exponential
// a pair; blocks are 128 keys wide, so a window of W keys costs up to W + 255 keys and the
// sinks one block.
#pragma once

#include <cuda_bf16.h>

#include "flash_attention.cuh"

namespace gemmrelu {
namespace attn {

struct WindowParams {
    const uint16_t *q, *k, *v;
    int64_t qs[3], ks[3], vs[3];   // sequence, token, head
    uint16_t *o;                   // [batch][n_q][q_heads][d]
    int n_q, n_kv, q_heads, group;
    int q_tiles, items;            // items = q_tiles * group: tiles of one K/V head
    int pairs, window, sinks;
    float scale;                   // log2(e) / sqrt(d)
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
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
    if constexpr (kBf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        return pack_half2(a, b);
    }
}

template <bool kBf16>
__device__ __forceinline__ float load_x16(const uint16_t *p) {
    if constexpr (kBf16)
        return __uint_as_float((uint32_t)*p << 16);
    else
        return __half2float(*reinterpret_cast<const __half *>(p));
}

// One row from its visible keys alone, by a warp: the plain one-pass softmax, a key at a
// time.  Only rows whose result was not finite come here.
template <int HD, bool kBf16>
__device__ __noinline__ void window_row(const WindowParams &p, int batch, int head, int qi,
                                        int lane) {
    const int pos = qi + p.n_kv - p.n_q, kvh = head / p.group;
    constexpr int E = HD / 32;
    float q[E], o[E], m = -INFINITY, l = 0.0f;
    const uint16_t *src = p.q + batch * p.qs[0] + qi * p.qs[1] + head * p.qs[2] + lane;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = load_x16<kBf16>(src + 32 * e);
        o[e] = 0.0f;
    }
    const int low = p.window > 0 && pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
    for (int j = p.sinks < low ? 0 : low; j <= pos; ++j) {
        if (j < low && j >= p.sinks)
            j = low;
        const uint16_t *k = p.k + batch * p.ks[0] + j * p.ks[1] + kvh * p.ks[2] + lane;
        const uint16_t *v = p.v + batch * p.vs[0] + j * p.vs[1] + kvh * p.vs[2] + lane;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            s += q[e] * load_x16<kBf16>(k + 32 * e);
#pragma unroll
        for (int x = 16; x; x >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= p.scale;
        const float to = fmaxf(m, s);
        const float f = to > m ? exp2f(m - to) : 1.0f, w = exp2f(s - to);
        l = l * f + w;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = o[e] * f + w * load_x16<kBf16>(v + 32 * e);
        m = to;
        if (l != l)
            break;   // a NaN score: the row is NaN
    }
    uint16_t *dst = p.o + (((int64_t)batch * p.n_q + qi) * p.q_heads + head) * HD + lane;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float x = l == 0.0f ? 0.0f : o[e] / l + (l != l ? l : 0.0f);
        dst[32 * e] = (uint16_t)(pack_pair<kBf16>(x, 0.0f) & 0xffffu);
    }
}

template <int HD, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    flash_attention_window_kernel(const __grid_constant__ CUtensorMap tmQ,
                                  const __grid_constant__ CUtensorMap tmK,
                                  const __grid_constant__ CUtensorMap tmV,
                                  const __grid_constant__ WindowParams p) {
    using G = Cfg<HD>;
    constexpr uint32_t kIdescS = with_type(G::kIdescS, kBf16);
    constexpr uint32_t kIdescO = with_type(G::kIdescO, kBf16);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);

    const uint32_t bar0 = base + G::kOffBar;
    const uint32_t q_full = bar0;
    auto k_full = [&](uint32_t s) { return bar0 + 8u * (1 + s); };
    auto v_full = [&](uint32_t s) { return bar0 + 8u * (1 + kKV + s); };
    auto kv_empty = [&](uint32_t s) { return bar0 + 8u * (1 + 2 * kKV + s); };
    auto s_full = [&](uint32_t t) { return bar0 + 8u * (1 + 3 * kKV + t); };
    auto p_full = [&](uint32_t t) { return bar0 + 8u * (3 + 3 * kKV + t); };
    const uint32_t o_full = bar0 + 8u * (5 + 3 * kKV);
    const uint32_t drain_bar = bar0 + 8u * (6 + 3 * kKV);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + G::kOffMisc);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + G::kOffMisc + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int kvh = blockIdx.y, batch = blockIdx.z;
    const int off = p.n_kv - p.n_q;
    // the last queries see the most keys: they go first
    const int item0 = 2 * (p.pairs - 1 - (int)blockIdx.x);
    const bool two = item0 + 1 < p.items;
    const int tile0 = item0 / p.group, tile1 = (item0 + 1) / p.group;
    const int head0 = kvh * p.group + item0 % p.group, head1 = kvh * p.group + (item0 + 1) % p.group;
    auto seen_by = [&](int tile) {
        const int last = min(tile * BM + BM, p.n_q) - 1;
        return blocks_seen(tile * BM + off, last + off, p.window, p.sinks);
    };
    const Blocks s0 = seen_by(tile0);
    const Blocks s1 = two ? seen_by(tile1) : Blocks{0, 0, 0};
    // the list: the union, in order
    Blocks all = s0;
    if (s1.count() > 0) {
        if (s0.count() == 0) {
            all = s1;
        } else {
            all.low = min(s0.low, s1.low);
            all.high = max(s0.high, s1.high);
            all.sinks = min(max(s0.sinks, s1.sinks), all.low);
        }
    }
    const int nb = all.count();
    auto block_of = [&](int j) { return j < all.sinks ? j : all.low + (j - all.sinks); };

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1u);
        for (uint32_t s = 0; s < (uint32_t)kKV; ++s) {
            mbar_init(k_full(s), 1u);
            mbar_init(v_full(s), 1u);
            mbar_init(kv_empty(s), 1u);
        }
        for (uint32_t t = 0; t < (uint32_t)kTiles; ++t) {
            mbar_init(s_full(t), 1u);
            mbar_init(p_full(t), 4u);
        }
        mbar_init(o_full, 1u);
        mbar_init(drain_bar, 1u);
        *abort_flag = 0u;
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

    if (warp == kProducerWarp) {
        // ============================================================ TMA producer
        if (lane == 0 && nb > 0) {
            uint32_t issued = 0, parity = 0;  // K/V stages with copies in flight
            bool q_issued = false;
            if (!(p.drop_arrive && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)) {
                mbar_arrive_expect_tx(q_full, (two ? 2u : 1u) * G::kQBytes);
                for (int t = 0; t < (two ? 2 : 1); ++t)
#pragma unroll
                    for (int d = 0; d < G::kDSub; ++d)
                        tma_load_4d(&tmQ, base + G::kOffQ + t * G::kQBytes + d * kSub, q_full,
                                    64 * d, t ? head1 : head0, (t ? tile1 : tile0) * BM, batch);
                q_issued = true;
            }
            for (int j = 0; j < nb; ++j) {
                const uint32_t st = (uint32_t)(j % kKV), ph = (uint32_t)((j / kKV) & 1);
                if (!wait_bounded_eager(kv_empty(st), ph ^ 1u, p.wait_limit_ns, abort_flag,
                                  kSiteProducerEmpty))
                    break;
                const int key = block_of(j) * BN;
                mbar_arrive_expect_tx(k_full(st), G::kKBytes);
#pragma unroll
                for (int d = 0; d < G::kDSub; ++d)
                    tma_load_4d(&tmK, base + G::kOffK + st * G::kKBytes + d * kSub, k_full(st),
                                64 * d, kvh, key, batch);
                mbar_arrive_expect_tx(v_full(st), G::kVBytes);
#pragma unroll
                for (int d = 0; d < G::kDSub; ++d)
                    tma_load_4d(&tmV, base + G::kOffV + st * G::kVBytes + d * kSub, v_full(st),
                                64 * d, kvh, key, batch);
                issued |= 1u << st;
                parity = (parity & ~(1u << st)) | (ph << st);
            }
            // every copy issued must have landed before the CTA may exit
            if (q_issued)
                wait_drain(q_full, 0u, p.wait_limit_ns, abort_flag);
            for (uint32_t s = 0; s < (uint32_t)kKV; ++s)
                if (issued & (1u << s)) {
                    wait_drain(k_full(s), (parity >> s) & 1u, p.wait_limit_ns, abort_flag);
                    wait_drain(v_full(s), (parity >> s) & 1u, p.wait_limit_ns, abort_flag);
                }
        }
    } else if (warp == kMmaWarp) {
        // ============================================================ MMA issuer
        if (lane == 0 && nb > 0) {
            bool ok = wait_bounded_eager(q_full, 0u, p.wait_limit_ns, abort_flag, kSiteMmaFull);
            uint32_t done0 = 0, done1 = 0;   // P V products of each tile so far
            // S_t = Q_t K_j^T
            auto score = [&](int t, int j) -> bool {
                const uint32_t st = (uint32_t)(j % kKV), ph = (uint32_t)((j / kKV) & 1);
                if (!wait_bounded_eager(k_full(st), ph, p.wait_limit_ns, abort_flag, kSiteMmaFull))
                    return false;
                tc_fence_after_sync();
                const uint64_t qd = make_sdesc_sw128(base + G::kOffQ + t * G::kQBytes, 16, 1024);
                const uint64_t kd = make_sdesc_sw128(base + G::kOffK + st * G::kKBytes, 16, 1024);
                const uint32_t d_s = tmem_base + G::kTmemS + t * BN;
#pragma unroll
                for (int kk = 0; kk < HD / UKA; ++kk) {
                    const uint64_t o = (uint64_t)((kk / 4) * (kSub >> 4) + (kk % 4) * 2);
                    umma_f16(d_s, qd + o, kd + o, kIdescS, kk > 0 ? 1u : 0u);
                }
                umma_commit(s_full(t));
                return true;
            };
            // O_t += P_t V_j, P_t from TMEM (over S_t)
            auto pv = [&](int t, int j, uint32_t &done) -> bool {
                const uint32_t st = (uint32_t)(j % kKV), ph = (uint32_t)((j / kKV) & 1);
                if (!wait_bounded_eager(p_full(t), done & 1u, p.wait_limit_ns, abort_flag,
                                  kSiteMmaAccEmpty) ||
                    !wait_bounded_eager(v_full(st), ph, p.wait_limit_ns, abort_flag, kSiteMmaFull))
                    return false;
                tc_fence_after_sync();
                const uint64_t vd = make_sdesc_sw128(base + G::kOffV + st * G::kVBytes, kSub, 1024);
                const uint32_t d_o = tmem_base + G::kTmemO + t * HD;
                const uint32_t a_p = tmem_base + G::kTmemS + t * BN;
#pragma unroll
                for (int kk = 0; kk < BN / UKA; ++kk)
                    umma_f16_ts(d_o, a_p + kk * (UKA / 2), vd + (uint64_t)(kk * ((UKA * 128) >> 4)),
                                kIdescO, (done > 0 || kk > 0) ? 1u : 0u);
                ++done;
                return true;
            };
            if (ok && s0.has(block_of(0)))
                ok = score(0, 0);
            if (ok && s1.has(block_of(0)))
                ok = score(1, 0);
            for (int j = 0; ok && j < nb; ++j) {
                const int blk = block_of(j), next = j + 1 < nb ? block_of(j + 1) : -1;
                if (s0.has(blk))
                    ok = pv(0, j, done0);
                if (ok && next >= 0 && s0.has(next))
                    ok = score(0, j + 1);
                if (ok && s1.has(blk))
                    ok = pv(1, j, done1);
                if (!ok)
                    break;
                umma_commit(kv_empty((uint32_t)(j % kKV)));
                if (next >= 0 && s1.has(next))
                    ok = score(1, j + 1);
            }
            if (ok)
                umma_commit(o_full);
            // all MMAs of this thread complete before TMEM can be released
            umma_commit(drain_bar);
            wait_drain(drain_bar, 0u, p.wait_limit_ns, abort_flag);
        }
    } else {
        // ============================================================ softmax / output
        const int t = warp >> 2;                        // tile
        const int q = warp & 3;                         // TMEM lanes 32q .. 32q+31
        const int tile = t ? tile1 : tile0, head = t ? head1 : head0;
        const Blocks mine = t ? s1 : s0;
        const int qi = tile * BM + 32 * q + lane;       // query index
        const int pos = qi + off;
        const int first = tile * BM + off, last = min(tile * BM + BM, p.n_q) - 1 + off;
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        const uint32_t s_addr = tmem_base + lane_base + G::kTmemS + t * BN;
        const uint32_t o_addr = tmem_base + lane_base + G::kTmemO + t * HD;
        float m = -INFINITY, l = 0.0f;
        bool alive = true;
        uint32_t turn = 0;
        for (int j = 0; j < nb; ++j) {
            const int blk = block_of(j);
            if (!mine.has(blk))
                continue;
            const bool ok = wait_bounded_eager(s_full((uint32_t)t), turn & 1u, p.wait_limit_ns,
                                         abort_flag, kSiteEpiAccFull);
            if (!__all_sync(0xffffffffu, ok)) {
                alive = false;
                break;
            }
            tc_fence_after_sync();
            const int key0 = blk * BN;
            // some row does not see some key of the block
            const bool masked = key0 + BN - 1 > first ||
                                (p.window > 0 && key0 <= last - p.window && key0 + BN > p.sinks);
            uint32_t v[BN];
#pragma unroll
            for (int c0 = 0; c0 < BN; c0 += 32)
                tmem_ld_x32(s_addr + c0, *reinterpret_cast<uint32_t(*)[32]>(&v[c0]));
#pragma unroll
            for (int c0 = 0; c0 < BN; c0 += 32)
                tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&v[c0]));
            if (masked) {
                const int hi = pos - key0;
                const int lo = p.window > 0 ? hi - p.window : -1;   // seen above it, or below `head`
                const int head_end = p.sinks - key0;
#pragma unroll
                for (int i = 0; i < BN; ++i)
                    v[i] = i <= hi && (i > lo || i < head_end) ? v[i] : __float_as_uint(-INFINITY);
            }
            float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
            for (int i = 0; i < BN; i += 2) {
                mx0 = fmaxf(mx0, __uint_as_float(v[i]));
                mx1 = fmaxf(mx1, __uint_as_float(v[i + 1]));
            }
            const float m_blk = fmaxf(mx0, mx1) * p.scale;   // scale > 0
            // move the reference only when the maximum grew by more than kRescaleLog2;
            // -infinity until the row has seen a key
            const bool move = m_blk > m + kRescaleLog2;
            const float m_new = move ? m_blk : m;
            const float alpha = move ? fast_exp2(m - m_new) : 1.0f;   // 0 at the first block
            const float m_ref = m_new == -INFINITY ? 0.0f : m_new;
            const float2 sc2 = make_float2(p.scale, p.scale), nm2 = make_float2(-m_ref, -m_ref);
            float2 sa = make_float2(0.0f, 0.0f), sb = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int c0 = 0; c0 < BN; c0 += 32) {
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
            if (turn > 0 && __any_sync(0xffffffffu, move)) {
#pragma unroll 1
                for (int c0 = 0; c0 < HD; c0 += 32) {
                    uint32_t w[32];
                    tmem_ld_x32_sync(o_addr + c0, w);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
                    tmem_st_x32(o_addr + c0, w);
                }
            }
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(p_full((uint32_t)t));
            ++turn;
        }
        // the last P V of both tiles, then O / l rounded once
        if (alive && (t == 0 || two)) {
            const bool done = turn == 0 || wait_bounded_eager(o_full, 0u, p.wait_limit_ns, abort_flag,
                                                              kSiteEpiAccFull);
            if (__all_sync(0xffffffffu, done)) {
                tc_fence_after_sync();
                const float inv_l = l == 0.0f ? 0.0f : 1.0f / l;
                uint16_t *dst = p.o + (((int64_t)batch * p.n_q + qi) * p.q_heads + head) * HD;
                bool fine = true;
#pragma unroll 1
                for (int c0 = 0; c0 < HD; c0 += 32) {
                    uint32_t w[32];
                    uint32_t h[16];
                    if (turn > 0)
                        tmem_ld_x32_sync(o_addr + c0, w);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float x = turn > 0 ? __uint_as_float(w[2 * i]) * inv_l : 0.0f;
                        const float y = turn > 0 ? __uint_as_float(w[2 * i + 1]) * inv_l : 0.0f;
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
                uint32_t again = __ballot_sync(0xffffffffu, !fine && qi < p.n_q);
                while (again) {
                    const int r = __ffs(again) - 1;
                    again &= again - 1;
                    __syncwarp();
                    window_row<HD, kBf16>(p, batch, head, tile * BM + 32 * q + r, lane);
                }
            }
        }
    }

    // ---------------------------------------------------------------- teardown
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, G::kTmemCols);
    }
}

}  // namespace attn
}  // namespace gemmrelu
