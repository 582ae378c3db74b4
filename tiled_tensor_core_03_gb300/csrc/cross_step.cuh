// cross_step.cuh -- attention of a few query rows to an encoder's states:
//
//   O[r] = sum_j softmax_j(q_r . k_j / sqrt(D)) v_j  over the keys j < n of the row's sequence,
//
// for fp16 or bf16 tensors with strides.  The rows of one K/V head are its group's query heads of every query
// token, at most 16: a step of an answer.
//
// Bound: the keys and values are read once, 4 D bytes a key and head, for 4 D flops a row.  So nothing is gained from
// tiles of 128 rows: a block streams a part of one head's states through a ring of 64-key stages (TMA),
// four warps take 16 keys of a stage each, and the products run on mma.sync.m16n8k16 with keys in M and 8 query
// rows in N, S^T = K Q^T and O^T += V^T P^T (operands by ldmatrix, V's transposed; P turned with movmatrix).  A
// head's states are cut into equal parts as long as there are fewer heads than fill the GPU; the block that
// comes last joins the parts, in order: no block waits for another, and the same call gives the same bits.
//
// Scores, softmax statistics and sums are fp32; the weights are rounded to the inputs' type for the second product, which
// takes both operands in one type (against 64 bits: fp16 0.00025 of the result, 0.00020 with weights in 32 bits; bf16 0.0023,
// 0.0017).
//
// Measured, up to 1500 states (times and the bytes' floor): 48 sequences, 16 heads of 64: 36 us (31.9), 6.1 TB/s, 41 with 16
// rows a head; of 128: 71 (63.8), 80; 32 sequences, 8 heads of 128: 26.9 (20.7), 30.1; 4 sequences, 8 heads of 64: 7.6, 9.4; of 128:
// 8.0, 11.0.  2 of up to 700, 8 heads of 64: 6.5, where a launch that does nothing takes 2.
//
// More than 16 rows go to the tiles of the long form, which does not cut a head's states and takes about the same time
// from 17 rows to 256: 70 us for the first of these, 93 at heads of 128, 35 for the second; where there are few heads its few
// CTAs walk over all states alone (one sequence of 8192 states, 1 to 8 heads of 64: 12 us with 16 rows, 73 with 17; of 128: 17 and 88).
#pragma once

#include "kv_attention.cuh"

namespace gemmrelu {
namespace attn {

constexpr int kStepKeys = 64;        // keys of a stage
constexpr int kStepWarps = 4;        // computing warps; one more feeds
constexpr int kStepThreads = 32 * (kStepWarps + 1);
constexpr int kStepMostRows = 16;
constexpr int kStepCounters = GEMMRELU_CROSS_COUNTER_BYTES / (int)sizeof(unsigned);

template <int D, int kN>
struct StepCfg {
    static constexpr int kRows = 8 * kN;
    static constexpr int kStages = D == 64 ? 4 : 3;
    static constexpr uint32_t kSub8 = kStepKeys * 128;           // [64 keys][64] 16-bit, 128-byte swizzle
    static constexpr uint32_t kTile = D / 64 * kSub8;            // K (or V) of a stage
    static constexpr uint32_t kOffV = kStages * kTile;
    static constexpr uint32_t kOffBar = 2 * kStages * kTile;
    static constexpr uint32_t kOffMisc = kOffBar + 2 * kStages * 8;
    static constexpr uint32_t kOffStat = kOffMisc + 16;          // m and l, [4 warps][kRows] each
    static constexpr int kPitch = D + 4;
    static constexpr uint32_t kOffJoin = kOffStat + 2 * kStepWarps * kRows * 4;   // [4 warps][kRows][kPitch]
    static constexpr uint32_t kSmem = kOffJoin + kStepWarps * kRows * kPitch * 4 + 1024;
    // Blocks that an SM's 228 KB of shared memory hold, 1 KB of it reserved for each: heads of 64 three with 8 rows and two
    // with 16, heads of 128 one.
    static constexpr int kBlocksPerSm = 228 * 1024 / ((int)kSmem + 1024);
    // What the compiler is told: with one block an SM it took more registers, and heads of 128 with 16 rows were 1 to 3% slower.
    static constexpr int kBlocksToCompileFor = kBlocksPerSm < 2 ? 2 : kBlocksPerSm;
};

struct StepParams {
    const uint16_t *q;
    int64_t qs[3];                  // sequence, token, head
    uint16_t *o;                    // [batch][n_q][q_heads][D]
    const int32_t *states;          // or nullptr: n_kv keys each
    int n_q, n_kv, q_heads, kv_heads, group, rows;
    int parts;
    float scale;                    // log2(e) / sqrt(D)
    float slack;                    // how far a score may exceed the reference: 8 / scale
    float shift;                    // bf16: weights are 2^-shift times as large, so that their sums with V stay in fp32
    float *partial;                 // [batch * kv_heads][parts][kRows][D + 4]: sums, then m and l
    unsigned *arrived;              // [batch * kv_heads]; all 0 between calls
    int drop_arrive;
    uint64_t wait_limit_ns;
};

template <bool kBf16>
__device__ __forceinline__ void mma_step(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kBf16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        kvc::mma_f16(d, a[0], a[1], a[2], a[3], b0, b1);
}

template <bool kTrans>
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t addr) {
    if constexpr (kTrans)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// The numbers of states where no sequence has any: another number than 0 is out of range.
__global__ void cross_no_states_kernel(const int32_t *states, int batch) {
    pdl_launch_dependents();
    pdl_wait_primary();
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < batch && states[b] != 0)
        atomicCAS(&g_status, 0u, kStatusLength);
}

template <int D, int kN, bool kBf16>
__global__ void __launch_bounds__(kStepThreads, StepCfg<D, kN>::kBlocksToCompileFor)
    cross_step_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const StepParams p) {
    using G = StepCfg<D, kN>;
    constexpr int kRows = G::kRows;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t bar0 = base + G::kOffBar;
    auto full = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty = [&](uint32_t s) { return bar0 + 8u * (G::kStages + s); };
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + G::kOffMisc);
    volatile uint32_t *last_flag = reinterpret_cast<volatile uint32_t *>(gbase + G::kOffMisc + 4);
    float *stat_m = reinterpret_cast<float *>(gbase + G::kOffStat), *stat_l = stat_m + kStepWarps * kRows;
    float *join = reinterpret_cast<float *>(gbase + G::kOffJoin);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (uint32_t s = 0; s < (uint32_t)G::kStages; ++s) {
            mbar_init(full(s), 1u);
            mbar_init(empty(s), kStepWarps);
        }
        *abort_flag = 0u;
        fence_mbar_init();
        pdl_launch_dependents();
    }
    if (tid == 32 * kStepWarps) {
        tma_prefetch_map(&tmK);
        tma_prefetch_map(&tmV);
    }
    __syncthreads();
    pdl_wait_primary();

    const int bh = blockIdx.x / p.parts, part = blockIdx.x - bh * p.parts;
    const int b = bh / p.kv_heads, h = bh - b * p.kv_heads;
    int n = p.states ? p.states[b] : p.n_kv;
    if (n < 0 || n > p.n_kv) {
        atomicCAS(&g_status, 0u, kStatusLength);
        n = 0;
    }
    const int units = (n + kStepKeys - 1) / kStepKeys;
    const int u0 = (int)((int64_t)units * part / p.parts), u1 = (int)((int64_t)units * (part + 1) / p.parts);

    if (warp == kStepWarps) {
        // ============================================================ the feed
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            int i = 0;
            const int count = p.drop_arrive && blockIdx.x == 0 ? 0 : u1 - u0;
            for (; i < count; ++i) {
                if (!wait_bounded(empty(stage), phase ^ 1u, p.wait_limit_ns, abort_flag, kSiteProducerEmpty))
                    break;
                mbar_arrive_expect_tx(full(stage), 2u * G::kTile);
                const int key = (u0 + i) * kStepKeys;
#pragma unroll
                for (int d = 0; d < D / 64; ++d) {
                    tma_load_4d(&tmK, base + stage * G::kTile + d * G::kSub8, full(stage), 64 * d, h, key, b);
                    tma_load_4d(&tmV, base + G::kOffV + stage * G::kTile + d * G::kSub8, full(stage), 64 * d, h, key, b);
                }
                if (++stage == (uint32_t)G::kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            // every copy issued has landed before the block may exit
            for (int x = i > G::kStages ? i - G::kStages : 0; x < i; ++x)
                wait_drain(full(x % G::kStages), x / G::kStages & 1u, p.wait_limit_ns, abort_flag);
        }
        return;
    }

    // ================================================================ the products
    const int g = lane >> 2, c = lane & 3;
    uint32_t q[kN][D / 16][2];
#pragma unroll
    for (int t = 0; t < kN; ++t) {
        const int r = 8 * t + g, token = r / p.group;
        const uint16_t *src = p.q + b * p.qs[0] + token * p.qs[1] + (h * p.group + r - token * p.group) * p.qs[2];
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                q[t][k][e] = r < p.rows ? *reinterpret_cast<const uint32_t *>(src + 16 * k + 8 * e + 2 * c) : 0u;
    }
    // o[t][j]: elements 16 j + g (0, 1) and 16 j + g + 8 (2, 3), rows 2c and 2c + 1
    float o[kN][D / 16][4], m[kN][2], l[kN][2];
#pragma unroll
    for (int t = 0; t < kN; ++t) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
            o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.0f;
        m[t][0] = m[t][1] = -INFINITY;
        l[t][0] = l[t][1] = 0.0f;
    }
    // this lane's rows in ldmatrix: of K rows and chunks (lane / 8: 0, 1 rows 0-7, 8-15 of a chunk; 2, 3 the next chunk), of
    // V the other way round
    const int k_row = 16 * warp + (lane & 15), k_chunk = lane >> 4;
    const int v_row = 16 * warp + (lane & 7) + (lane >> 4) * 8, v_chunk = lane >> 3 & 1;
    bool alive = true;
    uint32_t stage = 0, phase = 0;
    for (int u = u0; u < u1; ++u) {
        const int key0 = u * kStepKeys + 16 * warp;
        alive = alive && wait_bounded_eager(full(stage), phase, p.wait_limit_ns, abort_flag, kSiteMmaFull);
        alive = __all_sync(0xffffffffu, alive);
        if (!alive)
            break;
        if (key0 < n) {
            const uint32_t k_at = base + stage * G::kTile, v_at = base + G::kOffV + stage * G::kTile;
            float acc[kN][4];
#pragma unroll
            for (int t = 0; t < kN; ++t)
                acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const int chunk = 2 * k + k_chunk;
                uint32_t a[4];
                load_matrices<false>(a, k_at + (chunk >> 3) * G::kSub8 + k_row * 128 + (((chunk & 7) ^ (k_row & 7)) << 4));
#pragma unroll
                for (int t = 0; t < kN; ++t)
                    mma_step<kBf16>(acc[t], a, q[t][k][0], q[t][k][1]);
            }
            if (key0 + 16 > n) {   // the sequence's last keys
#pragma unroll
                for (int t = 0; t < kN; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[t][i] = key0 + g + 8 * (i >> 1) < n ? acc[t][i] : -INFINITY;
                // what stands behind them in V may be NaN, and 0 times that too
                for (int i = lane; i < 16 * (D / 8); i += 32) {
                    const int r = 16 * warp + i / (D / 8), x = i % (D / 8);
                    if (u * kStepKeys + r >= n)
                        st_shared_v4(v_at + (x >> 3) * G::kSub8 + r * 128 + ((x & 7) << 4), 0u, 0u, 0u, 0u);
                }
                __syncwarp();
            }
            // the reference moves when a score exceeds it by 2^8, and with the first scores
            bool high = false;
#pragma unroll
            for (int t = 0; t < kN; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    high = high || acc[t][i] > m[t][i & 1] + p.slack;
            if (__any_sync(0xffffffffu, high)) {
#pragma unroll
                for (int t = 0; t < kN; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = fmaxf(acc[t][e], acc[t][2 + e]);
#pragma unroll
                        for (int s = 4; s < 32; s <<= 1)
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, s));
                        const bool move = x > m[t][e] + p.slack;
                        const float alpha = move ? fast_exp2((m[t][e] - x) * p.scale) : 1.0f;   // 0 at the first scores
                        m[t][e] = move ? x : m[t][e];
                        l[t][e] *= alpha;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            o[t][j][e] *= alpha;
                            o[t][j][2 + e] *= alpha;
                        }
                    }
            }
            uint32_t pb[kN][2];
#pragma unroll
            for (int t = 0; t < kN; ++t) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float ref = m[t][i & 1] == -INFINITY ? 0.0f : m[t][i & 1];
                    w[i] = fast_exp2(fmaf(acc[t][i] - ref, p.scale, -p.shift));
                    l[t][i & 1] += w[i];
                }
                pb[t][0] = kvc::turned(pack_pair<kBf16>(w[0], w[1]));
                pb[t][1] = kvc::turned(pack_pair<kBf16>(w[2], w[3]));
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                const int chunk = 2 * j + v_chunk;
                uint32_t a[4];
                load_matrices<true>(a, v_at + (chunk >> 3) * G::kSub8 + v_row * 128 + (((chunk & 7) ^ (v_row & 7)) << 4));
#pragma unroll
                for (int t = 0; t < kN; ++t)
                    mma_step<kBf16>(o[t][j], a, pb[t][0], pb[t][1]);
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(empty(stage));
        if (++stage == (uint32_t)G::kStages) {
            stage = 0;
            phase ^= 1u;
        }
    }

    // ---------------------------------------------------------------- the warps' results together
    // (a warp whose wait expired brings what it has: the status says that the output is not to be used)
#pragma unroll
    for (int t = 0; t < kN; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float sum = l[t][e];
#pragma unroll
            for (int s = 4; s < 32; s <<= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, s);
            const int row = 8 * t + 2 * c + e;
            if (g == 0) {
                stat_m[warp * kRows + row] = m[t][e];
                stat_l[warp * kRows + row] = sum;
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                join[(warp * kRows + row) * G::kPitch + 16 * j + g] = o[t][j][e];
                join[(warp * kRows + row) * G::kPitch + 16 * j + g + 8] = o[t][j][2 + e];
            }
        }
    named_bar_sync(1, 32 * kStepWarps);
    auto write_out = [&](int row, int d, float4 y, float sum) {
        const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;   // 0: there are no keys
        const int token = row / p.group;
        uint16_t *dst = p.o + (((int64_t)b * p.n_q + token) * p.q_heads + h * p.group + row - token * p.group) * D + d;
        *reinterpret_cast<uint2 *>(dst) =
            make_uint2(pack_pair<kBf16>(y.x * inv, y.y * inv), pack_pair<kBf16>(y.z * inv, y.w * inv));
    };
    // a reference of -infinity counts for nothing, but a NaN among its weights
    auto weight = [&](float m, float ref) { return m == -INFINITY ? 1.0f : exp2f((m - ref) * p.scale); };
    float *mine = p.partial + ((int64_t)bh * p.parts + part) * kRows * (D + 4);
    for (int i = tid; i < p.rows * (D / 4); i += 32 * kStepWarps) {
        const int row = i / (D / 4), d = i % (D / 4) * 4;
        float top = -INFINITY, sum = 0.0f;
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kStepWarps; ++w)
            top = fmaxf(top, stat_m[w * kRows + row]);
        const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int w = 0; w < kStepWarps; ++w) {
            const float a = weight(stat_m[w * kRows + row], ref);
            const float4 x = *reinterpret_cast<const float4 *>(join + (w * kRows + row) * G::kPitch + d);
            sum = fmaf(stat_l[w * kRows + row], a, sum);
            y = make_float4(fmaf(x.x, a, y.x), fmaf(x.y, a, y.y), fmaf(x.z, a, y.z), fmaf(x.w, a, y.w));
        }
        if (p.parts == 1) {
            write_out(row, d, y, sum);
        } else {
            __stcg(reinterpret_cast<float4 *>(mine + row * (D + 4) + d), y);
            if (d == 0)
                __stcg(reinterpret_cast<float4 *>(mine + row * (D + 4) + D), make_float4(top, sum, 0.0f, 0.0f));
        }
    }
    if (p.parts == 1)
        return;

    // ---------------------------------------------------------------- the parts together
    named_bar_sync(1, 32 * kStepWarps);
    if (tid == 0)
        *last_flag = kvc::count_part(p.arrived + bh, (unsigned)(p.parts - 1)) == (unsigned)(p.parts - 1);
    named_bar_sync(1, 32 * kStepWarps);
    if (*last_flag == 0u)
        return;
    const float *all = p.partial + (int64_t)bh * p.parts * kRows * (D + 4);
    for (int i = tid; i < p.rows * (D / 4); i += 32 * kStepWarps) {
        const int row = i / (D / 4), d = i % (D / 4) * 4;
        float top = -INFINITY, sum = 0.0f;
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int x = 0; x < p.parts; ++x) {
            const float *at = all + ((int64_t)x * kRows + row) * (D + 4);
            const float4 s = __ldcg(reinterpret_cast<const float4 *>(at + D));
            const float4 z = __ldcg(reinterpret_cast<const float4 *>(at + d));
            const float now = fmaxf(top, s.x), ref = now == -INFINITY ? 0.0f : now;
            const float old = top == now ? 1.0f : weight(top, ref), a = weight(s.x, ref);
            sum = fmaf(sum, old, s.y * a);
            y = make_float4(fmaf(y.x, old, z.x * a), fmaf(y.y, old, z.y * a), fmaf(y.z, old, z.z * a),
                            fmaf(y.w, old, z.w * a));
            top = now;
        }
        write_out(row, d, y, sum);
    }
}

}  // namespace attn
}  // namespace gemmrelu
