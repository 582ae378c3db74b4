// kv_attention.cuh -- attention of a few new tokens over the paged 8-bit cache:
//
//   O[r] = sum_t softmax_t(q_r . k_t / sqrt(D)) v_t,  k_t = ks * K8[t], v_t = vs * V8[t]
//
// over the tokens t that row r sees (t <= p_r; with a window W also t > p_r - W
// or t < sinks), p_r the row's position.  The rows of one K/V head are
// its group's query heads of every new token, 8 rows a tile (16 for heads of 64).
//
// What bounds it: every visible token's 2 D bytes are read once per row tile and
// used for 4 D flops a row, so one tile is a stream from HBM: 64 sequences of up to 32768
// tokens, 8 heads of 128, 3.1 GB in 468 us, 6.6 TB/s (0.98 of a measured copy).  About 13 us of a
// call are fixed: 3 to the first bytes (lengths, page numbers, pages, one after the other), 5 between
// the first and the last block's end, 4 for counting and joining; so 32 sequences of up to 4096
// tokens, 183 MB, take 42 us, and one sequence of 1000 tokens 9.7 us.  More row tiles are bound by
// the chain of conversions and products of a unit: 25 us for every further 8 rows at those 183 MB.  The
// kernel is built around the stream:
//
//  - Work is cut into units of 64 tokens of one (sequence, head); the
//    units of all of them, in order, are dealt to the blocks in equal contiguous
//    ranges whatever the lengths are.  Each range has a block per row tile (grid.y, up to 16; further
//    tiles in further passes): they read the same units at about the same time, from
//    HBM once, and their strips of the scores meet in L2.  With the tiles one after the other in one
//    block's range 32 sequences of up to 4096 tokens, 8 heads of 128, took 66.3 us, not 64.3, with 16 rows,
//    222 and 216 with 64, and with weights 202 and 165 with 28; one tile pays 0.3 us of 41.  (Now 65.4,
//    217.6 and 170: references of their own for O, and scores before their factor.)
//    A block finishes what lies
//    inside its range; a (sequence, head, row tile) that is cut leaves one fp32
//    partial (O, m, l) per block in the workspace, and the block that comes last joins
//    them, in the order of the ranges.  No block waits for another and nothing depends on
//    the order in which they come: the same call gives the same bits.  Parts are counted and
//    joined after a block's last unit: done where they arise, between two segments, a
//    block's copies stood still for up to 10 us.
//  - One warp feeds a ring of 64-token stages by TMA (a page or a part of one per
//    copy), reading page numbers and scales 32 pieces ahead.
//  - Four warps take 16 tokens of a stage each.  The products run on mma.sync.m16n8k16
//    with fp16 operands, tokens in the M of 16 and query rows in the N of 8:
//    S^T = K Q^T and O^T += V^T P^T.  Eight rows are all that a decode step with up to
//    8 heads a group has, far below the 128 of a tcgen05.mma, and e4m3 has to become
//    fp16 (exact) on the way, which happens in registers here.  The operand layouts are
//    chosen so that the bytes a lane loads from shared memory are the ones its fragment
//    needs (see key_of / piece_of below); P^T is turned with movmatrix.
//    Rows in M instead (S = Q K^T, 16 rows) took twice the products, accumulators and
//    exponentials and 168 registers: 729 us at 64 sequences of up to 32768 tokens (8 K/V
//    heads of 128), 4.25 TB/s, at 1.3 instructions a cycle from 10 warps an SM.
//  - Softmax in one pass, base 2, a running reference m per row that moves only when
//    a score exceeds it by 2^8; fp32 statistics and accumulators.  P is
//    rounded to fp16 for the second product (relative 2^-11, like the output's own
//    rounding).  V's scale is folded into P, and O has a reference of its own, r above m and moved
//    likewise: P = 2^(7 - r) * vs * weight stays below 2^15 and normal down to 2^-21 of the row's
//    largest weight times scale, whatever scales come in what order (but for weights below 2^-111 under
//    scales 2^111 above the others).  (With P relative to the largest scale met so far a
//    page with the weight but a scale 2^30 below another's lost its bits.)
//    m is a score before its factor log2(e) / sqrt(D), which multiplies differences alone: with scales that
//    are powers of two the largest score's difference is then 0 at any size.  (Multiplied first, the
//    reference is rounded and the fused product is not: off by half a unit at 2^24, an overflow at 2^31.  The
//    multiplication more costs 0 to 1%.)
#pragma once

#include "kv_cache.cuh"

namespace gemmrelu {
namespace kvc {

constexpr int kUnit = 64;            // tokens of a stage
constexpr int kWarps = 4;            // computing warps
constexpr int kFeedWarp = 4;
constexpr int kAttnThreads = 160;
constexpr int kMostAbreast = 16;     // row tiles that share the stream of a head
constexpr float kMoveLog2 = 8.0f;    // the reference moves when a score exceeds it by more
constexpr float kPLog2 = 7.0f;       // see above

// kN groups of 8 query rows a tile (two for heads of 64 only).  Two blocks an SM (168 registers a
// thread); three (128) for 64 elements and one group.  Measured, one group: 32 sequences of up to
// 4096 tokens, 8 heads of 128, 42.2 us with two blocks and 45.3 with three; 16 sequences of up
// to 8192, window 2000, 16 heads of 64, 4 tokens each, 33.2 and 27.7 us.
template <int D, int kN>
struct AttnCfg {
    static constexpr int kRows = 8 * kN;
    static constexpr int kBlocksPerSm = kN == 1 && D == 64 ? 3 : 2;
    static constexpr uint32_t kTile = kUnit * D;                 // bytes of K (or V) in a stage
    static constexpr int kStages = D == 128 ? 4 : kN == 1 ? 6 : 8;
    static constexpr uint32_t kOffK = 0;
    static constexpr uint32_t kOffV = kOffK + kStages * kTile;
    static constexpr int kPitch = D + 4;                         // floats a row of the join buffer
    static constexpr uint32_t kOffJoin = kOffV + kStages * kTile;   // [4 warps][kRows][kPitch]
    static constexpr uint32_t kOffStat = kOffJoin + kWarps * kRows * kPitch * 4;   // m, l, r [4][kRows]
    static constexpr uint32_t kOffMeta = kOffStat + 3 * kWarps * kRows * 4;
    static constexpr uint32_t kOffScan = kOffMeta + kStages * 4 * 8;   // (ks, log2 vs) per 16 tokens
    static constexpr uint32_t kOffBar = kOffScan + 16 * 4;
    static constexpr uint32_t kOffMisc = kOffBar + 2 * kStages * 8;
    static constexpr uint32_t kSmem = kOffMisc + 16 + 1024;
};

struct AttnParams {
    Pool pool;
    const uint16_t *q;
    int64_t q_stride[3];               // sequence, token, head
    uint16_t *out;                     // [batch][tokens][q_heads][D]
    const int32_t *pages, *lengths;
    int64_t max_pages;
    int batch, tokens, q_heads, group;
    int rows;                          // tokens * group, in tiles of 8 or 16: `abreast` at a time,
    int abreast, passes;               // `passes` times
    int window, sinks;
    float scale_log2;                  // log2(e) / sqrt(D)
    float *partial;                    // [2 * grid][kRows][D], then [2 * grid][kRows][4] (m, l, r, unused)
    int grid;                          // ranges * abreast
    unsigned *arrived;                 // [ranges][abreast] parts that are there of the segment that
                                       // leaves the block's range; all 0 between calls
    float *scores;                     // with weights: [batch][kv_heads][width][rows], base 2
    float *lse;                        //               [batch][kv_heads][rows], base 2
    float *weights;                    // [batch][kv_heads][width]
    int64_t width;
    int drop_arrive;
    uint64_t wait_limit_ns;
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------- which units there are

// The units of 64 tokens that some row of a sequence of n tokens sees: those of the
// sinks left of the first row's window, then all from that window on.
struct Span {
    int sink_units, low_unit, units;
    __host__ __device__ __forceinline__ int chunk(int u) const {
        return u < sink_units ? u : low_unit + (u - sink_units);
    }
};

__host__ __device__ __forceinline__ Span span_of(int n, int tokens, int window, int sinks) {
    Span s{0, 0, (n + kUnit - 1) / kUnit};
    const int first = n > tokens ? n - tokens : 0;   // position of the first row
    if (window > 0 && first >= window) {
        const int low = first - window + 1;
        const int head = sinks < low ? sinks : low;
        s.low_unit = low / kUnit;
        s.sink_units = (head + kUnit - 1) / kUnit;
        if (s.sink_units > s.low_unit)
            s.sink_units = s.low_unit;
        s.units = s.units - s.low_unit + s.sink_units;
    }
    return s;
}

__device__ __forceinline__ bool sees(int t, int pos, int window, int sinks) {
    return t <= pos && (window == 0 || t > pos - window || t < sinks);
}

// Sequence b's length as this call takes it: 0 where it is out of range.
__device__ __forceinline__ int length_of(const AttnParams &p, int b) {
    return checked_length(p.lengths, b, p.max_pages * p.pool.page);
}

// First unit of block c of `grid`, of `total`: equal ranges (the first ones one unit
// longer), and the block that owns unit x.  (The host keeps the units of a call below 2^31.)
__host__ __device__ __forceinline__ int range_start(int c, int total, int grid) {
    const int q = total / grid, r = total % grid;
    return c * q + (c < r ? c : r);
}
__host__ __device__ __forceinline__ int range_owner(int x, int total, int grid) {
    const int q = total / grid, r = total % grid, longer = r * (q + 1);
    return x < longer ? x / (q + 1) : r + (x - longer) / q;
}

// How many of the launched ranges have work: each has a unit at least, and a (sequence, head,
// pass) is cut into about sqrt(4 units) parts at most.  A part costs its block's start
// and, in the join, a read of its O by one block; a unit in sequence costs its copy.
__device__ __forceinline__ int blocks_used(int total, int segments, int grid) {
    const float most = sqrtf(4.0f * (float)total * (float)segments);
    int n = total < grid ? total : grid;
    if (most < (float)n)
        n = (int)most;
    return n > 1 ? n : 1;
}

// ---------------------------------------------------------------- layouts
// A stage's K and V are rows of D bytes, one per token, with the 16-byte chunks of a row
// permuted by the TMA swizzle (128-byte swizzle: chunk ^ row mod 8; 64-byte rows: chunk ^
// row / 2 mod 4).
template <int D>
__device__ __forceinline__ uint32_t at_chunk(int row, int chunk) {
    if constexpr (D == 128)
        return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4));
    else
        return (uint32_t)(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}

// In fragments of mma.m16n8k16 lane = 4 g + c.  S^T = K Q^T: token row i of 16 is token
// key_of(i), so that eight lanes that load together touch eight different chunks, here and
// in V, where lane c takes the rows 2c, 2c + 1, 2c + 8, 2c + 9: tokens c, c + 4, c + 8, c + 12.
__device__ __forceinline__ int key_of(int i) { return (i & 8) | (i >> 1 & 3) | ((i & 1) << 2); }

// The k index of S^T = K Q^T runs over the D elements in an order of its own: lane c's
// k-steps are the consecutive fours of its chunk(s) c (and c + 4), so a K fragment is 4
// consecutive bytes.  Q's fragment uses the same order.
//
// O^T += V^T P^T: lane g's rows of the D / 16 row groups are D / 8 consecutive elements,
// those of piece piece_of(g) (16 bytes for D = 128, 8 for D = 64), two per group.
template <int D>
__device__ __forceinline__ int piece_of(int g) {
    if constexpr (D == 128)
        return (g >> 1) | ((g & 1) << 2);
    else
        return ((g >> 1) & 1) << 2 | (g >> 2) << 1 | (g & 1);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose an 8 x 8 matrix of 16-bit elements held two a lane (row g, columns 2c, 2c + 1).
__device__ __forceinline__ uint32_t turned(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

// Bytes of w that are an e4m3 NaN (0x7f or 0xff), as 0x80 in their place.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Sixteen (or for D = 64 the lane's sixteen) elements of a query row as fp16 pairs in the
// order of the fragments.  bf16 rows are scaled by a power of two that
// brings their largest element to [2^14, 2^15), within fp16; `back` undoes it.
template <int D, bool kBf16>
__device__ __forceinline__ void load_row(const uint16_t *row, int c, uint32_t (&x)[D / 8],
                                         float &back) {
    uint4 v[D / 32];
    back = 1.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        v[i] = make_uint4(0, 0, 0, 0);
    if (row != nullptr) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i)   // elements 16 c + 8 (i & 1) of half i / 2
            v[i] = *reinterpret_cast<const uint4 *>(row + (i >> 1) * 64 + 16 * c + 8 * (i & 1));
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        x[4 * i] = v[i].x;
        x[4 * i + 1] = v[i].y;
        x[4 * i + 2] = v[i].z;
        x[4 * i + 3] = v[i].w;
    }
    if constexpr (kBf16) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            top = max(top, max(x[i] & 0x7fffu, (x[i] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int e = (int)(top >> 7) - 127;
        e = e < -100 ? -100 : e > 127 ? 127 : e;
        const float to = __uint_as_float((uint32_t)(14 - e + 127) << 23);
        back = __uint_as_float((uint32_t)(e - 14 + 127) << 23);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            const float2 f = pair_to_float2<true>(x[i]);
            x[i] = half2_of(f.x * to, f.y * to);
        }
    }
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pack_out(float a, float b) {
    if constexpr (kBf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        return half2_of(a, b);
    }
}

__device__ __forceinline__ int64_t out_row(const AttnParams &p, int b, int h, int row) {
    return ((int64_t)b * p.tokens + row / p.group) * p.q_heads + h * p.group + row % p.group;
}

// a - b, but -infinity less anything is -infinity.
__device__ __forceinline__ float less(float a, float b) { return a - (b == -INFINITY ? 0.0f : b); }

// kF elements of a row of the result from the row's sum of weights, relative to the reference ref, and their
// own sum y, whose reference is r above that; with scores also the row's log-sum-exp.
template <int D, int kF, bool kBf16, bool kScores>
__device__ __forceinline__ void write_row(const AttnParams &p, int b, int h, int row, int d0,
                                          const float (&y)[kF], float ref, float r, float sum) {
    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;   // 0: the row sees nothing
    // (its square: r may span the range of all scales)
    const float f = r == -INFINITY ? 0.0f : exp2f(0.5f * (r - kPLog2));
    uint16_t *dst = p.out + out_row(p, b, h, row) * D + d0;
#pragma unroll
    for (int j = 0; j < kF; j += 4)
        *reinterpret_cast<uint2 *>(dst + j) =
            make_uint2(pack_out<kBf16>(y[j] * inv * f * f, y[j + 1] * inv * f * f),
                       pack_out<kBf16>(y[j + 2] * inv * f * f, y[j + 3] * inv * f * f));
    if (kScores && d0 == 0)
        p.lse[((int64_t)b * p.pool.kv_heads + h) * p.rows + row] = sum == 0.0f ? INFINITY : ref * p.scale_log2 + log2f(sum);
}

// Count a part of a segment of n + 1: the number counted before; wraps to 0 with the last.
// Releases this block's part (whose writers a barrier precedes), acquires the others'.
__device__ __forceinline__ unsigned count_part(unsigned *word, unsigned n) {
    unsigned old;
    asm volatile("fence.acq_rel.gpu;\n\tatom.relaxed.gpu.global.inc.u32 %0, [%1], %2;\n\tfence.acq_rel.gpu;"
                 : "=r"(old)
                 : "l"(word), "r"(n)
                 : "memory");
    return old;
}

// ---------------------------------------------------------------- the stream

template <int D, int kN, bool kBf16, bool kScores>
__global__ void __launch_bounds__(kAttnThreads, AttnCfg<D, kN>::kBlocksPerSm)
    kv_attention_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const AttnParams p) {
    using G = AttnCfg<D, kN>;
    constexpr int kRows = G::kRows;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t bar0 = base + G::kOffBar;
    auto full = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty = [&](uint32_t s) { return bar0 + 8u * (G::kStages + s); };
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + G::kOffMisc);
    int *scan = reinterpret_cast<int *>(gbase + G::kOffScan);   // 5 warps' units, then what was found
    float2 *meta = reinterpret_cast<float2 *>(gbase + G::kOffMeta);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (uint32_t s = 0; s < (uint32_t)G::kStages; ++s) {
            mbar_init(full(s), 2u);   // the copies, and the scales
            mbar_init(empty(s), kWarps);
        }
        *abort_flag = 0u;
        fence_mbar_init();
        pdl_launch_dependents();
    }
    if (tid == 32 * kFeedWarp) {
        tma_prefetch_map(&tmK);
        tma_prefetch_map(&tmV);
    }
    // Warm L2 with what the start depends on, one load after the other: the lengths and the page
    // table (L2 is where all writes meet, so fetching early returns nothing stale).
    {
        const int64_t i = ((int64_t)blockIdx.x * kAttnThreads + tid) * 32;
        if (i < p.batch * p.max_pages)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.pages + i));
        if (i < p.batch)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.lengths + i));
    }
    pdl_wait_primary();

    // this block's range of units of 64 tokens, and the sequence that it starts in: every thread counts a
    // slice of the sequences
    const int range = blockIdx.x, lane_tile = blockIdx.y;
    const int per_seq = p.pool.kv_heads * p.passes;   // (head, pass) pairs
    const int slice = (p.batch + kAttnThreads - 1) / kAttnThreads;
    const int b0 = min(tid * slice, p.batch), b1 = min(b0 + slice, p.batch);
    int mine = 0;
    for (int i = b0; i < b1; ++i)
        mine += span_of(length_of(p, i), p.tokens, p.window, p.sinks).units;
    int run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, run, o);
        run += lane >= o ? x : 0;
    }
    if (lane == 31)
        scan[warp] = run;
    __syncthreads();
    int total = 0, seq_at = run - mine;
#pragma unroll
    for (int w = 0; w < kAttnThreads / 32; ++w) {
        seq_at += w < warp ? scan[w] : 0;
        total += scan[w];
    }
    total *= per_seq;
    seq_at *= per_seq;
    const int ranges = blocks_used(total, p.batch * per_seq, gridDim.x);
    const int start = range < ranges ? range_start(range, total, ranges) : total;
    const int stop = range < ranges ? range_start(range + 1, total, ranges) : total;
    if (start < stop && start >= seq_at && start < seq_at + mine * per_seq) {
        int i = b0;
        for (; slice > 1; ++i) {
            const int u = span_of(length_of(p, i), p.tokens, p.window, p.sinks).units * per_seq;
            if (start < seq_at + u)
                break;
            seq_at += u;
        }
        scan[8] = i;
        scan[9] = seq_at;
    }
    __syncthreads();
    int b = scan[8];
    seq_at = scan[9];   // first unit of sequence b

    if (start < stop && warp == kFeedWarp) {
        // ============================================================ the feed
        // A stage is `pieces` copies each of K and V; lane l describes piece l % pieces of
        // unit l / pieces of a batch of 32 / pieces units.
        const int piece_tokens = min(p.pool.page, kUnit);
        const int pieces = kUnit / piece_tokens, per_batch = 32 / pieces;
        uint32_t issued = 0, parity = 0;
        bool ok = !(p.drop_arrive && blockIdx.x == 0);
        int u0 = start;
        uint32_t stage = 0, phase = 0;
        while (ok && u0 < stop) {
            const int unit = u0 + lane / pieces;
            float ks = -1.0f, vs = -1.0f;   // < 0: no such page
            int id = -1, slot = 0, h = 0;
            if (unit < stop) {
                int n = length_of(p, b);
                Span s = span_of(n, p.tokens, p.window, p.sinks);
                int lb = b, lat = seq_at;
                while (unit >= lat + s.units * per_seq) {
                    lat += s.units * per_seq;
                    n = length_of(p, ++lb);
                    s = span_of(n, p.tokens, p.window, p.sinks);
                }
                const int local = (unit - lat) / s.units;
                h = local / p.passes;
                const int token = s.chunk((unit - lat) % s.units) * kUnit +
                                  (lane % pieces) * piece_tokens;
                slot = token & (p.pool.page - 1);
                // (a page of 16 or 32 tokens may lie in a unit that rows see and be seen by none itself: the
                // sequence may have given it up)
                const bool seen = p.window == 0 || token < p.sinks ||
                                  token + piece_tokens > max(n - p.tokens, 0) - p.window + 1;
                if (token < n && seen) {
                    id = p.pages[lb * p.max_pages + (token >> p.pool.page_shift)];
                    if (id < 0 || id >= p.pool.num_pages) {
                        record_page_error();
                        id = -1;
                    } else {
                        ks = p.pool.scales[0][(int64_t)id * p.pool.kv_heads + h];
                        vs = p.pool.scales[1][(int64_t)id * p.pool.kv_heads + h];
                    }
                }
                b = lb;
                seq_at = lat;
            }
            const float lv = log2f(fmaxf(vs, kMinScale));
            // the next batch starts in the sequence of this one's last unit
            const int last = min(per_batch, stop - u0) * pieces - 1;
            b = __shfl_sync(0xffffffffu, b, last);
            seq_at = __shfl_sync(0xffffffffu, seq_at, last);
            for (int i = 0; i < per_batch && u0 + i < stop; ++i) {
                if (!wait_bounded(empty(stage), phase ^ 1u, p.wait_limit_ns, abort_flag,
                                  kSiteProducerEmpty)) {
                    ok = false;
                    break;
                }
                const bool in = lane / pieces == i;
                const uint32_t copies = __popc(__ballot_sync(0xffffffffu, in && id >= 0));
                if (lane == 0)
                    mbar_arrive_expect_tx(full(stage), copies * 2u * piece_tokens * D);
                __syncwarp();
                if (in && id >= 0) {
                    const uint32_t off = stage * G::kTile + (lane % pieces) * piece_tokens * D;
                    tma_load_4d(&tmK, base + G::kOffK + off, full(stage), 0, slot, h, id);
                    tma_load_4d(&tmV, base + G::kOffV + off, full(stage), 0, slot, h, id);
                }
                if (in)
                    for (int s = 0; s < piece_tokens / 16; ++s)
                        meta[stage * 4 + (lane % pieces) * (piece_tokens / 16) + s] = make_float2(ks, lv);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(full(stage));
                issued |= 1u << stage;
                parity = (parity & ~(1u << stage)) | (phase << stage);
                if (++stage == (uint32_t)G::kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            u0 += per_batch;
        }
        // every copy issued has landed before the block may exit
        for (uint32_t s = 0; s < (uint32_t)G::kStages; ++s)
            if (issued & (1u << s))
                wait_drain(full(s), (parity >> s) & 1u, p.wait_limit_ns, abort_flag);
    } else if (start < stop && warp < kWarps) {
        // ============================================================ the products
        const int g = lane >> 2, c = lane & 3;
        float *join = reinterpret_cast<float *>(gbase + G::kOffJoin);
        float *stat = reinterpret_cast<float *>(gbase + G::kOffStat);
        float *stat_m = stat, *stat_l = stat + kWarps * kRows, *stat_r = stat + 2 * kWarps * kRows;
        float *stats = p.partial + (int64_t)p.grid * 2 * kRows * D;   // the parts' (m, l, r)
        bool alive = true;
        uint32_t stage = 0, phase = 0;
        int unit = start;
        // the segments that this block has a part of, at most two: the one that it starts in
        // and the one that it ends in
        int cut_b[2], cut_local[2], cut_seg0[2], cut_seg1[2], cuts = 0;
        while (unit < stop) {
            // the (sequence, head, pass) of this unit, and its units in this block
            int n = length_of(p, b);
            Span s = span_of(n, p.tokens, p.window, p.sinks);
            while (unit >= seq_at + s.units * per_seq) {
                seq_at += s.units * per_seq;
                n = length_of(p, ++b);
                s = span_of(n, p.tokens, p.window, p.sinks);
            }
            const int local = (unit - seq_at) / s.units;
            const int h = local / p.passes, tile = local % p.passes * p.abreast + lane_tile;
            const int seg0 = seq_at + local * s.units, seg1 = seg0 + s.units;
            const int end = seg1 < stop ? seg1 : stop;
            const int row0 = tile * kRows;

            // the query rows as fragments (lane g's row of each group of 8), and what the lane
            // knows of the rows of its scores, 2c and 2c + 1: position (-1: sees nothing), scale (a power of two)
            uint32_t q[kN][D / 8];
            int pos[kN][2];
            float row_scale[kN][2];
#pragma unroll
            for (int t = 0; t < kN; ++t) {
                const int r = row0 + 8 * t + g, token = r / p.group;
                const uint16_t *src = p.q + b * p.q_stride[0] + token * p.q_stride[1] +
                                      (h * p.group + r % p.group) * p.q_stride[2];
                float back;
                load_row<D, kBf16>(r < p.rows ? src : nullptr, c, q[t], back);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = row0 + 8 * t + 2 * c + e;
                    pos[t][e] = row < p.rows ? n - p.tokens + row / p.group : -1;
                    row_scale[t][e] = 1.0f;
                    if constexpr (kBf16)
                        row_scale[t][e] = __shfl_sync(0xffffffffu, back, 4 * (2 * c + e));
                }
            }
            const int pos_min = n - p.tokens + row0 / p.group;
            const int pos_max = n - p.tokens + (min(row0 + kRows, p.rows) - 1) / p.group;

            // o[t][j]: elements 2j (0, 1) and 2j + 1 (2, 3) of the lane's piece, rows 2c, 2c + 1
            float o[kN][D / 16][4];
            float m[kN][2], md[kN][2], l[kN][2];   // (md: 7 - r)
#pragma unroll
            for (int t = 0; t < kN; ++t) {
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.0f;
                m[t][0] = m[t][1] = -INFINITY;
                md[t][0] = md[t][1] = 0.0f;
                l[t][0] = l[t][1] = 0.0f;
            }
            const int units_here = end - unit, u0 = unit - seg0;
            for (int u = 0; u < units_here; ++u) {
                const int t0 = s.chunk(u0 + u) * kUnit + 16 * warp;
                if (alive)
                    alive = wait_bounded_eager(full(stage), phase, p.wait_limit_ns, abort_flag,
                                               kSiteMmaFull);
                alive = __all_sync(0xffffffffu, alive);
                const float2 sc = meta[stage * 4 + warp];
                if (kScores && alive && !(sc.x > 0.0f)) {   // a page that is not there
                    for (int k = lane; k < 16 * kRows; k += 32)
                        if (t0 + k / kRows < n && row0 + k % kRows < p.rows)
                            p.scores[(((int64_t)b * p.pool.kv_heads + h) * p.width + t0 + k / kRows) * p.rows +
                                     row0 + k % kRows] = -INFINITY;
                }
                if (alive && sc.x > 0.0f && t0 <= pos_max &&
                    (p.window == 0 || t0 + 15 > pos_min - p.window || t0 < p.sinks)) {
                    const uint32_t k_at = base + G::kOffK + stage * G::kTile + 16 * warp * D;
                    const uint32_t v_at = base + G::kOffV + stage * G::kTile + 16 * warp * D;
                    // ---- S^T = K Q^T; acc[t][2 i + e]: token row g + 8 i, query row 2c + e
                    float acc[kN][4];
                    {
                        float part[kN][2][4];   // two chains of products
#pragma unroll
                        for (int t = 0; t < kN; ++t)
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                part[t][x][0] = part[t][x][1] = part[t][x][2] = part[t][x][3] = 0.0f;
#pragma unroll
                        for (int half = 0; half < D / 64; ++half) {
                            const uint4 lo = ld_shared_v4(k_at + at_chunk<D>(key_of(g), c + 4 * half));
                            const uint4 hi = ld_shared_v4(k_at + at_chunk<D>(8 + key_of(g), c + 4 * half));
                            const uint32_t k0[4] = {lo.x, lo.y, lo.z, lo.w};
                            const uint32_t k1[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                            for (int st = 0; st < 4; ++st) {
                                const uint32_t a0 = e4m3x2_to_half2(k0[st] & 0xffffu);
                                const uint32_t a1 = e4m3x2_to_half2(k1[st] & 0xffffu);
                                const uint32_t a2 = e4m3x2_to_half2(k0[st] >> 16);
                                const uint32_t a3 = e4m3x2_to_half2(k1[st] >> 16);
#pragma unroll
                                for (int t = 0; t < kN; ++t)
                                    mma_f16(part[t][st & 1], a0, a1, a2, a3, q[t][8 * half + 2 * st],
                                            q[t][8 * half + 2 * st + 1]);
                            }
                        }
#pragma unroll
                        for (int t = 0; t < kN; ++t)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                acc[t][x] = part[t][0][x] + part[t][1][x];
                    }
                    // ---- scores in base 2 relative to the rows' references, masked
                    const bool masked = !(t0 + 15 <= pos_min &&
                                          (p.window == 0 || t0 > pos_max - p.window || t0 + 15 < p.sinks));
                    const int ta = t0 + key_of(g), tb = ta + 8;   // the lane's tokens
                    float x[kN][4], d[kN][2];   // exponents of the weights, and what P's exceed them by
                    bool high = false;
#pragma unroll
                    for (int t = 0; t < kN; ++t) {
                        if constexpr (kScores) {
                            float *dst = p.scores + (((int64_t)b * p.pool.kv_heads + h) * p.width + ta) * p.rows +
                                         row0 + 8 * t + 2 * c;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (pos[t][i & 1] >= 0 && (i < 2 ? ta : tb) < n)
                                    dst[(i >> 1) * 8 * p.rows + (i & 1)] =
                                        acc[t][i] * (sc.x * row_scale[t][i & 1]) * p.scale_log2;
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = i & 1;
                            x[t][i] = fmaf(acc[t][i], sc.x * row_scale[t][e], -m[t][e]) * p.scale_log2;
                            if (masked && !sees(i < 2 ? ta : tb, pos[t][e], p.window, p.sinks))
                                x[t][i] = acc[t][i] = -INFINITY;
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            d[t][e] = fminf(md[t][e] + sc.y, 126.0f);
                            high |= fmaxf(x[t][e], x[t][2 + e]) > fminf(kMoveLog2, kMoveLog2 + kPLog2 - d[t][e]);
                        }
                    }
                    if (__any_sync(0xffffffffu, high)) {
                        // move the rows' references to their largest score so far
#pragma unroll
                        for (int t = 0; t < kN; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float f = sc.x * row_scale[t][e];
                                float top = fmaxf(acc[t][e] * f, acc[t][2 + e] * f);
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                                const float to = fmaxf(m[t][e], top);
                                const float a = to > m[t][e] ? exp2_fast((m[t][e] - to) * p.scale_log2) : 1.0f;   // 0 at first
                                l[t][e] *= a;
                                // o's old reference and this unit's, from the new m
                                const float ref = to == -INFINITY ? 0.0f : to;
                                const float r0 = (m[t][e] - ref) * p.scale_log2 + (kPLog2 - md[t][e]);
                                const float r1 = fmaxf(r0, rintf((top - ref) * p.scale_log2 + sc.y));
                                const float ao = r1 > r0 ? exp2_fast(r0 - r1) : 1.0f;
#pragma unroll
                                for (int j = 0; j < D / 16; ++j) {
                                    o[t][j][e] *= ao;
                                    o[t][j][2 + e] *= ao;
                                }
                                m[t][e] = to;
                                md[t][e] = less(kPLog2, r1);
                                d[t][e] = fminf(md[t][e] + sc.y, 126.0f);
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    x[t][2 * i + e] = acc[t][2 * i + e] == -INFINITY
                                                          ? -INFINITY
                                                          : fmaf(acc[t][2 * i + e], f, -ref) * p.scale_log2;
                            }
                    }
                    // ---- P^T as the second product's B operand: {rows 2c, 2c + 1} of a token to
                    // {tokens 2c, 2c + 1} of a row
                    uint32_t pt[kN][2];
#pragma unroll
                    for (int t = 0; t < kN; ++t) {
                        const float e0 = exp2_fast(x[t][0]), e1 = exp2_fast(x[t][1]);
                        const float e2 = exp2_fast(x[t][2]), e3 = exp2_fast(x[t][3]);
                        const float f0 = exp2_fast(d[t][0]), f1 = exp2_fast(d[t][1]);
                        l[t][0] += e0 + e2;
                        l[t][1] += e1 + e3;
                        pt[t][0] = turned(half2_of(e0 * f0, e1 * f1));
                        pt[t][1] = turned(half2_of(e2 * f0, e3 * f1));
                    }
                    // ---- O^T += V^T P^T: the lane's four tokens c, c + 4, c + 8, c + 12
                    constexpr int kW = D / 32;   // words of a lane's piece
                    uint32_t v[4][kW];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = c + 4 * k, piece = piece_of<D>(g);
                        if constexpr (D == 128) {
                            const uint4 w = ld_shared_v4(v_at + at_chunk<D>(row, piece));
                            v[k][0] = w.x, v[k][1] = w.y, v[k][2] = w.z, v[k][3] = w.w;
                        } else {
                            const uint2 w = ld_shared_v2(v_at + at_chunk<D>(row, piece >> 1) + 8 * (piece & 1));
                            v[k][0] = w.x, v[k][1] = w.y;
                        }
                    }
                    if (masked) {
                        // slots that no row sees may hold anything, NaN included: 0 * NaN
                        uint32_t bad = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int at = t0 + c + 4 * k;
                            const bool any = at <= pos_max && (p.window == 0 || at > pos_min - p.window || at < p.sinks);
#pragma unroll
                            for (int w = 0; w < kW; ++w) {
                                v[k][w] = any ? v[k][w] : 0u;
                                bad |= nan_bytes(v[k][w]);
                            }
                        }
                        if (__any_sync(0xffffffffu, bad != 0)) {
                            // a NaN that some rows see and others do not: count it for
                            // the rows that see it, then take it out
                            const uint32_t one = 0x3c00u;
#pragma unroll
                            for (int t = 0; t < kN; ++t) {
                                const int row = row0 + 8 * t + g;
                                const int at = row < p.rows ? n - p.tokens + row / p.group : -1;
                                uint32_t seen[2];
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    seen[i] = (sees(t0 + c + 8 * i, at, p.window, p.sinks) ? one : 0u) |
                                              (sees(t0 + c + 8 * i + 4, at, p.window, p.sinks) ? one << 16 : 0u);
#pragma unroll
                                for (int j = 0; j < D / 16; ++j) {
                                    uint32_t a[4];   // elements 2j, 2j + 1 (i & 1), tokens k, k + 1 (k = i & 2)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const int sh = 8 * ((2 * j + (i & 1)) & 3) + 7;
                                        const int k = i & 2;
                                        a[i] = (nan_bytes(v[k][j >> 1]) >> sh & 1u ? one : 0u) |
                                               (nan_bytes(v[k + 1][j >> 1]) >> sh & 1u ? one << 16 : 0u);
                                    }
                                    float count[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                    mma_f16(count, a[0], a[1], a[2], a[3], seen[0], seen[1]);
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        if (count[i] > 0.0f)
                                            o[t][j][i] = __uint_as_float(0x7fffffffu);
                                }
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k)
#pragma unroll
                                for (int w = 0; w < kW; ++w)
                                    v[k][w] &= ~((nan_bytes(v[k][w]) >> 7) * 0xffu);
                        }
                    }
#pragma unroll
                    for (int w = 0; w < kW; ++w)
#pragma unroll
                        for (int pair = 0; pair < 2; ++pair) {
                            // bytes 2 pair, 2 pair + 1 of two tokens each: {token, token} of both elements
                            const uint32_t sel = pair ? 0x7362u : 0x5140u;
                            const uint32_t y = __byte_perm(v[0][w], v[1][w], sel);
                            const uint32_t z = __byte_perm(v[2][w], v[3][w], sel);
                            const uint32_t a0 = e4m3x2_to_half2(y & 0xffffu), a1 = e4m3x2_to_half2(y >> 16);
                            const uint32_t a2 = e4m3x2_to_half2(z & 0xffffu), a3 = e4m3x2_to_half2(z >> 16);
#pragma unroll
                            for (int t = 0; t < kN; ++t)
                                mma_f16(o[t][2 * w + pair], a0, a1, a2, a3, pt[t][0], pt[t][1]);
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
            unit = end;

            // ---- join the four warps: each leaves (O, m, l, r), then 16 / kN threads take a row
#pragma unroll
            for (int t = 0; t < kN; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 4);
                    l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 8);
                    l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 16);
                    const int row = warp * kRows + 8 * t + 2 * c + e;
                    float *dst = join + row * G::kPitch + piece_of<D>(g) * (D / 8);
#pragma unroll
                    for (int j = 0; j < D / 16; j += 2)
                        *reinterpret_cast<float4 *>(dst + 2 * j) =
                            make_float4(o[t][j][e], o[t][j][2 + e], o[t][j + 1][e], o[t][j + 1][2 + e]);
                    if (g == 0) {
                        stat_m[row] = m[t][e];
                        stat_l[row] = l[t][e];
                        stat_r[row] = kPLog2 - md[t][e];
                    }
                }
            named_bar_sync(1, 32 * kWarps);
            {
                constexpr int kF = D * kN / 16;   // elements a thread
                const int r = tid * kN / 16, d0 = tid % (16 / kN) * kF;
                float top = -INFINITY, top_r = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    top = fmaxf(top, stat_m[w * kRows + r]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    top_r = fmaxf(top_r, less(stat_m[w * kRows + r], top) * p.scale_log2 + stat_r[w * kRows + r]);
                float y[kF];
#pragma unroll
                for (int j = 0; j < kF; ++j)
                    y[j] = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float below = less(stat_m[w * kRows + r], top) * p.scale_log2;
                    const float fv = exp2_fast(less(below + stat_r[w * kRows + r], top_r));
                    sum += exp2_fast(below) * stat_l[w * kRows + r];
                    const float4 *src = reinterpret_cast<const float4 *>(
                        join + (w * kRows + r) * G::kPitch + d0);
#pragma unroll
                    for (int j = 0; j < kF / 4; ++j) {
                        const float4 z = src[j];
                        y[4 * j] += fv * z.x;
                        y[4 * j + 1] += fv * z.y;
                        y[4 * j + 2] += fv * z.z;
                        y[4 * j + 3] += fv * z.w;
                    }
                }
                if (seg0 >= start && seg1 <= stop) {   // the whole of it
                    if (alive && row0 + r < p.rows)
                        write_row<D, kF, kBf16, kScores>(p, b, h, row0 + r, d0, y, top, top_r, sum);
                } else {
                    // a part: slot 0 where it starts this block's range, else slot 1
                    const int64_t at = ((int64_t)(range * p.abreast + lane_tile) * 2 + (seg0 > start ? 1 : 0)) * kRows + r;
                    float *dst = p.partial + at * D + d0;
#pragma unroll
                    for (int j = 0; j < kF; j += 4)
                        *reinterpret_cast<float4 *>(dst + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
                    if (d0 == 0)
                        *reinterpret_cast<float4 *>(stats + at * 4) = make_float4(top, sum, top_r, 0.0f);
                    cut_b[cuts & 1] = b;
                    cut_local[cuts & 1] = local;
                    cut_seg0[cuts & 1] = seg0;
                    cut_seg1[cuts & 1] = seg1;
                    ++cuts;
                }
            }
            named_bar_sync(1, 32 * kWarps);
        }

        // ---- count the parts; who counts the last one of a segment joins it
        if (cuts > 0) {
            int *last = reinterpret_cast<int *>(stat_r);
            named_bar_sync(1, 32 * kWarps);
            if (lane == 0 && warp < cuts) {
                const int i = warp;
                const int c0 = range_owner(i ? cut_seg0[1] : cut_seg0[0], total, ranges);
                const int c1 = range_owner((i ? cut_seg1[1] : cut_seg1[0]) - 1, total, ranges);
                last[i] = count_part(p.arrived + c0 * p.abreast + lane_tile, (unsigned)(c1 - c0)) ==
                          (unsigned)(c1 - c0);
            }
            named_bar_sync(1, 32 * kWarps);
#pragma unroll 1
            for (int i = 0; i < cuts; ++i) {
                if (!last[i])
                    continue;
                const int seg0 = i ? cut_seg0[1] : cut_seg0[0], seg1 = i ? cut_seg1[1] : cut_seg1[0];
                const int local = i ? cut_local[1] : cut_local[0], bb = i ? cut_b[1] : cut_b[0];
                const int c0 = range_owner(seg0, total, ranges), c1 = range_owner(seg1 - 1, total, ranges);
                constexpr int kF = D * kN / 16;
                const int r = tid * kN / 16, d0 = tid % (16 / kN) * kF;
                // a part's row: only the first part can start inside its block's range
                const int first = seg0 > range_start(c0, total, ranges) ? 1 : 0;
                auto slot = [&](int c) {
                    return (int64_t)((c * p.abreast + lane_tile) * 2 + (c == c0 ? first : 0)) * kRows + r;
                };
                float ref = -INFINITY, ref_r = -INFINITY, sum = 0.0f, y[kF];
#pragma unroll
                for (int j = 0; j < kF; ++j)
                    y[j] = 0.0f;
                // a few parts are read at a time: each round waits for L2 once
                constexpr int kAtOnce = kN == 1 ? 8 : 4;
                for (int c = c0; c <= c1; c += kAtOnce) {
                    float4 ml[kAtOnce];   // (m, l, r)
                    float4 z[kAtOnce][kF / 4];
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k) {
                        ml[k] = make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
                        if (c + k <= c1) {
                            const int64_t at = slot(c + k);
                            ml[k] = __ldcg(reinterpret_cast<const float4 *>(stats + at * 4));
#pragma unroll
                            for (int j = 0; j < kF / 4; ++j)
                                z[k][j] = __ldcg(reinterpret_cast<const float4 *>(p.partial + at * D + d0) + j);
                        }
                    }
                    float top = ref;
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k)
                        top = fmaxf(top, ml[k].x);
                    const float r0 = less(ref, top) * p.scale_log2 + ref_r;   // (-infinity at first, as in ref)
                    float r1 = r0;
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k)
                        r1 = fmaxf(r1, less(ml[k].x, top) * p.scale_log2 + ml[k].z);
                    sum *= exp2_fast(less(ref, top) * p.scale_log2);
                    const float fy = exp2_fast(less(r0, r1));
#pragma unroll
                    for (int j = 0; j < kF; ++j)
                        y[j] *= fy;
                    ref = top;
                    ref_r = r1;
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k) {
                        if (c + k > c1)
                            break;
                        const float below = less(ml[k].x, ref) * p.scale_log2;
                        sum += exp2_fast(below) * ml[k].y;
                        const float f = exp2_fast(less(below + ml[k].z, ref_r));
#pragma unroll
                        for (int j = 0; j < kF / 4; ++j) {
                            y[4 * j] += f * z[k][j].x;
                            y[4 * j + 1] += f * z[k][j].y;
                            y[4 * j + 2] += f * z[k][j].z;
                            y[4 * j + 3] += f * z[k][j].w;
                        }
                    }
                }
                const int row = (local % p.passes * p.abreast + lane_tile) * kRows + r;
                if (alive && row < p.rows)
                    write_row<D, kF, kBf16, kScores>(p, bb, local / p.passes, row, d0, y, ref, ref_r, sum);
            }
        }
    }

    // sequences without tokens
    for (int i = blockIdx.x; i < p.batch; i += gridDim.x) {
        if (length_of(p, i) > 0)
            continue;
        uint4 *dst = reinterpret_cast<uint4 *>(p.out + (int64_t)i * p.tokens * p.q_heads * D);
        for (int j = tid; j < p.tokens * p.q_heads * (D / 8); j += kAttnThreads)
            dst[j] = make_uint4(0, 0, 0, 0);
    }
}

// weights[t] += sum over the rows that see t of softmax_t, from the scores and each row's
// log-sum-exp; a thread per token, the rows kVec at a time.  All that it reads is asked for
// before the length is known (scores and weights have room for every slot of the table).
constexpr int kWeightThreads = 256;

template <int kVec>
__global__ void __launch_bounds__(kWeightThreads) kv_attention_weights_kernel(const AttnParams p) {
    pdl_launch_dependents();
    const int blocks = (int)((p.width + kWeightThreads - 1) / kWeightThreads);
    const int bh = blockIdx.x / blocks, b = bh / p.pool.kv_heads;
    const int t = (blockIdx.x - bh * blocks) * kWeightThreads + threadIdx.x;
    pdl_wait_primary();
    if (t >= p.width)
        return;
    const float *s = p.scores + ((int64_t)bh * p.width + t) * p.rows;
    const float *lse = p.lse + (int64_t)bh * p.rows;
    float *w = p.weights + (int64_t)bh * p.width + t;
    const float before = *w;
    const int n = length_of(p, b);
    float sum = 0.0f;
    for (int r = 0; r < p.rows; r += kVec) {
        float x[kVec], y[kVec];
        if constexpr (kVec == 4) {
            const float4 u = *reinterpret_cast<const float4 *>(s + r);
            const float4 v = *reinterpret_cast<const float4 *>(lse + r);
            x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
            y[0] = v.x, y[1] = v.y, y[2] = v.z, y[3] = v.w;
        } else {
            x[0] = s[r], y[0] = lse[r];
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (sees(t, n - p.tokens + (r + i) / p.group, p.window, p.sinks))   // (else x is anything)
                sum += exp2_fast(x[i] - y[i]);
    }
    if (t < n)
        *w = before + sum;
}

}  // namespace kvc
}  // namespace gemmrelu
