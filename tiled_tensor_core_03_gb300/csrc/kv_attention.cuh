// kv_attention.cuh -- attention of a few new tokens over the paged 8-bit cache:
//
//   O[r] = sum_t softmax_t(q_r . k_t / sqrt(D)) v_t,  k_t = ks * K8[t], v_t = vs * V8[t]
//
// over the tokens t that row r sees (t <= p_r; with a window W also t > p_r - W
// or t < sinks), p_r the row's position.  The rows of one K/V head are
// its group's query heads of every new token, 16 rows a tile.
//
// What bounds it: every visible token's 2 D bytes are read once per 16 rows and
// used for 4 D flops a row, so up to some tens of rows it is a stream from HBM.  The
// kernel is built around that stream:
//
//  - Work is cut into units of 64 tokens of one (sequence, head, row tile); the
//    units of all of them, in order, are dealt to the blocks in equal contiguous
//    ranges whatever the lengths are, two blocks an SM.  A block finishes what lies
//    inside its range; a (sequence, head, row tile) that is cut leaves one fp32
//    partial (O, m, l) per block in the workspace, and a second kernel joins them in
//    order.  Nothing depends on the order in which blocks run: the same call gives
//    the same bits.
//  - One warp feeds a ring of 64-token stages by TMA (a page or a part of one per
//    copy), reading page numbers and scales 32 pieces ahead.
//  - Four warps take 16 tokens of a stage each.  The products run on
//    mma.sync.m16n8k16 with fp16 operands: 16 rows are all there is, far below the
//    128 of a tcgen05.mma, and e4m3 has to become fp16 (exact) on the way, which
//    happens in registers here.  The operand layouts are chosen so that the bytes a
//    lane loads from shared memory are the ones its fragment needs, with no
//    shuffle (see key_of / chunk_of below).
//  - Softmax in one pass, base 2, a running reference m per row that moves only when
//    a score exceeds it by 2^8; fp32 statistics and accumulators.  P is
//    rounded to fp16 for the second product (relative 2^-11, like the output's own
//    rounding).  V's scale is folded into P relative to the
//    largest scale met so far, 2^7 above one: P stays below 2^15 and normal down to
//    2^-21 of the row's largest weight.
#pragma once

#include "kv_cache.cuh"

namespace gemmrelu {
namespace kvc {

constexpr int kUnit = 64;            // tokens of a stage
constexpr int kRows = 16;            // query rows of a tile
constexpr int kWarps = 4;            // computing warps
constexpr int kFeedWarp = 4;
constexpr int kAttnThreads = 160;
constexpr int kAttnBlocksPerSm = 2;
constexpr float kMoveLog2 = 8.0f;    // the reference moves when a score exceeds it by more
constexpr float kPShift = 128.0f;    // 2^7, see above

template <int D>
struct AttnCfg {
    static constexpr uint32_t kTile = kUnit * D;                 // bytes of K (or V) in a stage
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr uint32_t kOffK = 0;
    static constexpr uint32_t kOffV = kOffK + kStages * kTile;
    static constexpr int kPitch = D + 4;                         // floats a row of the join buffer
    static constexpr uint32_t kOffJoin = kOffV + kStages * kTile;   // [4 warps][16][kPitch]
    static constexpr uint32_t kOffStat = kOffJoin + kWarps * kRows * kPitch * 4;   // m, l [4][16], vref [4]
    static constexpr uint32_t kOffMeta = kOffStat + (2 * kWarps * kRows + kWarps) * 4;
    static constexpr uint32_t kOffScan = kOffMeta + kStages * 4 * 8;   // (ks, vs) per 16 tokens
    static constexpr uint32_t kOffBar = kOffScan + (kAttnThreads + 8) * 8;
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
    int rows, row_tiles;               // tokens * group, in tiles of 16
    int window, sinks;
    float scale_log2;                  // log2(e) / sqrt(D)
    float *partial;                    // [2 * grid][16][D], then [2 * grid][16][2] (m, l)
    int grid;
    int64_t *before;                   // [batch + 1] units of the sequences before
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

// First unit of block c of `grid`, of `total`: equal ranges, and the block that owns unit x.
__host__ __device__ __forceinline__ int64_t range_start(int64_t c, int64_t total, int grid) {
    return c * total / grid;
}
__host__ __device__ __forceinline__ int range_owner(int64_t x, int64_t total, int grid) {
    return (int)(((x + 1) * grid - 1) / total);
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

// In fragments of mma.m16n8k16 lane = 4 g + c.  S = Q K^T: column g of an 8-token group is
// token key_of(g), so that the score fragment's columns 2c, 2c+1 are tokens c, c + 4 and
// eight lanes that load together touch eight different chunks.
__device__ __forceinline__ int key_of(int g) { return (g >> 1) | ((g & 1) << 2); }

// The k index of S = Q K^T runs over the D elements in an order of its own: lane c's
// k-steps are the consecutive fours of its chunk(s) c (and c + 4), so a K fragment is 4
// consecutive bytes.  Q's fragment uses the same order.
//
// O += P V: lane g's columns of the D / 8 column groups are D / 8 consecutive elements,
// those of piece piece_of(g) (16 bytes for D = 128, 8 for D = 64).
template <int D>
__device__ __forceinline__ int piece_of(int g) {
    if constexpr (D == 128)
        return (g >> 1) | ((g & 1) << 2);
    else
        return ((g >> 1) & 1) << 2 | (g >> 2) << 1 | (g & 1);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t half2_of(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
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

// ---------------------------------------------------------------- the stream

template <int D, bool kBf16, bool kScores>
__global__ void __launch_bounds__(kAttnThreads, kAttnBlocksPerSm)
    kv_attention_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const AttnParams p) {
    using G = AttnCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t bar0 = base + G::kOffBar;
    auto full = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty = [&](uint32_t s) { return bar0 + 8u * (G::kStages + s); };
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + G::kOffMisc);
    int64_t *scan = reinterpret_cast<int64_t *>(gbase + G::kOffScan);
    float2 *meta = reinterpret_cast<float2 *>(gbase + G::kOffMeta);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (uint32_t s = 0; s < (uint32_t)G::kStages; ++s) {
            mbar_init(full(s), 1u);
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
    pdl_wait_primary();

    // this block's range of units, and the sequence that it starts in
    const int per_seq = p.pool.kv_heads * p.row_tiles;   // (head, row tile) pairs
    const int slice = (p.batch + kAttnThreads - 1) / kAttnThreads;
    const int b0 = min(tid * slice, p.batch), b1 = min(b0 + slice, p.batch);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b)
        mine += span_of(length_of(p, b), p.tokens, p.window, p.sinks).units;
    scan[tid] = mine;
    __syncthreads();
    if (warp == 0) {   // exclusive sums of the 160 slices
        int64_t v[5], sum = 0;
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            v[i] = scan[lane * 5 + i];
            sum += v[i];
        }
        int64_t run = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, run, o);
            run += lane >= o ? x : 0;
        }
        int64_t at = run - sum;
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            scan[lane * 5 + i] = at;
            at += v[i];
        }
        if (lane == 31)
            scan[kAttnThreads] = run;
    }
    __syncthreads();
    const int64_t total = scan[kAttnThreads] * per_seq;
    const int64_t start = range_start(blockIdx.x, total, p.grid);
    const int64_t stop = range_start(blockIdx.x + 1, total, p.grid);
    {
        int64_t at = scan[tid];
        for (int b = b0; b < b1; ++b) {
            const int64_t u = span_of(length_of(p, b), p.tokens, p.window, p.sinks).units;
            if (blockIdx.x == 0)
                p.before[b] = at;
            if (start < stop && start >= at * per_seq && start < (at + u) * per_seq) {
                scan[kAttnThreads + 1] = b;
                scan[kAttnThreads + 2] = at * per_seq;
            }
            at += u;
        }
        if (blockIdx.x == 0 && tid == 0)
            p.before[p.batch] = scan[kAttnThreads];
    }
    __syncthreads();
    int b = (int)scan[kAttnThreads + 1];
    int64_t seq_at = scan[kAttnThreads + 2];   // first unit of sequence b

    if (start < stop && warp == kFeedWarp) {
        // ============================================================ the feed
        // A stage is `pieces` copies each of K and V; lane l describes piece l % pieces of
        // unit l / pieces of a batch of 32 / pieces units.
        const int piece_tokens = min(p.pool.page, kUnit);
        const int pieces = kUnit / piece_tokens, per_batch = 32 / pieces;
        uint32_t issued = 0, parity = 0;
        bool ok = !(p.drop_arrive && blockIdx.x == 0);
        int64_t u0 = start;
        uint32_t stage = 0, phase = 0;
        while (ok && u0 < stop) {
            const int64_t unit = u0 + lane / pieces;
            float ks = -1.0f, vs = -1.0f;   // < 0: no such page
            int id = -1, slot = 0, h = 0;
            if (unit < stop) {
                int n = length_of(p, b);
                Span s = span_of(n, p.tokens, p.window, p.sinks);
                int lb = b;
                int64_t lat = seq_at;
                while (unit >= lat + (int64_t)s.units * per_seq) {
                    lat += (int64_t)s.units * per_seq;
                    n = length_of(p, ++lb);
                    s = span_of(n, p.tokens, p.window, p.sinks);
                }
                const int local = (int)((unit - lat) / s.units);
                h = local / p.row_tiles;
                const int token = s.chunk((int)((unit - lat) % s.units)) * kUnit +
                                  (lane % pieces) * piece_tokens;
                slot = token & (p.pool.page - 1);
                if (token < n) {
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
            // the next batch starts in the sequence of this one's last unit
            const int last = (int)min((int64_t)per_batch, stop - u0) * pieces - 1;
            b = __shfl_sync(0xffffffffu, b, last);
            seq_at = __shfl_sync(0xffffffffu, seq_at, last);
            for (int i = 0; i < per_batch && u0 + i < stop; ++i) {
                if (!wait_bounded(empty(stage), phase ^ 1u, p.wait_limit_ns, abort_flag,
                                  kSiteProducerEmpty)) {
                    ok = false;
                    break;
                }
                const bool in = lane / pieces == i;
                if (in)
                    for (int s = 0; s < piece_tokens / 16; ++s)
                        meta[stage * 4 + (lane % pieces) * (piece_tokens / 16) + s] = make_float2(ks, vs);
                const uint32_t copies = __popc(__ballot_sync(0xffffffffu, in && id >= 0));
                if (lane == 0)
                    mbar_arrive_expect_tx(full(stage), copies * 2u * piece_tokens * D);
                __syncwarp();
                if (in && id >= 0) {
                    const uint32_t off = stage * G::kTile + (lane % pieces) * piece_tokens * D;
                    tma_load_4d(&tmK, base + G::kOffK + off, full(stage), 0, slot, h, id);
                    tma_load_4d(&tmV, base + G::kOffV + off, full(stage), 0, slot, h, id);
                }
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
        float *stat_m = stat, *stat_l = stat + kWarps * kRows, *stat_v = stat + 2 * kWarps * kRows;
        bool alive = true;
        uint32_t stage = 0, phase = 0;
        int64_t unit = start;
        while (unit < stop) {
            // the (sequence, head, row tile) of this unit, and its units in this block
            int n = length_of(p, b);
            Span s = span_of(n, p.tokens, p.window, p.sinks);
            while (unit >= seq_at + (int64_t)s.units * per_seq) {
                seq_at += (int64_t)s.units * per_seq;
                n = length_of(p, ++b);
                s = span_of(n, p.tokens, p.window, p.sinks);
            }
            const int local = (int)((unit - seq_at) / s.units);
            const int h = local / p.row_tiles, tile = local % p.row_tiles;
            const int64_t seg0 = seq_at + (int64_t)local * s.units, seg1 = seg0 + s.units;
            const int64_t end = seg1 < stop ? seg1 : stop;
            const int row0 = tile * kRows;

            // this lane's rows g and g + 8: position (-1: sees nothing) and query
            int pos[2];
            uint32_t q[2][D / 8];
            float row_scale[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = row0 + g + 8 * i, token = r / p.group;
                const bool there = r < p.rows;
                pos[i] = there ? n - p.tokens + token : -1;
                const uint16_t *src = p.q + b * p.q_stride[0] + token * p.q_stride[1] +
                                      (h * p.group + r % p.group) * p.q_stride[2];
                float back;
                load_row<D, kBf16>(there ? src : nullptr, c, q[i], back);
                row_scale[i] = back * p.scale_log2;
            }
            const int pos_min = n - p.tokens + row0 / p.group;
            const int pos_max = n - p.tokens + (min(row0 + kRows, p.rows) - 1) / p.group;

            float o[D / 8][4];
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
                o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
            float vref = 0.0f, vinv = 0.0f;

            for (; unit < end; ++unit) {
                const int t0 = s.chunk((int)(unit - seg0)) * kUnit + 16 * warp;
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
                    // ---- S = Q K^T, two groups of 8 tokens
                    float acc[2][4];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
                        const int row = 8 * j + key_of(g);
#pragma unroll
                        for (int half = 0; half < D / 64; ++half) {
                            const uint4 k4 = ld_shared_v4(k_at + at_chunk<D>(row, c + 4 * half));
                            const uint32_t kw[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                            for (int st = 0; st < 4; ++st) {
                                const int x = 8 * half + 2 * st;
                                const uint32_t a[4] = {q[0][x], q[1][x], q[0][x + 1], q[1][x + 1]};
                                mma_f16(acc[j], a, e4m3x2_to_half2(kw[st] & 0xffffu),
                                        e4m3x2_to_half2(kw[st] >> 16));
                            }
                        }
                    }
                    // ---- scores in base 2, masked; acc[j][2 i + e]: row i, token 8 j + c + 4 e
                    const bool masked = !(t0 + 15 <= pos_min &&
                                          (p.window == 0 || t0 > pos_max - p.window || t0 + 15 < p.sinks));
                    const float f0 = sc.x * row_scale[0], f1 = sc.x * row_scale[1];
                    bool high = false;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float &x = acc[j][2 * i + e];
                                x *= i ? f1 : f0;
                                if (masked && !sees(t0 + 8 * j + c + 4 * e, pos[i], p.window, p.sinks))
                                    x = -INFINITY;
                                high |= x > m[i] + kMoveLog2;
                            }
                    if constexpr (kScores) {
                        float *dst = p.scores + (((int64_t)b * p.pool.kv_heads + h) * p.width + t0) * p.rows + row0;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (pos[i] >= 0 && t0 + 8 * j + c + 4 * e < n)
                                        dst[(int64_t)(8 * j + c + 4 * e) * p.rows + g + 8 * i] = acc[j][2 * i + e];
                    }
                    if (__any_sync(0xffffffffu, high)) {
                        // move the rows' references to their largest score so far
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float x = fmaxf(fmaxf(acc[0][2 * i], acc[0][2 * i + 1]),
                                            fmaxf(acc[1][2 * i], acc[1][2 * i + 1]));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                            const float to = fmaxf(m[i], x);
                            const float f = to > m[i] ? exp2_fast(m[i] - to) : 1.0f;   // 0 at first
                            l[i] *= f;
#pragma unroll
                            for (int j = 0; j < D / 8; ++j) {
                                o[j][2 * i] *= f;
                                o[j][2 * i + 1] *= f;
                            }
                            m[i] = to;
                        }
                    }
                    const float vs = fmaxf(sc.y, kMinScale);
                    if (vs > vref) {   // uniform in the warp
                        const float f = vref / vs;
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            o[j][0] *= f;
                            o[j][1] *= f;
                            o[j][2] *= f;
                            o[j][3] *= f;
                        }
                        vref = vs;
                        vinv = kPShift / vs;
                    }
                    // ---- P
                    const float m0 = m[0] == -INFINITY ? 0.0f : m[0], m1 = m[1] == -INFINITY ? 0.0f : m[1];
                    const float pf = vs * vinv;
                    uint32_t a[4];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float e0 = exp2_fast(acc[j][0] - m0), e1 = exp2_fast(acc[j][1] - m0);
                        const float e2 = exp2_fast(acc[j][2] - m1), e3 = exp2_fast(acc[j][3] - m1);
                        l[0] += e0 + e1;
                        l[1] += e2 + e3;
                        a[2 * j] = half2_of(e0 * pf, e1 * pf);
                        a[2 * j + 1] = half2_of(e2 * pf, e3 * pf);
                    }
                    // ---- O += P V: the lane's four tokens c, c + 4, c + 8, c + 12
                    constexpr int kW = D / 32;   // words of a lane's piece
                    uint32_t v[4][kW];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = c + 4 * k, piece = piece_of<D>(g);
                        if constexpr (D == 128) {
                            const uint4 x = ld_shared_v4(v_at + at_chunk<D>(row, piece));
                            v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
                        } else {
                            const uint2 x = ld_shared_v2(v_at + at_chunk<D>(row, piece >> 1) + 8 * (piece & 1));
                            v[k][0] = x.x, v[k][1] = x.y;
                        }
                    }
                    if (masked) {
                        // slots that no row sees may hold anything, NaN included: 0 * NaN
                        uint32_t bad = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int t = t0 + c + 4 * k;
                            const bool any = t <= pos_max && (p.window == 0 || t > pos_min - p.window || t < p.sinks);
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
                            uint32_t seen[4];
#pragma unroll
                            for (int j = 0; j < 2; ++j)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const int t = t0 + 8 * j + c;
                                    seen[2 * j + i] = (sees(t, pos[i], p.window, p.sinks) ? one : 0u) |
                                                      (sees(t + 4, pos[i], p.window, p.sinks) ? one << 16 : 0u);
                                }
#pragma unroll
                            for (int j = 0; j < D / 8; ++j) {
                                const int sh = 8 * (j & 3) + 7;
                                uint32_t n4[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    n4[k] = (nan_bytes(v[k][j >> 2]) >> sh) & 1u ? one : 0u;
                                float count[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                mma_f16(count, seen, n4[0] | n4[1] << 16, n4[2] | n4[3] << 16);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (count[e] > 0.0f)
                                        o[j][e] = __uint_as_float(0x7fffffffu);
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k)
#pragma unroll
                                for (int w = 0; w < kW; ++w) {
                                    const uint32_t z = nan_bytes(v[k][w]);
                                    v[k][w] &= ~((z >> 7) * 0xffu);
                                }
                        }
                    }
#pragma unroll
                    for (int w = 0; w < kW; ++w)
#pragma unroll
                        for (int pair = 0; pair < 2; ++pair) {
                            // bytes 2 pair, 2 pair + 1 of two tokens each: {t0, t1} of both columns
                            const uint32_t sel = pair ? 0x7362u : 0x5140u;
                            const uint32_t x = __byte_perm(v[0][w], v[1][w], sel);
                            const uint32_t y = __byte_perm(v[2][w], v[3][w], sel);
                            mma_f16(o[4 * w + 2 * pair], a, e4m3x2_to_half2(x & 0xffffu),
                                    e4m3x2_to_half2(y & 0xffffu));
                            mma_f16(o[4 * w + 2 * pair + 1], a, e4m3x2_to_half2(x >> 16),
                                    e4m3x2_to_half2(y >> 16));
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

            // ---- join the four warps: each leaves (O, m, l), then eight threads take a row
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
                float *row = join + (warp * kRows + g + 8 * i) * G::kPitch;
                // columns 2c and 2c + 1 of the groups: D / 8 consecutive elements each
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < D / 8; j += 4)
                        *reinterpret_cast<float4 *>(row + piece_of<D>(2 * c + e) * (D / 8) + j) =
                            make_float4(o[j][2 * i + e], o[j + 1][2 * i + e], o[j + 2][2 * i + e],
                                        o[j + 3][2 * i + e]);
                if (c == 0) {
                    stat_m[warp * kRows + g + 8 * i] = m[i];
                    stat_l[warp * kRows + g + 8 * i] = l[i];
                }
            }
            if (lane == 0)
                stat_v[warp] = vref / kPShift;
            named_bar_sync(1, 32 * kWarps);
            {
                const int r = tid >> 3, d0 = (tid & 7) * (D / 8);
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    top = fmaxf(top, stat_m[w * kRows + r]);
                const float ref = top == -INFINITY ? 0.0f : top;
                float x[D / 8];
#pragma unroll
                for (int j = 0; j < D / 8; ++j)
                    x[j] = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = exp2_fast(stat_m[w * kRows + r] - ref);
                    const float fv = f * stat_v[w];
                    sum += f * stat_l[w * kRows + r];
                    const float4 *src = reinterpret_cast<const float4 *>(
                        join + (w * kRows + r) * G::kPitch + d0);
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) {
                        const float4 y = src[j];
                        x[4 * j] += fv * y.x;
                        x[4 * j + 1] += fv * y.y;
                        x[4 * j + 2] += fv * y.z;
                        x[4 * j + 3] += fv * y.w;
                    }
                }
                if (alive && seg0 >= start && seg1 <= stop) {
                    // the whole of it: the result
                    const int row = row0 + r;
                    if (row < p.rows) {
                        const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
                        uint16_t *dst = p.out + out_row(p, b, h, row) * D + d0;
#pragma unroll
                        for (int j = 0; j < D / 8; j += 8)
                            *reinterpret_cast<uint4 *>(dst + j) = make_uint4(
                                pack_out<kBf16>(x[j] * inv, x[j + 1] * inv),
                                pack_out<kBf16>(x[j + 2] * inv, x[j + 3] * inv),
                                pack_out<kBf16>(x[j + 4] * inv, x[j + 5] * inv),
                                pack_out<kBf16>(x[j + 6] * inv, x[j + 7] * inv));
                        if (kScores && d0 == 0)
                            p.lse[((int64_t)b * p.pool.kv_heads + h) * p.rows + row] =
                                sum == 0.0f ? INFINITY : ref + log2f(sum);
                    }
                } else if (alive) {
                    // a part: slot 0 where it starts this block's range, else slot 1
                    const int64_t at = ((int64_t)blockIdx.x * 2 + (seg0 > start ? 1 : 0)) * kRows + r;
                    float *dst = p.partial + at * D + d0;
#pragma unroll
                    for (int j = 0; j < D / 8; j += 4)
                        *reinterpret_cast<float4 *>(dst + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                    if (d0 == 0)
                        *reinterpret_cast<float2 *>(p.partial + (int64_t)p.grid * 2 * kRows * D + at * 2) =
                            make_float2(top, sum);
                }
            }
            named_bar_sync(1, 32 * kWarps);
        }
    }
}

// ---------------------------------------------------------------- joining the parts

constexpr int kJoinThreads = 128;

// One block per (sequence, head, row): joins the partials of the blocks that the row's
// (sequence, head, row tile) was cut between, in their order; 0 for a row of a sequence
// without tokens.
template <int D, bool kBf16, bool kScores>
__global__ void __launch_bounds__(kJoinThreads) kv_attention_join_kernel(const AttnParams p) {
    __shared__ float wide[kJoinThreads / 32][2];
    __shared__ float acc[kJoinThreads / 32][D];
    pdl_launch_dependents();
    pdl_wait_primary();
    int64_t i = blockIdx.x;
    const int row = (int)(i % p.rows);
    i /= p.rows;
    const int h = (int)(i % p.pool.kv_heads), b = (int)(i / p.pool.kv_heads);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t at = p.before[b], units = p.before[b + 1] - at;
    const int per_seq = p.pool.kv_heads * p.row_tiles;
    const int64_t total = p.before[p.batch] * per_seq;
    const int64_t seg0 = at * per_seq + (h * p.row_tiles + row / kRows) * units, seg1 = seg0 + units;
    uint16_t *dst = p.out + out_row(p, b, h, row) * D;
    float *lse = kScores ? p.lse + ((int64_t)b * p.pool.kv_heads + h) * p.rows + row : nullptr;
    if (units == 0) {
        for (int d = tid; d < D; d += kJoinThreads)
            dst[d] = 0;
        if (kScores && tid == 0)
            *lse = INFINITY;   // no token has a weight
        return;
    }
    const int c0 = range_owner(seg0, total, p.grid), c1 = range_owner(seg1 - 1, total, p.grid);
    if (c0 == c1)
        return;   // one block had all of it
    const float *stats = p.partial + (int64_t)p.grid * 2 * kRows * D;
    auto slot_of = [&](int c) -> int64_t {   // -1: a block without units
        const int64_t lo = range_start(c, total, p.grid), hi = range_start(c + 1, total, p.grid);
        return lo == hi ? -1 : ((int64_t)c * 2 + (seg0 > lo ? 1 : 0)) * kRows + row % kRows;
    };
    float top = -INFINITY;
    for (int c = c0 + tid; c <= c1; c += kJoinThreads) {
        const int64_t s = slot_of(c);
        if (s >= 0)
            top = fmaxf(top, stats[s * 2]);
    }
    for (int o = 16; o; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0)
        wide[warp][0] = top;
    __syncthreads();
    top = fmaxf(fmaxf(wide[0][0], wide[1][0]), fmaxf(wide[2][0], wide[3][0]));
    const float ref = top == -INFINITY ? 0.0f : top;
    // warp w takes the parts c0 + w, c0 + w + 4, ...; then the four sums in order
    float x[D / 32], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
        x[j] = 0.0f;
    for (int c = c0 + warp; c <= c1; c += kJoinThreads / 32) {
        const int64_t s = slot_of(c);
        if (s < 0)
            continue;
        const float f = exp2_fast(stats[s * 2] - ref);
        sum += f * stats[s * 2 + 1];
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
            x[j] += f * p.partial[s * D + 32 * j + lane];
    }
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
        acc[warp][32 * j + lane] = x[j];
    if (lane == 0)
        wide[warp][1] = sum;
    __syncthreads();
    sum = (wide[0][1] + wide[1][1]) + (wide[2][1] + wide[3][1]);
    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    for (int d = tid; d < D; d += kJoinThreads) {
        const float y = ((acc[0][d] + acc[1][d]) + (acc[2][d] + acc[3][d])) * inv;
        dst[d] = (uint16_t)(pack_out<kBf16>(y, 0.0f) & 0xffffu);
    }
    if (kScores && tid == 0)
        *lse = sum == 0.0f ? INFINITY : ref + log2f(sum);
}

// weights[t] += sum over the rows that see t of softmax_t, from the scores and each row's
// log-sum-exp; a thread per token.
constexpr int kWeightThreads = 256;

__global__ void __launch_bounds__(kWeightThreads) kv_attention_weights_kernel(const AttnParams p) {
    pdl_launch_dependents();
    pdl_wait_primary();
    const int64_t blocks = (p.width + kWeightThreads - 1) / kWeightThreads;
    const int64_t bh = blockIdx.x / blocks;
    const int b = (int)(bh / p.pool.kv_heads);
    const int64_t t = (blockIdx.x % blocks) * kWeightThreads + threadIdx.x;
    const int n = length_of(p, b);
    if (t >= n)
        return;
    const float *s = p.scores + (bh * p.width + t) * p.rows;
    const float *lse = p.lse + bh * p.rows;
    float sum = 0.0f;
    for (int r = 0; r < p.rows; ++r) {
        const int pos = n - p.tokens + r / p.group;
        if (sees((int)t, pos, p.window, p.sinks))
            sum += exp2_fast(s[r] - lse[r]);
    }
    p.weights[bh * p.width + t] += sum;
}

}  // namespace kvc
}  // namespace gemmrelu
