// kv_ragged.cuh -- attention of a batch of chunks over the paged 8-bit cache:
//
//   O[r] = sum_t softmax_t(q_r . k_t / sqrt(D)) v_t,  k_t = ks * K8[t], v_t = vs * V8[t]
//
// over the tokens t that row r sees, rows packed: sequence b has the query tokens starts[b] ..
// starts[b + 1] - 1, the last of its lengths[b] tokens.  The rows of one K/V head are its group's query
// heads of every new token, token by token; 128 of them are a tile, two neighbouring tiles an item.
//
// The work: items go over the 128-key blocks that some row of theirs sees, a CTA to an SM has a run of consecutive blocks of
// the whole call (ragged_plan, from starts and lengths on the device: no host knows them), and items that several CTAs have
// parts of are joined by the one that comes last, in the CTAs' order: no CTA waits for another, and the same call
// gives the same bits.
//
// A block: the feed's warp looks the pages up and copies K's and V's bytes (a bulk copy per page and head), a warpgroup turns
// them to fp16 in the products' layout, one warp issues S = Q K^T and O += P V (tcgen05, Q from shared memory, P from TMEM),
// and a warpgroup per tile makes P of S, a row a thread.  e4m3 is exact in fp16, and so is a power of two beside it: K's
// scales within a block go into the keys and V's into the values as long as they lie near each other (RaggedMeta), so
// that a row has one factor a block.
//
// Two references a row: m, the largest score, for the sum of weights, and rr, the largest score plus log2 of V's scale above
// it, for P and O.  A reference moves when it is exceeded by 2^8, so P = 2^(score + log2 vs - m - rr + 7) is at most 2^15 whatever
// the scales are: fp16 holds it, to half a step down to 2^-21 of the largest, and the fp32 sums of a block do not overflow.  Sums,
// references and O are fp32; P in fp16 is the only rounding besides the result's.
//
// V's bytes may be NaN where no row looks (0 * NaN is NaN): the conversion takes NaN out of blocks that are masked in part, and
// ragged_add_nan gives them back to the rows that see them.
//
// Bound, 2048 new tokens that end 32768, 32 heads on 8 of 128 (1.07 TFLOP, 555 us of products at the measured rate): 854 us,
// 1.25 PFLOP/s.  A block of two tiles takes about 4000 cycles for 2048 of products: S, softmax and P V of a tile
// follow each other, the other tile's fill the gaps, and a tile's softmax (2250 cycles: 128 reads from TMEM, 128 exponentials
// at 16 a cycle of an SM for both tiles, packing) is longer than the other's products; S reads both
// operands from shared memory, all 128 bytes a cycle, which the conversion's reads and writes interrupt.  Measured beside it, same
// case: no exponentials and no conversion 680 us.  Not kept: two threads a row 1004; S in steps of 64 keys, twice buffered
// 1095 (Q is read twice); P handed over in halves 1258 (the issuer goes in order); the rare paths unrolled or inlined 1016
// (instruction fetch: the loops of the four roles have to stay in the cache together); two converting warps 1018.
// 16 sequences of up to 8000 tokens, 1000 of them new: 809 us; 6 of 12000, 2000 new, 16 heads of 64 with a window of 1024: 117; 4 of
// 700 with up to 5 new: 18, most of it loads that wait for one another: counts, pages, keys, the other CTAs' parts.  Over fourteen
// sizes of this kind (fp16, 32 heads on 8 of 128) a call took 14 us, 2.09 us a block of a CTA and 14.7 us an item (pages of 32; 13,
// 2.00 and 14.9 at pages of 128), within 6% but for one (11%).
#pragma once

#include "flash_attention_window.cuh"
#include "kv_attention.cuh"

namespace gemmrelu {
namespace kvc {

using attn::BM;
using attn::BN;
using attn::kSub;

// Four warpgroups: two of softmax, one with the feed's and the issuer's warp, one that converts.  512 threads launch
// with 128 registers: 2 * 168 + 2 * 88 = 4 * 128.
constexpr int kRaggedThreads = 512;
constexpr int kConvWarp = 12, kConvWarps = 4;
constexpr int kRaggedSoftmaxRegs = 168, kRaggedFeedRegs = 88, kRaggedConvRegs = 88;
static_assert(2 * kRaggedSoftmaxRegs + kRaggedFeedRegs + kRaggedConvRegs <= 4 * 128, "registers given back cover those taken");
// Segments of a tile whose flags (NaN of V were taken out) are kept.  A tile's flags are numbered by the segments that it has
// rows in.  When those of its segment n are written, the P V two blocks before are done, with them one at least of
// its segment n - 2, whose P each of its warps brought after it had read the flags of segment n - 3: three would do, a
// power of two is quicker to index.
constexpr int kDirty = 4;
static_assert(kDirty >= 3, "flags stay until they have been read");
constexpr int kGroups = BN / 16;                // pieces of 16 tokens of a block: the smallest page
constexpr int kRaggedMaxCtas = GEMMRELU_RAGGED_COUNTER_BYTES / (8 * (int)sizeof(unsigned));
constexpr int kRaggedMaxBatch = 16384;          // sequences whose units fit the scratch of the start
static_assert(kPLog2 + attn::kRescaleLog2 <= 15.0f, "P stays below fp16's largest, 2^16 (1 - 2^-11), its exponent's rounding included");
constexpr float kBigLog2 = 2048.0f;             // 2^11: scores from here on are referred before V's scale is added

// What the feed says of a block.
//
// Where its scales are powers of two at most 2^14 apart (kNearScales) the conversion to fp16 brings all keys
// to the largest of K and the largest of V, exactly: e4m3's least value 2^-9 becomes 2^-23 at least.  Elsewhere
// the conversion leaves the values alone and every 16 keys have scales of their own.
enum RaggedFlags : uint32_t {
    kNearScales = 1,
    kInPart = 4,                        // some row of the item does not see some key
    kFirst = 8, kLast = 16,             // of its segment
    kBothTiles = 32,                    // the item has rows in its second tile
};

struct RaggedMeta {
    uint32_t flags;
    float ks, lv;                  // kNearScales: the block's scale of K, log2 of that of V
    uint32_t missing;              // a bit for every 16 keys that are not there
    int valid;                     // keys up to the sequence's end
    uint32_t pad[3];
    uint32_t mul[2][kGroups];      // kNearScales: the factors of K and V, twice fp16
    float2 scale[kGroups];         // (ks, log2 vs)
};

template <int HD>
struct RaggedCfg {
    static constexpr int kDSub = HD / 64;
    static constexpr int kRaw = HD == 128 ? 1 : 4;               // stages of e4m3 bytes
    // Blocks whose scales are kept.  Block i's are written when the bytes of block i - kRaw have been converted: then the
    // scores of block i - kRaw - 2 are done, and with them both tiles' softmax of block i - kRaw - 3.
    static constexpr int kMetas = HD == 128 ? 4 : 8;
    static_assert(kMetas >= kRaw + 3, "scales stay until they have been read");
    static constexpr uint32_t kTile16 = kDSub * kSub;            // a block of K or V in fp16; a tile of Q
    static constexpr uint32_t kTile8 = BN * HD;                  // in e4m3
    static constexpr uint32_t kOffQ = 0;
    static constexpr uint32_t kOffK = kOffQ + 2 * kTile16;
    static constexpr uint32_t kOffV = kOffK + 2 * kTile16;
    static constexpr uint32_t kOffRawK = kOffV + 2 * kTile16;
    static constexpr uint32_t kOffRawV = kOffRawK + kRaw * kTile8;
    static constexpr uint32_t kOffMeta = kOffRawV + kRaw * kTile8;
    static constexpr uint32_t kOffBar = kOffMeta + kMetas * (uint32_t)sizeof(RaggedMeta);
    // raw_k_full, raw_v_full, raw_k_empty, raw_v_empty [kRaw]; k_full, v_full, k_empty, v_empty [2];
    // meta_full[kMetas]; q_full, s_full, p_full, o_full [2]; drain
    static constexpr uint32_t kNumBars = 4 * kRaw + 8 + kMetas + 8 + 1;
    static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
    static constexpr uint32_t kOffDirty = kOffMisc + 16;         // [tiles][converting warps][kDirty]
    static constexpr uint32_t kOffPlan = (kOffDirty + 2 * kConvWarps * kDirty * 4 + 7) / 8 * 8;
    static constexpr uint32_t kOffSums = kOffPlan + 56;          // [2][warps], 64 bits each
    static constexpr uint32_t kSmem = kOffSums + 256 + 1024;
    static constexpr uint32_t kTmemS = 0, kTmemO = 2 * BN;
    static constexpr uint32_t kIdescS = make_idesc_f16_f32(BM, BN, 0, 0);
    static constexpr uint32_t kIdescO = make_idesc_f16_f32(BM, HD, 0, 1);
    static_assert(kSmem <= 232448, "shared memory of a block");
};

struct RaggedParams {
    Pool pool;
    const uint16_t *q;
    int64_t q_stride[2];               // token, head
    uint16_t *out;                     // [rows][q_heads][D]
    const int32_t *pages, *lengths, *starts;
    int64_t max_pages;
    int batch, rows, q_heads, group;
    attn::Divisor by_group;
    int window, sinks;
    float scale_log2;                  // log2(e) / sqrt(D)
    float4 *partial;                   // [2 * CTAs][8 warps][D / 4 of O, then (m, l, rr, unused)][32 rows]
    unsigned *arrived;                 // [CTAs][8 warps]; all 0 between calls
    int drop_arrive;
    uint64_t wait_limit_ns;
};

// ---------------------------------------------------------------- the work

// A sequence's part of the call: rows [start, start + count), tokens [0, n), items of one head.
struct RaggedSeq {
    int start, count, n, items;
};

// (what is out of range is taken as nothing, and reported where `report` is set)
__device__ __forceinline__ RaggedSeq ragged_seq(const RaggedParams &p, int b, bool report) {
    RaggedSeq s{0, 0, 0, 0};
    const int s0 = p.starts[b], s1 = p.starts[b + 1], n = p.lengths[b];
    bool ok = s0 >= 0 && s1 >= s0 && s1 <= p.rows;
    if (ok) {
        s.start = s0;
        s.count = s1 - s0;
    }
    if (n < 0 || n > p.max_pages * p.pool.page)
        ok = false;
    else
        s.n = n;
    if (!ok && report)
        record_page_error();
    s.items = (s.count * p.group + 2 * BM - 1) / (2 * BM);
    return s;
}

// Positions of an item's (or a tile's) first and last row, and the blocks that some row of it sees; an item
// whose rows see nothing has one block all the same, so that somebody writes its output.
struct RaggedItem {
    int first, last;
    attn::Blocks blocks;
    __device__ __forceinline__ int count() const { return max(1, blocks.count()); }
    __device__ __forceinline__ int key0(int j) const {
        return (j < blocks.sinks ? j : blocks.low + (j - blocks.sinks)) * BN;
    }
};

__device__ __forceinline__ RaggedItem ragged_item(const RaggedParams &p, const RaggedSeq &s, int item) {
    RaggedItem it;
    const int r0 = item * 2 * BM, r1 = min(r0 + 2 * BM, s.count * p.group) - 1;
    it.first = s.n - s.count + p.by_group.quotient(r0);
    it.last = s.n - s.count + p.by_group.quotient(r1);
    it.blocks = attn::blocks_seen(it.first, it.last, p.window, p.sinks);
    return it;
}

// Some row at positions first .. last does not see some key of the block.
__device__ __forceinline__ bool ragged_masked(const RaggedParams &p, int first, int last, int key0) {
    return key0 + BN - 1 > first || (p.window > 0 && key0 <= last - p.window && key0 + BN > p.sinks);
}

// Whether some row of the item sees some of `tokens` tokens from `token` on.
__device__ __forceinline__ bool ragged_sees(const RaggedParams &p, const RaggedItem &it, int token, int tokens) {
    return token <= it.last && (p.window == 0 || token < p.sinks ||
                                token + tokens > max(it.first, 0) - p.window + 1);
}

// How the work is cut.  The blocks of all items in order are dealt to the CTAs in equal ranges (part = 0): each finishes
// what lies inside its range, and what it has of the items at its two ends are parts that are joined.  With fewer items than
// CTAs every CTA would have two such ends and little between them: there each item is cut into equal parts of `part` blocks
// at most, and a CTA has one.  A unit is a block, or such a part.
__device__ __forceinline__ int ragged_units(int blocks, int part) { return part ? (blocks + part - 1) / part : blocks; }

// `part` for so many blocks and items: blocks / part + items parts at most, which fit.  0, ranges, with no fewer items
// than CTAs, and with so few blocks that a CTA has one or two of them in any case.
__device__ __forceinline__ int ragged_part(int blocks, int items, int grid) {
    return items < grid && blocks >= 4 * grid ? (blocks + grid - items - 1) / (grid - items) : 0;
}

// Whether to cut that way, given the blocks of the longest part: where it takes no more than an equal range and its two
// ends, about 8 blocks' time.
__device__ __forceinline__ bool ragged_cut_pays(int longest, int blocks, int grid) { return longest <= blocks / grid + 8; }

// The segments (runs of blocks of one item) of a CTA's range of units, in order.
struct RaggedWalk {
    int b, head, item, j, left;      // where it stands; blocks left of the range, this segment's too
    int unit0;                       // first unit of the item
    RaggedSeq seq;
    RaggedItem it;
    int j1, nb;                      // this segment is the blocks j .. j1 - 1 of nb
    __device__ __forceinline__ void describe(const RaggedParams &p) {
        it = ragged_item(p, seq, item);
        nb = it.count();
        j1 = min(nb, j + left);
    }
    __device__ __forceinline__ int rows(const RaggedParams &p) const { return seq.count * p.group - item * 2 * BM; }
    // The next segment; false at the end of the range.
    __device__ __forceinline__ bool next(const RaggedParams &p) {
        left -= j1 - j;
        if (left <= 0)
            return false;
        unit0 += nb;
        j = 0;
        if (++item == seq.items) {
            item = 0;
            if (++head == p.pool.kv_heads) {
                head = 0;
                do
                    seq = ragged_seq(p, ++b, false);
                while (seq.items == 0);
            }
        }
        describe(p);
        return true;
    }
};

// How many CTAs get a range: an item of n blocks is cut into about sqrt(2.5 n) parts at most.  (4 sequences of up to 700
// tokens with up to 5 new ones, 32 heads on 8, 5 blocks an item: 17.8 us so, 20.3 with a CTA a block, 25.7 with sqrt(n)
// parts.)
__device__ __forceinline__ int ragged_ranges(int total, int items, int grid) {
    const float most = sqrtf(2.5f * (float)total * (float)items);
    return max(1, min(min(total, grid), most < (float)grid ? (int)most : grid));
}

// What the start works out, in shared memory: where the CTA's range begins, its blocks, and how units are dealt.
struct RaggedPlan {
    int b, head, item, j, unit0, blocks, part, total, ranges;
    RaggedSeq seq;
};

// The sum over a warp of values in [0, 2^31).
__device__ __forceinline__ int64_t warp_sum(int x) {
    return ((int64_t)__reduce_add_sync(0xffffffffu, (unsigned)x >> 16) << 16) +
           __reduce_add_sync(0xffffffffu, (unsigned)x & 0xffffu);
}

// This CTA's range of units: sums over all sequences, a lane each (those of long chunks by a warp), by one warp or, with more
// than 32 sequences, by all; then one warp looks up where the range begins.  `units`: those of one head of each sequence.
__device__ __noinline__ void ragged_plan(const RaggedParams &p, RaggedPlan *plan, int *units, int64_t *sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grid = gridDim.x;
    const bool alone = p.batch <= 32;
    if (alone && warp > 0)
        return;
    int part = 0, total = 0, blocks = 0, all_items = 0;
    for (int pass = 0;; ++pass) {   // in blocks, in parts, and in blocks again where parts do not pay
        int64_t mine = 0, items = 0;
        int longest = 0;
        for (int b0 = warp * 32; b0 < p.batch; b0 += alone ? 32 : kRaggedThreads) {
            const int b = b0 + lane;
            RaggedSeq s{0, 0, 0, 0};
            if (b < p.batch)
                s = ragged_seq(p, b, pass == 0 && blockIdx.x == 0);
            int u = 0;   // (the host keeps a sequence's units below 2^31)
            auto add = [&](const RaggedSeq &x, int i) {
                const int n = ragged_item(p, x, i).count(), parts = ragged_units(n, part);
                if (part)
                    longest = max(longest, (n + parts - 1) / parts);
                return parts;
            };
            if (s.items <= 4)
                for (int i = 0; i < s.items; ++i)
                    u += add(s, i);
            for (uint32_t m = __ballot_sync(0xffffffffu, s.items > 4); m; m &= m - 1) {
                const int from = __ffs(m) - 1;
                RaggedSeq x;
                x.count = __shfl_sync(0xffffffffu, s.count, from);
                x.n = __shfl_sync(0xffffffffu, s.n, from);
                x.items = __shfl_sync(0xffffffffu, s.items, from);
                int sum = 0;
                for (int i = lane; i < x.items; i += 32)
                    sum += add(x, i);
                sum = (int)warp_sum(sum);
                u = lane == from ? sum : u;
            }
            if (b < p.batch)
                units[b] = u;
            mine += warp_sum(u);
            items += warp_sum(s.items);
        }
        longest = __reduce_max_sync(0xffffffffu, longest);
        if (!alone) {
            if (lane == 0) {
                sums[warp] = mine;
                sums[16 + warp] = items << 32 | longest;
            }
            __syncthreads();
            mine = items = 0;
            for (int w = 0; w < kRaggedThreads / 32; ++w) {
                mine += sums[w];
                items += sums[16 + w] >> 32;
                longest = max(longest, (int)sums[16 + w]);
            }
            __syncthreads();   // (the sums have been read)
        }
        mine *= p.pool.kv_heads;
        items *= p.pool.kv_heads;
        if (mine > 0x7fffffff) {   // rows that several sequences claim
            record_page_error();
            mine = 0;
        }
        total = (int)mine;
        if (pass == 0) {
            blocks = total;
            all_items = (int)(items < grid ? items : grid);   // (more make no difference)
            part = ragged_part(total, all_items, grid);
        } else if (pass == 1 && !ragged_cut_pays(longest, blocks, grid)) {
            part = 0;
            continue;
        }
        if (part == 0 || pass == 1)
            break;
    }
    if (warp > 0)
        return;
    __syncwarp();
    const int ranges = part ? max(total, 1) : ragged_ranges(total, all_items, grid), c = blockIdx.x;
    const int start = c < ranges ? range_start(c, total, ranges) : total;
    const int stop = c < ranges ? range_start(c + 1, total, ranges) : total;
    if (start >= stop) {
        if (lane == 0)
            *plan = RaggedPlan{0, 0, 0, 0, 0, 0, 0, 0, 1, RaggedSeq{0, 0, 0, 0}};
        return;
    }
    int at = 0, b = 0, u = 0;
    for (int b0 = 0;; b0 += 32) {   // the sequence that the range starts in
        const int x = b0 + lane < p.batch ? units[b0 + lane] * p.pool.kv_heads : 0;
        int run = x;
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, run, o);
            run += lane >= o ? y : 0;
        }
        const uint32_t m = __ballot_sync(0xffffffffu, start < at + run);
        if (m) {
            const int l = __ffs(m) - 1;
            b = b0 + l;
            u = __shfl_sync(0xffffffffu, x, l);
            at += __shfl_sync(0xffffffffu, run, l) - u;
            break;
        }
        at += __shfl_sync(0xffffffffu, run, 31);
    }
    u /= p.pool.kv_heads;
    const int head = (start - at) / u;
    at += head * u;
    const RaggedSeq s = ragged_seq(p, b, false);
    int item = 0, nb = 0;
    for (int i0 = 0;; i0 += 32) {   // the item of that head
        const int n = i0 + lane < s.items ? ragged_item(p, s, i0 + lane).count() : 0;
        const int x = ragged_units(n, part);
        int run = x;
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, run, o);
            run += lane >= o ? y : 0;
        }
        const uint32_t m = __ballot_sync(0xffffffffu, start < at + run);
        if (m) {
            const int l = __ffs(m) - 1;
            item = i0 + l;
            nb = __shfl_sync(0xffffffffu, n, l);
            at += __shfl_sync(0xffffffffu, run - x, l);
            break;
        }
        at += __shfl_sync(0xffffffffu, run, 31);
    }
    int j = start - at, here = stop - start;
    if (part) {   // part j of the item
        const int x = ragged_units(nb, part), j0 = range_start(j, nb, x);
        here = range_start(j + 1, nb, x) - j0;
        j = j0;
    }
    if (lane == 0)
        *plan = RaggedPlan{b, head, item, j, at, here, part, total, ranges, s};
}

// ---------------------------------------------------------------- V that is not finite

// The NaN of V in blocks that some row sees in part were taken out (0 in their place); the rows that see one get
// it back here, in the warp's 32 rows of O in TMEM: blocks j0 .. j1 - 1 of an item, `pos` the lane's row's position.
template <int HD>
__device__ __noinline__ void ragged_add_nan(const RaggedParams &p, int b, int head, int item, int j0, int j1, int pos,
                                            uint32_t o_addr) {
    const int lane = threadIdx.x & 31, page = p.pool.page;
    const RaggedSeq seq = ragged_seq(p, b, false);
    const RaggedItem it = ragged_item(p, seq, item);
#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
#pragma unroll 1
        for (int k0 = it.key0(j); k0 < it.key0(j) + BN; k0 += 32) {
            const int key = k0 + lane;
            const uint8_t *row = nullptr;
            if (key < seq.n && ragged_sees(p, it, key & ~(page - 1), page)) {
                const int64_t id = p.pages[b * p.max_pages + (key >> p.pool.page_shift)];
                if (id >= 0 && id < p.pool.num_pages)
                    row = p.pool.values[1] + ((id * p.pool.kv_heads + head) * page + (key & (page - 1))) * HD;
            }
            uint32_t bad = 0;
            if (row != nullptr)
#pragma unroll 1
                for (int c = 0; c < HD; c += 16) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(row + c);
                    bad |= nan_bytes(x.x) | nan_bytes(x.y) | nan_bytes(x.z) | nan_bytes(x.w);
                }
            const uint32_t low = (uint32_t)reinterpret_cast<uintptr_t>(row);
            const uint32_t high = (uint32_t)(reinterpret_cast<uintptr_t>(row) >> 32);
#pragma unroll 1
            for (uint32_t keys = __ballot_sync(0xffffffffu, bad != 0); keys; keys &= keys - 1) {
                const int i = __ffs(keys) - 1;
                const uintptr_t at = (uintptr_t)__shfl_sync(0xffffffffu, low, i) |
                                     (uintptr_t)__shfl_sync(0xffffffffu, high, i) << 32;
                const bool mine = sees(k0 + i, pos, p.window, p.sinks);
#pragma unroll 1
                for (int c0 = 0; c0 < HD; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld_x32_sync(o_addr + c0, o);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const uint32_t x = nan_bytes(reinterpret_cast<const uint32_t *>(at + c0)[c]);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[4 * c + e] = mine && x & (0x80u << 8 * e) ? 0x7fffffffu : o[4 * c + e];
                    }
                    tmem_st_x32(o_addr + c0, o);
                    tmem_st_wait();
                }
            }
        }
    }
}

// ---------------------------------------------------------------- weights, the rare cases

// What scores of keys with scale ks are multiplied by: neither 0, which would make a NaN of a score of -infinity, nor an
// infinity, which would make one of a score of 0.
__device__ __forceinline__ float score_factor(float c_row, float ks) {
    return fminf(fmaxf(c_row * ks, 1.17549435e-38f), 3.40282347e+38f);
}

// What brings a sum of P (weights times V's scale, relative to O's reference) back to weights relative to m; bounded, so
// that no sum of 0 meets an infinity.
__device__ __forceinline__ float back_of(float rr, float lv) { return attn::fast_exp2(fminf(rr - kPLog2 - lv, 126.0f)); }

// A block whose scales are far apart: its largest score (x), and the largest score plus log2 of V's scale (y) relative to
// m_ref.
__device__ __forceinline__ float2 ragged_top(uint32_t s_addr, const RaggedMeta &meta, float c_row, float m_ref) {
    float mx = -INFINITY, over = -INFINITY;
#pragma unroll 1
    for (int g = 0; g < kGroups; ++g) {
        uint32_t v[16];
        tmem_ld_x16(s_addr + 16 * g, v);
        tmem_ld_wait_regs16(v);
        float a = -INFINITY;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            a = fmaxf(a, __uint_as_float(v[e]));
        const float2 sc = meta.scale[g];
        const float x = __fmul_rn(a, score_factor(c_row, sc.x));
        mx = fmaxf(mx, x);
        over = fmaxf(over, (x - m_ref) + sc.y);
    }
    return make_float2(mx, over);
}

// P and its sum for a block whose scales are far apart, or for scores of 2^11 and more: there the product and the
// reference are rounded before they are subtracted, and V's scale comes last.
__device__ __forceinline__ float ragged_weights(uint32_t s_addr, const RaggedMeta &meta, float c_row, float m_ref, float rr) {
    const bool near = meta.flags & kNearScales;
    float sum = 0.0f;
#pragma unroll 1
    for (int g = 0; g < kGroups; ++g) {
        const float2 sc = near ? make_float2(meta.ks, meta.lv) : meta.scale[g];
        const float c = score_factor(c_row, sc.x), a = sc.y + kPLog2 - rr;
        uint32_t v[16], ph[8];
        tmem_ld_x16(s_addr + 16 * g, v);
        tmem_ld_wait_regs16(v);
        float part = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const float x = attn::fast_exp2(__fsub_rn(__fmul_rn(__uint_as_float(v[e]), c), m_ref) + a);
            const float y = attn::fast_exp2(__fsub_rn(__fmul_rn(__uint_as_float(v[e + 1]), c), m_ref) + a);
            part += x + y;
            ph[e / 2] = half2_of(x, y);
        }
        tmem_st_x8(s_addr + 8 * g, ph);   // (over scores that have been read)
        sum = fmaf(part, back_of(rr, sc.y), sum);
    }
    return sum;
}

// 32 elements of a row of the result: inv f^2 times its sums (f's square spans the range of all scales).
template <bool kBf16>
__device__ __forceinline__ void write_row32(uint16_t *dst, const float (&y)[32], float inv, float f) {
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            h[k] = pack_out<kBf16>(y[e + 2 * k] * inv * f * f, y[e + 2 * k + 1] * inv * f * f);
        *reinterpret_cast<uint4 *>(dst + e) = make_uint4(h[0], h[1], h[2], h[3]);
    }
}

// A (sequence, head, item) that several CTAs have parts of, for one lane's row.
struct RaggedCut {
    uint16_t *dst;         // where the row goes; nullptr: there is no such row
    int first, last;       // CTAs
    bool mid;              // it begins behind the start of the first one's range: in that one's second part
};

// What CTA c has of a cut item in the workspace, for one warp's 32 rows: HD / 4 times 4 columns of O, then m, l and rr, a
// lane's row each.
template <int HD>
__device__ __forceinline__ float4 *ragged_part_of(const RaggedParams &p, const RaggedCut &cut, int warp, int lane, int c) {
    return p.partial + ((int64_t)(2 * c + (c == cut.first && cut.mid ? 1 : 0)) * 8 + warp) * (HD / 4 + 1) * 32 + lane;
}

// The parts of a lane's row joined, in the order of the CTAs.
template <int HD, bool kBf16>
__device__ __forceinline__ void ragged_join(const RaggedParams &p, const RaggedCut cut, int warp, int lane) {
    // the largest references, and the sum of weights
    float mm = -INFINITY, yy = -INFINITY, ll = 0.0f;
#pragma unroll 4
    for (int c = cut.first; c <= cut.last; ++c) {
        const float4 x = __ldcg(ragged_part_of<HD>(p, cut, warp, lane, c) + HD / 4 * 32);   // m, l, rr
        const float top = fmaxf(mm, x.x);
        ll *= mm == top ? 1.0f : exp2f(mm - top);
        yy = mm == -INFINITY ? -INFINITY : (mm - top) + yy;
        yy = fmaxf(yy, x.x == -INFINITY ? -INFINITY : (x.x - top) + x.z);
        ll += x.y != x.y ? x.y : x.x == -INFINITY ? 0.0f : x.y * exp2f(x.x - top);
        mm = top;
    }
    const float ref = mm == -INFINITY ? 0.0f : mm;
    const float inv = ll > 0.0f || ll != ll ? 1.0f / ll : 0.0f;
    const float f = yy == -INFINITY ? 0.0f : exp2f(0.5f * (yy - kPLog2));
#pragma unroll 1
    for (int c0 = 0; c0 < HD; c0 += 64) {
        float s[64];
#pragma unroll
        for (int e = 0; e < 64; ++e)
            s[e] = 0.0f;
#pragma unroll 1
        for (int c = cut.first; c <= cut.last; c += 2) {   // two parts' loads are under way at once
            const bool both = c < cut.last;
            const float4 *x = ragged_part_of<HD>(p, cut, warp, lane, c), *y = ragged_part_of<HD>(p, cut, warp, lane, both ? c + 1 : c);
            float4 o[2][16];
            const float4 xs = __ldcg(x + HD / 4 * 32), ys = __ldcg(y + HD / 4 * 32);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                o[0][e] = __ldcg(x + (c0 / 4 + e) * 32);
                o[1][e] = __ldcg(y + (c0 / 4 + e) * 32);
            }
            const float a = xs.x == -INFINITY ? 1.0f : exp2f((xs.x - ref) + xs.z - yy);
            const float d = ys.x == -INFINITY ? 1.0f : exp2f((ys.x - ref) + ys.z - yy);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                s[4 * e] = fmaf(o[0][e].x, a, s[4 * e]);
                s[4 * e + 1] = fmaf(o[0][e].y, a, s[4 * e + 1]);
                s[4 * e + 2] = fmaf(o[0][e].z, a, s[4 * e + 2]);
                s[4 * e + 3] = fmaf(o[0][e].w, a, s[4 * e + 3]);
            }
            if (both)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    s[4 * e] = fmaf(o[1][e].x, d, s[4 * e]);
                    s[4 * e + 1] = fmaf(o[1][e].y, d, s[4 * e + 1]);
                    s[4 * e + 2] = fmaf(o[1][e].z, d, s[4 * e + 2]);
                    s[4 * e + 3] = fmaf(o[1][e].w, d, s[4 * e + 3]);
                }
        }
#pragma unroll
        for (int e = 0; e < 64; e += 32)
            write_row32<kBf16>(cut.dst + c0 + e, reinterpret_cast<const float(&)[32]>(s[e]), inv, f);
    }
}

// The same for a warp with no more than 8 rows: four lanes a row, HD / 4 columns each (every fourth of the float4), so that
// the parts' loads are few and many parts' are under way at once.  `row_dst` is the row's.  (One token after 1000, 32 heads on
// 8: 17.0 us so, 21.0 with a lane a row; after 30000: 45.7 and 55.2.)
template <int HD, bool kBf16>
__device__ __noinline__ void ragged_join_few(const RaggedParams &p, const RaggedCut cut, uint16_t *row_dst, int warp, int lane) {
    const int row = lane & 7, nth = lane >> 3;
    float mm = -INFINITY, yy = -INFINITY, ll = 0.0f;
    float4 s[HD / 16];
#pragma unroll
    for (int e = 0; e < HD / 16; ++e)
        s[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
    for (int c = cut.first; c <= cut.last; ++c) {
        const float4 *at = ragged_part_of<HD>(p, cut, warp, row, c);
        const float4 x = __ldcg(at + HD / 4 * 32);   // m, l, rr
        float4 o[HD / 16];
#pragma unroll
        for (int e = 0; e < HD / 16; ++e)
            o[e] = __ldcg(at + (4 * e + nth) * 32);
        const float top = fmaxf(mm, x.x), ref = top == -INFINITY ? 0.0f : top;
        const float shrink = mm == top ? 1.0f : exp2f(mm - top);
        ll = ll * shrink + (x.y != x.y ? x.y : x.x == -INFINITY ? 0.0f : x.y * exp2f(x.x - ref));
        const float mine = x.x == -INFINITY ? -INFINITY : (x.x - ref) + x.z;
        const float old = mm == -INFINITY ? -INFINITY : (mm - top) + yy;
        const float now = fmaxf(old, mine), base = now == -INFINITY ? 0.0f : now;
        const float a = x.x == -INFINITY ? 1.0f : exp2f(mine - base), d = old == -INFINITY ? 1.0f : exp2f(old - base);
#pragma unroll
        for (int e = 0; e < HD / 16; ++e)
            s[e] = make_float4(fmaf(o[e].x, a, s[e].x * d), fmaf(o[e].y, a, s[e].y * d), fmaf(o[e].z, a, s[e].z * d),
                               fmaf(o[e].w, a, s[e].w * d));
        mm = top;
        yy = now;
    }
    const float inv = ll > 0.0f || ll != ll ? 1.0f / ll : 0.0f;
    const float f = yy == -INFINITY ? 0.0f : exp2f(0.5f * (yy - kPLog2));
    if (row_dst != nullptr)
#pragma unroll
        for (int e = 0; e < HD / 16; ++e)
            *reinterpret_cast<uint2 *>(row_dst + 4 * (4 * e + nth)) =
                make_uint2(pack_out<kBf16>(s[e].x * inv * f * f, s[e].y * inv * f * f),
                           pack_out<kBf16>(s[e].z * inv * f * f, s[e].w * inv * f * f));
}

// ---------------------------------------------------------------- e4m3 to fp16

// Rows [row0, row0 + BN / kConvWarps) of a block: bytes at `src` (rows of HD) become fp16 in the sub-tiles of 64
// columns at `dst`, 128-byte swizzled, the layout of both products' B operands.  Four lanes take 64 bytes
// of an even row and four the other half of the next one, so that eight lanes that load or store
// together touch all banks once.  Row r is multiplied by mul[r / 16].  kCheck: rows past the sequence's end or of pages
// that are not there become 0 and so do NaN; true if the lane met one.
template <int HD, bool kCheck>
__device__ __forceinline__ bool convert_rows(uint32_t src, uint32_t dst, int row0, const uint32_t *mul, int valid,
                                             uint32_t missing) {
    const int lane = threadIdx.x & 31;
    const int odd = (lane >> 2) & 1, c4 = lane & 3, row1 = row0 + 2 * (lane >> 3) + odd;
    constexpr int kHalves = HD / 64;
    uint32_t bad = 0;
    src += row1 * HD + c4 * 16;
    dst += row1 * 128 + ((uint32_t)((2 * c4) ^ (row1 & 7)) << 4);   // (row & 7 does not change below)
#pragma unroll 1
    for (int i = 0; i < BN / kConvWarps / 8; ++i) {
        const int row = row1 + 8 * i;
        const uint32_t m = mul[row >> 4];
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            const int half = kHalves == 1 ? 0 : (odd ^ h);
            const uint4 x = ld_shared_v4(src + 8 * i * HD + half * 64);
            uint32_t w[4] = {x.x, x.y, x.z, x.w};
            if constexpr (kCheck) {
                const bool there = row < valid && !(missing >> (row >> 4) & 1u);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = there ? w[e] : 0u;
                    const uint32_t n = nan_bytes(w[e]);
                    bad |= n;
                    w[e] &= ~((n >> 7) * 0xffu);
                }
            }
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[2 * e] = e4m3x2_to_half2(w[e] & 0xffffu);
                y[2 * e + 1] = e4m3x2_to_half2(w[e] >> 16);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(y[e]) : "r"(m));
            const uint32_t at = dst + 1024 * i + half * kSub;
            st_shared_v4(at, y[0], y[1], y[2], y[3]);
            st_shared_v4(at ^ 16u, y[4], y[5], y[6], y[7]);
        }
    }
    return bad != 0;
}

// ---------------------------------------------------------------- the kernel

template <int HD, bool kBf16>
__global__ void __launch_bounds__(kRaggedThreads, 1)
    kv_attention_ragged_kernel(const __grid_constant__ RaggedParams p) {
    using G = RaggedCfg<HD>;
    using namespace attn;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);

    const uint32_t bar0 = base + G::kOffBar;
    auto raw_full = [&](int kv, uint32_t s) { return bar0 + 8u * (kv * G::kRaw + s); };
    auto raw_empty = [&](int kv, uint32_t s) { return bar0 + 8u * ((2 + kv) * G::kRaw + s); };
    constexpr uint32_t kB1 = 4 * G::kRaw;
    auto full = [&](int kv, uint32_t s) { return bar0 + 8u * (kB1 + 2 * kv + s); };
    auto empty = [&](int kv, uint32_t s) { return bar0 + 8u * (kB1 + 4 + 2 * kv + s); };
    auto meta_full = [&](uint32_t s) { return bar0 + 8u * (kB1 + 8 + s); };
    constexpr uint32_t kB2 = kB1 + 8 + G::kMetas;
    auto q_full = [&](uint32_t t) { return bar0 + 8u * (kB2 + t); };
    auto s_full = [&](uint32_t t) { return bar0 + 8u * (kB2 + 2 + t); };
    auto p_full = [&](uint32_t t) { return bar0 + 8u * (kB2 + 4 + t); };
    auto o_full = [&](uint32_t t) { return bar0 + 8u * (kB2 + 6 + t); };
    const uint32_t drain_bar = bar0 + 8u * (kB2 + 8);
    RaggedMeta *metas = reinterpret_cast<RaggedMeta *>(gbase + G::kOffMeta);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + G::kOffMisc);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + G::kOffMisc + 4);
    volatile uint32_t *dirty = reinterpret_cast<volatile uint32_t *>(gbase + G::kOffDirty);
    RaggedPlan *plan = reinterpret_cast<RaggedPlan *>(gbase + G::kOffPlan);
    static_assert(sizeof(RaggedPlan) <= 56 && G::kOffPlan % 8 == 0, "the plan and the sums behind it");
    int64_t *sums = reinterpret_cast<int64_t *>(gbase + G::kOffSums);

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);   // uniform
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < (uint32_t)G::kRaw; ++s)
            for (int kv = 0; kv < 2; ++kv) {
                mbar_init(raw_full(kv, s), 1u);
                mbar_init(raw_empty(kv, s), kConvWarps);
            }
        for (uint32_t s = 0; s < 2; ++s) {
            for (int kv = 0; kv < 2; ++kv) {
                mbar_init(full(kv, s), kConvWarps);
                mbar_init(empty(kv, s), 1u);
            }
            mbar_init(q_full(s), 4u);
            mbar_init(s_full(s), 1u);
            mbar_init(p_full(s), 4u);
            mbar_init(o_full(s), 1u);
        }
        for (uint32_t s = 0; s < (uint32_t)G::kMetas; ++s)
            mbar_init(meta_full(s), 1u);
        mbar_init(drain_bar, 1u);
        *abort_flag = 0u;
        fence_mbar_init();
        pdl_launch_dependents();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
    }
    // Warm L2 with what the start depends on, one load after the other (L2 is where all writes meet, so fetching early
    // returns nothing stale)
    {
        const int64_t i = ((int64_t)blockIdx.x * kRaggedThreads + threadIdx.x) * 32;
        if (i < p.batch * p.max_pages)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.pages + i));
        if (i < p.batch) {
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.lengths + i));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.starts + i));
        }
    }
    pdl_wait_primary();
    ragged_plan(p, plan, reinterpret_cast<int *>(gbase + G::kOffK), sums);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
    const int blocks_here = plan->blocks;
    auto first_segment = [&]() {
        RaggedWalk w;
        w.b = plan->b;
        w.head = plan->head;
        w.item = plan->item;
        w.j = plan->j;
        w.left = blocks_here;
        w.unit0 = plan->unit0;
        w.seq = plan->seq;
        w.describe(p);
        return w;
    };

    if (warp >= kProducerWarp) {
        if (warp >= kConvWarp)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRaggedConvRegs));
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRaggedFeedRegs));
        if (blocks_here > 0 && warp == kProducerWarp) {
            // ======================================================== the feed
            // A block is `pieces` pages, a copy each of K and of V; lane l describes page l % pieces of block
            // l / pieces of a batch of 32 / pieces blocks.
            const int piece = p.pool.page, pieces = BN / piece, per_batch = 32 / pieces;
            uint32_t blocks = 0, segment = 0;
            bool ok = !(p.drop_arrive && blockIdx.x == 0);
            RaggedWalk w = first_segment();
            do {
                // The item's rows into L2, the softmax warps load them some blocks later (816 -> 808 us, and 120.3 -> 118.9 under the
                // window; a segment's change costs 7000 to 9000 cycles, 3200 of them for its rows).
                if (segment > 0) {
                    const int rows = min(w.rows(p), 2 * BM);
#pragma unroll 1
                    for (int r = lane; r < rows; r += 32) {
                        const int token = p.by_group.quotient(w.item * 2 * BM + r), g = w.item * 2 * BM + r - token * p.group;
                        const uint16_t *at = p.q + (w.seq.start + token) * p.q_stride[0] + (w.head * p.group + g) * p.q_stride[1];
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
                        if (HD == 128)
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(at + 64));
                    }
                }
                for (int j0 = w.j; ok && j0 < w.j1; j0 += per_batch) {
                    const int j = j0 + lane / pieces;
                    int64_t id = -1;
                    float ks = 0.0f, vs = 0.0f, ks_top, lv, lv_top;
                    uint32_t k_mul, v_mul;
                    bool all_fit = false;
                    if (j < w.j1) {
                        const int token = w.it.key0(j) + (lane % pieces) * piece;
                        if (token < w.seq.n && ragged_sees(p, w.it, token, piece)) {
                            id = p.pages[w.b * p.max_pages + (token >> p.pool.page_shift)];
                            if (id < 0 || id >= p.pool.num_pages) {
                                record_page_error();
                                id = -1;
                            } else {
                                ks = p.pool.scales[0][id * p.pool.kv_heads + w.head];
                                vs = p.pool.scales[1][id * p.pool.kv_heads + w.head];
                            }
                        }
                    }
                    const uint32_t there = __ballot_sync(0xffffffffu, id >= 0), block = (1u << pieces) - 1;
                    const int64_t at = (id * p.pool.kv_heads + w.head) * p.pool.page * HD;
                    for (int i = 0; i < per_batch && j0 + i < w.j1; ++i, ++blocks) {
                        const uint32_t s = blocks % G::kRaw, ph = blocks / G::kRaw & 1u;
                        const bool in = lane / pieces == i;
                        const uint32_t mine = there >> (i * pieces) & block;
                        const uint32_t bytes = __popc(mine) * piece * HD;
                        const uint32_t off = s * G::kTile8 + (lane % pieces) * piece * HD;
                        if (!wait_warp(raw_empty(0, s), ph ^ 1u, p.wait_limit_ns, abort_flag, kSiteProducerEmpty)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0)
                            mbar_arrive_expect_tx(raw_full(0, s), bytes);
                        __syncwarp();
                        if (in && id >= 0)
                            bulk_load(base + G::kOffRawK + off, p.pool.values[0] + at, piece * HD, raw_full(0, s));
                        if (i == 0) {
                            // the blocks' largest scales, and how far the pages' are below (read while the first copies are under way)
                            ks_top = ks;
                            float vs_top = vs;
                            for (int o = 1; o < pieces; o <<= 1) {
                                ks_top = fmaxf(ks_top, __shfl_xor_sync(0xffffffffu, ks_top, o));
                                vs_top = fmaxf(vs_top, __shfl_xor_sync(0xffffffffu, vs_top, o));
                            }
                            if (id < 0) {
                                ks = ks_top > 0.0f ? ks_top : 1.0f;
                                vs = vs_top > 0.0f ? vs_top : 1.0f;
                            }
                            ks_top = fmaxf(ks_top, ks);
                            vs_top = fmaxf(vs_top, vs);
                            const uint32_t k_bits = __float_as_uint(ks), v_bits = __float_as_uint(vs);
                            const int k_below = (int)(__float_as_uint(ks_top) - k_bits) >> 23;
                            const int v_below = (int)(__float_as_uint(vs_top) - v_bits) >> 23;
                            const bool fits = ks > 0.0f && vs > 0.0f && ((k_bits | v_bits) & 0x7fffffu) == 0 &&
                                              k_below <= 14 && v_below <= 14;
                            const uint32_t near = __ballot_sync(0xffffffffu, fits);
                            all_fit = (near >> (lane & ~(pieces - 1)) & block) == block;
                            k_mul = (uint32_t)(all_fit ? 15 - k_below : 15) << 10;   // 2^-k_below, or 1
                            v_mul = (uint32_t)(all_fit ? 15 - v_below : 15) << 10;
                            lv = log2f(fmaxf(vs, kMinScale));
                            lv_top = log2f(fmaxf(vs_top, kMinScale));
                        }
                        RaggedMeta &m = metas[blocks % G::kMetas];
                        if (in) {
                            for (int x = 0; x < piece / 16; ++x) {
                                const int g = (lane % pieces) * (piece / 16) + x;
                                m.scale[g] = make_float2(ks, lv);
                                m.mul[0][g] = k_mul * 0x10001u;
                                m.mul[1][g] = v_mul * 0x10001u;
                            }
                            if (lane % pieces == 0) {
                                const int at = j0 + i, key0 = w.it.key0(at);
                                uint32_t gone = 0;
                                for (int g = 0; g < kGroups; ++g)
                                    gone |= (mine >> (g * 16 / piece) & 1u) ? 0u : 1u << g;
                                const bool part = gone || ragged_masked(p, w.it.first, w.it.last, key0);
                                m.flags = (all_fit ? kNearScales : 0) | (part ? kInPart : 0) | (at == w.j ? kFirst : 0) |
                                          (at + 1 == w.j1 ? kLast : 0) | (w.rows(p) > BM ? kBothTiles : 0);
                                m.ks = ks_top;
                                m.lv = lv_top;
                                m.missing = gone;
                                m.valid = w.seq.n - key0;
                            }
                        }
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(meta_full(blocks % G::kMetas));
                        if (!wait_warp(raw_empty(1, s), ph ^ 1u, p.wait_limit_ns, abort_flag, kSiteProducerEmpty)) {
                            ok = false;
                            ++blocks;   // its K is on its way
                            break;
                        }
                        if (lane == 0)
                            mbar_arrive_expect_tx(raw_full(1, s), bytes);
                        __syncwarp();
                        if (in && id >= 0)
                            bulk_load(base + G::kOffRawV + off, p.pool.values[1] + at, piece * HD, raw_full(1, s));
                    }
                }
                ++segment;
            } while (ok && w.next(p));
            // Every copy issued has landed before the block may exit.  (After a wait that expired the last
            // block's V was not asked for; waiting for it only runs into the limit again.)
            for (uint32_t i = blocks > (uint32_t)G::kRaw ? blocks - G::kRaw : 0u; i < blocks; ++i) {
                wait_drain(raw_full(0, i % G::kRaw), i / G::kRaw & 1u, p.wait_limit_ns, abort_flag);
                if (ok || i + 1 < blocks)
                    wait_drain(raw_full(1, i % G::kRaw), i / G::kRaw & 1u, p.wait_limit_ns, abort_flag);
            }
        } else if (blocks_here > 0 && warp >= kConvWarp) {
            // ======================================================== e4m3 to fp16
            const int mine = warp - kConvWarp, row0 = BN / kConvWarps * mine;
            bool ok = true, bad = false;
            uint32_t segments0 = 0, segments1 = 0;   // of the tiles
            for (uint32_t i = 0; ok && i < (uint32_t)blocks_here; ++i) {
                const uint32_t rs = i % G::kRaw, rp = i / G::kRaw & 1u, st = i & 1u, ph = i >> 1 & 1u;
                ok = wait_warp(meta_full(i % G::kMetas), i / G::kMetas & 1u, p.wait_limit_ns, abort_flag,
                               kSiteMmaFull);
                if (!ok)
                    break;
                const RaggedMeta &meta = metas[i % G::kMetas];
                const uint32_t flags = meta.flags;
#pragma unroll 1
                for (int kv = 0; ok && kv < 2; ++kv) {
                    ok = wait_warp(raw_full(kv, rs), rp, p.wait_limit_ns, abort_flag, kSiteMmaFull) &&
                         wait_warp(empty(kv, st), ph ^ 1u, p.wait_limit_ns, abort_flag, kSiteProducerEmpty);
                    if (!ok)
                        break;
                    const uint32_t src = base + (kv ? G::kOffRawV : G::kOffRawK) + rs * G::kTile8;
                    const uint32_t dst = base + (kv ? G::kOffV : G::kOffK) + st * G::kTile16;
                    if (kv && flags & kInPart) {
                        bad = convert_rows<HD, true>(src, dst, row0, meta.mul[1], meta.valid, meta.missing) ||
                              (bad && !(flags & kFirst));
                    } else {
                        bad = bad && !(kv && flags & kFirst);
                        convert_rows<HD, false>(src, dst, row0, meta.mul[kv], BN, 0u);
                    }
                    if (kv && flags & kLast) {
                        const bool any = __any_sync(0xffffffffu, bad), both = flags & kBothTiles;
                        if (lane == 0) {
                            dirty[kDirty * mine + segments0 % kDirty] = any ? 1u : 0u;
                            if (both)
                                dirty[kDirty * (kConvWarps + mine) + segments1 % kDirty] = any ? 1u : 0u;
                        }
                        ++segments0;
                        segments1 += both;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(raw_empty(kv, rs));
                        mbar_arrive(full(kv, st));
                    }
                }
            }
        } else if (blocks_here > 0 && warp == kMmaWarp) {
            // ======================================================== products
            // (one elected thread issues, the whole warp walks along)
            const bool leader = elect_one();
            const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
            const uint64_t q_desc = make_sdesc_sw128(base + G::kOffQ, 16, 1024);
            const uint64_t k_desc = make_sdesc_sw128(base + G::kOffK, 16, 1024);
            const uint64_t v_desc = make_sdesc_sw128(base + G::kOffV, kSub, 1024);
            uint32_t turns0 = 0, turns1 = 0, segs0 = 0, segs1 = 0;
            // S_t = Q_t K^T of block number i
            auto score = [&](const uint32_t t, uint32_t i) {
                const uint64_t qd = q_desc + t * (G::kTile16 >> 4), kd = k_desc + (i & 1u) * (G::kTile16 >> 4);
#pragma unroll
                for (int kk = 0; kk < HD / UKA; ++kk) {
                    const uint32_t o = (kk / 4) * (kSub >> 4) + (kk % 4) * 2;
                    if (leader)
                        umma_f16(tmem + G::kTmemS + t * BN, qd + o, kd + o, G::kIdescS, kk > 0 ? 1u : 0u);
                }
                if (leader)
                    umma_commit(s_full(t));
            };
            auto wait_q = [&](const uint32_t t, uint32_t &segs) {
                const bool ok = wait_warp(q_full(t), segs++ & 1u, p.wait_limit_ns, abort_flag, kSiteMmaFull);
                tc_fence_after_sync();
                return ok;
            };
            auto wait_k = [&](uint32_t i) {
                const bool ok = wait_warp(full(0, i & 1u), i >> 1 & 1u, p.wait_limit_ns, abort_flag, kSiteMmaFull);
                tc_fence_after_sync();
                return ok;
            };
            // O_t (+)= P_t V of block number i, P_t from TMEM (over S_t)
            auto pv = [&](const uint32_t t, uint32_t i, bool fresh, bool complete, uint32_t &turns) {
                if (!wait_warp(p_full(t), turns++ & 1u, p.wait_limit_ns, abort_flag, kSiteMmaAccEmpty))
                    return false;
                tc_fence_after_sync();
                const uint64_t vd = v_desc + (i & 1u) * (G::kTile16 >> 4);
                const uint32_t d_o = tmem + G::kTmemO + t * HD, a_p = tmem + G::kTmemS + t * BN;
#pragma unroll
                for (int kk = 0; kk < BN / UKA; ++kk)
                    if (leader)
                        umma_f16_ts(d_o, a_p + kk * (UKA / 2), vd + kk * ((UKA * 128) >> 4), G::kIdescO,
                                    kk > 0 || !fresh ? 1u : 0u);
                if (complete && leader)
                    umma_commit(o_full(t));
                return true;
            };
            // Both tiles' scores of block i; the first ones of a segment wait for its rows
            auto flags_of = [&](uint32_t i) { return __shfl_sync(0xffffffffu, metas[i % G::kMetas].flags, 0); };
            const uint32_t blocks = (uint32_t)blocks_here;
            bool ok = wait_k(0) && wait_q(0, segs0);
            uint32_t flags = 0;
            if (ok) {
                flags = flags_of(0);
                score(0, 0);
                if (flags & kBothTiles) {
                    ok = wait_q(1, segs1);
                    if (ok)
                        score(1, 0);
                }
                if (ok && leader)
                    umma_commit(empty(0, 0));
            }
            for (uint32_t i = 0; ok && i < blocks; ++i) {
                const bool first = i == 0 || flags & kFirst, last = i + 1 == blocks || flags & kLast;
                const bool more = i + 1 < blocks, two = flags & kBothTiles;
                ok = wait_warp(full(1, i & 1u), i >> 1 & 1u, p.wait_limit_ns, abort_flag, kSiteMmaFull) &&
                     pv(0, i, first, last, turns0);
                // within a segment the first tile's next scores go ahead of the second tile's P V
                if (ok && !last) {
                    ok = wait_k(i + 1);
                    if (ok)
                        score(0, i + 1);
                }
                if (ok && two)
                    ok = pv(1, i, first, last, turns1);
                if (!ok)
                    break;
                if (leader)
                    umma_commit(empty(1, i & 1u));
                if (!more)
                    break;
                if (last) {
                    ok = wait_k(i + 1) && wait_q(0, segs0);
                    if (!ok)
                        break;
                    score(0, i + 1);
                }
                flags = flags_of(i + 1);
                if (flags & kBothTiles) {
                    ok = !last || wait_q(1, segs1);
                    if (!ok)
                        break;
                    score(1, i + 1);
                }
                if (leader)
                    umma_commit(empty(0, (i + 1) & 1u));
            }
            // all MMAs of this thread complete before TMEM can be released
            if (leader)
                umma_commit(drain_bar);
            wait_drain(drain_bar, 0u, p.wait_limit_ns, abort_flag);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRaggedSoftmaxRegs));
        if (blocks_here > 0) {
            // ======================================================== softmax / output
            const int t = warp >> 2;                        // tile
            const int q = warp & 3;                         // TMEM lanes 32q .. 32q+31
            const uint32_t lane_base = (uint32_t)(32 * q) << 16;
            const uint32_t s_addr = tmem_base + lane_base + G::kTmemS + t * BN;
            const uint32_t o_addr = tmem_base + lane_base + G::kTmemO + t * HD;
            const int my_row = t * BM + 32 * q + lane;      // row of the item
            // The warp's 32 rows of Q into shared memory: HD / 8 lanes a row.  bf16 rows are scaled by a power of
            // two that brings their largest element to [2^14, 2^15), within fp16; returned: what undoes it.
            auto load_q = [&](const RaggedWalk &w) -> float {
                constexpr int kLanes = HD / 8, kRows = 32 / kLanes;
                // Loads on their way at once: all; of bf16, whose conversion is long, a quarter, so that the loop is rolled (the
                // feed has brought the rows into L2).  Measured: bf16 858 -> 851 us, under the window 118.7 -> 116.3; fp16 a quarter
                // at a time 808 -> 825.
                constexpr int kLoads = 32 / kRows / (kBf16 ? 4 : 1);
                const int rows = w.rows(p), sub = lane % kLanes;
                float mine = 1.0f;
#pragma unroll 1
                for (int i0 = 0; i0 < 32 / kRows; i0 += kLoads) {
                    uint4 x[kLoads];
#pragma unroll
                    for (int i = 0; i < kLoads; ++i) {
                        const int row = t * BM + 32 * q + (i0 + i) * kRows + lane / kLanes;   // of the item
                        x[i] = make_uint4(0, 0, 0, 0);
                        if (row < rows) {
                            const int token = p.by_group.quotient(w.item * 2 * BM + row);
                            const int g = w.item * 2 * BM + row - token * p.group;
                            x[i] = *reinterpret_cast<const uint4 *>(p.q + (w.seq.start + token) * p.q_stride[0] +
                                                                    (w.head * p.group + g) * p.q_stride[1] + sub * 8);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kLoads; ++i) {
                        const int r = 32 * q + (i0 + i) * kRows + lane / kLanes;   // of the tile
                        if constexpr (kBf16) {
                            uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                            uint32_t top = 0;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                top = max(top, max(v[e] & 0x7fffu, (v[e] >> 16) & 0x7fffu));
#pragma unroll
                            for (int o = 1; o < kLanes; o <<= 1)
                                top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                            int e2 = (int)(top >> 7) - 127;
                            e2 = e2 < -100 ? -100 : e2 > 127 ? 127 : e2;
                            const float to = __uint_as_float((uint32_t)(14 - e2 + 127) << 23);
                            const float back = __uint_as_float((uint32_t)(e2 - 14 + 127) << 23);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 f = pair_to_float2<true>(v[e]);
                                v[e] = half2_of(f.x * to, f.y * to);
                            }
                            x[i] = make_uint4(v[0], v[1], v[2], v[3]);
                            const float got = __shfl_sync(0xffffffffu, back, (lane % kRows) * kLanes);
                            mine = lane / kRows == i0 + i ? got : mine;
                        }
                        st_shared_v4(base + G::kOffQ + t * G::kTile16 + (sub >> 3) * kSub + r * 128 +
                                         ((uint32_t)((sub & 7) ^ (r & 7)) << 4), x[i].x, x[i].y, x[i].z, x[i].w);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(q_full((uint32_t)t));
                return mine;
            };
            uint32_t turns = 0, blocks = 0, outputs = 0;
            bool alive = true;
            RaggedCut cuts[2];
            int num_cuts = 0;
            RaggedWalk w = first_segment();
            float row_scale = t == 0 || w.rows(p) > BM ? load_q(w) : 1.0f;
            // (after a wait that expired the rest is walked through without it, so that every part is counted and the counters
            // go back to 0; the status says that the output is not to be used)
            for (bool more = true; more;) {
                const RaggedWalk cur = w;
                const int rows = cur.rows(p);
                const bool here = t == 0 || rows > BM;
                const int row = cur.item * 2 * BM + my_row;     // of the sequence and head
                const int token = p.by_group.quotient(row);
                const int off = cur.seq.n - cur.seq.count;
                const int pos = my_row < rows ? off + token : -1;
                const int first = off + p.by_group.quotient(cur.item * 2 * BM + t * BM);
                const int last = off + p.by_group.quotient(min(cur.item * 2 * BM + t * BM + BM, cur.seq.count * p.group) - 1);
                const float c_row = row_scale * p.scale_log2;
                auto factor = [&](float ks) { return score_factor(c_row, ks); };
                float m = -INFINITY, l = 0.0f;   // reference of the weights, their sum
                float rr = -INFINITY;            // O's reference above m
                float m_ref = 0.0f, rr_ref = 0.0f;   // both, 0 as long as there are none
                bool big = false;
                for (int j = cur.j; alive && here && j < cur.j1; ++j) {
                    const uint32_t i = blocks + (j - cur.j);
                    const bool ok = wait_bounded_eager(s_full((uint32_t)t), turns & 1u, p.wait_limit_ns, abort_flag,
                                                       kSiteEpiAccFull) &&
                                    wait_bounded_eager(meta_full(i % G::kMetas), i / G::kMetas & 1u, p.wait_limit_ns,
                                                       abort_flag, kSiteEpiAccFull);
                    if (!__all_sync(0xffffffffu, ok)) {
                        alive = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const RaggedMeta &meta = metas[i % G::kMetas];
                    const int key0 = cur.it.key0(j);
                    const uint32_t missing = meta.missing, flags = meta.flags;
                    // The scores are read twice: all at once for the largest, then 32 at a time, the next ones while these are
                    // worked on, for the weights.  (Kept in registers, with the weights' pass unrolled over all 128, the loop
                    // was 10 KB of code, and fetching it the bound: 2048 tokens in
                    // 32768 957 us, so 854; the largest 32 at a time, too, 922.)
                    // First, what the row does not see becomes -infinity.
                    const bool masked = missing || ragged_masked(p, first, last, key0);
                    const int hi = pos - key0, lo = p.window > 0 ? hi - p.window : -1, head = p.sinks - key0;
                    auto mask = [&](uint32_t (&x)[32], int c0) {   // a bit per key
                        uint32_t seen = keys_below(hi + 1 - c0) & (~keys_below(lo + 1 - c0) | keys_below(head - c0));
                        seen &= ~((missing >> (c0 / 16) & 1u ? 0x0000ffffu : 0u) |
                                  (missing >> (c0 / 16 + 1) & 1u ? 0xffff0000u : 0u));
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            x[e] = seen & (1u << e) ? x[e] : __float_as_uint(-INFINITY);
                        tmem_st_x32(s_addr + c0, x);
                    };
                    if (masked) {
#pragma unroll 1
                        for (int c0 = 0; c0 < BN; c0 += 32) {
                            uint32_t x[32];
                            tmem_ld_x32_sync(s_addr + c0, x);
                            mask(x, c0);
                        }
                        tmem_st_wait();
                    }
                    uint32_t xa[32], xb[32];
                    float ma = -INFINITY, mb = -INFINITY, mc = -INFINITY, md = -INFINITY;
                    {
                        uint32_t v[BN];
#pragma unroll
                        for (int c0 = 0; c0 < BN; c0 += 32)
                            tmem_ld_x32(s_addr + c0, *reinterpret_cast<uint32_t(*)[32]>(&v[c0]));
#pragma unroll
                        for (int c0 = 0; c0 < BN; c0 += 32)
                            tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&v[c0]));
#pragma unroll
                        for (int e = 0; e < BN; e += 4) {
                            ma = fmaxf(ma, __uint_as_float(v[e]));
                            mb = fmaxf(mb, __uint_as_float(v[e + 1]));
                            mc = fmaxf(mc, __uint_as_float(v[e + 2]));
                            md = fmaxf(md, __uint_as_float(v[e + 3]));
                        }
                        ma = fmaxf(ma, mc);
                        mb = fmaxf(mb, md);
                    }
                    const float c_blk = factor(meta.ks);
                    float mx = __fmul_rn(fmaxf(ma, mb), c_blk);
                    const float lv = meta.lv;
                    // the row's largest product with V's scale, above the reference of the weights
                    float over = (mx - m_ref) + lv;
                    const bool near = flags & kNearScales;
                    if (!near) {
                        const float2 top = ragged_top(s_addr, meta, c_row, m_ref);
                        mx = top.x;
                        over = top.y;
                    }
                    // The references of the weights (m) and of O (rr above m) move when a score or a product exceeds them by
                    // 2^8, and with the first scores.  Mostly none does: one vote and one jump.
                    if (__any_sync(0xffffffffu, mx > m + kRescaleLog2 || over > rr + kRescaleLog2)) {
                        const bool move = mx > m + kRescaleLog2;
                        const float m_new = move ? mx : m;
                        m_ref = m_new == -INFINITY ? 0.0f : m_new;
                        over = near ? (mx - m_ref) + lv : ragged_top(s_addr, meta, c_row, m_ref).y;
                        const float rr_old = move ? (m - m_new) + rr : rr;
                        const bool turn = over > rr_old + kRescaleLog2;
                        l *= move ? fast_exp2(m - m_new) : 1.0f;
                        m = m_new;
                        rr = turn ? over : rr_old;
                        rr_ref = rr == -INFINITY ? 0.0f : rr;
                        big = __any_sync(0xffffffffu, fabsf(m_ref) >= kBigLog2);
                        if (j > cur.j && __any_sync(0xffffffffu, turn)) {   // (the P V before this block is done)
                            const float alpha = turn ? fast_exp2(rr_old - rr) : 1.0f;
#pragma unroll 1
                            for (int c0 = 0; c0 < HD; c0 += 32) {
                                uint32_t o[32];
                                tmem_ld_x32_sync(o_addr + c0, o);
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st_x32(o_addr + c0, o);
                            }
                        }
                    }
                    float sum;
                    if (near && !big) {
                        tmem_ld_x32(s_addr, xa);
                        const float a = (lv + kPLog2 - rr_ref) - m_ref;
                        const float2 c2 = make_float2(c_blk, c_blk), a2 = make_float2(a, a);
                        float2 sa = make_float2(0.0f, 0.0f), sb = make_float2(0.0f, 0.0f);
                        auto weigh = [&](const uint32_t (&x)[32], int c0) {
                            uint32_t ph[16];
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float2 x01 = __ffma2_rn(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])),
                                                              c2, a2);
                                const float2 x23 = __ffma2_rn(make_float2(__uint_as_float(x[e + 2]),
                                                                          __uint_as_float(x[e + 3])), c2, a2);
                                const float2 e01 = make_float2(fast_exp2(x01.x), fast_exp2(x01.y));
                                const float2 e23 = make_float2(fast_exp2(x23.x), fast_exp2(x23.y));
                                sa = __fadd2_rn(sa, e01);
                                sb = __fadd2_rn(sb, e23);
                                ph[e / 2] = half2_of(e01.x, e01.y);
                                ph[e / 2 + 1] = half2_of(e23.x, e23.y);
                            }
                            tmem_st_x16(s_addr + c0 / 2, ph);   // (over scores that have been read)
                        };
#pragma unroll 1
                        for (int c0 = 0; c0 < BN; c0 += 64) {
                            tmem_ld_wait_regs(xa);
                            tmem_ld_x32(s_addr + c0 + 32, xb);
                            weigh(xa, c0);
                            tmem_ld_wait_regs(xb);
                            if (c0 + 64 < BN)
                                tmem_ld_x32(s_addr + c0 + 64, xa);
                            weigh(xb, c0 + 32);
                        }
                        sum = ((sa.x + sa.y) + (sb.x + sb.y)) * back_of(rr_ref, lv);
                    } else {
                        sum = ragged_weights(s_addr, meta, c_row, m_ref, rr_ref);
                    }
                    l += sum;
                    tmem_st_wait();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(p_full((uint32_t)t));
                    ++turns;
                }
                blocks += cur.j1 - cur.j;
                // the next item's rows (the last scores of this one are done with Q)
                more = w.next(p);
                if (alive && more && (t == 0 || w.rows(p) > BM))
                    row_scale = load_q(w);
                if (!here)
                    continue;
                if (alive)
                    alive = __all_sync(0xffffffffu, wait_bounded_eager(o_full((uint32_t)t), outputs & 1u, p.wait_limit_ns,
                                                                       abort_flag, kSiteEpiAccFull));
                tc_fence_after_sync();
                bool taken = false;
                for (int x = 0; x < kConvWarps; ++x)
                    taken = taken || dirty[kDirty * (kConvWarps * t + x) + outputs % kDirty];
                ++outputs;
                if (alive && taken)
                    ragged_add_nan<HD>(p, cur.b, cur.head, cur.item, cur.j, cur.j1, pos, o_addr);
                const bool valid = my_row < rows;
                uint16_t *dst = p.out + ((int64_t)(cur.seq.start + token) * p.q_heads + cur.head * p.group +
                                         (row - token * p.group)) * HD;
                const bool whole = cur.j == 0 && cur.j1 == cur.nb;
                if (whole) {
                    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;   // 0: the row sees nothing
                    const float f = exp2f(0.5f * (rr - kPLog2));
#pragma unroll 1
                    for (int c0 = 0; alive && c0 < HD; c0 += 32) {
                        uint32_t o[32];
                        tmem_ld_x32_sync(o_addr + c0, o);
                        if (valid)
                            write_row32<kBf16>(dst + c0, reinterpret_cast<const float(&)[32]>(o), inv, f);
                    }
                } else {
                    // a part: O, m, l and rr to the workspace
                    RaggedCut &cut = cuts[num_cuts++];
                    cut.dst = valid ? dst : nullptr;
                    cut.first = range_owner(cur.unit0, plan->total, plan->ranges);
                    cut.last = range_owner(cur.unit0 + ragged_units(cur.nb, plan->part) - 1, plan->total, plan->ranges);
                    cut.mid = cur.unit0 != range_start(cut.first, plan->total, plan->ranges);
                    float4 *part = ragged_part_of<HD>(p, cut, warp, lane, blockIdx.x);
#pragma unroll 1
                    for (int c0 = 0; alive && c0 < HD; c0 += 32) {
                        uint32_t o[32];
                        tmem_ld_x32_sync(o_addr + c0, o);
                        if (valid)
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                __stcg(part + (c0 + e) / 4 * 32,
                                       make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                                   __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3])));
                    }
                    if (alive && valid)
                        __stcg(part + HD / 4 * 32, make_float4(m, l, rr, 0.0f));
                }
            }
            // The parts of cut items (the one that the range starts in and the one that it ends in) are counted now; the warp
            // that comes last joins those of its rows, in the order of the ranges.
            for (int k = 0; k < num_cuts; ++k) {
                const RaggedCut cut = cuts[k];
                __syncwarp();
                unsigned before = 0;
                if (lane == 0)
                    before = count_part(p.arrived + cut.first * 8 + warp, (unsigned)(cut.last - cut.first));
                before = __shfl_sync(0xffffffffu, before, 0);
                __syncwarp();
                if (before != (unsigned)(cut.last - cut.first))
                    continue;
                const uint32_t rows = __ballot_sync(0xffffffffu, cut.dst != nullptr);
                if (rows >> 8) {
                    if (cut.dst != nullptr)
                        ragged_join<HD, kBf16>(p, cut, warp, lane);
                } else if (rows) {
                    const uint64_t at = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(cut.dst), lane & 7);
                    ragged_join_few<HD, kBf16>(p, cut, reinterpret_cast<uint16_t *>(at), warp, lane);
                }
            }
        }
    }

    // ---------------------------------------------------------------- teardown
    __syncwarp();
    tc_fence_before_sync();
    named_bar_sync(1, kRaggedThreads);
    tc_fence_after_sync();
    if (warp == kMmaWarp)
        tmem_dealloc(tmem_base, 512);
}

}  // namespace kvc
}  // namespace gemmrelu
