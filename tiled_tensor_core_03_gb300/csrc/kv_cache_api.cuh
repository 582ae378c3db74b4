// kv_cache_api.cuh -- host side of kv_cache.h: argument checks and launches
// (part of the translation unit of gemm_relu_api.cu, whose helpers it uses).
#pragma once

#include "kv_cache.h"
#include "kv_cache.cuh"
#include "kv_attention.cuh"

namespace {

namespace KC = gemmrelu::kvc;

constexpr int64_t kMaxTokens = (int64_t)1 << 30;   // of a sequence: 32-bit positions with room
constexpr int64_t kMaxGrid = 0x7fffffff;

bool pool_ok(const kv_cache_pool *c) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !aligned(c->k, 16) ||
        !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return false;
    if (c->head_dim != 64 && c->head_dim != 128)
        return false;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)
        return false;
    return c->num_pages > 0 && c->num_pages <= kMaxDim && c->kv_heads > 0 && c->kv_heads <= 65535;
}

KC::Pool device_pool(const kv_cache_pool *c) {
    KC::Pool p{};
    p.values[0] = static_cast<uint8_t *>(c->k);
    p.values[1] = static_cast<uint8_t *>(c->v);
    p.scales[0] = c->k_scale;
    p.scales[1] = c->v_scale;
    p.num_pages = c->num_pages;
    p.kv_heads = (int)c->kv_heads;
    p.page = (int)c->page;
    p.page_shift = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
    return p;
}

// A page table's row and the batch it serves.
bool table_ok(const int32_t *pages, int64_t batch, int64_t max_pages, int64_t page) {
    return pages && aligned(pages, 4) && max_pages > 0 && max_pages <= kMaxTokens / page &&
           batch <= 65535;
}

// {sequence, token, head} strides of a 16-bit tensor whose heads start on
// 16-byte boundaries.  A stride of 0 (a broadcast axis) is one.
bool strides_ok(const int64_t *s) {
    if (!s)
        return false;
    for (int i = 0; i < 3; ++i)
        if (s[i] < 0 || s[i] % 8 != 0 || s[i] > ((int64_t)1 << 39))
            return false;
    return true;
}

// Launch `kern` on a 1-D grid (a count beyond the grid limit is the caller's
// to refuse).
template <typename P>
int launch_kv(void (*kern)(P), int64_t grid, int threads, cudaStream_t s, const P &p) {
    return launch_kernel(kern, (unsigned)grid, (unsigned)threads, 0u, s, false, 1u, p);
}

template <int D, int kVec>
int launch_append(const KC::AppendParams &p, int64_t grid, int dtype, cudaStream_t s) {
    return dtype == GEMMRELU_BF16
               ? launch_kv(KC::kv_append_kernel<D, kVec, true>, grid, KC::kAppendThreads, s, p)
               : launch_kv(KC::kv_append_kernel<D, kVec, false>, grid, KC::kAppendThreads, s, p);
}

template <int D, int kVec>
int launch_move_vec(const KC::EvictParams &p, int sms, cudaStream_t s) {
    // blocks walk over the items; two rounds of them even out their ends (608 blocks 74.1 us, 1216 72.3)
    const int64_t grid = std::min<int64_t>(p.items, (int64_t)sms * 8);
    return launch_kv(KC::kv_evict_move_kernel<D, kVec>, grid, KC::kMoveThreads, s, p);
}

template <int D>
int launch_move(const KC::EvictParams &p, int sms, cudaStream_t s) {
    // vectors of 16 elements a thread
    const int vectors = p.from.page * D / 16;
    return vectors > 2 * KC::kMoveThreads ? launch_move_vec<D, 4>(p, sms, s)
           : vectors > KC::kMoveThreads   ? launch_move_vec<D, 2>(p, sms, s)
                                          : launch_move_vec<D, 1>(p, sms, s);
}

// A cluster of blocks holds a sequence's keys in registers as far as 8 blocks go.
int launch_select(KC::EvictParams &p, int64_t heads, cudaStream_t s) {
    constexpr int kSmall = 8, kLarge = 32;   // keys a thread
    const int64_t most = p.max_pages * p.from.page;
    p.cluster = 1;
    if (most <= (int64_t)kSmall * KC::kSelectThreads)
        return launch_kv(KC::kv_evict_select_kernel<kSmall>, heads, KC::kSelectThreads, s, p);
    while (p.cluster < KC::kMaxSelectCluster && most > (int64_t)p.cluster * kLarge * KC::kSelectThreads)
        p.cluster *= 2;
    return launch_kernel(KC::kv_evict_select_kernel<kLarge>, (unsigned)(heads * p.cluster),
                         KC::kSelectThreads, 0u, s, false, (unsigned)p.cluster, p);
}

// K or V of a pool as a 4-D tensor of bytes {head_dim, page, kv_heads, num_pages}; boxes
// of one head's `box_tokens` tokens, swizzled by the row's width.
bool make_pool_map(CUtensorMap *map, const void *ptr, const kv_cache_pool *c, uint32_t box_tokens) {
    EncodeTiledFn enc = encode_fn();
    if (!enc)
        return false;
    const cuuint64_t d = (cuuint64_t)c->head_dim, row = d * (cuuint64_t)c->page;
    cuuint64_t dims[4] = {d, (cuuint64_t)c->page, (cuuint64_t)c->kv_heads, (cuuint64_t)c->num_pages};
    cuuint64_t strides[3] = {d, row, row * (cuuint64_t)c->kv_heads};
    cuuint32_t box[4] = {(cuuint32_t)d, box_tokens, 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(ptr), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workspace of kv_cache_attention_x16: the counters of cut segments, one per block at most, at a
// place that no call's sizes move; partials; with weights every row's log-sum-exp and scores.
struct AttnSpace {
    size_t partial, lse, scores, total;   // byte offsets; counters at 0
};

AttnSpace attention_space(int64_t batch, int64_t rows, int64_t kv_heads, int64_t head_dim,
                          int64_t weights_width, int sms) {
    AttnSpace a{};
    const size_t slots = 2 * (size_t)sms * std::max(KC::AttnCfg<64, 1>::kBlocksPerSm * 8,
                                                    KC::AttnCfg<64, 2>::kBlocksPerSm * 16);
    size_t at = a.partial = GEMMRELU_KV_COUNTER_BYTES;
    at += slots * (head_dim + 4) * 4;
    a.lse = at = round256(at);
    if (weights_width > 0) {
        at += (size_t)batch * kv_heads * rows * 4;
        a.scores = at = round256(at);
        at += (size_t)batch * kv_heads * weights_width * rows * 4;
    }
    a.total = round256(at);
    return a;
}

// batch, tokens and heads of an attention call; their products stay far from 2^63.
bool attention_sizes_ok(int64_t batch, int64_t tokens, int64_t q_heads, int64_t kv_heads,
                        int64_t head_dim, int64_t weights_width) {
    return batch >= 0 && batch <= 65535 && tokens >= 0 && tokens <= 65535 && kv_heads > 0 &&
           kv_heads <= 65535 && q_heads > 0 && q_heads <= 65535 && q_heads % kv_heads == 0 &&
           (head_dim == 64 || head_dim == 128) && weights_width >= 0 && weights_width <= kMaxTokens &&
           batch * kv_heads <= kMaxGrid && tokens * q_heads <= (int64_t)1 << 24 &&
           batch * kv_heads * (tokens * (q_heads / kv_heads)) <= kMaxGrid;
}

template <int D, int kN, bool kBf16, bool kScores>
int launch_kv_attention(const CUtensorMap &mK, const CUtensorMap &mV, KC::AttnParams &p,
                        cudaStream_t s, int sms, bool *attr) {
    using G = KC::AttnCfg<D, kN>;
    auto kern = KC::kv_attention_kernel<D, kN, kBf16, kScores>;
    bool &attr_done = attr[(D == 128 ? 8 : 0) + (kN == 2 ? 4 : 0) + (kBf16 ? 2 : 0) + (kScores ? 1 : 0)];
    if (!ensure_smem_attr(attr_done, kern, G::kSmem))
        return GEMMRELU_ERR_LAUNCH;
    const int tiles = (p.rows + G::kRows - 1) / G::kRows;
    p.passes = (tiles + KC::kMostAbreast - 1) / KC::kMostAbreast;
    p.abreast = (tiles + p.passes - 1) / p.passes;
    const int ranges = std::max(1, std::min(sms * G::kBlocksPerSm,
                                            (int)(GEMMRELU_KV_COUNTER_BYTES / sizeof(unsigned))) / p.abreast);
    p.grid = ranges * p.abreast;
    const int rc = launch_kernel(kern, dim3((unsigned)ranges, (unsigned)p.abreast), KC::kAttnThreads, G::kSmem, s,
                                 false, 1u, mK, mV, p);
    if (rc != GEMMRELU_OK || !kScores)
        return rc;
    const int64_t blocks = (p.width + KC::kWeightThreads - 1) / KC::kWeightThreads;
    const int64_t grid = (int64_t)p.batch * p.pool.kv_heads * blocks;
    return p.rows % 4 == 0 ? launch_kv(KC::kv_attention_weights_kernel<4>, grid, KC::kWeightThreads, s, p)
                           : launch_kv(KC::kv_attention_weights_kernel<1>, grid, KC::kWeightThreads, s, p);
}

template <int D, int kN>
int launch_kv_attention_as(bool bf16, const CUtensorMap &mK, const CUtensorMap &mV, KC::AttnParams &p,
                           cudaStream_t s, int sms, bool *attr) {
    if (p.weights)
        return bf16 ? launch_kv_attention<D, kN, true, true>(mK, mV, p, s, sms, attr)
                    : launch_kv_attention<D, kN, false, true>(mK, mV, p, s, sms, attr);
    return bf16 ? launch_kv_attention<D, kN, true, false>(mK, mV, p, s, sms, attr)
                : launch_kv_attention<D, kN, false, false>(mK, mV, p, s, sms, attr);
}

}  // namespace

extern "C" {

int kv_cache_append_x16(const kv_cache_pool *cache, const void *k, const void *v, int dtype,
                        int64_t batch, int64_t tokens, const int64_t *k_strides,
                        const int64_t *v_strides, const int32_t *pages, int64_t max_pages,
                        const int32_t *lengths, const int32_t *counts, void *stream) {
    if (!pool_ok(cache) || (dtype != GEMMRELU_F16 && dtype != GEMMRELU_BF16) || batch < 0 ||
        tokens < 0 || tokens > kMaxTokens)
        return GEMMRELU_ERR_INVALID_ARG;
    if (batch == 0 || tokens == 0)
        return GEMMRELU_OK;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !strides_ok(k_strides) ||
        !strides_ok(v_strides) || !table_ok(pages, batch, max_pages, cache->page) || !lengths ||
        !aligned(lengths, 4) || !aligned(counts, 4))
        return GEMMRELU_ERR_INVALID_ARG;
    KC::AppendParams p{};
    p.pool = device_pool(cache);
    p.x[0] = static_cast<const uint16_t *>(k);
    p.x[1] = static_cast<const uint16_t *>(v);
    for (int i = 0; i < 3; ++i) {
        p.stride[0][i] = k_strides[i];
        p.stride[1][i] = v_strides[i];
    }
    p.pages = pages;
    p.lengths = lengths;
    p.counts = counts;
    p.max_pages = max_pages;
    p.batch = (int)batch;
    p.tokens = (int)tokens;
    p.touched = (int)((tokens + cache->page - 2) / cache->page + 1);
    const int64_t grid = batch * p.touched * cache->kv_heads * 2;
    if (grid > kMaxGrid)
        return GEMMRELU_ERR_INVALID_ARG;
    DeviceState *ds = nullptr;
    const int rc = current_device_state(&ds);
    if (rc != GEMMRELU_OK)
        return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t vectors = cache->page * cache->head_dim / 8;   // 128 .. 2048
    if (cache->head_dim == 64)
        return vectors <= 256   ? launch_append<64, 1>(p, grid, dtype, s)
               : vectors <= 512 ? launch_append<64, 2>(p, grid, dtype, s)
                                : launch_append<64, 4>(p, grid, dtype, s);
    return vectors <= 256    ? launch_append<128, 1>(p, grid, dtype, s)
           : vectors <= 512  ? launch_append<128, 2>(p, grid, dtype, s)
           : vectors <= 1024 ? launch_append<128, 4>(p, grid, dtype, s)
                             : launch_append<128, 8>(p, grid, dtype, s);
}

int kv_cache_evict_e4m3(const kv_cache_pool *cache, const float *weights, int64_t weights_width,
                        const int32_t *pages, int64_t max_pages, const int32_t *lengths,
                        int64_t batch, int64_t budget, int64_t sinks, int64_t recent,
                        const kv_cache_pool *to, const int32_t *to_pages, int64_t to_max_pages,
                        int32_t *to_lengths, float *to_weights, int32_t *kept, void *stream) {
    if (!pool_ok(cache) || !pool_ok(to) || to->kv_heads != cache->kv_heads ||
        to->page != cache->page || to->head_dim != cache->head_dim || batch < 0 || budget < 1 ||
        budget > kMaxTokens || sinks < 0 || recent < 0 || sinks > budget || recent > budget - sinks)
        return GEMMRELU_ERR_INVALID_ARG;
    if (batch == 0)
        return GEMMRELU_OK;
    if (!table_ok(pages, batch, max_pages, cache->page) ||
        !table_ok(to_pages, batch, to_max_pages, cache->page) ||
        to_max_pages * cache->page < budget || weights_width < max_pages * cache->page ||
        !weights || !lengths || !to_lengths || !to_weights || !kept || !aligned(weights, 4) ||
        !aligned(lengths, 4) || !aligned(to_lengths, 4) || !aligned(to_weights, 4) ||
        !aligned(kept, 4))
        return GEMMRELU_ERR_INVALID_ARG;
    const int64_t heads = batch * cache->kv_heads, moves = heads * to_max_pages;
    if (heads > kMaxGrid / KC::kMaxSelectCluster || moves > kMaxGrid)
        return GEMMRELU_ERR_INVALID_ARG;
    KC::EvictParams p{};
    p.from = device_pool(cache);
    p.to = device_pool(to);
    p.weights = weights;
    p.width = weights_width;
    p.pages = pages;
    p.lengths = lengths;
    p.to_pages = to_pages;
    p.max_pages = max_pages;
    p.to_max_pages = to_max_pages;
    p.batch = (int)batch;
    p.budget = (int)budget;
    p.sinks = (int)sinks;
    p.recent = (int)recent;
    p.items = (int)moves;
    p.to_lengths = to_lengths;
    p.to_weights = to_weights;
    p.kept = kept;
    DeviceState *ds = nullptr;
    int rc = current_device_state(&ds);
    if (rc != GEMMRELU_OK)
        return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    rc = launch_select(p, heads, s);
    if (rc != GEMMRELU_OK)
        return rc;
    return cache->head_dim == 64 ? launch_move<64>(p, ds->sms, s) : launch_move<128>(p, ds->sms, s);
}

size_t kv_cache_attention_x16_workspace_bytes(int64_t batch, int64_t tokens, int64_t q_heads,
                                              int64_t kv_heads, int64_t head_dim,
                                              int64_t weights_width) {
    if (!attention_sizes_ok(batch, tokens, q_heads, kv_heads, head_dim, weights_width))
        return 0;
    DeviceState *ds = nullptr;
    if (current_device_state(&ds) != GEMMRELU_OK)
        return 0;
    return attention_space(batch, tokens * (q_heads / kv_heads), kv_heads, head_dim, weights_width,
                           ds->sms).total;
}

int kv_cache_attention_x16(const kv_cache_pool *cache, const void *q, int dtype, int64_t batch,
                           int64_t tokens, int64_t q_heads, const int64_t *q_strides, void *out,
                           const int32_t *pages, int64_t max_pages, const int32_t *lengths,
                           int64_t window, int64_t sinks, float *weights, int64_t weights_width,
                           void *workspace, size_t workspace_bytes, void *stream) {
    if (!pool_ok(cache) || (dtype != GEMMRELU_F16 && dtype != GEMMRELU_BF16) || window < 0 ||
        sinks < 0 ||
        !attention_sizes_ok(batch, tokens, q_heads, cache->kv_heads, cache->head_dim,
                            weights ? weights_width : 0))
        return GEMMRELU_ERR_INVALID_ARG;
    if (batch == 0 || tokens == 0)
        return GEMMRELU_OK;
    if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !strides_ok(q_strides) ||
        !table_ok(pages, batch, max_pages, cache->page) || !lengths || !aligned(lengths, 4) ||
        !aligned(weights, 4) || (weights && weights_width < max_pages * cache->page) ||
        (weights && batch * cache->kv_heads * ((weights_width + KC::kWeightThreads - 1) /
                                               KC::kWeightThreads) > kMaxGrid))
        return GEMMRELU_ERR_INVALID_ARG;
    DeviceState *ds = nullptr;
    const int rc = current_device_state(&ds);
    if (rc != GEMMRELU_OK)
        return rc;
    const int64_t rows = tokens * (q_heads / cache->kv_heads);
    // units of 64 tokens, counted in 32 bits
    if (batch * cache->kv_heads * ((rows + 7) / 8) > kMaxGrid / ((max_pages * cache->page + 63) / 64))
        return GEMMRELU_ERR_INVALID_ARG;
    const AttnSpace sp = attention_space(batch, rows, cache->kv_heads, cache->head_dim,
                                         weights ? weights_width : 0, ds->sms);
    if (!workspace || workspace_bytes < sp.total || !aligned(workspace, 16))
        return GEMMRELU_ERR_WORKSPACE;
    const uint32_t box = (uint32_t)std::min<int64_t>(cache->page, KC::kUnit);
    CUtensorMap mK, mV;
    if (!make_pool_map(&mK, cache->k, cache, box) || !make_pool_map(&mV, cache->v, cache, box))
        return GEMMRELU_ERR_LAUNCH;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    KC::AttnParams p{};
    p.pool = device_pool(cache);
    p.q = static_cast<const uint16_t *>(q);
    for (int i = 0; i < 3; ++i)
        p.q_stride[i] = q_strides[i];
    p.out = static_cast<uint16_t *>(out);
    p.pages = pages;
    p.lengths = lengths;
    p.max_pages = max_pages;
    p.batch = (int)batch;
    p.tokens = (int)tokens;
    p.q_heads = (int)q_heads;
    p.group = (int)(q_heads / cache->kv_heads);
    p.rows = (int)rows;
    p.window = (int)std::min<int64_t>(window, kMaxTokens);
    p.sinks = (int)std::min<int64_t>(sinks, kMaxTokens);
    p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)cache->head_dim));
    p.partial = reinterpret_cast<float *>(ws + sp.partial);
    p.arrived = reinterpret_cast<unsigned *>(ws);
    if (weights) {
        p.lse = reinterpret_cast<float *>(ws + sp.lse);
        p.scores = reinterpret_cast<float *>(ws + sp.scores);
        p.weights = weights;
        p.width = weights_width;
    }
    p.drop_arrive = g_drop_arrive.load();
    p.wait_limit_ns = wait_limit_ns();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == GEMMRELU_BF16;
    // Up to 8 rows fit one group of 8.  Beyond, two groups a tile share the conversion of K and V, which
    // pays for heads of 64 (32 sequences of up to 4096 tokens, 8 K/V heads: 16 rows 42.5 us with two
    // groups, 46.5 with a tile per group; 64 rows 131 and 147) but not for heads of 128, whose
    // accumulators and query fragments spill at 168 registers (16 rows 76 to 107 us with two
    // groups, 65.4 with a tile per group; 64 rows 233 to 365 and 218).
    if (cache->head_dim == 128)
        return launch_kv_attention_as<128, 1>(bf16, mK, mV, p, s, ds->sms, ds->attr_kv);
    return rows <= 8 ? launch_kv_attention_as<64, 1>(bf16, mK, mV, p, s, ds->sms, ds->attr_kv)
                     : launch_kv_attention_as<64, 2>(bf16, mK, mV, p, s, ds->sms, ds->attr_kv);
}

int kv_cache_debug_span(int64_t length, int64_t tokens, int64_t window, int64_t sinks, int *out) {
    if (length < 0 || length > kMaxTokens || tokens < 1 || tokens > kMaxTokens || window < 0 ||
        window > kMaxTokens || sinks < 0 || sinks > kMaxTokens || !out)
        return GEMMRELU_ERR_INVALID_ARG;
    const KC::Span s = KC::span_of((int)length, (int)tokens, (int)window, (int)sinks);
    out[0] = s.sink_units;
    out[1] = s.low_unit;
    out[2] = s.units;
    return GEMMRELU_OK;
}

int kv_cache_debug_range(int x, int total, int grid, int owner) {
    if (x < 0 || total < 1 || grid < 1)
        return -1;
    return owner ? KC::range_owner(x, total, grid) : KC::range_start(x, total, grid);
}

}  // extern "C"
