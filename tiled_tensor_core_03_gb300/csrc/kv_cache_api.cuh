// kv_cache_api.cuh -- host side of kv_cache.h: argument checks and launches
// (part of the translation unit of gemm_relu_api.cu, whose helpers it uses).
#pragma once

#include "kv_cache.h"
#include "kv_cache.cuh"

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

template <int D>
int launch_move(const KC::EvictParams &p, int64_t grid, cudaStream_t s) {
    // vectors of 16 elements a thread
    if (p.from.page * D / 16 > 2 * KC::kMoveThreads)
        return launch_kv(KC::kv_evict_move_kernel<D, 4>, grid, KC::kMoveThreads, s, p);
    if (p.from.page * D / 16 > KC::kMoveThreads)
        return launch_kv(KC::kv_evict_move_kernel<D, 2>, grid, KC::kMoveThreads, s, p);
    return launch_kv(KC::kv_evict_move_kernel<D, 1>, grid, KC::kMoveThreads, s, p);
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
    if (heads > kMaxGrid || moves > kMaxGrid)
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
    p.to_lengths = to_lengths;
    p.to_weights = to_weights;
    p.kept = kept;
    DeviceState *ds = nullptr;
    int rc = current_device_state(&ds);
    if (rc != GEMMRELU_OK)
        return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    rc = launch_kv(KC::kv_evict_select_kernel, heads, KC::kSelectThreads, s, p);
    if (rc != GEMMRELU_OK)
        return rc;
    return cache->head_dim == 64 ? launch_move<64>(p, moves, s) : launch_move<128>(p, moves, s);
}

}  // extern "C"
