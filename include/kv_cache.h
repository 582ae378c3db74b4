/*
 * kv_cache.h -- a paged K/V cache held in 8 bits, C ABI of libgemmrelu.so
 * (GB300, sm_103a; status codes, the device watchdog and gemm_relu_status /
 * gemm_relu_strerror are shared with gemm_relu.h).
 *
 * The cache is a pool of pages.  A page holds `page` consecutive tokens of one
 * sequence for every K/V head, as e4m3 values with one fp32 scale per page
 * and head: token value = e4m3 value * scale.  A sequence's row of the page
 * table lists its pages in token order: token t is slot t % page of page
 * pages[t / page].
 *
 * Scales are powers of two, at least 2^-100: the smallest s with
 * amax <= 448 s, amax the largest finite magnitude of the page and head (448
 * the largest e4m3 value).  e4m3 is a floating format, so a finer scale would
 * only move the values by less than one binade; a power of two makes a page
 * whose scale grows a change of exponents.  NaN and infinities are stored
 * as e4m3 NaN; nothing else is.
 *
 * Conventions shared by the entry points
 * --------------------------------------
 *  - All array pointers are DEVICE pointers on the current device, owned by
 *    the caller; the descriptor itself is a host structure, read during the
 *    call.  Calls are asynchronous on `stream` (a cudaStream_t, NULL = the
 *    legacy default stream), allocate nothing and can be captured in a graph.
 *  - `dtype` GEMMRELU_F16 or GEMMRELU_BF16 is the type of the 16-bit tensors.
 *    Those have head_dim contiguous elements per head; `strides` counts elements
 *    from one sequence, token and head to the next, each a multiple of 8, and
 *    bases are 16-byte aligned.
 *  - head_dim is 64 or 128, page 16, 32, 64 or 128.
 *  - What only the device can see is checked there: a page number outside the
 *    pool, a length that is negative or beyond the page table's row, a count
 *    outside [0, min(tokens, length)] makes the call skip those tokens and
 *    gemm_relu_status report GEMMRELU_ERR_PAGE; nothing out of range is read
 *    or written.  That sequences own different pages, and that outputs do
 *    not overlap inputs, is not checked.
 */
#ifndef KV_CACHE_H
#define KV_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "gemm_relu.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMMRELU_KV_COUNTER_BYTES 4096   /* of kv_cache_attention_x16's workspace */
#define GEMMRELU_RAGGED_COUNTER_BYTES 8192   /* of kv_cache_attention_ragged_x16's */

typedef struct {
    void *k, *v;               /* e4m3 [num_pages][kv_heads][page][head_dim], 16-byte aligned */
    float *k_scale, *v_scale;  /* [num_pages][kv_heads] */
    int64_t num_pages, kv_heads, page, head_dim;
} kv_cache_pool;

/*
 * kv_cache_append_x16 -- write the K and V of new tokens into their pages.
 *
 * k, v     : [batch][tokens][kv_heads][head_dim] of `dtype`; k_strides and
 *            v_strides hold {sequence, token, head}.
 * pages    : int32 [batch][max_pages], the page table.
 * lengths  : int32 [batch], each sequence's length INCLUDING the new tokens.
 * counts   : int32 [batch], how many of the `tokens` rows are new tokens (the
 *            first counts[b] of them), or NULL: all of them.
 *
 * New token i of sequence b becomes token lengths[b] - counts[b] + i.  A page
 * that already holds tokens of the sequence keeps them; where its scale has to
 * grow, they are rounded again to the new scale (exact but for values that
 * become subnormal).  A page whose first slot is written starts afresh.  Slots
 * past the length keep what they hold.
 */
int kv_cache_append_x16(const kv_cache_pool *cache, const void *k, const void *v, int dtype,
                        int64_t batch, int64_t tokens, const int64_t *k_strides,
                        const int64_t *v_strides, const int32_t *pages, int64_t max_pages,
                        const int32_t *lengths, const int32_t *counts, void *stream);

/*
 * kv_cache_attention_x16_workspace_bytes -- bytes of device workspace that
 * kv_cache_attention_x16 needs for these sizes on the current device (its SM
 * count decides the partials); weights_width 0 when no weights are collected.
 * 0 for invalid arguments, or when no CUDA device is available.
 */
size_t kv_cache_attention_x16_workspace_bytes(int64_t batch, int64_t tokens, int64_t q_heads,
                                              int64_t kv_heads, int64_t head_dim,
                                              int64_t weights_width);

/*
 * kv_cache_attention_x16 -- attention of the last `tokens` tokens of every
 * sequence over the cache: O = softmax(q K^T / sqrt(head_dim)) V over the
 * tokens that each one sees.
 *
 * q        : [batch][tokens][q_heads][head_dim] of `dtype`, q_strides its
 *            {sequence, token, head}; q_heads a multiple of kv_heads: query head h
 *            reads K/V head h / (q_heads / kv_heads).
 * out      : [batch][tokens][q_heads][head_dim] of `dtype`, contiguous, 16-byte
 *            aligned.
 * lengths  : int32 [batch], each sequence's length including these tokens: query
 *            token i has position p = length - tokens + i.  It sees the tokens
 *            t <= p; with a window > 0 only those with t > p - window or
 *            t < sinks.  A token at a negative position (a sequence shorter
 *            than `tokens`) sees nothing: its output is 0.  Pages of which no
 *            query sees a token are not looked up: their numbers may be anything.
 * weights  : fp32 [batch][kv_heads][weights_width] or NULL.  weights[t] grows by the
 *            sum, over the query tokens and the head's group of query heads,
 *            of the softmax weight of token t; weights_width >= max_pages * page.
 * workspace: at least kv_cache_attention_x16_workspace_bytes(...), 16-byte
 *            aligned.  Its first GEMMRELU_KV_COUNTER_BYTES must be 0 before its
 *            first call; every call leaves them 0, whatever its sizes.  Calls
 *            that may overlap on the GPU need different workspaces.
 *
 * Sizes whose 64-token units, batch * kv_heads * ceil(tokens * group / 8) *
 * ceil(max_pages * page / 64), reach 2^31 are refused.
 *
 * Scores, softmax statistics and sums are fp32.  For the product with V a softmax weight
 * times its page's scale is rounded to fp16, relative to the largest such product of
 * the row: exact to 2^-11 of itself down to 2^-21 of that, and to 2^-32 of that
 * below.  The order of all sums is fixed: the same call gives the same bits.
 */
int kv_cache_attention_x16(const kv_cache_pool *cache, const void *q, int dtype, int64_t batch,
                           int64_t tokens, int64_t q_heads, const int64_t *q_strides, void *out,
                           const int32_t *pages, int64_t max_pages, const int32_t *lengths,
                           int64_t window, int64_t sinks, float *weights, int64_t weights_width,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * kv_cache_attention_ragged_x16_workspace_bytes -- bytes of device workspace that
 * kv_cache_attention_ragged_x16 needs on the current device for heads of
 * head_dim elements, whatever the call's other sizes.  0 for invalid
 * arguments, or when no CUDA device is available.
 */
size_t kv_cache_attention_ragged_x16_workspace_bytes(int64_t head_dim);

/*
 * kv_cache_attention_ragged_x16 -- kv_cache_attention_x16 for sequences that bring different
 * numbers of tokens (chunks of prompts, drafts and single tokens in one call):
 * each query token attends over its sequence's pages.
 *
 * q        : [rows][q_heads][head_dim] of `dtype`, q_strides its {token, head},
 *            multiples of 8 (0 among them); q_heads a multiple of kv_heads.
 * out      : [rows][q_heads][head_dim] of `dtype`, contiguous, 16-byte aligned.
 * starts   : int32 [batch + 1], ascending: sequence b's query tokens are the rows
 *            starts[b] .. starts[b + 1] - 1 (none where they are equal).  Rows of no
 *            sequence keep what they hold in `out`.
 * lengths  : int32 [batch], each sequence's length including its query tokens, which
 *            are its last ones: row starts[b] + i has position lengths[b] -
 *            (starts[b + 1] - starts[b]) + i and sees what kv_cache_attention_x16 says.
 *            Rows that see nothing become 0.
 * workspace: at least kv_cache_attention_ragged_x16_workspace_bytes(head_dim), 16-byte aligned.
 *            Its first GEMMRELU_RAGGED_COUNTER_BYTES must be 0 before its first
 *            call; every call leaves them 0, whatever its sizes.  Calls that may
 *            overlap on the GPU need different workspaces.
 *
 * batch is at most 16384, rows at most 2^24, rows * q_heads at most 2^30; sizes whose blocks of 128 tokens,
 * (rows * group / 256 + batch) * kv_heads * (max_pages * page / 128 + 1), reach 2^31 are
 * refused.  A sequence whose rows are not inside [0, rows) or descend is skipped and
 * reported as GEMMRELU_ERR_PAGE, and so is the whole call where rows that several sequences claim
 * make that many blocks.
 *
 * Scores, softmax statistics and sums are fp32.  For the products bf16 queries become
 * fp16, scaled by a power of two per row (exact but for elements below 2^-29 of the row's
 * largest), and a softmax weight times its page's scale is rounded to fp16, relative to the
 * largest such product of the row, as in kv_cache_attention_x16.  A weight whose product
 * with its page's V scale is below 2^-132 of the row's largest is left out of the sum of
 * weights.  NaN of V reach exactly the rows that see them.  The order of all sums is
 * fixed: the same call gives the same bits.
 */
int kv_cache_attention_ragged_x16(const kv_cache_pool *cache, const void *q, int dtype, int64_t rows,
                                  int64_t q_heads, const int64_t *q_strides, void *out,
                                  int64_t batch, const int32_t *starts, const int32_t *pages,
                                  int64_t max_pages, const int32_t *lengths, int64_t window,
                                  int64_t sinks, void *workspace, size_t workspace_bytes, void *stream);

/*
 * kv_cache_evict_e4m3 -- keep `budget` tokens of every sequence and head, by
 * accumulated attention weight, in new pages.
 *
 * weights  : fp32 [batch][kv_heads][weights_width], as kv_cache_attention_x16
 *            accumulates them; weights_width >= max_pages * page.
 * budget   : tokens kept.  A sequence of at most `budget` tokens keeps all of
 *            them.  Otherwise the first `sinks` tokens, the last `recent`, and of
 *            the others the budget - sinks - recent with the largest weights
 *            stay: ties go to the earlier token, NaN counts as -infinity.
 *            sinks, recent >= 0, sinks + recent <= budget, budget >= 1.
 * to       : the pool that receives them (may be `cache`), same kv_heads, page
 *            and head_dim; to_pages int32 [batch][to_max_pages] names pages
 *            that no sequence uses, to_max_pages * page >= budget.
 * to_lengths : int32 [batch], receives min(length, budget).
 * to_weights : fp32 [batch][kv_heads][to_max_pages * page], receives the kept
 *            tokens' weights, 0 past them.
 * kept     : int32 [batch][kv_heads][budget], receives the kept tokens' former
 *            positions in ascending order, -1 past them.
 *
 * Tokens keep their order.  The values that the kept tokens stand for are
 * stored as kv_cache_append_x16 stores a fresh page; the slots past them in a
 * sequence's last page become 0, pages past that are left alone.
 */
int kv_cache_evict_e4m3(const kv_cache_pool *cache, const float *weights, int64_t weights_width,
                        const int32_t *pages, int64_t max_pages, const int32_t *lengths,
                        int64_t batch, int64_t budget, int64_t sinks, int64_t recent,
                        const kv_cache_pool *to, const int32_t *to_pages, int64_t to_max_pages,
                        int32_t *to_lengths, float *to_weights, int32_t *kept, void *stream);

/*
 * Host-only test hooks.  kv_cache_debug_span: out[0] units of 64 tokens from the
 * first on, then those from out[1], out[2] in all -- what kv_cache_attention_x16
 * reads of a sequence.  kv_cache_debug_range: first of `total` units that block
 * x of `grid` takes, or (owner != 0) the block that takes unit x; -1 for
 * invalid arguments.
 */
int kv_cache_debug_span(int64_t length, int64_t tokens, int64_t window, int64_t sinks, int *out);
int kv_cache_debug_range(int x, int total, int grid, int owner);

#ifdef __cplusplus
}
#endif

#endif /* KV_CACHE_H */
