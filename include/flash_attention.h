/*
 * flash_attention.h -- attention forward on GB300 (sm_103a), C ABI of
 * libgemmrelu.so (the same library as gemm_relu.h; status codes, the device
 * watchdog and gemm_relu_status / gemm_relu_strerror are shared).
 */
#ifndef FLASH_ATTENTION_H
#define FLASH_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#include "gemm_relu.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * flash_attention_f16 -- O = softmax(Q K^T / sqrt(d)) V for every batch and
 * head, the FlashAttention forward of the TileLang tutorial pages (section
 * "FlashAttention": online softmax over blocks of keys, base-2 exponentials
 * with log2(e) / sqrt(d) folded in, fp32 accumulation, P rounded to fp16 for
 * the second product, causal mode cut at the diagonal).
 *
 * Q, K, V, O : DEVICE pointers to fp16 arrays of shape [batch][seq][heads][d]
 *              (row-major; the pages' "bshd"), 16-byte aligned, on the
 *              current CUDA device; the caller owns them.  O must not overlap
 *              Q, K or V (not checked).
 * batch, seq, heads >= 0 (0 in any of them: nothing to do, returns OK);
 *              batch and heads at most 65535.
 * head_dim   : 64 or 128 (else GEMMRELU_ERR_INVALID_ARG).
 * causal     : nonzero -> query i attends to keys 0..i only.
 * stream     : cudaStream_t to launch on (NULL = legacy default stream).
 *
 * One CTA per 128-row query tile of one (batch, head): TMA loads of Q and of
 * 128-key blocks of K and V, tcgen05.mma for S = Q K^T and O += P V with both
 * accumulators in TMEM, one thread per query row for the softmax.  The
 * summation order is fixed: the same call gives the same bits.
 *
 * Returns GEMMRELU_OK or an error code; asynchronous on `stream`.  Device-side
 * timeouts surface through gemm_relu_status.
 */
int flash_attention_f16(const void *Q, const void *K, const void *V, void *O,
                        int64_t batch, int64_t seq, int64_t heads, int64_t head_dim,
                        int causal, void *stream);

/*
 * flash_attention_window_x16 -- attention forward of a prompt with a sliding
 * window and first tokens that stay visible: query i stands at position
 * p = i + kv_seq - q_seq and sees the keys j <= p; with window > 0 only those
 * with j > p - window or j < sinks (window 0: causal attention).  A query that
 * sees nothing (p < 0) gets 0.
 *
 * Q, O       : [batch][q_seq][q_heads][head_dim], K, V
 *              [batch][kv_seq][kv_heads][head_dim], DEVICE pointers, all of
 *              `dtype` (GEMMRELU_F16 or GEMMRELU_BF16), 16-byte aligned.  O is
 *              contiguous and must not overlap the inputs (not checked).
 * q_heads    : a multiple of kv_heads; query head h reads K/V head
 *              h / (q_heads / kv_heads).  head_dim: 64 or 128.
 * *_strides  : {sequence, token, head} strides of Q, K and V in elements,
 *              positive multiples of 8 (any value for an axis of one
 *              element); head_dim elements are contiguous.
 * sizes      : batch and heads at most 65535, sequences at most 2^30.
 *
 * Softmax statistics and sums are fp32; the softmax weights are rounded to
 * `dtype` for the product with V, the result once.  NaN and infinities
 * reach exactly the queries that see them, and finite V give finite results
 * but for those that round past the type's largest number.  (bf16 scores that
 * leave fp32 are infinities; bf16 V below 2^-117 times the number of visible
 * keys may lose bits.)  The summation order is fixed: the
 * same call gives the same bits.  Asynchronous on `stream`, allocates nothing.
 */
int flash_attention_window_x16(const void *Q, const void *K, const void *V, void *O, int dtype,
                               int64_t batch, int64_t q_seq, int64_t kv_seq, int64_t q_heads,
                               int64_t kv_heads, int64_t head_dim, const int64_t *q_strides,
                               const int64_t *k_strides, const int64_t *v_strides, int64_t window,
                               int64_t sinks, void *stream);

#define GEMMRELU_CROSS_COUNTER_BYTES 4096   /* of flash_attention_cross_x16's workspace */

/*
 * flash_attention_cross_x16_workspace_bytes -- bytes of device workspace that
 * flash_attention_cross_x16 needs for these sizes on the current device: 0 unless few query
 * rows meet fewer heads than fill the GPU (and for invalid arguments, or when no CUDA device is available).
 */
size_t flash_attention_cross_x16_workspace_bytes(int64_t batch, int64_t q_seq, int64_t kv_seq,
                                                 int64_t q_heads, int64_t kv_heads, int64_t head_dim);

/*
 * flash_attention_cross_x16 -- attention to an encoder's states: O = softmax(Q K^T / sqrt(d)) V,
 * where query i of sequence b sees the keys j < lengths[b], whatever i is.
 *
 * Arguments, types, numerics and errors are flash_attention_window_x16's, but:
 * lengths    : DEVICE int32 [batch], each in [0, kv_seq], or NULL: all kv_seq.  A
 *              sequence without keys gets 0; a number out of range counts as 0, and
 *              gemm_relu_status reports GEMMRELU_ERR_PAGE.
 * q_heads    : at most 128 times kv_heads.
 * workspace  : at least flash_attention_cross_x16_workspace_bytes(...), 16-byte aligned (any
 *              value where that is 0).  Its first GEMMRELU_CROSS_COUNTER_BYTES must be 0
 *              before its first call; every call leaves them 0, whatever its sizes.
 *              Calls that may overlap on the GPU need different workspaces.
 * What stands behind a sequence's keys in K and V, NaN and infinities among it, reaches no query.
 */
int flash_attention_cross_x16(const void *Q, const void *K, const void *V, void *O, int dtype,
                              int64_t batch, int64_t q_seq, int64_t kv_seq, int64_t q_heads,
                              int64_t kv_heads, int64_t head_dim, const int64_t *q_strides,
                              const int64_t *k_strides, const int64_t *v_strides,
                              const int32_t *lengths, void *workspace, size_t workspace_bytes,
                              void *stream);

/*
 * Host-only test hook: the blocks of 128 keys that flash_attention_window_x16 visits
 * for rows at positions first .. last: [0, out[0]) and [out[1], out[2]).
 */
int flash_attention_window_debug_blocks(int64_t first, int64_t last, int64_t window, int64_t sinks,
                                        int *out);

#ifdef __cplusplus
}
#endif

#endif /* FLASH_ATTENTION_H */
