/*
 * rotary.h -- rotary positions of queries and keys on GB300 (sm_103a), C ABI of
 * libgemmrelu.so (status codes are shared with gemm_relu.h).
 */
#ifndef ROTARY_H
#define ROTARY_H

#include <stdint.h>

#include "gemm_relu.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMMRELU_POS_I32 0
#define GEMMRELU_POS_I64 1
#define GEMMRELU_FREQ_F32 0
#define GEMMRELU_FREQ_F64 1

/*
 * One tensor to rotate: [batch][tokens][heads][head_dim] of 16-bit elements, `heads` of it (0: no such
 * tensor).  x and y are 16-byte aligned, head_dim elements contiguous, strides {sequence, token, head}
 * multiples of 8 elements (0 among x's).  y may be x, with the same strides.
 */
typedef struct {
    const void *x;
    void *y;
    int64_t heads;
    int64_t x_strides[3], y_strides[3];
} rotary_tensor;

/*
 * rotary_x16 -- turn the pairs of the first `rot` elements of every head of q and k by angles that grow
 * with the token's position:
 *
 *   y1 = a (x1 cos t - x2 sin t),  y2 = a (x2 cos t + x1 sin t),  t = positions[b][i] * inv_freq[p]
 *
 * for pair p = 0 .. rot / 2 - 1: elements p and p + rot / 2, or with `interleaved` 2p and 2p + 1; a is
 * `amplitude`.  Elements from rot on are copied.  `inverse` turns by -t: with the same amplitude the
 * gradient with respect to x, given that with respect to y.
 *
 * q, k       : host structures, read during the call; all pointers in them are DEVICE pointers.
 * dtype      : GEMMRELU_F16 or GEMMRELU_BF16.
 * positions  : [batch][tokens], int32 or int64 (pos_type), any values.
 * inv_freq   : [rot / 2], radians a token, fp32 or fp64 (freq_type), finite, magnitudes below 2^31.
 * head_dim   : a multiple of 8, at most 512; rot even, 2 .. head_dim.
 * sizes      : batch * tokens at most 2^31 - 1, heads together at most 65535.
 *
 * A position times a frequency is formed as a 64-bit fraction of a turn: the angle is off by at most
 * 2^-52 of itself, 2^-64 turns a position and 2^-26 of a turn, however far the position is.  Sines,
 * cosines and products are fp32, the result is rounded once.  Asynchronous on `stream`, allocates nothing.
 */
int rotary_x16(const rotary_tensor *q, const rotary_tensor *k, int dtype, int64_t batch, int64_t tokens,
               int64_t head_dim, int64_t rot, int interleaved, const void *positions, int pos_type,
               const void *inv_freq, int freq_type, double amplitude, int inverse, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ROTARY_H */
