// rotary_api.cuh -- host side of rotary.h: argument checks and launch (part of the translation
// unit of gemm_relu_api.cu).
#pragma once

#include "rotary.h"
#include "rotary.cuh"

namespace {

namespace RO = gemmrelu::rot;

bool rotary_tensor_ok(const rotary_tensor *t) {
    if (t->heads == 0)
        return true;
    if (t->heads < 0 || t->heads > 65535 || !t->x || !t->y || !aligned(t->x, 16) || !aligned(t->y, 16) ||
        !strides_ok(t->x_strides) || !strides_ok(t->y_strides))
        return false;
    return true;
}

template <bool kBf16, bool kInterleaved>
int launch_rotary(const RO::RotaryParams &p, bool vector, int64_t blocks, cudaStream_t s) {
    return vector ? launch_kv(RO::rotary_kernel<kBf16, kInterleaved, true>, blocks, RO::kRotThreads, s, p)
                  : launch_kv(RO::rotary_kernel<kBf16, kInterleaved, false>, blocks, RO::kRotThreads, s, p);
}

}  // namespace

extern "C" int rotary_x16(const rotary_tensor *q, const rotary_tensor *k, int dtype, int64_t batch, int64_t tokens,
                          int64_t head_dim, int64_t rot, int interleaved, const void *positions, int pos_type,
                          const void *inv_freq, int freq_type, double amplitude, int inverse, void *stream) {
    if (!q || !k || (dtype != GEMMRELU_F16 && dtype != GEMMRELU_BF16) || batch < 0 || tokens < 0 ||
        batch > kMaxDim || tokens > kMaxDim || batch * tokens > kMaxDim || head_dim < 8 || head_dim > 512 ||
        head_dim % 8 != 0 || rot < 2 || rot > head_dim || rot % 2 != 0 ||
        (pos_type != GEMMRELU_POS_I32 && pos_type != GEMMRELU_POS_I64) ||
        (freq_type != GEMMRELU_FREQ_F32 && freq_type != GEMMRELU_FREQ_F64) || !(std::fabs(amplitude) <= 3e38) ||
        q->heads < 0 || k->heads < 0)
        return GEMMRELU_ERR_INVALID_ARG;
    if (batch == 0 || tokens == 0 || q->heads + k->heads == 0)
        return GEMMRELU_OK;
    if (!rotary_tensor_ok(q) || !rotary_tensor_ok(k) || q->heads + k->heads > 65535 || !positions ||
        !aligned(positions, pos_type == GEMMRELU_POS_I64 ? 8 : 4) || !inv_freq ||
        !aligned(inv_freq, freq_type == GEMMRELU_FREQ_F64 ? 8 : 4))
        return GEMMRELU_ERR_INVALID_ARG;
    DeviceState *ds = nullptr;
    const int rc = current_device_state(&ds);
    if (rc != GEMMRELU_OK)
        return rc;
    RO::RotaryParams p{};
    const rotary_tensor *t[2] = {q, k};
    for (int i = 0; i < 2; ++i) {
        p.x[i] = static_cast<const uint16_t *>(t[i]->x);
        p.y[i] = static_cast<uint16_t *>(t[i]->y);
        for (int j = 0; j < 3; ++j) {
            p.xs[i][j] = t[i]->x_strides[j];
            p.ys[i][j] = t[i]->y_strides[j];
        }
        p.copy = p.copy || (t[i]->heads > 0 && t[i]->x != t[i]->y);
    }
    p.heads0 = (int)q->heads;
    p.heads = (int)(q->heads + k->heads);
    p.rows = batch * tokens;
    p.tokens = (int)tokens;
    p.head_dim = (int)head_dim;
    p.half = (int)(rot / 2);
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.pos64 = pos_type == GEMMRELU_POS_I64;
    p.freq64 = freq_type == GEMMRELU_FREQ_F64;
    // vectors of 8 pairs where both halves are made of whole vectors
    const bool vector = rot % 16 == 0;
    p.turned = vector ? (int)rot / 16 : p.half;
    p.items = p.turned + (p.copy ? (int)((head_dim - rot) / 8 + 1) / 2 : 0);   // two vectors an item
    p.amplitude = (float)amplitude;
    p.sine = inverse ? -p.amplitude : p.amplitude;
    // Rows of a block: as many as give its threads an angle each, but two blocks an SM first.  The other
    // threads are head lanes.
    const int slots = RO::kRotThreads / p.items;   // (row, head lane) pairs
    p.rows_block = 1;
    while (p.rows_block * 2 <= slots && p.rows_block * 2 * p.half <= RO::kRotThreads &&
           p.rows >= (int64_t)p.rows_block * 4 * ds->sms)
        p.rows_block *= 2;
    p.lanes = std::min(slots / p.rows_block, p.heads);
    const int64_t blocks = (p.rows + p.rows_block - 1) / p.rows_block;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == GEMMRELU_BF16)
        return interleaved ? launch_rotary<true, true>(p, vector, blocks, s)
                           : launch_rotary<true, false>(p, vector, blocks, s);
    return interleaved ? launch_rotary<false, true>(p, vector, blocks, s)
                       : launch_rotary<false, false>(p, vector, blocks, s);
}
