// flash_attention_window_api.cuh -- host side of flash_attention_window_x16: argument checks,
// tensor maps and launch (part of the translation unit of gemm_relu_api.cu).
#pragma once

#include "flash_attention_window.cuh"

namespace {

// A [batch][seq][heads][d] tensor of 16-bit elements with strides {sequence, token,
// head}: boxes of 64 d x 1 head x 128 tokens, 128-byte swizzle, zero fill outside.  An axis of
// one element is never stepped over, whatever its stride.
bool make_strided_map(CUtensorMap *map, const void *ptr, int dtype, int64_t batch, int64_t seq,
                      int64_t heads, int64_t d, const int64_t *strides) {
    EncodeTiledFn enc = encode_fn();
    if (!enc)
        return false;
    auto bytes = [&](int64_t n, int64_t stride) { return (cuuint64_t)(n == 1 ? d : stride) * 2; };
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)seq, (cuuint64_t)batch};
    cuuint64_t step[3] = {bytes(heads, strides[2]), bytes(seq, strides[1]), bytes(batch, strides[0])};
    cuuint32_t box[4] = {64, 1, (cuuint32_t)FA::BM, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, dtype == GEMMRELU_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
               4, const_cast<void *>(ptr), dims, step, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Strides that TMA can describe: positive multiples of 8 elements below 2^40 bytes where
// the axis has more than one element.
bool window_strides_ok(const int64_t *s, int64_t batch, int64_t seq, int64_t heads) {
    if (!s)
        return false;
    const int64_t n[3] = {batch, seq, heads};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (s[i] <= 0 || s[i] % 8 != 0 || s[i] >= ((int64_t)1 << 39)))
            return false;
    return true;
}

template <int HD, bool kBf16>
int launch_window(const CUtensorMap &mQ, const CUtensorMap &mK, const CUtensorMap &mV,
                  const FA::WindowParams &p, int sms, cudaStream_t stream, bool &attr_done) {
    auto kern = FA::flash_attention_window_kernel<HD, kBf16>;
    if (!ensure_smem_attr(attr_done, kern, FA::WindowCfg<HD>::kSmemBytes))
        return GEMMRELU_ERR_LAUNCH;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(sms, (int64_t)p.pairs * p.kv_heads * p.batch));
    cfg.blockDim = dim3(FA::kWindowThreads);
    cfg.dynamicSmemBytes = FA::WindowCfg<HD>::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = GEMMRELU_PDL ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, kern, mQ, mK, mV, p));
}

}  // namespace

// The order of the work.  The first queries see fewer keys than the last, and with one head after the
// other a CTA whose stride shares a factor with a head's items gets the same few places in each.  So
// heads go together, the last queries of all of them first, as many heads as have K and V in 96 MB
// of the L2 cache (129 MB).  Measured, 32 heads on 8 of 128, one head after the other against this: 4 x 4096
// tokens without a window 440 -> 405 us, with 1024 237 -> 223; 2048 tokens 51.3 -> 40.9; 16384 tokens
// without a window 1590 -> 1444 us, with 4096 710 -> 666; 4 x 4096 and 32 heads on 32 557 -> 453 us
// (485 with all heads together).  What it costs: 16384 tokens with a window of 512 173 -> 186 us.
constexpr int64_t kWindowChunkBytes = (int64_t)96 << 20;

extern "C" int flash_attention_window_x16(const void *Q, const void *K, const void *V, void *O,
                                          int dtype, int64_t batch, int64_t q_seq, int64_t kv_seq,
                                          int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                          const int64_t *q_strides, const int64_t *k_strides,
                                          const int64_t *v_strides, int64_t window, int64_t sinks,
                                          void *stream) {
    if ((dtype != GEMMRELU_F16 && dtype != GEMMRELU_BF16) || batch < 0 || batch > 65535 ||
        q_seq < 0 || kv_seq < 0 || q_seq > ((int64_t)1 << 30) || kv_seq > ((int64_t)1 << 30) ||
        q_heads < 0 || q_heads > 65535 || kv_heads < 0 || kv_heads > 65535 ||
        (head_dim != 64 && head_dim != 128) || window < 0 || sinks < 0)
        return GEMMRELU_ERR_INVALID_ARG;
    if (batch == 0 || q_seq == 0 || q_heads == 0)
        return GEMMRELU_OK;
    if (kv_heads == 0 || q_heads % kv_heads != 0 || !O || !aligned(O, 16) ||
        q_seq > ((int64_t)1 << 40) / (batch * q_heads * head_dim))
        return GEMMRELU_ERR_INVALID_ARG;
    if (kv_seq > 0 && (!Q || !K || !V || !aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) ||
                       !window_strides_ok(q_strides, batch, q_seq, q_heads) ||
                       !window_strides_ok(k_strides, batch, kv_seq, kv_heads) ||
                       !window_strides_ok(v_strides, batch, kv_seq, kv_heads)))
        return GEMMRELU_ERR_INVALID_ARG;
    DeviceState *ds = nullptr;
    const int rc = current_device_state(&ds);
    if (rc != GEMMRELU_OK)
        return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (kv_seq == 0)   // nobody sees anything
        return launch_status(cudaMemsetAsync(O, 0, (size_t)(batch * q_seq * q_heads * head_dim) * 2, s));
    CUtensorMap mQ, mK, mV;
    if (!make_strided_map(&mQ, Q, dtype, batch, q_seq, q_heads, head_dim, q_strides) ||
        !make_strided_map(&mK, K, dtype, batch, kv_seq, kv_heads, head_dim, k_strides) ||
        !make_strided_map(&mV, V, dtype, batch, kv_seq, kv_heads, head_dim, v_strides))
        return GEMMRELU_ERR_LAUNCH;
    FA::WindowParams p{};
    p.v = static_cast<const uint16_t *>(V);
    p.o = static_cast<uint16_t *>(O);
    for (int i = 0; i < 3; ++i)
        p.vs[i] = v_strides[i];
    p.n_q = (int)q_seq;
    p.n_kv = (int)kv_seq;
    p.q_heads = (int)q_heads;
    p.group = (int)(q_heads / kv_heads);
    p.q_tiles = (int)((q_seq + FA::BM - 1) / FA::BM);
    const int64_t items = (int64_t)p.q_tiles * p.group;
    if (items >= kMaxDim / (batch * kv_heads))
        return GEMMRELU_ERR_INVALID_ARG;
    p.kv_heads = (int)kv_heads;
    p.batch = (int)batch;
    p.items = (int)items;
    p.pairs = (int)((items + 1) / 2);
    const int64_t heads = batch * kv_heads;
    const int64_t fit = std::max<int64_t>(1, kWindowChunkBytes / (kv_seq * head_dim * 4));
    const int64_t chunks = (heads + fit - 1) / fit;
    p.chunk = (int)((heads + chunks - 1) / chunks);
    p.chunk_items = p.chunk * p.pairs;
    p.by_chunk = FA::Divisor::of(p.chunk);
    p.by_last = FA::Divisor::of(heads % p.chunk ? heads % p.chunk : p.chunk);
    p.by_chunk_items = FA::Divisor::of(p.chunk_items);
    p.by_kv_heads = FA::Divisor::of(p.kv_heads);
    p.by_group = FA::Divisor::of(p.group);
    p.window = (int)std::min<int64_t>(window, (int64_t)1 << 30);
    p.sinks = (int)std::min<int64_t>(sinks, (int64_t)1 << 30);
    p.scale = (float)(1.4426950408889634 / std::sqrt((double)head_dim));
    // Weights stay below 2^8 times a row's largest: 9 + log2(keys that a row can see) keeps their sum
    // below 1/2.  fp16 values are far from fp32's range, and its weights have none to spare.
    const int64_t seen = window > 0 ? std::min(kv_seq, std::min(window, kv_seq) + std::min(sinks, kv_seq)) : kv_seq;
    p.shift = dtype == GEMMRELU_BF16 ? 9.0f + std::ceil(std::log2((float)seen)) : 0.0f;
    p.drop_arrive = g_drop_arrive.load();
    p.wait_limit_ns = wait_limit_ns();
    if (head_dim == 64)
        return dtype == GEMMRELU_BF16
                   ? launch_window<64, true>(mQ, mK, mV, p, ds->sms, s, ds->attr_window[0])
                   : launch_window<64, false>(mQ, mK, mV, p, ds->sms, s, ds->attr_window[1]);
    return dtype == GEMMRELU_BF16
               ? launch_window<128, true>(mQ, mK, mV, p, ds->sms, s, ds->attr_window[2])
               : launch_window<128, false>(mQ, mK, mV, p, ds->sms, s, ds->attr_window[3]);
}

extern "C" int flash_attention_window_debug_blocks(int64_t first, int64_t last, int64_t window,
                                                   int64_t sinks, int *out) {
    const int64_t most = (int64_t)1 << 30;
    if (first < -most || last < first || last >= most || window < 0 || window > most || sinks < 0 ||
        sinks > most || !out)
        return GEMMRELU_ERR_INVALID_ARG;
    const FA::Blocks b = FA::blocks_seen((int)first, (int)last, (int)window, (int)sinks);
    out[0] = b.sinks;
    out[1] = b.low;
    out[2] = b.high;
    return GEMMRELU_OK;
}
