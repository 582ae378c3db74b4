// flash_attention_window_api.cuh -- host side of flash_attention_window_x16: argument checks,
// tensor maps and launch (part of the translation unit of gemm_relu_api.cu).
#pragma once

#include "flash_attention_window.cuh"
#include "cross_step.cuh"

namespace {

// A [batch][seq][heads][d] tensor of 16-bit elements with strides {sequence, token,
// head}: boxes of 64 d x 1 head x 128 tokens (or box_heads x box_tokens), 128-byte swizzle, zero fill
// outside.  An axis of one element is never stepped over, whatever its stride.
bool make_strided_map(CUtensorMap *map, const void *ptr, int dtype, int64_t batch, int64_t seq,
                      int64_t heads, int64_t d, const int64_t *strides, int box_heads = 1,
                      int box_tokens = FA::BM) {
    EncodeTiledFn enc = encode_fn();
    if (!enc)
        return false;
    auto bytes = [&](int64_t n, int64_t stride) { return (cuuint64_t)(n == 1 ? d : stride) * 2; };
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)seq, (cuuint64_t)batch};
    cuuint64_t step[3] = {bytes(heads, strides[2]), bytes(seq, strides[1]), bytes(batch, strides[0])};
    cuuint32_t box[4] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens, 1};
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

template <int HD, bool kBf16, bool kCross>
int launch_window(const CUtensorMap &mQ, const CUtensorMap &mK, const CUtensorMap &mV,
                  const FA::WindowParams &p, int sms, cudaStream_t stream, bool &attr_done) {
    auto kern = FA::flash_attention_window_kernel<HD, kBf16, kCross>;
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

// How a step of cross attention is cut: none (0) for more rows than a step has.
struct StepSplit {
    int rows, parts;      // rows of a head; parts of its states
    size_t bytes;         // of workspace
};

// Parts of a head's states: as many as run at once, a unit of 64 keys at least.  (13 sequences of up to 1500 states, 8 heads of
// 128: 14.9 us, and 19.5 cut for twice as many blocks; 16 rows a head 16.5 and 24.1.)
StepSplit step_split(int64_t batch, int64_t q_seq, int64_t kv_seq, int64_t q_heads, int64_t kv_heads,
                     int64_t head_dim, int sms) {
    StepSplit s{0, 1, 0};
    const int64_t group = q_heads / kv_heads;
    if (q_seq > FA::kStepMostRows || q_seq * group > FA::kStepMostRows)
        return s;
    s.rows = (int)(q_seq * group);
    const int64_t heads = batch * kv_heads, units = (kv_seq + FA::kStepKeys - 1) / FA::kStepKeys;
    const bool few = s.rows <= 8;
    const int64_t slots = (int64_t)sms * (head_dim == 64 ? few ? FA::StepCfg<64, 1>::kBlocksPerSm : FA::StepCfg<64, 2>::kBlocksPerSm
                                                         : few ? FA::StepCfg<128, 1>::kBlocksPerSm : FA::StepCfg<128, 2>::kBlocksPerSm);
    // One block joins all parts of a head, about as long a part as a stage of states takes: no more parts than stages of one.
    // (One row on 30000 states, one head of 64: 13.7 us, 57 with a block on every SM slot; 16 rows on 1774, 10 heads of 128: 12.7 and
    // 24; one on 700, 16 heads of 64: 6.6 and 7.6; twice the square root: 13.1, 12.0 and 7.0.)
    const int64_t most = (int64_t)std::ceil(std::sqrt((double)units));
    if (heads <= FA::kStepCounters)
        s.parts = (int)std::max<int64_t>(1, std::min({slots / heads, units, most}));
    if (s.parts > 1)
        s.bytes = GEMMRELU_CROSS_COUNTER_BYTES +
                  (size_t)heads * s.parts * (few ? 8 : 16) * (head_dim + 4) * sizeof(float);
    return s;
}

template <int D, int kN, bool kBf16>
int launch_step(const CUtensorMap &mK, const CUtensorMap &mV, const FA::StepParams &p, int64_t blocks, cudaStream_t s,
                bool &attr_done) {
    auto kern = FA::cross_step_kernel<D, kN, kBf16>;
    if (!ensure_smem_attr(attr_done, kern, FA::StepCfg<D, kN>::kSmem))
        return GEMMRELU_ERR_LAUNCH;
    return launch_kernel(kern, (unsigned)blocks, (unsigned)FA::kStepThreads, FA::StepCfg<D, kN>::kSmem, s, false, 1u, mK,
                         mV, p);
}

template <int D>
int launch_step_as(int dtype, const CUtensorMap &mK, const CUtensorMap &mV, const FA::StepParams &p, int64_t blocks,
                   cudaStream_t s, bool *attr) {
    if (p.rows <= 8)
        return dtype == GEMMRELU_BF16 ? launch_step<D, 1, true>(mK, mV, p, blocks, s, attr[0])
                                      : launch_step<D, 1, false>(mK, mV, p, blocks, s, attr[1]);
    return dtype == GEMMRELU_BF16 ? launch_step<D, 2, true>(mK, mV, p, blocks, s, attr[2])
                                  : launch_step<D, 2, false>(mK, mV, p, blocks, s, attr[3]);
}

template <bool kCross>
int launch_window_as(int dtype, int64_t head_dim, const CUtensorMap &mQ, const CUtensorMap &mK, const CUtensorMap &mV,
                     const FA::WindowParams &p, int sms, cudaStream_t s, bool *attr) {
    if (head_dim == 64)
        return dtype == GEMMRELU_BF16 ? launch_window<64, true, kCross>(mQ, mK, mV, p, sms, s, attr[0])
                                      : launch_window<64, false, kCross>(mQ, mK, mV, p, sms, s, attr[1]);
    return dtype == GEMMRELU_BF16 ? launch_window<128, true, kCross>(mQ, mK, mV, p, sms, s, attr[2])
                                  : launch_window<128, false, kCross>(mQ, mK, mV, p, sms, s, attr[3]);
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

// flash_attention_window_x16, and flash_attention_cross_x16 (kCross: no window or sinks; `states` keys a
// sequence).
template <bool kCross>
static int attention_strided(const void *Q, const void *K, const void *V, void *O, int dtype, int64_t batch,
                             int64_t q_seq, int64_t kv_seq, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                             const int64_t *q_strides, const int64_t *k_strides, const int64_t *v_strides,
                             int64_t window, int64_t sinks, const int32_t *states, void *workspace,
                             size_t workspace_bytes, void *stream) {
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
    const int64_t group = q_heads / kv_heads;
    if (kCross && (group > FA::BM || !aligned(states, 4)))
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
    if (kv_seq == 0) {   // nobody sees anything
        const int set = launch_status(cudaMemsetAsync(O, 0, (size_t)(batch * q_seq * q_heads * head_dim) * 2, s));
        if (set != GEMMRELU_OK || states == nullptr)
            return set;
        return launch_kernel(FA::cross_no_states_kernel, (unsigned)((batch + 255) / 256), 256u, 0u, s, false, 1u, states,
                             (int)batch);
    }
    const int tile_tokens = kCross ? (int)(FA::BM / group) : FA::BM;
    // Weights stay below 2^8 times a row's largest: 9 + log2(keys that a row can see) keeps their sum
    // below 1/2.  fp16 values are far from fp32's range, and its weights have none to spare.
    const int64_t seen = window > 0 ? std::min(kv_seq, std::min(window, kv_seq) + std::min(sinks, kv_seq)) : kv_seq;
    const float shift = dtype == GEMMRELU_BF16 ? 9.0f + std::ceil(std::log2((float)seen)) : 0.0f;
    const double scale = 1.4426950408889634 / std::sqrt((double)head_dim);
    CUtensorMap mQ, mK, mV;
    const StepSplit step = kCross ? step_split(batch, q_seq, kv_seq, q_heads, kv_heads, head_dim, ds->sms) : StepSplit{0, 1, 0};
    if (step.rows > 0) {
        const int64_t blocks = batch * kv_heads * step.parts;
        if (blocks > 0x7fffffff)
            return GEMMRELU_ERR_INVALID_ARG;
        if (step.bytes > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < step.bytes))
            return GEMMRELU_ERR_WORKSPACE;
        if (!make_strided_map(&mK, K, dtype, batch, kv_seq, kv_heads, head_dim, k_strides, 1, FA::kStepKeys) ||
            !make_strided_map(&mV, V, dtype, batch, kv_seq, kv_heads, head_dim, v_strides, 1, FA::kStepKeys))
            return GEMMRELU_ERR_LAUNCH;
        FA::StepParams p{};
        p.q = static_cast<const uint16_t *>(Q);
        const int64_t n[3] = {batch, q_seq, q_heads};
        for (int i = 0; i < 3; ++i)
            p.qs[i] = n[i] > 1 ? q_strides[i] : 0;
        p.o = static_cast<uint16_t *>(O);
        p.states = states;
        p.n_q = (int)q_seq;
        p.n_kv = (int)kv_seq;
        p.q_heads = (int)q_heads;
        p.kv_heads = (int)kv_heads;
        p.group = (int)group;
        p.rows = step.rows;
        p.parts = step.parts;
        p.scale = (float)scale;
        p.slack = (float)(FA::kRescaleLog2 / scale);
        p.shift = shift;
        p.arrived = static_cast<unsigned *>(workspace);
        p.partial = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + GEMMRELU_CROSS_COUNTER_BYTES);
        p.drop_arrive = g_drop_arrive.load();
        p.wait_limit_ns = wait_limit_ns();
        return head_dim == 64 ? launch_step_as<64>(dtype, mK, mV, p, blocks, s, ds->attr_step)
                              : launch_step_as<128>(dtype, mK, mV, p, blocks, s, ds->attr_step + 4);
    }
    if (!make_strided_map(&mQ, Q, dtype, batch, q_seq, q_heads, head_dim, q_strides, kCross ? (int)group : 1,
                          tile_tokens) ||
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
    p.group = (int)group;
    p.states = states;
    p.tile_tokens = tile_tokens;
    p.q_tiles = (int)((q_seq + tile_tokens - 1) / tile_tokens);
    const int64_t items = kCross ? p.q_tiles : (int64_t)p.q_tiles * p.group;
    if (items >= kMaxDim / (batch * kv_heads))
        return GEMMRELU_ERR_INVALID_ARG;
    p.kv_heads = (int)kv_heads;
    p.batch = (int)batch;
    p.items = (int)items;
    p.pairs = (int)((items + 1) / 2);
    const int64_t heads = batch * kv_heads;
    // (cross attention: a head's items see the same keys, so one head after the other falls in cost over all of them, as
    // the order by length has it)
    const int64_t fit = kCross ? 1 : std::max<int64_t>(1, kWindowChunkBytes / (kv_seq * head_dim * 4));
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
    p.scale = (float)scale;
    p.shift = shift;
    p.drop_arrive = g_drop_arrive.load();
    p.wait_limit_ns = wait_limit_ns();
    return launch_window_as<kCross>(dtype, head_dim, mQ, mK, mV, p, ds->sms, s,
                                    kCross ? ds->attr_cross : ds->attr_window);
}

extern "C" int flash_attention_window_x16(const void *Q, const void *K, const void *V, void *O,
                                          int dtype, int64_t batch, int64_t q_seq, int64_t kv_seq,
                                          int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                          const int64_t *q_strides, const int64_t *k_strides,
                                          const int64_t *v_strides, int64_t window, int64_t sinks,
                                          void *stream) {
    return attention_strided<false>(Q, K, V, O, dtype, batch, q_seq, kv_seq, q_heads, kv_heads, head_dim, q_strides,
                                    k_strides, v_strides, window, sinks, nullptr, nullptr, 0, stream);
}

extern "C" int flash_attention_cross_x16(const void *Q, const void *K, const void *V, void *O, int dtype,
                                         int64_t batch, int64_t q_seq, int64_t kv_seq, int64_t q_heads,
                                         int64_t kv_heads, int64_t head_dim, const int64_t *q_strides,
                                         const int64_t *k_strides, const int64_t *v_strides,
                                         const int32_t *lengths, void *workspace, size_t workspace_bytes,
                                         void *stream) {
    return attention_strided<true>(Q, K, V, O, dtype, batch, q_seq, kv_seq, q_heads, kv_heads, head_dim, q_strides,
                                   k_strides, v_strides, 0, 0, lengths, workspace, workspace_bytes, stream);
}

extern "C" size_t flash_attention_cross_x16_workspace_bytes(int64_t batch, int64_t q_seq, int64_t kv_seq,
                                                            int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
    DeviceState *ds = nullptr;
    if (batch < 1 || batch > 65535 || q_seq < 1 || kv_seq < 1 || kv_seq > ((int64_t)1 << 30) || q_heads < 1 ||
        q_heads > 65535 || kv_heads < 1 || q_heads % kv_heads != 0 || (head_dim != 64 && head_dim != 128) ||
        current_device_state(&ds) != GEMMRELU_OK)
        return 0;
    return step_split(batch, q_seq, kv_seq, q_heads, kv_heads, head_dim, ds->sms).bytes;
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
