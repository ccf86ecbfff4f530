// C ABI of the layer operators (include/ep_layer.h): argument checks and
// launches. Nothing is kept between calls.
#include <cmath>
#include <cstdint>

#include <nvtx3/nvToolsExt.h>

#include "ep_layer.cuh"

namespace {

struct ApiRange {
    explicit ApiRange(const char* name) { nvtxRangePushA(name); }
    ~ApiRange() { nvtxRangePop(); }
    ApiRange(const ApiRange&) = delete;
    ApiRange& operator=(const ApiRange&) = delete;
};

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline ep_status_t status_of(cudaError_t err) { return err == cudaSuccess ? EP_OK : EP_ERR_CUDA; }
inline bool half_type(int d) { return d == EP_DTYPE_BF16 || d == EP_DTYPE_FP16; }
inline bool router_type(int d) { return half_type(d) || d == EP_DTYPE_FP32; }
inline size_t type_bytes(int d) { return d == EP_DTYPE_FP32 ? 4 : d == EP_DTYPE_FP8_E4M3 ? 1 : 2; }

constexpr int kMostSide = INT32_MAX - 511;   // rows, inputs and outputs of the experts: whole tiles of them are counted in an int

bool router_config_ok(const ep_router_config_t* c) {
    return c && router_type(c->logits_dtype) && (c->score == EP_SCORE_SOFTMAX || c->score == EP_SCORE_SIGMOID) &&
           std::isfinite(c->scale);
}

// A cache whose rows of `dim` elements all start on 16 bytes.
bool cache_ok(const ep_cache_t* c, int dtype, int dim) {
    if (!c || (c->dtype != dtype && c->dtype != EP_DTYPE_FP8_E4M3)) return false;
    const int64_t unit = 16 / static_cast<int64_t>(type_bytes(c->dtype));
    if (dim % unit != 0 || c->page_size < 1 || c->num_pages < 0 ||
        c->num_pages >= (int64_t{1} << 40) / c->page_size || c->num_pages >= (int64_t{1} << 31))
        return false;
    for (const int64_t s : {c->k_page_stride, c->k_slot_stride, c->k_head_stride, c->v_page_stride, c->v_slot_stride,
                            c->v_head_stride})
        if (s < 0 || s % unit != 0) return false;
    if (c->dtype == EP_DTYPE_FP8_E4M3 && !(std::isfinite(c->k_scale) && c->k_scale > 0 && std::isfinite(c->v_scale) &&
                                           c->v_scale > 0))
        return false;
    return true;
}

}  // namespace

extern "C" {

ep_status_t ep_router_topk(const void* logits, int64_t logits_ld, const float* bias, int T, int E, int K,
                           const ep_router_config_t* config, int64_t* topk_idx, float* topk_weights, void* stream) {
    ApiRange range("ep_router_topk");
    if (!router_config_ok(config) || T < 0 || E < 1 || E > EP_MAX_EXPERTS || K < 1 || K > EP_MAX_TOPK || logits_ld < E)
        return EP_ERR_INVALID_ARG;
    const int groups = config->num_groups > 0 ? config->num_groups : 1;
    if (config->num_groups < 0 || groups > 32 || E % groups != 0 || config->group_top < 0 || config->group_top > 2 ||
        (groups > 1 && (config->topk_groups < 1 || config->topk_groups > groups)))
        return EP_ERR_INVALID_ARG;
    if (T == 0) return EP_OK;
    if (!logits || !topk_idx || !topk_weights || !aligned(logits, type_bytes(config->logits_dtype)) ||
        !aligned(bias, 4) || !aligned(topk_idx, 8) || !aligned(topk_weights, 4))
        return EP_ERR_INVALID_ARG;
    ep::RouterArgs a{};
    a.logits = logits;
    a.ld = logits_ld;
    a.bias = bias;
    a.T = T;
    a.E = E;
    a.K = K;
    a.score = config->score;
    a.renormalize = config->renormalize;
    a.scale = config->scale;
    a.num_groups = groups;
    a.topk_groups = config->topk_groups;
    a.group_top = config->group_top ? config->group_top : 1;
    a.idx = topk_idx;
    a.weights = topk_weights;
    return status_of(ep::launch_router_topk(a, config->logits_dtype, static_cast<cudaStream_t>(stream)));
}

ep_status_t ep_router_topk_backward(const void* logits, int64_t logits_ld, const int64_t* topk_idx, int64_t topk_ld,
                                    const float* grad_weights, int T, int E, int K, const ep_router_config_t* config,
                                    void* grad_logits, int64_t grad_ld, void* stream) {
    ApiRange range("ep_router_topk_backward");
    if (!router_config_ok(config) || T < 0 || E < 1 || E > EP_MAX_EXPERTS || K < 1 || K > EP_MAX_TOPK ||
        logits_ld < E || grad_ld < E || topk_ld < K)
        return EP_ERR_INVALID_ARG;
    if (T == 0) return EP_OK;
    const size_t bytes = type_bytes(config->logits_dtype);
    if (!logits || !topk_idx || !grad_weights || !grad_logits || !aligned(logits, bytes) ||
        !aligned(grad_logits, bytes) || !aligned(topk_idx, 8) || !aligned(grad_weights, 4))
        return EP_ERR_INVALID_ARG;
    ep::RouterBackwardArgs a{};
    a.logits = logits;
    a.ld = logits_ld;
    a.idx = topk_idx;
    a.idx_ld = topk_ld;
    a.grad_w = grad_weights;
    a.T = T;
    a.E = E;
    a.K = K;
    a.score = config->score;
    a.renormalize = config->renormalize;
    a.scale = config->scale;
    a.grad = grad_logits;
    a.grad_ld = grad_ld;
    return status_of(ep::launch_router_topk_backward(a, config->logits_dtype, static_cast<cudaStream_t>(stream)));
}

ep_status_t ep_kv_append(const void* q, const void* k, const void* v, const int64_t* positions, const int64_t* slots,
                         const float* cos_sin, int T, const ep_append_config_t* config, void* q_out, void* k_cache,
                         void* v_cache, const ep_cache_t* cache, int32_t* device_error, void* stream) {
    ApiRange range("ep_kv_append");
    if (!config || !half_type(config->dtype) || T < 0) return EP_ERR_INVALID_ARG;
    const int D = config->head_dim, rot = config->rotary_dim;
    if (D < 8 || D > 1024 || D % 8 != 0 || rot < 0 || rot > D || rot % 2 != 0 || config->num_heads < 0 ||
        config->num_kv_heads < 1 || !cache_ok(cache, config->dtype, D) || !aligned(device_error, 4) ||
        (rot > 0 && config->max_position < 1))
        return EP_ERR_INVALID_ARG;
    const bool fp8 = cache->dtype == EP_DTYPE_FP8_E4M3;
    if (fp8 && !(std::isfinite(1.0f / cache->k_scale) && std::isfinite(1.0f / cache->v_scale))) return EP_ERR_INVALID_ARG;
    const int64_t q_row = static_cast<int64_t>(config->num_heads) * D, kv_row = static_cast<int64_t>(config->num_kv_heads) * D;
    if (q_row + 2 * kv_row >= (int64_t{1} << 28) || config->k_ld < kv_row || config->v_ld < kv_row ||
        config->k_ld % 8 != 0 || config->v_ld % 8 != 0)
        return EP_ERR_INVALID_ARG;
    if (config->num_heads > 0 && (config->q_ld < q_row || config->q_out_ld < q_row || config->q_ld % 8 != 0 ||
                                  config->q_out_ld % 8 != 0))
        return EP_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T > 0) {
        if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return EP_ERR_INVALID_ARG;
        if (rot > 0 && (!positions || !cos_sin)) return EP_ERR_INVALID_ARG;
        if (!aligned(positions, 8) || !aligned(cos_sin, 4)) return EP_ERR_INVALID_ARG;
        if (config->num_heads > 0 && (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16)))
            return EP_ERR_INVALID_ARG;
        if (cache->num_pages > 0 && (!k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16)))
            return EP_ERR_INVALID_ARG;
    }
    if (device_error && cudaMemsetAsync(device_error, 0, sizeof(int32_t), s) != cudaSuccess) return EP_ERR_CUDA;
    if (T == 0) return EP_OK;
    ep::AppendArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.positions = positions;
    a.slots = slots;
    a.cos_sin = cos_sin;
    a.T = T;
    a.num_heads = config->num_heads;
    a.num_kv_heads = config->num_kv_heads;
    a.head_dim = D;
    a.rotary_dim = rot;
    a.interleaved = config->interleaved;
    a.q_ld = config->q_ld;
    a.k_ld = config->k_ld;
    a.v_ld = config->v_ld;
    a.q_out_ld = config->q_out_ld;
    a.max_position = config->max_position;
    a.q_out = q_out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.page_size = cache->page_size;
    a.num_slots = cache->num_pages * cache->page_size;
    a.k_page = cache->k_page_stride;
    a.k_slot = cache->k_slot_stride;
    a.k_head = cache->k_head_stride;
    a.v_page = cache->v_page_stride;
    a.v_slot = cache->v_slot_stride;
    a.v_head = cache->v_head_stride;
    a.k_inv_scale = fp8 ? 1.0f / cache->k_scale : 1.0f;
    a.v_inv_scale = fp8 ? 1.0f / cache->v_scale : 1.0f;
    a.error = device_error;
    return status_of(ep::launch_kv_append(a, config->dtype, cache->dtype, s));
}

int64_t ep_paged_attention_workspace(int B, int num_heads, int num_kv_heads, int head_dim) {
    if (B < 0 || num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads != 0 || head_dim < 8 ||
        head_dim > 256 || head_dim % 8 != 0 || static_cast<int64_t>(B) * num_heads >= (int64_t{1} << 31))
        return -1;
    return ep::paged_attention_workspace(B, num_heads, num_kv_heads, head_dim);
}

ep_status_t ep_paged_attention(const void* q, const void* k_cache, const void* v_cache, const ep_cache_t* cache,
                               const int32_t* block_table, const int32_t* seq_lens, int B,
                               const ep_attention_config_t* config, void* out, float* lse, void* workspace,
                               int64_t workspace_bytes, void* stream) {
    ApiRange range("ep_paged_attention");
    if (!config || !half_type(config->dtype) || B < 0) return EP_ERR_INVALID_ARG;
    const int D = config->head_dim, H = config->num_heads;
    if (D < 8 || D > 256 || D % 8 != 0 || H < 1 || config->num_kv_heads < 1 || H % config->num_kv_heads != 0 ||
        static_cast<int64_t>(B) * H >= (int64_t{1} << 31) || static_cast<int64_t>(H) * D >= (int64_t{1} << 28) ||
        !cache_ok(cache, config->dtype, D) || config->max_pages < 0 ||
        static_cast<int64_t>(config->max_pages) * cache->page_size >= (int64_t{1} << 31) || config->window < 0 ||
        !std::isfinite(config->scale))
        return EP_ERR_INVALID_ARG;
    const int64_t row = static_cast<int64_t>(H) * D;
    if (config->q_ld < row || config->out_ld < row || config->q_ld % 8 != 0 || config->out_ld % 8 != 0 ||
        config->table_ld < config->max_pages)
        return EP_ERR_INVALID_ARG;
    if (B == 0) return EP_OK;
    if (!q || !out || !seq_lens || !aligned(q, 16) || !aligned(out, 16) || !aligned(seq_lens, 4) || !aligned(lse, 4) ||
        !aligned(workspace, 16) || !aligned(block_table, 4) || (config->max_pages > 0 && !block_table))
        return EP_ERR_INVALID_ARG;
    if (cache->num_pages > 0 && (!k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16)))
        return EP_ERR_INVALID_ARG;
    const int64_t need = ep::paged_attention_workspace(B, H, config->num_kv_heads, D);
    if (need < 0) return EP_ERR_CUDA;
    if (need > 0 && (!workspace || workspace_bytes < need)) return EP_ERR_INVALID_ARG;
    ep::AttentionArgs a{};
    a.q = q;
    a.k = k_cache;
    a.v = v_cache;
    a.table = block_table;
    a.lens = seq_lens;
    a.B = B;
    a.num_heads = H;
    a.num_kv_heads = config->num_kv_heads;
    a.head_dim = D;
    a.page_size = cache->page_size;
    a.max_pages = config->max_pages;
    a.window = config->window;
    a.num_pages = cache->num_pages;
    a.table_ld = config->table_ld;
    a.q_ld = config->q_ld;
    a.out_ld = config->out_ld;
    a.k_page = cache->k_page_stride;
    a.k_slot = cache->k_slot_stride;
    a.k_head = cache->k_head_stride;
    a.v_page = cache->v_page_stride;
    a.v_slot = cache->v_slot_stride;
    a.v_head = cache->v_head_stride;
    const bool fp8 = cache->dtype == EP_DTYPE_FP8_E4M3;
    a.score_scale = fp8 ? config->scale * cache->k_scale : config->scale;
    a.v_scale = fp8 ? cache->v_scale : 1.0f;
    a.out = out;
    a.lse = lse;
    a.workspace = workspace;
    return status_of(ep::launch_paged_attention(a, config->dtype, cache->dtype, static_cast<cudaStream_t>(stream)));
}

int64_t ep_expert_w4_workspace(int64_t rows, int I, int group_size, int dtype) {
    if (rows < 0 || rows > kMostSide || (group_size != 32 && group_size != 64 && group_size != 128) ||
        I < group_size || I > kMostSide || I % group_size != 0 || !half_type(dtype))
        return -1;
    return ep::expert_w4_workspace(rows, I, group_size, dtype);
}

ep_status_t ep_expert_w4(const void* x, int64_t rows, int I, const uint8_t* weights, const void* scales,
                         const uint8_t* zeros, const int32_t* expert_offsets, const int32_t* expert_counts, int E,
                         int O, const ep_w4_config_t* config, void* y, void* workspace, int64_t workspace_bytes,
                         void* stream) {
    ApiRange range("ep_expert_w4");
    if (!config || !half_type(config->dtype) || rows < 0) return EP_ERR_INVALID_ARG;
    const int group = config->group_size;
    const bool swiglu = config->activation == EP_ACT_SWIGLU;
    if ((group != 32 && group != 64 && group != 128) || I < group || I % group != 0 || O < 1 ||
        (!swiglu && config->activation != EP_ACT_NONE) || (swiglu && O % 2 != 0) || E < 1 || E > EP_MAX_EXPERTS)
        return EP_ERR_INVALID_ARG;
    if (rows > kMostSide || I > kMostSide || O > kMostSide) return EP_ERR_INVALID_ARG;
    if (config->x_ld < I || config->x_ld % 8 != 0 || config->y_ld < (swiglu ? O / 2 : O)) return EP_ERR_INVALID_ARG;
    if (!expert_offsets && (E != 1 || expert_counts)) return EP_ERR_INVALID_ARG;
    if (rows == 0) return EP_OK;
    if (!x || !weights || !scales || !y || !aligned(x, 16) || !aligned(weights, 16) || !aligned(scales, 2) ||
        !aligned(y, 2) || !aligned(expert_offsets, 4) || !aligned(expert_counts, 4))
        return EP_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < ep::expert_w4_workspace(rows, I, group, config->dtype))
        return EP_ERR_INVALID_ARG;
    ep::W4Args a{};
    a.x = x;
    a.w = weights;
    a.scales = scales;
    a.zeros = zeros;
    a.offsets = expert_offsets;
    a.counts = expert_counts;
    a.rows = static_cast<int>(rows);
    a.I = I;
    a.E = E;
    a.O = O;
    a.group = group;
    a.swiglu = swiglu;
    a.x_ld = config->x_ld;
    a.y_ld = config->y_ld;
    a.y = y;
    return status_of(ep::launch_expert_w4(a, workspace, config->dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
