// Declarations shared by the translation units of the layer operators
// (include/ep_layer.h): argument blocks, launchers and element conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "../../include/ep_layer.h"
#include "ep_internal.cuh"

namespace ep {

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(float v) { return v; }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }

// Eight 16-bit values as loaded by one 16-byte access.
template <typename T>
union Vec8 {
    uint4 raw;
    T v[8];
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

struct RouterArgs {
    const void* logits;
    int64_t ld;
    const float* bias;
    int T, E, K;
    int score, renormalize;
    float scale;
    int num_groups, topk_groups, group_top;
    int64_t* idx;
    float* weights;
};
cudaError_t launch_router_topk(const RouterArgs& a, int dtype, cudaStream_t stream);

struct RouterBackwardArgs {
    const void* logits;
    int64_t ld;
    const int64_t* idx;
    int64_t idx_ld;
    const float* grad_w;
    int T, E, K;
    int score, renormalize;
    float scale;
    void* grad;
    int64_t grad_ld;
};
cudaError_t launch_router_topk_backward(const RouterBackwardArgs& a, int dtype, cudaStream_t stream);

struct AppendArgs {
    const void *q, *k, *v;
    const int64_t *positions, *slots;
    const float* cos_sin;
    int T, num_heads, num_kv_heads, head_dim, rotary_dim, interleaved;
    int64_t q_ld, k_ld, v_ld, q_out_ld, max_position;
    void *q_out, *k_cache, *v_cache;
    int page_size;
    int64_t num_slots;
    int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;
    float k_inv_scale, v_inv_scale;
    int32_t* error;
};
cudaError_t launch_kv_append(const AppendArgs& a, int dtype, int cache_dtype, cudaStream_t stream);

struct AttentionArgs {
    const void *q, *k, *v;
    const int32_t* table;
    const int32_t* lens;
    int B, num_heads, num_kv_heads, head_dim;
    int page_size, max_pages, window;
    int64_t num_pages, table_ld, q_ld, out_ld;
    int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;
    float score_scale;   // scale * k_scale
    float v_scale;
    void* out;
    float* lse;
    void* workspace;
};
cudaError_t launch_paged_attention(const AttentionArgs& a, int dtype, int cache_dtype, cudaStream_t stream);
// Bytes of workspace for these sizes on the current device, -1 on a CUDA error.
int64_t paged_attention_workspace(int B, int num_heads, int num_kv_heads, int head_dim);

struct W4Args {
    const void* x;
    const uint8_t* w;
    const void* scales;
    const uint8_t* zeros;
    const int32_t* offsets;
    const int32_t* counts;
    int rows, I, E, O;
    int group, swiglu;
    int64_t x_ld, y_ld;
    void* y;
};
cudaError_t launch_expert_w4(const W4Args& a, void* workspace, int dtype, cudaStream_t stream);
int64_t expert_w4_workspace(int64_t rows, int I, int group, int dtype);

}  // namespace ep
