// Attention of one new token per sequence over a paged key-value cache.
#include <math.h>

#include "ep_layer.cuh"

namespace ep {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxDim = 256;

__device__ __forceinline__ float cache_float(__nv_fp8_e4m3 v) { return static_cast<float>(v); }
__device__ __forceinline__ float cache_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float cache_float(__half v) { return __half2float(v); }

// One block per (sequence, query head): each warp takes every kWarps-th key
// with a running maximum and sum, lanes over the head's values; the warps'
// parts are joined at the end.
template <typename T, typename C>
__global__ void __launch_bounds__(32 * kWarps) paged_attention_kernel(AttentionArgs a) {
    __shared__ float part[kWarps][kMaxDim];
    __shared__ float part_m[kWarps], part_l[kWarps];
    dependent_entry();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / a.num_heads, h = blockIdx.x % a.num_heads;
    const int kvh = h / (a.num_heads / a.num_kv_heads);
    const int64_t most = static_cast<int64_t>(a.max_pages) * a.page_size;
    const int64_t len = min(static_cast<int64_t>(max(a.lens[b], 0)), most);
    const int64_t low = a.window > 0 ? max(int64_t{0}, len - a.window) : 0;
    const T* q = static_cast<const T*>(a.q) + b * a.q_ld + h * a.head_dim;
    float qf[kMaxDim / 32], acc[kMaxDim / 32] = {};
#pragma unroll
    for (int j = 0; j < kMaxDim / 32; ++j)
        qf[j] = lane + 32 * j < a.head_dim ? to_float(q[lane + 32 * j]) * a.score_scale : 0.0f;
    float m = -INFINITY, l = 0.0f;
    for (int64_t i = low + warp; i < len; i += kWarps) {
        const int32_t page = a.table[b * a.table_ld + i / a.page_size];
        if (page < 0 || page >= a.num_pages) continue;
        const int64_t place = i % a.page_size;
        const C* k = static_cast<const C*>(a.k) + page * a.k_page + place * a.k_slot + kvh * a.k_head;
        const C* v = static_cast<const C*>(a.v) + page * a.v_page + place * a.v_slot + kvh * a.v_head;
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < kMaxDim / 32; ++j)
            if (lane + 32 * j < a.head_dim) s += qf[j] * cache_float(k[lane + 32 * j]);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
        const float top = fmaxf(m, s);
        const float keep = m == top ? 1.0f : expf(m - top), p = s == top ? 1.0f : expf(s - top);
        m = top;
        l = l * keep + p;
#pragma unroll
        for (int j = 0; j < kMaxDim / 32; ++j)
            if (lane + 32 * j < a.head_dim) acc[j] = acc[j] * keep + p * cache_float(v[lane + 32 * j]);
    }
#pragma unroll
    for (int j = 0; j < kMaxDim / 32; ++j) part[warp][lane + 32 * j] = acc[j];
    if (lane == 0) part_m[warp] = m, part_l[warp] = l;
    __syncthreads();
    float top = -INFINITY, total = 0.0f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_m[w]);
    for (int w = 0; w < kWarps; ++w) total += part_l[w] * (part_m[w] == top ? 1.0f : expf(part_m[w] - top));
    T* out = static_cast<T*>(a.out) + b * a.out_ld + h * a.head_dim;
    for (int d = threadIdx.x; d < a.head_dim; d += 32 * kWarps) {
        float o = 0.0f;
        for (int w = 0; w < kWarps; ++w) o += part[w][d] * (part_m[w] == top ? 1.0f : expf(part_m[w] - top));
        out[d] = from_float<T>(total > 0.0f || total != total ? o / total * a.v_scale : 0.0f);
    }
    if (threadIdx.x == 0 && a.lse) a.lse[blockIdx.x] = total == 0.0f ? -INFINITY : top + logf(total);
}

}  // namespace

int64_t paged_attention_workspace(int, int, int, int) { return 0; }

cudaError_t launch_paged_attention(const AttentionArgs& a, int dtype, int cache_dtype, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(a.B) * a.num_heads), block(32 * kWarps);
    const bool fp8 = cache_dtype == EP_DTYPE_FP8_E4M3;
    auto* kernel = dtype == EP_DTYPE_BF16
                       ? (fp8 ? paged_attention_kernel<__nv_bfloat16, __nv_fp8_e4m3>
                              : paged_attention_kernel<__nv_bfloat16, __nv_bfloat16>)
                       : (fp8 ? paged_attention_kernel<__half, __nv_fp8_e4m3> : paged_attention_kernel<__half, __half>);
    return launch_dependent(kernel, grid, block, 0, stream, a);
}

}  // namespace ep
