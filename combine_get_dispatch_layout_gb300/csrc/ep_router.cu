// Router: top-k experts per token from the logits, their weights, and the
// gradient of the weights back to the logits.
#include <math.h>

#include "ep_layer.cuh"

namespace ep {
namespace {

constexpr int kWarps = 4;   // tokens per block

// A key as an unsigned integer in the same order (-0 with +0); 0 stands for
// an expert that cannot be used (-infinity and NaN: the lowest finite value
// maps above 0, so a row of lowest values still yields experts).
__device__ __forceinline__ uint32_t ordered(float f) {
    if (!(f > -INFINITY)) return 0u;
    const uint32_t u = __float_as_uint(f + 0.0f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

// exp(l - m) for l <= m with m possibly infinite: the logits that equal the
// maximum count 1, so a row of +infinities shares its weight.
__device__ __forceinline__ float exp_below(float l, float m) { return l == m ? 1.0f : expf(l - m); }

__device__ __forceinline__ float usable(float l) { return l == l ? l : -INFINITY; }

// sigmoid(l) without overflow on either side.
__device__ __forceinline__ float sigmoid(float l) {
    const float e = expf(-fabsf(l));
    return (l >= 0.0f ? 1.0f : e) / (1.0f + e);
}

// The scores of a token's chosen experts, one per lane (lane < K, `on` where
// an expert was chosen), up to a factor common to the token when only ratios
// count (renormalize): sigmoid(l) * exp(-c) with c = min(0, largest logit)
// cannot underflow for all of them at once.
__device__ __forceinline__ float chosen_score(float l, bool on, int score, int renormalize, float row_max,
                                              float row_sum) {
    if (score == EP_SCORE_SOFTMAX) {
        if (!renormalize) return on ? exp_below(l, row_max) / row_sum : 0.0f;
        const float m = warp_max(on ? l : -INFINITY);
        return on ? exp_below(l, m) : 0.0f;
    }
    if (!renormalize) return on ? sigmoid(l) : 0.0f;
    const float c = fminf(0.0f, warp_max(on ? l : -INFINITY));
    if (!on) return 0.0f;
    return l >= 0.0f ? 1.0f / (1.0f + expf(-l)) : expf(l - c) / (1.0f + expf(l));
}

// Largest logit of the row and the sum of exp(logit - largest), one warp.
template <typename T>
__device__ __forceinline__ void row_statistics(const T* row, int E, int lane, float& m, float& sum) {
    m = -INFINITY;
    for (int e = lane; e < E; e += 32) m = fmaxf(m, usable(to_float(row[e])));
    m = warp_max(m);
    sum = 0.0f;
    if (m > -INFINITY)
        for (int e = lane; e < E; e += 32) sum += exp_below(usable(to_float(row[e])), m);
    sum = warp_sum(sum);
}

// One warp per token; the token's keys live in shared memory. K rounds of a
// warp-wide maximum, each lane scanning its own keys.
template <typename T>
__global__ void router_topk_kernel(RouterArgs a) {
    extern __shared__ uint32_t keys_all[];
    dependent_entry();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    uint32_t* keys = keys_all + (threadIdx.x >> 5) * a.E;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    const bool by_score = a.bias != nullptr || (a.num_groups > 1 && a.group_top == 2);

    float m = 0.0f, sum = 1.0f;
    if (a.score == EP_SCORE_SOFTMAX && (by_score || !a.renormalize)) row_statistics(row, a.E, lane, m, sum);
    for (int e = lane; e < a.E; e += 32) {
        const float l = usable(to_float(row[e]));
        float key = l;
        if (by_score && l > -INFINITY) {
            key = a.score == EP_SCORE_SOFTMAX ? exp_below(l, m) / sum : sigmoid(l);
            if (a.bias) key += a.bias[e];
        }
        keys[e] = ordered(key);
    }
    __syncwarp();
    if (a.num_groups > 1) {
        // lane g scores group g, reading it from a start of its own (the
        // groups' sizes are mostly powers of two, one bank otherwise)
        const int n = a.E / a.num_groups;
        uint32_t first = 0, second = 0;
        if (lane < a.num_groups)
            for (int i = 0; i < n; ++i) {
                const uint32_t k = keys[lane * n + (i + lane) % n];
                if (k > first) second = first, first = k;
                else if (k > second) second = k;
            }
        uint32_t g = first;
        if (a.group_top == 2 && first) {
            const auto value = [](uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k); };
            g = ordered(value(first) + (second ? value(second) : 0.0f));
        }
        int before = 0;   // groups that come before this one
        for (int j = 0; j < a.num_groups; ++j) {
            const uint32_t o = __shfl_sync(kFullMask, g, j);
            before += o > g || (o == g && j < lane);
        }
        const unsigned kept = __ballot_sync(kFullMask, lane < a.num_groups && before < a.topk_groups);
        for (int e = lane; e < a.E; e += 32)
            if (!((kept >> (e / n)) & 1)) keys[e] = 0;
        __syncwarp();
    }
    int mine = -1;
    for (int k = 0; k < a.K; ++k) {
        uint32_t best = 0;
        int at = 0;
        for (int e = lane; e < a.E; e += 32)
            if (keys[e] > best) best = keys[e], at = e;
        const uint32_t top = __reduce_max_sync(kFullMask, best);
        if (top == 0) break;
        const int e = __reduce_min_sync(kFullMask, best == top ? at : 0x7fffffff);
        if (lane == k) mine = e;
        if (e == at && best == top) keys[e] = 0;
        __syncwarp();
    }
    const bool on = mine >= 0;
    const float l = on ? usable(to_float(row[mine])) : 0.0f;
    float w = chosen_score(l, on, a.score, a.renormalize, m, sum);
    if (a.renormalize) {
        const float total = warp_sum(w);
        if (on) w /= total;
    }
    if (lane < a.K) {
        a.idx[static_cast<int64_t>(t) * a.K + lane] = mine;
        a.weights[static_cast<int64_t>(t) * a.K + lane] = on ? w * a.scale : 0.0f;
    }
}

// One warp per token. A dense row first (zeros, or -p_j sum_k g_k p_k for the
// plain softmax), then each chosen expert's full gradient over it.
template <typename T>
__global__ void router_backward_kernel(RouterBackwardArgs a) {
    dependent_entry();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    T* out = static_cast<T*>(a.grad) + t * a.grad_ld;
    int64_t e64 = -1;
    float g = 0.0f;
    if (lane < a.K) {
        e64 = a.idx[static_cast<int64_t>(t) * a.K + lane];
        g = a.grad_w[static_cast<int64_t>(t) * a.K + lane] * a.scale;
    }
    const bool on = e64 >= 0 && e64 < a.E;
    const int e = on ? static_cast<int>(e64) : -1 - lane;
    const float l = on ? usable(to_float(row[e])) : 0.0f;
    if (!on) g = 0.0f;

    const bool dense = a.score == EP_SCORE_SOFTMAX && !a.renormalize;
    float m = 0.0f, sum = 1.0f;
    if (dense) row_statistics(row, a.E, lane, m, sum);
    float p = chosen_score(l, on, a.score, a.renormalize, m, sum);
    if (a.renormalize) {
        const float total = warp_sum(p);
        p = on ? p / total : 0.0f;
    }
    const float mean = warp_sum(g * p);   // sum_k g_k p_k
    float d;
    if (a.score == EP_SCORE_SOFTMAX) d = a.renormalize ? p * (g - mean) : p * g;
    else d = (a.renormalize ? p * (g - mean) : g * p) * sigmoid(-l);
    // terms of an expert named more than once, in ascending k
    float total = 0.0f;
    for (int k = 0; k < a.K; ++k) {
        const float dk = __shfl_sync(kFullMask, d, k);
        if (__shfl_sync(kFullMask, e, k) == e) total += dk;
    }
    for (int j = lane; j < a.E; j += 32)
        out[j] = from_float<T>(dense && m > -INFINITY ? -mean * exp_below(usable(to_float(row[j])), m) / sum : 0.0f);
    __syncwarp();
    if (on) out[e] = from_float<T>(dense ? total - mean * p : total);
}

}  // namespace

cudaError_t launch_router_topk(const RouterArgs& a, int dtype, cudaStream_t stream) {
    const dim3 grid((a.T + kWarps - 1) / kWarps), block(32 * kWarps);
    const size_t smem = sizeof(uint32_t) * kWarps * a.E;
    auto* kernel = dtype == EP_DTYPE_BF16   ? router_topk_kernel<__nv_bfloat16>
                   : dtype == EP_DTYPE_FP16 ? router_topk_kernel<__half>
                                            : router_topk_kernel<float>;
    if (smem > 48 * 1024) {
        const cudaError_t err =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (err != cudaSuccess) return err;
    }
    return launch_dependent(kernel, grid, block, smem, stream, a);
}

cudaError_t launch_router_topk_backward(const RouterBackwardArgs& a, int dtype, cudaStream_t stream) {
    const dim3 grid((a.T + kWarps - 1) / kWarps), block(32 * kWarps);
    auto* kernel = dtype == EP_DTYPE_BF16   ? router_backward_kernel<__nv_bfloat16>
                   : dtype == EP_DTYPE_FP16 ? router_backward_kernel<__half>
                                            : router_backward_kernel<float>;
    return launch_dependent(kernel, grid, block, 0, stream, a);
}

}  // namespace ep
