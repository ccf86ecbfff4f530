// Router: top-k experts per token from the logits, their weights, and the
// gradient of the weights back to the logits.
//
// One warp a token. Up to 512 experts the token's keys stay in registers (V a
// lane, expert 32 j + lane), so the row is read once; K rounds of a warp-wide
// maximum pick the experts, each lane rescanning its own V keys. Larger rows go
// through shared memory. Memory bounds neither (a row is a kilobyte): what
// counts is the chain of each warp's steps, and with few tokens the launch.
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

// The number that a key above 0 stands for.
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k); }

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

// A group's score from its largest and second largest keys.
__device__ __forceinline__ uint32_t group_score(uint32_t first, uint32_t second, int group_top) {
    if (group_top != 2 || first == 0) return first;
    return ordered(value_of(first) + (second ? value_of(second) : 0.0f));
}
// Lane g holds group g's score: the groups with the largest ones, equal ones in order, as a mask.
__device__ __forceinline__ unsigned kept_groups(uint32_t score, int groups, int keep, int lane) {
    int before = 0;
    for (int j = 0; j < groups; ++j) {
        const uint32_t o = __shfl_sync(kFullMask, score, j);
        before += o > score || (o == score && j < lane);
    }
    return __ballot_sync(kFullMask, lane < groups && before < keep);
}

// The weights of the chosen experts (lane k: the k-th, its logit l), and both outputs.
__device__ __forceinline__ void write_choice(const RouterArgs& a, int t, int lane, int mine, float l, float row_max, float row_sum) {
    const bool on = mine >= 0;
    float w = chosen_score(l, on, a.score, a.renormalize, row_max, row_sum);
    if (a.renormalize) {
        const float total = warp_sum(w);
        if (on) w /= total;
    }
    if (lane < a.K) {
        a.idx[static_cast<int64_t>(t) * a.K + lane] = mine;
        a.weights[static_cast<int64_t>(t) * a.K + lane] = on ? w * a.scale : 0.0f;
    }
}

// Keys in registers. Groups of experts that are not a power of two up to 32 go through router_topk_kernel.
template <typename T, int V>
__global__ void __launch_bounds__(32 * kWarps) router_topk_registers_kernel(RouterArgs a) {
    dependent_entry();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    const bool by_score = a.bias != nullptr || (a.num_groups > 1 && a.group_top == 2);
    float l[V];
#pragma unroll
    for (int j = 0; j < V; ++j) l[j] = 32 * j + lane < a.E ? usable(to_float(row[32 * j + lane])) : -INFINITY;
    float m = 0.0f, sum = 1.0f;
    if (a.score == EP_SCORE_SOFTMAX && (by_score || !a.renormalize)) {
        m = l[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
        m = warp_max(m);
        sum = 0.0f;
        if (m > -INFINITY) {
#pragma unroll
            for (int j = 0; j < V; ++j) sum += exp_below(l[j], m);
        }
        sum = warp_sum(sum);
    }
    uint32_t keys[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float key = l[j];
        if (by_score && key > -INFINITY) {
            key = a.score == EP_SCORE_SOFTMAX ? exp_below(l[j], m) / sum : sigmoid(l[j]);
            if (a.bias) key += a.bias[32 * j + lane];
        }
        keys[j] = ordered(key);
    }
    if (a.num_groups > 1) {
        // n neighbouring lanes hold a group: its two largest keys by exchange, then lane g takes group g's
        const int n = a.E / a.num_groups;
        uint32_t score = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            uint32_t first = keys[j], second = 0;
            for (int o = 1; o < n; o <<= 1) {
                const uint32_t f = __shfl_xor_sync(kFullMask, first, o), s = __shfl_xor_sync(kFullMask, second, o);
                second = max(min(first, f), max(second, s));
                first = max(first, f);
            }
            const uint32_t g = group_score(first, second, a.group_top);
            const uint32_t taken = __shfl_sync(kFullMask, g, lane * n & 31);
            if (lane * n >> 5 == j) score = taken;
        }
        const unsigned kept = kept_groups(score, a.num_groups, a.topk_groups, lane);
        const int log = 31 - __clz(n);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (!((kept >> min(31, (32 * j + lane) >> log)) & 1)) keys[j] = 0;
    }
    int mine = -1;
    uint32_t my_key = 0;
    uint32_t best = 0;
    int at = 0;
    const auto scan = [&]() {
        best = 0;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (keys[j] > best) best = keys[j], at = 32 * j + lane;
    };
    scan();
    for (int k = 0; k < a.K; ++k) {
        const uint32_t top = __reduce_max_sync(kFullMask, best);
        if (top == 0) break;
        const int e = __reduce_min_sync(kFullMask, best == top ? at : 0x7fffffff);
        if (lane == k) mine = e, my_key = top;
        if (e == at && best == top) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (32 * j + lane == e) keys[j] = 0;
            scan();
        }
    }
    // (a key that is the logit gives it back; otherwise the row has it)
    const float chosen = mine < 0 ? 0.0f : by_score ? usable(to_float(row[mine])) : value_of(my_key);
    write_choice(a, t, lane, mine, chosen, m, sum);
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
            for (int i = 0, at = lane % n; i < n; ++i, at = at + 1 == n ? 0 : at + 1) {
                const uint32_t k = keys[lane * n + at];
                if (k > first) second = first, first = k;
                else if (k > second) second = k;
            }
        const uint32_t g = group_score(first, second, a.group_top);
        const unsigned kept = kept_groups(g, a.num_groups, a.topk_groups, lane);
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
    write_choice(a, t, lane, mine, mine >= 0 ? usable(to_float(row[mine])) : 0.0f, m, sum);
}

// One warp per token. A dense row first (zeros, or -p_j sum_k g_k p_k for the plain softmax), then each chosen expert's
// full gradient over it. V > 0: the row's logits stay in registers (V a lane); 0: they are read again.
template <typename T, int V>
__global__ void __launch_bounds__(32 * kWarps) router_backward_kernel(RouterBackwardArgs a) {
    dependent_entry();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    T* out = static_cast<T*>(a.grad) + t * a.grad_ld;
    const bool dense = a.score == EP_SCORE_SOFTMAX && !a.renormalize;
    constexpr int kHeld = V > 0 ? V : 1;
    float held[kHeld];
    if (dense && V > 0) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) held[j] = 32 * j + lane < a.E ? usable(to_float(row[32 * j + lane])) : -INFINITY;
    }
    int64_t e64 = -1;
    float g = 0.0f;
    if (lane < a.K) {
        e64 = a.idx[t * a.idx_ld + lane];
        g = a.grad_w[static_cast<int64_t>(t) * a.K + lane] * a.scale;
    }
    const bool on = e64 >= 0 && e64 < a.E;
    const int e = on ? static_cast<int>(e64) : -1 - lane;
    const float l = on ? usable(to_float(row[e])) : 0.0f;
    if (!on) g = 0.0f;

    float m = 0.0f, sum = 1.0f;
    if (dense) {
        if constexpr (V > 0) {
            m = held[0];
#pragma unroll
            for (int j = 1; j < kHeld; ++j) m = fmaxf(m, held[j]);
            m = warp_max(m);
            sum = 0.0f;
#pragma unroll
            for (int j = 0; j < kHeld; ++j) {
                held[j] = m > -INFINITY ? exp_below(held[j], m) : 0.0f;   // from here on p times the sum
                sum += held[j];
            }
            sum = warp_sum(sum);
        } else {
            row_statistics(row, a.E, lane, m, sum);
        }
    }
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
    float total = d;
    const unsigned same = __match_any_sync(kFullMask, e);
    if (__any_sync(kFullMask, on && (same & (same - 1)) != 0)) {
        total = 0.0f;
        for (int k = 0; k < a.K; ++k) {
            const float dk = __shfl_sync(kFullMask, d, k);
            if (__shfl_sync(kFullMask, e, k) == e) total += dk;
        }
    }
    if constexpr (V > 0) {
        const float slope = dense && m > -INFINITY ? -mean / sum : 0.0f;
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (32 * j + lane < a.E) out[32 * j + lane] = from_float<T>(dense ? slope * held[j] : 0.0f);
    } else {
        for (int j = lane; j < a.E; j += 32)
            out[j] = from_float<T>(dense && m > -INFINITY ? -mean * exp_below(usable(to_float(row[j])), m) / sum : 0.0f);
    }
    __syncwarp();
    if (on) out[e] = from_float<T>(dense ? total - mean * p : total);
}

template <typename T>
cudaError_t launch_topk(const RouterArgs& a, cudaStream_t stream) {
    const dim3 grid((a.T + kWarps - 1) / kWarps), block(32 * kWarps);
    const int n = a.E / a.num_groups;
    if (a.E <= 512 && (a.num_groups == 1 || (n <= 32 && (n & (n - 1)) == 0))) {
        auto* kernel = a.E <= 64    ? router_topk_registers_kernel<T, 2>
                       : a.E <= 128 ? router_topk_registers_kernel<T, 4>
                       : a.E <= 256 ? router_topk_registers_kernel<T, 8>
                                    : router_topk_registers_kernel<T, 16>;
        return launch_dependent(kernel, grid, block, 0, stream, a);
    }
    const size_t smem = sizeof(uint32_t) * kWarps * a.E;
    if (smem > 48 * 1024) {
        const cudaError_t err = cudaFuncSetAttribute(router_topk_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(smem));
        if (err != cudaSuccess) return err;
    }
    return launch_dependent(router_topk_kernel<T>, grid, block, smem, stream, a);
}

template <typename T>
cudaError_t launch_backward(const RouterBackwardArgs& a, cudaStream_t stream) {
    auto* kernel = a.E <= 64    ? router_backward_kernel<T, 2>
                   : a.E <= 128 ? router_backward_kernel<T, 4>
                   : a.E <= 256 ? router_backward_kernel<T, 8>
                   : a.E <= 512 ? router_backward_kernel<T, 16>
                                : router_backward_kernel<T, 0>;
    return launch_dependent(kernel, dim3((a.T + kWarps - 1) / kWarps), dim3(32 * kWarps), 0, stream, a);
}

}  // namespace

cudaError_t launch_router_topk(const RouterArgs& a, int dtype, cudaStream_t stream) {
    return dtype == EP_DTYPE_BF16   ? launch_topk<__nv_bfloat16>(a, stream)
           : dtype == EP_DTYPE_FP16 ? launch_topk<__half>(a, stream)
                                    : launch_topk<float>(a, stream);
}

cudaError_t launch_router_topk_backward(const RouterBackwardArgs& a, int dtype, cudaStream_t stream) {
    return dtype == EP_DTYPE_BF16   ? launch_backward<__nv_bfloat16>(a, stream)
           : dtype == EP_DTYPE_FP16 ? launch_backward<__half>(a, stream)
                                    : launch_backward<float>(a, stream);
}

}  // namespace ep
