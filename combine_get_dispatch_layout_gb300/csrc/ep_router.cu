// Router: top-k experts per token from the logits, their weights, and the
// gradient of the weights back to the logits.
//
// Up to 512 experts a token's keys stay in registers, V neighbouring experts a
// lane, so the row is read once; K rounds of a maximum over the token's lanes
// pick the experts, the winning lane alone looking through its own keys again.
// Larger rows, and groups that are not a power of two of lanes, go through
// shared memory, a warp a token. Memory bounds neither (a row is a kilobyte):
// what counts is the instructions a token, the chain of each warp's steps, and
// with few tokens the launch. Measured, launches in a graph: 256 tokens, 256
// fp32 experts, top 8: 3.3 us; 16384 tokens, 64 bf16 experts in 8 groups, top 6:
// 8.4 us; the gradient for 8192 tokens, 256 fp32 experts: 6.1 us, 2.9 TB/s.
#include <math.h>
#include <string.h>

#include <type_traits>

#include "ep_layer.cuh"

namespace ep {
namespace {

constexpr int kWarps = 4;   // of a block
// From this many tokens on, rows of up to 128 experts share a warp (4 or 2 of them): the rounds' instructions are
// what counts then. Below, a token's own warp has the shorter chain. Two forms, a warp's share against a whole warp:
// 64 experts in groups, top 6: 8.4 / 10.6 us at 16384 tokens, 3.8 / 4.1 at 4096, 3.5 / 3.3 at 2048;
// 128 experts: 10.8 / 13.2 at 16384, 4.8 / 5.0 at 4096, 4.0 / 3.8 at 2048. (256 experts, two rows a warp: no gain.)
constexpr int kManyTokens = 4096;

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

// Over the LANES neighbouring lanes of a token; the whole warp calls them.
template <int LANES = 32>
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
    return v;
}
template <int LANES = 32>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

// N numbers from `p` on, in pieces of up to 16 bytes where `wide` says that p allows them.
template <int N, typename T>
__device__ __forceinline__ void load_row(const T* p, bool wide, T (&out)[N]) {
    constexpr int kBytes = N * static_cast<int>(sizeof(T));
    using Piece = std::conditional_t<(kBytes >= 16), uint4, std::conditional_t<kBytes == 8, uint2, uint32_t>>;
    if (wide) {
#pragma unroll
        for (int i = 0; i < kBytes / static_cast<int>(sizeof(Piece)); ++i) {
            const Piece piece = reinterpret_cast<const Piece*>(p)[i];
            memcpy(out + i * (sizeof(Piece) / sizeof(T)), &piece, sizeof(Piece));
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) out[i] = p[i];
    }
}
template <typename T>
__device__ __forceinline__ bool rows_aligned(const T* p, int64_t ld) {
    return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * sizeof(T))) & 15) == 0;
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
template <int LANES>
__device__ __forceinline__ float chosen_score(float l, bool on, int score, int renormalize, float row_max,
                                              float row_sum) {
    if (score == EP_SCORE_SOFTMAX) {
        if (!renormalize) return on ? exp_below(l, row_max) / row_sum : 0.0f;
        const float m = warp_max<LANES>(on ? l : -INFINITY);
        return on ? exp_below(l, m) : 0.0f;
    }
    if (!renormalize) return on ? sigmoid(l) : 0.0f;
    const float c = fminf(0.0f, warp_max<LANES>(on ? l : -INFINITY));
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

// Blocks of `tokens` tokens each.
dim3 blocks_of(int T, int tokens) { return dim3(static_cast<unsigned>((static_cast<int64_t>(T) + tokens - 1) / tokens)); }

// The weights of the chosen experts (lane k: the k-th, its logit l), and both outputs.
template <int LANES = 32>
__device__ __forceinline__ void write_choice(const RouterArgs& a, int t, int lane, int mine, float l, float row_max, float row_sum) {
    const bool on = mine >= 0;
    float w = chosen_score<LANES>(l, on, a.score, a.renormalize, row_max, row_sum);
    if (a.renormalize) {
        const float total = warp_sum<LANES>(w);
        if (on) w /= total;
    }
    if (lane < a.K && t < a.T) {
        a.idx[static_cast<int64_t>(t) * a.K + lane] = mine;
        a.weights[static_cast<int64_t>(t) * a.K + lane] = on ? w * a.scale : 0.0f;
    }
}

// Keys in registers: LANES lanes a token, 32 / LANES tokens a warp, experts V lane to V lane + V - 1 with lane `lane`,
// so that a lane's first largest key and the lowest lane that has it are the lowest expert of that key.
template <typename T, int LANES, int V>
__global__ void __launch_bounds__(32 * kWarps) router_topk_registers_kernel(RouterArgs a) {
    dependent_entry();
    const int lane = threadIdx.x % LANES;
    const int t = blockIdx.x * (kWarps * 32 / LANES) + threadIdx.x / LANES;   // (below 2^31: a block's tokens divide that)
    if ((t & ~(32 / LANES - 1)) >= a.T) return;   // (the warp's first token)
    // lanes past the last token go through the motions on its row
    const T* row = static_cast<const T*>(a.logits) + min(t, a.T - 1) * a.ld;
    const bool by_score = a.bias != nullptr || (a.num_groups > 1 && a.group_top == 2);
    const int first = V * lane;
    float l[V];
    if (first + V <= a.E) {
        T raw[V];
        load_row<V>(row + first, rows_aligned(static_cast<const T*>(a.logits), a.ld), raw);
#pragma unroll
        for (int j = 0; j < V; ++j) l[j] = usable(to_float(raw[j]));
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) l[j] = first + j < a.E ? usable(to_float(row[first + j])) : -INFINITY;
    }
    float m = 0.0f, sum = 1.0f;
    if (a.score == EP_SCORE_SOFTMAX && (by_score || !a.renormalize)) {
        m = l[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
        m = warp_max<LANES>(m);
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) sum += m > -INFINITY ? exp_below(l[j], m) : 0.0f;
        sum = warp_sum<LANES>(sum);
    }
    uint32_t keys[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float key = l[j];
        if (by_score && key > -INFINITY) {
            key = a.score == EP_SCORE_SOFTMAX ? exp_below(l[j], m) / sum : sigmoid(l[j]);
            if (a.bias) key += a.bias[first + j];
        }
        keys[j] = ordered(key);
    }
    if (a.num_groups > 1) {
        // a group is `span` whole lanes: the lane's two largest keys, then the span's by exchange
        const int span = a.E / a.num_groups / V;
        uint32_t one = 0, two = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            two = max(two, min(one, keys[j]));
            one = max(one, keys[j]);
        }
        for (int o = 1; o < span; o <<= 1) {
            const uint32_t f = __shfl_xor_sync(kFullMask, one, o), s = __shfl_xor_sync(kFullMask, two, o);
            two = max(min(one, f), max(two, s));
            one = max(one, f);
        }
        const uint32_t score = group_score(one, two, a.group_top);
        int before = 0;
        for (int j = 0; j < LANES; j += span) {
            const uint32_t o = __shfl_sync(kFullMask, score, j, LANES);
            before += o > score || (o == score && j + span <= lane);
        }
        if (before >= a.topk_groups) {
#pragma unroll
            for (int j = 0; j < V; ++j) keys[j] = 0;
        }
    }
    int mine = -1;
    uint32_t my_key = 0;
    uint32_t best = 0;
    const auto scan = [&]() {
        best = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) best = max(best, keys[j]);
    };
    scan();
    for (int k = 0; k < a.K; ++k) {
        // (no two lanes compare experts: the lowest lane with the largest key holds the lowest expert of it)
        uint32_t top = best;
        if constexpr (LANES == 32) {
            top = __reduce_max_sync(kFullMask, best);
        } else {
#pragma unroll
            for (int o = LANES / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(kFullMask, top, o));
        }
        const unsigned have = __ballot_sync(kFullMask, best == top) >> ((threadIdx.x & 31) - lane);
        const int winner = __ffs(have) - 1;
        if (!__any_sync(kFullMask, top != 0)) break;
        int at = 0;
        if (lane == winner) {
            bool found = false;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (!found && keys[j] == top) found = true, at = first + j, keys[j] = 0;
            scan();
        }
        const int e = __shfl_sync(kFullMask, at, winner, LANES);
        if (lane == k && top != 0) mine = e, my_key = top;
    }
    // (a key that is the logit gives it back; otherwise the row has it)
    const float chosen = mine < 0 ? 0.0f : by_score ? usable(to_float(row[mine])) : value_of(my_key);
    write_choice<LANES>(a, t, lane, mine, chosen, m, sum);
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
    // (an expert that the token cannot use has no score and no gradient, even where no other is left)
    float l = e64 >= 0 && e64 < a.E ? usable(to_float(row[e64])) : -INFINITY;
    const bool on = l > -INFINITY;
    const int e = on ? static_cast<int>(e64) : -1 - lane;
    if (!on) g = l = 0.0f;

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
    float p = chosen_score<32>(l, on, a.score, a.renormalize, m, sum);
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

template <typename T, int LANES, int V>
cudaError_t launch_topk_registers(const RouterArgs& a, cudaStream_t stream) {
    constexpr int kTokens = kWarps * 32 / LANES;
    return launch_dependent(router_topk_registers_kernel<T, LANES, V>, blocks_of(a.T, kTokens), dim3(32 * kWarps), 0,
                            stream, a);
}

template <typename T>
cudaError_t launch_topk(const RouterArgs& a, cudaStream_t stream) {
    // the register kernel wants a group to be a power of two of lanes
    const auto fits = [&](int V) {
        if (a.num_groups == 1) return true;
        const int n = a.E / a.num_groups, span = n / V;
        return n % V == 0 && (span & (span - 1)) == 0;
    };
    if (a.T >= kManyTokens) {
        if (a.E <= 64 && a.K <= 8 && fits(8)) return launch_topk_registers<T, 8, 8>(a, stream);
        if (a.E <= 128 && a.K <= 16 && fits(8)) return launch_topk_registers<T, 16, 8>(a, stream);
    }
    if (a.E <= 64 && fits(2)) return launch_topk_registers<T, 32, 2>(a, stream);
    if (a.E <= 128 && fits(4)) return launch_topk_registers<T, 32, 4>(a, stream);
    if (a.E <= 256 && fits(8)) return launch_topk_registers<T, 32, 8>(a, stream);
    if (a.E <= 512 && fits(16)) return launch_topk_registers<T, 32, 16>(a, stream);
    const dim3 grid = blocks_of(a.T, kWarps), block(32 * kWarps);
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
    return launch_dependent(kernel, blocks_of(a.T, kWarps), dim3(32 * kWarps), 0, stream, a);
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
