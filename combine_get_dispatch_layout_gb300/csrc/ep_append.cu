// Append of keys and values to a paged cache, the position's rotation applied
// to queries and keys on the way.
//
// Each value is read and written once, so memory bounds it. One block a token;
// a thread keeps its place in a head, and with it the place's cosines and sines
// in registers, and walks over the token's heads with three under way, the first
// of them before it knows the position. A pair is always one thread's, so queries
// may be turned in place. What counts is how much is on the way at once, for each
// token waits for its position, then its angles: 7 blocks of 128 threads a core (72
// registers) take 54.6 us for 8192 tokens of 64 + 8 + 8 heads of 128 (5.9 TB/s);
// 8 blocks with two heads 54.8, 6 with four 57.4, 8 with one 62.2; heads loaded
// behind the position, two at a time: 56.8.
#include <type_traits>

#include "ep_layer.cuh"

namespace ep {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 3;   // heads that a thread has under way

// How a head is cut up.
enum Mode {
    kHalves8,     // pairs (i, i + rot/2), rot/2 a multiple of 8: 8 values of either half together
    kHalves4,     // the same with a multiple of 4
    kNeighbours,  // pairs (2i, 2i + 1), rot a multiple of 8: 8 values
    kSingle       // any other rotary_dim: one pair, or one value behind them
};

// W neighbouring values, and their places in memory.
template <int W>
using Raw = std::conditional_t<W == 8, uint4, uint2>;

template <typename T, int W>
__device__ __forceinline__ void unpack(const Raw<W>& raw, float (&f)[W]) {
    const T* v = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = to_float(v[i]);
}
// fp32 values as a piece of a row of the destination type, times inv for e4m3.
template <typename C, int W>
__device__ __forceinline__ void store(C* dst, const float (&f)[W], float inv) {
    if constexpr (std::is_same_v<C, __nv_fp8_e4m3>) {
        uint32_t w[W / 4];
#pragma unroll
        for (int i = 0; i < W / 4; ++i)
            w[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i] * inv, f[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3) |
                   static_cast<uint32_t>(
                       __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2] * inv, f[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3))
                       << 16;
        if constexpr (W == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(dst) = w[0];
    } else {
        Raw<W> o;
#pragma unroll
        for (int i = 0; i < W; ++i) reinterpret_cast<C*>(&o)[i] = from_float<C>(f[i]);
        *reinterpret_cast<Raw<W>*>(dst) = o;
    }
}
template <typename C>
__device__ __forceinline__ void store1(C* dst, float f, float) {
    *dst = from_float<C>(f);
}
template <>
__device__ __forceinline__ void store1(__nv_fp8_e4m3* dst, float f, float inv) {
    dst->__x = __nv_cvt_float_to_fp8(f * inv, __NV_SATFINITE, __NV_E4M3);
}

template <typename T, typename C, Mode MODE>
__global__ void __launch_bounds__(kThreads, 7) kv_append_kernel(AppendArgs a) {
    dependent_entry();
    const int64_t t = blockIdx.x;
    const int D = a.head_dim, rot = a.rotary_dim, half = rot / 2, tid = threadIdx.x;
    const T* const q = static_cast<const T*>(a.q) + t * a.q_ld;
    const T* const k = static_cast<const T*>(a.k) + t * a.k_ld;
    const T* const v = static_cast<const T*>(a.v) + t * a.v_ld;
    T* const q_out = static_cast<T*>(a.q_out) + t * a.q_out_ld;

    constexpr bool kHalves = MODE == kHalves8 || MODE == kHalves4;
    constexpr int W = MODE == kHalves4 ? 4 : 8, kAngles = kHalves ? W : 4;
    // ---- a thread's first heads are under way before the position is known
    const int turned = half / kAngles, pieces = turned + (D - rot) / W;   // of a head
    const int step = MODE == kSingle ? 0 : kThreads / pieces, c = MODE == kSingle ? 0 : tid % pieces, h0 = MODE == kSingle ? 0 : tid / pieces;
    const bool turn = c < turned, two = kHalves && turn;
    const int first = turn ? c * W : rot + (c - turned) * W;
    Raw<W> one[kAhead], other[kAhead];
    const auto load = [&](int u, int h) {
        if (h >= a.num_heads + a.num_kv_heads) return;
        const T* from = (h >= a.num_heads ? k + (h - a.num_heads) * D : q + h * D) + first;
        one[u] = *reinterpret_cast<const Raw<W>*>(from);
        if (two) other[u] = *reinterpret_cast<const Raw<W>*>(from + half);
    };
    if constexpr (MODE != kSingle) {
        if (h0 < step) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) load(u, h0 + u * step);
        }
    }

    const int64_t pos = rot ? a.positions[t] : 0, slot = a.slots[t];
    const bool pos_ok = pos >= 0 && (rot == 0 || pos < a.max_position);
    const bool slot_ok = slot >= 0 && slot < a.num_slots;
    if (tid == 0 && a.error && (!pos_ok || (!slot_ok && slot != -1))) *a.error = EP_ERR_INVALID_ARG;
    const float* table = a.cos_sin + (pos_ok ? pos : 0) * rot;
    const int64_t page = slot_ok ? slot / a.page_size : 0, place = slot_ok ? slot - page * a.page_size : 0;
    const bool cached = pos_ok && slot_ok;
    C* const keys = static_cast<C*>(a.k_cache) + page * a.k_page + place * a.k_slot;
    C* const values = static_cast<C*>(a.v_cache) + page * a.v_page + place * a.v_slot;
    const int heads = a.num_heads + (cached ? a.num_kv_heads : 0);   // queries, then keys
    if constexpr (MODE == kSingle) {
        const int per_head = half + D - rot;
        for (int i = tid; i < heads * per_head; i += kThreads) {
            const int h = i / per_head, c = i % per_head;
            const bool key = h >= a.num_heads;
            const T* from = key ? k + (h - a.num_heads) * D : q + h * D;
            int first = c, second = -1;
            float x, y = 0.0f;
            if (c < half) {
                first = a.interleaved ? 2 * c : c;
                second = a.interleaved ? 2 * c + 1 : c + half;
                const float p = to_float(from[first]), r = to_float(from[second]), cs = table[c], sn = table[half + c];
                x = p * cs - r * sn;
                y = r * cs + p * sn;
            } else {
                first = c + half;
                x = to_float(from[first]);
            }
            if (key) {
                C* to = keys + (h - a.num_heads) * a.k_head;
                store1(to + first, x, a.k_inv_scale);
                if (second >= 0) store1(to + second, y, a.k_inv_scale);
            } else {
                q_out[h * D + first] = from_float<T>(pos_ok ? x : 0.0f);
                if (second >= 0) q_out[h * D + second] = from_float<T>(pos_ok ? y : 0.0f);
            }
        }
    } else {
        if (h0 < step) {
            float cs[kAngles], sn[kAngles];
            if (turn) {
#pragma unroll
                for (int i = 0; i < kAngles; ++i) cs[i] = table[c * kAngles + i], sn[i] = table[half + c * kAngles + i];
            }
            for (int base = h0; base < heads; base += kAhead * step) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int h = base + u * step;
                    if (h >= heads) break;
                    float x[W], y[W], p[W], r[W];
                    unpack<T, W>(one[u], p);
                    if (two) unpack<T, W>(other[u], r);
                    load(u, h + kAhead * step);
                    if (two) {
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            x[i] = p[i] * cs[i % kAngles] - r[i] * sn[i % kAngles];
                            y[i] = r[i] * cs[i % kAngles] + p[i] * sn[i % kAngles];
                        }
                    } else if (turn) {   // kNeighbours
#pragma unroll
                        for (int i = 0; i < W; i += 2) {
                            x[i] = p[i] * cs[i / 2] - p[i + 1] * sn[i / 2];
                            x[i + 1] = p[i + 1] * cs[i / 2] + p[i] * sn[i / 2];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < W; ++i) x[i] = p[i];
                    }
                    if (h >= a.num_heads) {
                        C* to = keys + (h - a.num_heads) * a.k_head + first;
                        store<C, W>(to, x, a.k_inv_scale);
                        if (two) store<C, W>(to + half, y, a.k_inv_scale);
                    } else {
                        if (!pos_ok) {
#pragma unroll
                            for (int i = 0; i < W; ++i) x[i] = y[i] = 0.0f;
                        }
                        store<T, W>(q_out + h * D + first, x, 1.0f);
                        if (two) store<T, W>(q_out + h * D + first + half, y, 1.0f);
                    }
                }
            }
        }
    }
    if (!cached) return;
    const int per_head = D / 8;
    for (int i = tid; i < a.num_kv_heads * per_head; i += kThreads) {
        const int h = i / per_head, c = i % per_head * 8;
        const uint4 raw = *reinterpret_cast<const uint4*>(v + h * D + c);
        C* to = values + h * a.v_head + c;
        if constexpr (sizeof(C) == 2) {
            *reinterpret_cast<uint4*>(to) = raw;
        } else {
            float f[8];
            unpack<T, 8>(raw, f);
            store<C, 8>(to, f, a.v_inv_scale);
        }
    }
}

template <typename T, typename C>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
    // a head is cut into at most kThreads pieces
    const int rot = a.rotary_dim;
    auto* kernel = a.interleaved   ? (rot % 8 == 0 ? kv_append_kernel<T, C, kNeighbours> : kv_append_kernel<T, C, kSingle>)
                   : rot % 16 == 0 ? kv_append_kernel<T, C, kHalves8>
                   : rot % 8 == 0 && a.head_dim <= 4 * kThreads ? kv_append_kernel<T, C, kHalves4>
                                                                : kv_append_kernel<T, C, kSingle>;
    return launch_dependent(kernel, dim3(a.T), dim3(kThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, int dtype, int cache_dtype, cudaStream_t stream) {
    const bool fp8 = cache_dtype == EP_DTYPE_FP8_E4M3;
    if (dtype == EP_DTYPE_BF16)
        return fp8 ? launch<__nv_bfloat16, __nv_fp8_e4m3>(a, stream) : launch<__nv_bfloat16, __nv_bfloat16>(a, stream);
    return fp8 ? launch<__half, __nv_fp8_e4m3>(a, stream) : launch<__half, __half>(a, stream);
}

}  // namespace ep
