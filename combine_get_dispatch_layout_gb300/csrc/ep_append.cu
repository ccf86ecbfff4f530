// Append of keys and values to a paged cache, the position's rotation applied
// to queries and keys on the way.
#include "ep_layer.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;

// Eight fp32 values as one row piece of the destination type.
template <typename C>
__device__ __forceinline__ void store8(C* dst, const float (&f)[8]) {
    Vec8<C> o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = from_float<C>(f[i]);
    *reinterpret_cast<uint4*>(dst) = o.raw;
}
template <>
__device__ __forceinline__ void store8(__nv_fp8_e4m3* dst, const float (&f)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i], f[4 * i + 1]), __NV_SATFINITE, __NV_E4M3) |
               static_cast<uint32_t>(
                   __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2], f[4 * i + 3]), __NV_SATFINITE, __NV_E4M3))
                   << 16;
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
}

template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&f)[8]) {
    Vec8<T> r;
    r.raw = *reinterpret_cast<const uint4*>(src);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_float(r.v[i]);
}

// Elements c .. c + 7 of a head, turned. table: the position's cosines, then
// sines. Element i of the turned part belongs to angle i mod half (halves
// paired) or i / 2 (neighbours paired); the first of a pair takes a cos - b
// sin, the second b cos + a sin.
template <typename T>
__device__ __forceinline__ void turned8(const T* head, int c, const float* table, int rot, int interleaved,
                                        float (&f)[8]) {
    load8(head + c, f);
    if (c >= rot) return;
    const int half = rot / 2;
    float own[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) own[i] = f[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = c + i;
        if (d >= rot) break;
        if (interleaved) {
            const float cs = table[d / 2], sn = table[half + d / 2];
            f[i] = (i & 1) ? own[i] * cs + own[i ^ 1] * sn : own[i] * cs - own[i ^ 1] * sn;
        } else {
            const bool first = d < half;
            const float other = to_float(head[first ? d + half : d - half]);
            const int g = first ? d : d - half;
            f[i] = first ? own[i] * table[g] - other * table[half + g] : own[i] * table[g] + other * table[half + g];
        }
    }
}

// One block per token: its threads share out the eight-element pieces of the
// token's query, key and value heads. (q_out may be q: a block's loads of a
// head end before its stores only within a thread, so queries are turned
// through shared memory.)
template <typename T, typename C>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendArgs a) {
    extern __shared__ char smem[];
    dependent_entry();
    const int64_t t = blockIdx.x;
    const int D = a.head_dim, per_head = D / 8;
    const int64_t pos = a.rotary_dim ? a.positions[t] : 0, slot = a.slots[t];
    const bool pos_ok = pos >= 0 && (a.rotary_dim == 0 || pos < a.max_position);
    const bool slot_ok = slot >= 0 && slot < a.num_slots;
    if (threadIdx.x == 0 && a.error && (!pos_ok || (!slot_ok && slot != -1))) *a.error = EP_ERR_INVALID_ARG;
    const float* table = a.cos_sin + (pos_ok ? pos : 0) * a.rotary_dim;

    T* heads = reinterpret_cast<T*>(smem);
    const T* q = static_cast<const T*>(a.q) + t * a.q_ld;
    for (int i = threadIdx.x; i < a.num_heads * per_head; i += kThreads)
        reinterpret_cast<uint4*>(heads)[i] = reinterpret_cast<const uint4*>(q)[i];
    __syncthreads();
    T* q_out = static_cast<T*>(a.q_out) + t * a.q_out_ld;
    for (int i = threadIdx.x; i < a.num_heads * per_head; i += kThreads) {
        float f[8] = {};
        if (pos_ok) turned8(heads + (i / per_head) * D, i % per_head * 8, table, a.rotary_dim, a.interleaved, f);
        store8(q_out + i * 8, f);
    }
    if (!pos_ok || !slot_ok) return;
    const int64_t page = slot / a.page_size, place = slot % a.page_size;
    for (int i = threadIdx.x; i < 2 * a.num_kv_heads * per_head; i += kThreads) {
        const bool key = i < a.num_kv_heads * per_head;
        const int j = key ? i : i - a.num_kv_heads * per_head;
        const int h = j / per_head, c = j % per_head * 8;
        float f[8];
        C* dst;
        float inv;
        if (key) {
            turned8(static_cast<const T*>(a.k) + t * a.k_ld + h * D, c, table, a.rotary_dim, a.interleaved, f);
            dst = static_cast<C*>(a.k_cache) + page * a.k_page + place * a.k_slot + h * a.k_head + c;
            inv = a.k_inv_scale;
        } else {
            load8(static_cast<const T*>(a.v) + t * a.v_ld + h * D + c, f);
            dst = static_cast<C*>(a.v_cache) + page * a.v_page + place * a.v_slot + h * a.v_head + c;
            inv = a.v_inv_scale;
        }
        if constexpr (sizeof(C) == 1) {
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] *= inv;
        }
        store8(dst, f);
    }
}

template <typename T, typename C>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(a.num_heads) * a.head_dim * sizeof(T);
    if (smem > 48 * 1024) {
        const cudaError_t err = cudaFuncSetAttribute(
            kv_append_kernel<T, C>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (err != cudaSuccess) return err;
    }
    return launch_dependent(kv_append_kernel<T, C>, dim3(a.T), dim3(kThreads), smem, stream, a);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, int dtype, int cache_dtype, cudaStream_t stream) {
    const bool fp8 = cache_dtype == EP_DTYPE_FP8_E4M3;
    if (dtype == EP_DTYPE_BF16)
        return fp8 ? launch<__nv_bfloat16, __nv_fp8_e4m3>(a, stream) : launch<__nv_bfloat16, __nv_bfloat16>(a, stream);
    return fp8 ? launch<__half, __nv_fp8_e4m3>(a, stream) : launch<__half, __half>(a, stream);
}

}  // namespace ep
