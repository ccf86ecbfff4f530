// Paged attention of one new token: choice of the kernel and its workspace.
#include "ep_attention_kernel.cuh"

namespace ep {
namespace {

// SMs of the current device (a fixed property: looked up once per device).
cudaError_t sm_count(int* sms) {
    constexpr int kDevices = 64;
    static int known[kDevices];   // 0: not yet; a benign race writes the same value
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < kDevices && (*sms = __atomic_load_n(&known[dev], __ATOMIC_RELAXED)) > 0) return cudaSuccess;
    err = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (err == cudaSuccess && dev < kDevices) __atomic_store_n(&known[dev], *sms, __ATOMIC_RELAXED);
    return err;
}

}  // namespace

// Two parts per CTA of the largest grid, each the heads of a unit
// with their statistics.
int64_t paged_attention_workspace(int, int num_heads, int num_kv_heads, int head_dim) {
    int sms = 0;
    if (sm_count(&sms) != cudaSuccess) return -1;
    const int dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
    const int eights = attn::eights(num_heads / num_kv_heads, dp);
    const int64_t grid = attn::kMaxResident * sms < attn::kMaxGrid ? attn::kMaxResident * sms : attn::kMaxGrid;
    return grid * static_cast<int64_t>(sizeof(attn::Cut)) +
           grid * 2 * 8 * eights * (dp + 2) * static_cast<int64_t>(sizeof(float));
}

cudaError_t launch_paged_attention(const AttentionArgs& a, int dtype, int cache_dtype, cudaStream_t stream) {
    int sms = 0;
    const cudaError_t err = sm_count(&sms);
    if (err != cudaSuccess) return err;
    const bool fp8 = cache_dtype == EP_DTYPE_FP8_E4M3;
    if (dtype == EP_DTYPE_BF16) return fp8 ? attn::launch_bf16_e4m3(a, sms, stream) : attn::launch_bf16(a, sms, stream);
    return fp8 ? attn::launch_fp16_e4m3(a, sms, stream) : attn::launch_fp16(a, sms, stream);
}

}  // namespace ep
