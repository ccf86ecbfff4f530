// The experts' products on dispatched rows: 4-bit weights, group scales.
#include "ep_layer.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8;

// The expert whose real rows hold row n, or -1.
__device__ __forceinline__ int expert_of(const W4Args& a, int n) {
    if (!a.offsets) return 0;
    int lo = 0, hi = a.E;   // last e with offsets[e] <= n
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (a.offsets[mid + 1] <= n) lo = mid + 1;
        else hi = mid;
    }
    if (lo >= a.E || a.offsets[lo] > n) return -1;
    if (a.counts && n - a.offsets[lo] >= a.counts[lo]) return -1;
    return lo;
}

// One weight row times one x row, one warp: each group's sum in fp32, then
// the group's scale.
template <typename T>
__device__ __forceinline__ float row_product(const W4Args& a, int e, int o, const T* x, int lane) {
    const uint8_t* w = a.w + (static_cast<int64_t>(e) * a.O + o) * (a.I / 2);
    const int groups = a.I / a.group;
    float acc = 0.0f;
    for (int g = 0; g < groups; ++g) {
        const int64_t at = (static_cast<int64_t>(e) * groups + g) * a.O + o;
        const float zero = a.zeros ? static_cast<float>(a.zeros[at]) : 8.0f;
        float sum = 0.0f;
        for (int i = g * a.group / 2 + lane; i < (g + 1) * a.group / 2; i += 32) {
            const int c = w[i];
            sum += (static_cast<float>(c & 15) - zero) * to_float(x[2 * i]);
            sum += (static_cast<float>(c >> 4) - zero) * to_float(x[2 * i + 1]);
        }
        acc += sum * to_float(static_cast<const T*>(a.scales)[at]);
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) acc += __shfl_xor_sync(kFullMask, acc, s);
    return acc;
}

// One warp per output element.
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) expert_w4_kernel(W4Args a) {
    dependent_entry();
    const int lane = threadIdx.x & 31;
    const int cols = a.swiglu ? a.O / 2 : a.O;
    const int j = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (j >= cols) return;
    for (int n = blockIdx.y; n < a.rows; n += gridDim.y) {
        const int e = expert_of(a, n);
        if (e < 0) continue;
        const T* x = static_cast<const T*>(a.x) + n * a.x_ld;
        float y = row_product(a, e, j, x, lane);
        if (a.swiglu) y = y / (1.0f + expf(-y)) * row_product(a, e, j + cols, x, lane);
        if (lane == 0) static_cast<T*>(a.y)[n * a.y_ld + j] = from_float<T>(y);
    }
}

}  // namespace

cudaError_t launch_expert_w4(const W4Args& a, int dtype, cudaStream_t stream) {
    const int cols = a.swiglu ? a.O / 2 : a.O;
    const dim3 grid((cols + kWarps - 1) / kWarps, a.rows < 1024 ? a.rows : 1024), block(32 * kWarps);
    auto* kernel = dtype == EP_DTYPE_BF16 ? expert_w4_kernel<__nv_bfloat16> : expert_w4_kernel<__half>;
    return launch_dependent(kernel, grid, block, 0, stream, a);
}

}  // namespace ep
