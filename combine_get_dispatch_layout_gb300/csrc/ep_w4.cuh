// What the two kernels of the 4-bit experts share.
#pragma once

#include "ep_layer.cuh"

namespace ep {

// First row and number of real rows of expert e, within [0, rows).
__device__ __forceinline__ int expert_rows(const W4Args& a, int e, int& first) {
    if (!a.offsets) {
        first = 0;
        return a.rows;
    }
    first = min(max(a.offsets[e], 0), a.rows);
    int n = min(max(a.offsets[e + 1], 0), a.rows) - first;
    if (a.counts) n = min(n, a.counts[e]);
    return max(n, 0);
}

// The kernel for few rows in all: whether it takes these sizes, and its launch (it needs no workspace).
constexpr int kFewRows = 8;
bool expert_w4_few(const W4Args& a);
cudaError_t launch_expert_w4_few(const W4Args& a, int dtype, cudaStream_t stream);

}  // namespace ep
