// What the two kernels of the 4-bit experts share.
#pragma once

#include <cuda.h>

#include "ep_layer.cuh"

namespace ep {

// Bytes [w][z][y][x] (x: 16-byte multiples), read in boxes of 128 x box_y x box_z with the 128-byte swizzle; zeros past the ends.
cudaError_t byte_map(CUtensorMap* map, const void* base, int64_t x, int64_t y, int64_t z, int64_t w, int box_y, int box_z);

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

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
