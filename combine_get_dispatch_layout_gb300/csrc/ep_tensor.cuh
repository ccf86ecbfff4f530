// What the kernels on the 5th-generation tensor cores share: PTX of barriers, tensor
// copies, TMEM and the products' descriptors, and the encoder of tensor maps.
#pragma once

#include <cuda.h>

#include "ep_layer.cuh"

namespace ep {
namespace {

// Shared memory barriers (mbarrier) and asynchronous copies.
__device__ __forceinline__ void barrier_init(uint32_t bar, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void barrier_expect(uint32_t bar, int bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool barrier_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}
// Every wait ends: after far more tries than any load takes, `dead` is set, the CTA runs through the rest
// without waiting, and its outputs are NaN.
static __device__ __noinline__ void barrier_wait_long(uint32_t bar, uint32_t parity, volatile int* dead) {
    for (int i = 0; i < (1 << 22); ++i) {
        if (barrier_try(bar, parity)) return;
        if ((i & 1023) == 1023 && *dead) return;
    }
    *dead = 1;
}
__device__ __forceinline__ void barrier_wait(uint32_t bar, uint32_t parity, volatile int* dead) {
    if (!barrier_try(bar, parity)) barrier_wait_long(bar, parity, dead);
}
// The same without a call, for warps whose registers were moved to them by setmaxnreg: the assembler finds no allocation
// for them around a function.
__device__ __forceinline__ void barrier_wait_inline(uint32_t bar, uint32_t parity, volatile int* dead) {
    for (int i = 0; i < (1 << 22); ++i) {
        if (barrier_try(bar, parity)) return;
        if ((i & 1023) == 1023 && *dead) return;
    }
    *dead = 1;
}
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_load8(uint32_t at, uint32_t (&u)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void multiply_done(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// Two fp32 numbers in one register pair, and arithmetic on both.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ uint64_t both(float v) { return pair(__float_as_uint(v), __float_as_uint(v)); }
__device__ __forceinline__ float2 apart(uint64_t v) {
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
    return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// Rows of 128 bytes along the inputs, 128-byte swizzle: 8 rows are 1024 bytes, the next 8 lie `stride` further on.
__device__ __forceinline__ uint64_t operand(uint32_t addr, int stride) {
    return static_cast<uint64_t>((addr >> 4) & 0x3fff) | (1ull << 16) | (static_cast<uint64_t>(stride >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
// Rows of 128 bytes along the lanes or columns, one a step of the contraction, 128-byte swizzle: 8 steps are 1024 bytes,
// the next 8 follow; the next 64 (16-bit) lanes or columns lie `stride` further on.
__device__ __forceinline__ uint64_t operand_outward(uint32_t addr, int stride) {
    return static_cast<uint64_t>((addr >> 4) & 0x3fff) | (static_cast<uint64_t>(stride >> 4) << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// One lane of a converged warp. The compiler then knows that what follows is one thread's, and issues a product every
// 16 clocks; behind `lane == 0` it took 54 to 150 (operands moved to uniform registers one by one).
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r != 0;
}

// ------------------------------------------------------------------ host

// cuTensorMapEncodeTiled, through the runtime (the library does not link the driver's).
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encoder() {
    static EncodeFn known = nullptr;   // a race writes the same value
    EncodeFn fn = __atomic_load_n(&known, __ATOMIC_RELAXED);
    if (fn) return fn;
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
        return nullptr;
    fn = reinterpret_cast<EncodeFn>(p);
    __atomic_store_n(&known, fn, __ATOMIC_RELAXED);
    return fn;
}

}  // namespace
}  // namespace ep
