// The experts' products on dispatched rows: 4-bit weights, group scales. (Up to
// 8 rows in all mostly go through ep_expert_w4_few.cu.)
//
// Mathematics. y[n, o] = sum over groups g of s[g, o] * sum over i in g of
// (code[o, i] - zero[g, o]) x[n, i]. The inner sums run through the 5th-generation
// tensor cores on 8-bit operands with fp32 sums:
//  - a code 0 .. 15 in a byte IS the e4m3 number code * 2^-9 (subnormal up to 7,
//    the first binade from 8 on), so unpacking eight codes is two masks and one
//    shift. (As bf16 operands of mma.sync they take 11 instructions, and that
//    kernel ran at 37 % of the memory rate, bound by instruction issue; e4m3
//    operands of mma.sync are converted to fp16 by further instructions.)
//  - x is taken as a sum of 8-bit numbers, two for bf16 and three for fp16, after
//    a power of two has brought the largest input of the group to [128, 256):
//    an e4m3 number with the 4 leading bits, then e5m2 ones, each with the 3
//    leading bits of what the ones before have left (rounded to nearest, so what
//    is left has a bit less). They make up the 8 or 11 bits of x exactly, but for
//    inputs so far below the group's largest that e5m2's smallest step counts:
//    at most 2^-24 of the largest is left off. All are multiplied into the same
//    sums, one after the other.
//  - the zero point enters as zero * (sum of the group's inputs), in fp32.
// Scales multiply a group's sum in fp32. y is rounded once.
//
// What bounds it: with few rows per expert each weight is used a few times, so
// reading the codes (half a byte each) once is the floor. Instruction issue is
// next: about 6 instructions a word of 8 codes of the 22 clocks that DRAM takes
// for 128 bytes an SM quarter.
//
// Layout. 128 weight rows are the product's 128 lanes: thread = weight row =
// TMEM lane, for unpacking (shared memory to TMEM operand A), for the scales
// (one a thread) and for the sums (tcgen05.ld, one column a row of x). One
// persistent CTA a core walks its items (an expert, 512 weight rows, at most NR
// rows of x). One warp fills the rings by TMA, straight on across items: stages
// of 256 inputs, 64 KB of codes; x, which comes from L2, is shared by all 512
// rows (with 128 rows it was half as much traffic again as the codes, and the
// ring alone could not pass 77 % of the memory rate). Four warpgroups take 128
// rows each: they unpack half a stage, hand it to the warp that issues the
// products, and take in the sums of the half before meanwhile. The first weights
// are on their way while split_kernel still runs. Where there are few items, the
// CTAs of a cluster share an item's inputs and join through distributed shared
// memory.
//
// Measured, launches in a graph, bf16, groups of 128, 256 experts of 4096 x 7168
// with the activation, top 8: 256 tokens 700 us (5.6 TB/s; groups of 64 771, of 32
// 1038; fp16 766), 128 tokens 636 us (6.0), 64 tokens 552 us (6.1). Parts of x as
// columns of one product instead: 706 (822, 1036; 779). Clusters of up to 16 instead of 8: 19.9 us against
// 12.0 for one 4096 x 4096 matrix.

#include <cuda.h>

#include <type_traits>

#include "ep_w4.cuh"

namespace ep {
namespace {

constexpr int kGroupsOfWarps = 4;                  // warpgroups
constexpr int kConsumers = 128 * kGroupsOfWarps;
constexpr int kLoader = kConsumers / 32, kIssuer = kLoader + 1;   // warps
constexpr int kThreads = kConsumers + 64;
constexpr int kTileRows = 128;                     // weight rows of a warpgroup
constexpr int kIn = 256;                           // inputs of a stage
constexpr int kTileBytes = kTileRows * kIn / 2;
constexpr int kWeightBytes = kGroupsOfWarps * kTileBytes;
constexpr int kWeightSlots = 3;
constexpr int kSplitThreads = 256;
constexpr int kMostSplit = 8;                      // CTAs of a cluster that share an item
constexpr int kTable = 1024;                       // entries of the table of experts' passes

// Parts that x is split into.
template <typename T>
constexpr int kParts = std::is_same_v<T, __half> ? 3 : 2;

// T: type of x, scales and y. NR: rows of x of an item. GROUP: inputs that share a scale.
template <typename T, int NR, int GROUP>
struct Shape {
    static_assert(NR == 16 || (NR == 8 && kParts<T> == 2), "");
    static constexpr int kN = 16;                              // columns of a product, the least there are: of 8 rows the others are garbage
    static constexpr int kGroups = 128 / GROUP;                // of half a stage
    static constexpr int kBlock = kParts<T> * 1024;            // 8 rows of x, 128 inputs: [part][8][128 bytes]
    static constexpr int kXBytes = NR / 8 * kBlock;            // x of half a stage
    static constexpr int kXSlots = kParts<T> == 3 ? 2 : 3;
    static constexpr int kStats = 2 * kGroups * NR * 2;        // floats of a stage
    static constexpr int kSumCols = kN * kGroups;
    // columns of TMEM of a warpgroup: operand A twice, sums twice where there is room
    static constexpr int kSumBuffers = 64 + 2 * kSumCols <= 128 ? 2 : 1;
    static constexpr int kCols = 64 + kSumBuffers * kSumCols;
    static_assert(kCols <= 128, "");
    static constexpr int kTmem = 512;
    static constexpr int kShared = 1024 + kWeightSlots * kWeightBytes + kXSlots * (2 * kXBytes + kStats * 4) + 512 + (kTable + 1) * 4;
    static_assert(kShared <= 227 * 1024 - 256, "");
};

struct Plan {
    int tiles;       // of kConsumers weight rows, of an expert
    int table_shift; // an entry of the table stands for 2^table_shift experts
    int slots;       // CTAs of the grid
    int split;       // CTAs that share an item
    int stages;      // of an item
    int groups;      // of a weight row
    const float* stats;    // [rows][groups][2]: power of two, 2^-9 * sum, of a group's inputs
};

// ------------------------------------------------------------------ PTX

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
// Arrives once this thread's copies so far are complete.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int real) {   // zeros where real is 0
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real) : "memory");
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); }
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
        "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
        "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
        "r"(r[31])
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_load8(uint32_t at, uint32_t (&u)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// sums [128 lanes][N] (+)= A [128 lanes][32 inputs, TMEM] * B [32 inputs][N, shared memory]^T
__device__ __forceinline__ void multiply(uint32_t sums, uint32_t a, uint64_t b, uint32_t shape, bool add) {
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p; }" ::"r"(sums),
                 "r"(a), "l"(b), "r"(shape), "r"(static_cast<uint32_t>(add))
                 : "memory");
}
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

// One lane of a converged warp. The compiler then knows that what follows is one thread's, and issues a product every
// 16 clocks; behind `lane == 0` it took 54 to 150 (operands moved to uniform registers one by one).
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r != 0;
}

// ------------------------------------------------------------------ rows and items

struct Item {
    int expert, row, rows, col;   // col: first output column of the tile
};

// Four values as 8-bit codes in a word, each reduced by what its code stands for.
__device__ __forceinline__ uint32_t take_part(float (&v)[4], __nv_fp8_interpretation_t type) {
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(make_float2(v[i], v[i + 1]), __NV_SATFINITE, type);
        const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, type)));
        v[i] -= f.x;
        v[i + 1] -= f.y;
        word |= static_cast<uint32_t>(c) << (8 * i);
    }
    return word;
}

// x as sums of 8-bit numbers, a plane [rows][I] for each part; of 8 neighbouring inputs the even ones come first, as
// masks leave the codes. A thread takes 8 inputs, GROUP / 8 threads share a power of two. An infinite or NaN
// input makes its group's power of two or sum NaN, and so every product with it.
template <typename T, int GROUP>
__global__ void __launch_bounds__(kSplitThreads) split_kernel(W4Args a, unsigned char* to, float2* stats) {
    dependent_entry();
    const int per_row = a.I / 8;
    const int last = a.offsets ? min(max(a.offsets[a.E], 0), a.rows) : a.rows;   // rows behind belong to nobody
    const int64_t all = static_cast<int64_t>(last) * per_row, plane = static_cast<int64_t>(a.rows) * a.I;
    // (a group's threads are of one warp: per_row is a multiple of GROUP / 8)
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kSplitThreads + threadIdx.x; i - threadIdx.x % 32 < all;
         i += static_cast<int64_t>(gridDim.x) * kSplitThreads) {
        const bool in = i < all;
        const int64_t row = in ? i / per_row : 0;
        const int c = in ? static_cast<int>(i - row * per_row) : 0;
        Vec8<T> v;
        v.raw = make_uint4(0, 0, 0, 0);
        if (in) v.raw = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + row * a.x_ld + c * 8);
        float big = 0.0f, even[4], odd[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            even[k] = to_float(v.v[2 * k]);
            odd[k] = to_float(v.v[2 * k + 1]);
            big = fmaxf(big, fmaxf(fabsf(even[k]), fabsf(odd[k])));
        }
#pragma unroll
        for (int o = 1; o < GROUP / 8; o <<= 1) big = fmaxf(big, __shfl_xor_sync(kFullMask, big, o));
        const bool finite = big < INFINITY;
        const int e = big > 0.0f && finite ? min(7 - ilogbf(big), 126) : 0;
        const float up = __int_as_float((e + 127) << 23);
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            even[k] *= up;
            odd[k] *= up;
            sum += even[k] + odd[k];
        }
#pragma unroll
        for (int k = 0; k < kParts<T>; ++k) {
            uint2 w;
            w.x = take_part(even, k == 0 ? __NV_E4M3 : __NV_E5M2);
            w.y = take_part(odd, k == 0 ? __NV_E4M3 : __NV_E5M2);
            if (in) *reinterpret_cast<uint2*>(to + k * plane + i * 8) = w;
        }
        // the sum of what the parts stand for: the inputs' less what is left of them
#pragma unroll
        for (int k = 0; k < 4; ++k) sum -= even[k] + odd[k];
#pragma unroll
        for (int o = 1; o < GROUP / 8; o <<= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
        if (in && c % (GROUP / 8) == 0)
            stats[row * (a.I / GROUP) + c / (GROUP / 8)] =
                make_float2(finite ? __int_as_float((127 - e) << 23) : __int_as_float(0x7fffffff), sum * 0.001953125f);
    }
}

template <typename T, int NR, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kThreads, 1)
    expert_w4_kernel(W4Args a, Plan p, const __grid_constant__ CUtensorMap weight_map, const __grid_constant__ CUtensorMap x_map) {
    using S = Shape<T, NR, GROUP>;
    constexpr int kGroups = S::kGroups, kXSlots = S::kXSlots;
    extern __shared__ unsigned char shared_bytes[];
    // weights: [kWeightSlots][warpgroup][128 rows][128 bytes], 128-byte swizzle; inputs: [kXSlots][half][NR / 8][part][8 rows]
    // [128 bytes], likewise; stats: [kXSlots][half][kGroups] of NR / 2 pairs of rows, a pair's two powers of two, then its
    // two sums; barriers; the table of passes
    unsigned char* const weights = shared_bytes + (1024 - smem_addr(shared_bytes) % 1024) % 1024;
    unsigned char* const inputs = weights + kWeightSlots * kWeightBytes;
    float* const stats = reinterpret_cast<float*>(inputs + kXSlots * 2 * S::kXBytes);
    uint64_t* const barriers = reinterpret_cast<uint64_t*>(stats + kXSlots * S::kStats);
    const uint32_t w_full = smem_addr(barriers), w_empty = w_full + 8 * kWeightSlots;
    const uint32_t x_full = w_empty + 8 * kWeightSlots, x_empty = x_full + 8 * kXSlots;
    const uint32_t ready = x_empty + 8 * kXSlots, done = ready + 16 * kGroupsOfWarps;   // [warpgroup][2 operand buffers]
    uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(barriers) + 120;
    volatile int* const dead = reinterpret_cast<volatile int*>(tmem_at + 1);
    int* const table = reinterpret_cast<int*>(barriers) + 128;
    static_assert((2 * kWeightSlots + 2 * kXSlots + 4 * kGroupsOfWarps) * 2 <= 120, "");
    __shared__ int warp_sum[kThreads / 32];
    // Everything before split_kernel, which this kernel follows, is complete once this one runs: split_kernel lets it
    // start only after it has waited for that itself. So all but split_kernel's own outputs can be read at once, and
    // griddepcontrol.wait comes before those (in the loading warp; the others see them through its barriers).

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cols = a.swiglu ? a.O / 2 : a.O;
    const int tile_cols = a.swiglu ? kTileRows / 2 : kTileRows;   // output columns of a warpgroup
    const int rank = blockIdx.x % p.split;

    if (warp == kLoader) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_at)), "n"(S::kTmem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        if (lane == 0) {
            *dead = 0;
            for (int i = 0; i < kWeightSlots; ++i) {
                barrier_init(w_full + 8 * i, 1);
                barrier_init(w_empty + 8 * i, kConsumers / 32);
            }
            for (int i = 0; i < kXSlots; ++i) {
                barrier_init(x_full + 8 * i, 33);                // the TMA loads' thread and 32 lanes' copies
                barrier_init(x_empty + 8 * i, kConsumers / 32);
            }
            for (int i = 0; i < 2 * kGroupsOfWarps; ++i) {
                barrier_init(ready + 8 * i, 4);
                barrier_init(done + 8 * i, 1);
            }
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    }
    // ---- items: an expert's rows in passes of NR, each pass over all tiles; a tile's passes follow each other, so
    // the weights of the second come from L2
    const auto passes_of = [&](int e) {
        int first;
        return (expert_rows(a, e, first) + NR - 1) / NR;
    };
    const int entries = ((a.E - 1) >> p.table_shift) + 1;
    {
        const int per = (entries + kThreads - 1) / kThreads, lo = min(entries, tid * per), hi = min(entries, lo + per);
        const int e0 = lo << p.table_shift, e1 = min(a.E, hi << p.table_shift);
        int own = 0;
        for (int e = e0; e < e1; ++e) own += passes_of(e);
        int scan = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFullMask, scan, o);
            if (lane >= o) scan += v;
        }
        if (lane == 31) warp_sum[warp] = scan;
        __syncthreads();
        int base = scan - own;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w)
            if (w < warp) base += warp_sum[w];
        for (int e = e0; e < e1; ++e) {
            if ((e & ((1 << p.table_shift) - 1)) == 0) table[e >> p.table_shift] = base;
            base += passes_of(e);
        }
        if (hi == entries && lo < hi) table[entries] = base;
        tmem_fence_before();
        __syncthreads();
        tmem_fence_after();
    }
    const uint32_t tmem = __shfl_sync(kFullMask, *tmem_at, 0);
    const bool leader = elected();
    const int64_t items = static_cast<int64_t>(table[entries]) * p.tiles;
    // as many clusters as share the items evenly: all of them wait on the same DRAM, so an idle SM costs nothing
    const int clusters = p.slots / p.split;
    const int64_t each = (items + clusters - 1) / clusters;
    const int64_t item0 = min(items, each * (blockIdx.x / p.split));
    // (a cluster joins once: more than one item for it come of offsets that contradict one another)
    const int64_t item1 = min(items, item0 + (p.split > 1 ? min(each, int64_t{1}) : each));
    // this CTA's stages of every item
    const int stage0 = p.stages * rank / p.split, stage1 = p.stages * (rank + 1) / p.split;

    const auto decode = [&](int64_t it) {
        int lo = 0, hi = entries - 1;   // the last entry whose first item is not behind `it`
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (static_cast<int64_t>(table[mid]) * p.tiles <= it) lo = mid;
            else hi = mid - 1;
        }
        int64_t in = it - static_cast<int64_t>(table[lo]) * p.tiles;
        int e = lo << p.table_shift, passes = passes_of(e);
        while (in >= static_cast<int64_t>(passes) * p.tiles && e + 1 < a.E) {   // (an entry of several experts)
            in -= static_cast<int64_t>(passes) * p.tiles;
            passes = passes_of(++e);
        }
        passes = max(passes, 1);   // (0, and an item behind the last one, come of offsets that contradict one another)
        Item r;
        int first;
        const int n = expert_rows(a, e, first), pass = static_cast<int>(in % passes);
        r.expert = e;
        r.row = first + pass * NR;
        r.rows = min(NR, n - pass * NR);
        r.col = static_cast<int>(in / passes) * (kGroupsOfWarps * tile_cols);
        return r;
    };
    const int64_t steps = (item1 - item0) * (stage1 - stage0);

    if (warp == kLoader) {
        const auto load_weights = [&](const Item& it, int stage, int slot) {
            const uint32_t bar = w_full + 8 * slot, to = smem_addr(weights) + slot * kWeightBytes;
            if (lane == 0) barrier_expect(bar, kWeightBytes);
            __syncwarp();
            // with an activation a box is the 16 gate and the 16 up rows of a warp, else the 128 rows of a warpgroup
            if (a.swiglu) {
                if (lane < kConsumers / 32)
                    load_box(to + lane * (kTileBytes / 4), &weight_map, stage * (kIn / 2), it.col + lane * 16, 0, it.expert, bar);
            } else if (lane < kGroupsOfWarps) {
                load_box(to + lane * kTileBytes, &weight_map, stage * (kIn / 2), it.col + lane * kTileRows, 0, it.expert, bar);
            }
        };
        const auto load_inputs = [&](const Item& it, int stage, int slot) {
            const uint32_t bar = x_full + 8 * slot;
            const int blocks = (it.rows + 7) / 8;   // (rows that are not there leave garbage in columns that are not written)
            if (lane == 0) barrier_expect(bar, 2 * blocks * S::kBlock);
            __syncwarp();
            if (lane < 2 * blocks)
                load_box(smem_addr(inputs) + (slot * 2 + lane / blocks) * S::kXBytes + lane % blocks * S::kBlock, &x_map,
                         stage * kIn + lane / blocks * 128, it.row + lane % blocks * 8, 0, 0, bar);
            for (int i = lane; i < S::kStats; i += 32) {
                const int n = i / 4 % (NR / 2) * 2 + (i & 1), which = (i >> 1) & 1, grp = stage * (kIn / GROUP) + i / (2 * NR);
                const bool in = n < it.rows && grp < p.groups;
                copy4(smem_addr(stats + slot * S::kStats + i),
                      p.stats + (in ? (static_cast<int64_t>(it.row + n) * p.groups + grp) * 2 + which : 0), in ? 4 : 0);
            }
            copies_arrive(bar);
        };
        struct Cursor {
            int64_t item;
            int stage, slot;
            uint32_t parity;
            Item at;
        };
        const auto advance = [&](Cursor& c, int slots) {
            if (++c.stage == stage1) c.stage = stage0, ++c.item;
            if (++c.slot == slots) c.slot = 0, c.parity ^= 1;
        };
        Cursor w{item0, stage0, 0, 1, {}}, x{item0, stage0, 0, 1, {}};   // (the first round of a ring waits for nothing)
        int64_t wi = 0;
        for (; wi < min(steps, static_cast<int64_t>(kWeightSlots)); ++wi, advance(w, kWeightSlots)) {
            if (w.stage == stage0) w.at = decode(w.item);
            load_weights(w.at, w.stage, w.slot);
        }
        dependent_entry();
        for (int64_t xi = 0; xi < steps; ++xi, advance(x, kXSlots)) {
            if (x.stage == stage0) x.at = decode(x.item);
            if (xi >= kXSlots) barrier_wait(x_empty + 8 * x.slot, x.parity, dead);
            load_inputs(x.at, x.stage, x.slot);
            // the weights of a stage are used up before its x is: they run ahead by their ring's length
            if (xi + 1 >= kXSlots && wi < steps) {
                if (w.stage == stage0) w.at = decode(w.item);
                barrier_wait(w_empty + 8 * w.slot, w.parity, dead);
                load_weights(w.at, w.stage, w.slot);
                ++wi;
                advance(w, kWeightSlots);
            }
        }
        for (; wi < steps; ++wi, advance(w, kWeightSlots)) {
            if (w.stage == stage0) w.at = decode(w.item);
            barrier_wait(w_empty + 8 * w.slot, w.parity, dead);
            load_weights(w.at, w.stage, w.slot);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == kIssuer) {
        if (leader) {
            constexpr uint32_t kShape = (1u << 4) | (static_cast<uint32_t>(S::kN / 8) << 17) | (static_cast<uint32_t>(kTileRows / 16) << 24);
            constexpr uint32_t kLaterShape = kShape | (1u << 10);   // x as e5m2
            // columns: 8 rows, then the next 8 (of an item of 8 rows whatever shared memory holds behind them)
            constexpr int kStride = S::kBlock;
            int slot = 0;
            uint32_t parity = 0, ready_parity = 0;
            for (int64_t i = 0; i < steps; ++i) {
                barrier_wait(x_full + 8 * slot, parity, dead);
                for (int half = 0; half < 2; ++half) {
                    const uint64_t b = operand(smem_addr(inputs) + (slot * 2 + half) * S::kXBytes, kStride);
                    for (int wg = 0; wg < kGroupsOfWarps; ++wg) {
                        barrier_wait(ready + 8 * (wg * 2 + half), ready_parity, dead);
                        tmem_fence_after();
                        const uint32_t a_at = tmem + wg * 128 + half * 32;
                        const uint32_t sums = tmem + wg * 128 + 64 + (S::kSumBuffers == 2 ? half * S::kSumCols : 0);
#pragma unroll
                        for (int part = 0; part < kParts<T>; ++part)
#pragma unroll
                            for (int k = 0; k < GROUP / 32; ++k)
#pragma unroll
                                for (int grp = 0; grp < kGroups; ++grp) {
                                    const int step = grp * (GROUP / 32) + k;
                                    multiply(sums + grp * S::kN, a_at + step * 8, b + step * 2 + part * (1024 / 16),
                                             part > 0 ? kLaterShape : kShape, part > 0 || k > 0);
                                }
                        multiply_done(done + 8 * (wg * 2 + half));
                    }
                }
                ready_parity ^= 1;
                if (++slot == kXSlots) slot = 0, parity ^= 1;
            }
        }
        __syncwarp();
    } else {
        // ---- a warpgroup: unpack half a stage, take in the sums of the half before
        const int wg = warp >> 2, row = tid & 127;      // row: of the tile; its TMEM lane
        const uint32_t mine = tmem + wg * 128 + (static_cast<uint32_t>(warp & 3) << 21);   // lane 32 * (warp % 4), upper half
        int w_slot = 0, x_slot = 0, stat_slot = 0;
        uint32_t w_parity = 0, x_parity = 0, done_parity = 0;
        for (int64_t item = item0; item < item1; ++item) {
            const Item it = decode(item);
            // this thread's output column and weight row; with an activation a warp's lanes are 16 gate and 16 up rows
            int col, o;
            if (a.swiglu) {
                col = it.col + warp * 16 + (lane & 15);
                o = lane < 16 ? col : cols + col;
            } else {
                o = col = it.col + wg * kTileRows + row;
            }
            const bool real = col < cols;
            // Scales are loaded half a stage ahead. A row past the tile's end takes another's, and a group past the inputs'
            // end the last one's: those sums are zero, or not written.
            int grp_next = stage0 * (kIn / GROUP);
            const int64_t scale_base = (static_cast<int64_t>(it.expert) * p.groups + grp_next) * a.O + (real ? o : 0);
            const T* scale_at = static_cast<const T*>(a.scales) + scale_base;
            const uint8_t* zero_at = ZEROS ? a.zeros + scale_base : nullptr;
            T scale[kGroups], scale_next[kGroups];
            uint8_t zero[kGroups] = {}, zero_next[kGroups] = {};
            const auto load_scales = [&]() {
#pragma unroll
                for (int i = 0; i < kGroups; ++i) {
                    const int64_t on = ++grp_next < p.groups ? a.O : 0;
                    scale_next[i] = *scale_at;
                    scale_at += on;
                    if constexpr (ZEROS) {
                        zero_next[i] = *zero_at;
                        zero_at += on;
                    }
                }
            };
            uint64_t acc2[NR / 2];   // rows 2 n, 2 n + 1
#pragma unroll
            for (int n = 0; n < NR / 2; ++n) acc2[n] = 0;
            // takes in the sums of half `half` of the stage whose x is in slot s
            const auto take_sums = [&](int half, int s) {
                barrier_wait(done + 8 * (wg * 2 + half), (done_parity >> half) & 1, dead);
                done_parity ^= 1u << half;
                tmem_fence_after();
#pragma unroll
                for (int i = 0; i < kGroups; ++i) {
                    const uint64_t sc = both(to_float(scale[i])), z = both(ZEROS ? -static_cast<float>(zero[i]) : -8.0f);
#pragma unroll
                    for (int b = 0; b < NR / 8; ++b) {   // 8 rows
                        if (b == 1 && it.rows <= 8) break;
                        uint32_t v[8];
                        tmem_load8(mine + 64 + (S::kSumBuffers == 2 ? half * S::kSumCols : 0) + i * S::kN + b * 8, v);
                        tmem_load_wait();
                        const float* st = stats + s * S::kStats + (half * kGroups + i) * (NR * 2) + b * 16;
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const uint64_t sum = pair(v[2 * n], v[2 * n + 1]);
                            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(st + 4 * n);
                            acc2[b * 4 + n] = fma2(mul2(sc, f.x), fma2(z, f.y, sum), acc2[b * 4 + n]);
                        }
                    }
                }
                tmem_fence_before();
                if (half == 1) {
                    __syncwarp();
                    if (lane == 0) barrier_arrive(x_empty + 8 * s);
                }
            };
            load_scales();
            bool before = false;
            for (int stage = stage0; stage < stage1; ++stage) {
                barrier_wait(w_full + 8 * w_slot, w_parity, dead);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t codes[32];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 v = *reinterpret_cast<const uint4*>(weights + w_slot * kWeightBytes + wg * kTileBytes + row * 128 + (((4 * half + j) ^ (row & 7)) << 4));
                        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            codes[8 * j + 2 * k] = u[k] & 0x0f0f0f0fu;
                            codes[8 * j + 2 * k + 1] = (u[k] >> 4) & 0x0f0f0f0fu;
                        }
                    }
                    // (the products that read this operand buffer last have been waited for in take_sums)
                    tmem_store32(mine + half * 32, codes);
                    if (S::kSumBuffers == 1 && before) take_sums(half ^ 1, half == 0 ? stat_slot : x_slot);
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        barrier_arrive(ready + 8 * (wg * 2 + half));
                        if (half == 1) barrier_arrive(w_empty + 8 * w_slot);
                    }
                    if (half == 0) {   // (the sums' statistics come with x)
                        barrier_wait(x_full + 8 * x_slot, x_parity, dead);
                    }
                    if (S::kSumBuffers == 2 && before) take_sums(half ^ 1, half == 0 ? stat_slot : x_slot);
#pragma unroll
                    for (int i = 0; i < kGroups; ++i) scale[i] = scale_next[i], zero[i] = zero_next[i];
                    load_scales();
                    before = true;
                }
                stat_slot = x_slot;
                if (++w_slot == kWeightSlots) w_slot = 0, w_parity ^= 1;
                if (++x_slot == kXSlots) x_slot = 0, x_parity ^= 1;
            }
            if (before) take_sums(1, stat_slot);

            // ---- the item's end: a cluster's CTAs join, in their order; codes count as code * 2^-9
            float acc[NR];
#pragma unroll
            for (int n = 0; n < NR / 2; ++n) {
                const float2 v = apart(acc2[n]);
                acc[2 * n] = 512.0f * v.x, acc[2 * n + 1] = 512.0f * v.y;
            }
            if (*dead) {
#pragma unroll
                for (int n = 0; n < NR; ++n) acc[n] = __int_as_float(0x7fffffff);
            }
            int n0 = 0, n1 = it.rows;   // the rows that this CTA writes
            if (p.split > 1) {   // (each cluster has one item at most: the ring is used up and serves the join)
                float* const join = reinterpret_cast<float*>(weights);   // [NR][kConsumers]
                consumers_sync();
#pragma unroll
                for (int n = 0; n < NR; ++n) join[n * kConsumers + tid] = acc[n];
                cluster_sync();
                n0 = NR / p.split * rank;   // (the split divides 8)
                n1 = min(it.rows, n0 + NR / p.split);
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    if (n < n0 || n >= n1) continue;
                    float v[kMostSplit];
#pragma unroll
                    for (int r = 0; r < kMostSplit; ++r) {
                        v[r] = 0.0f;
                        if (r >= p.split) continue;
                        uint32_t from;
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(smem_addr(join + n * kConsumers + tid)), "r"(r));
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[r]) : "r"(from) : "memory");
                    }
                    acc[n] = 0.0f;
#pragma unroll
                    for (int r = 0; r < kMostSplit; ++r) acc[n] += v[r];
                }
                cluster_sync();
            }
            T* y = static_cast<T*>(a.y) + static_cast<int64_t>(it.row) * a.y_ld + col;
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                if (n < n0 || n >= n1) continue;
                float v = acc[n];
                if (a.swiglu) v = v / (1.0f + expf(-v)) * __shfl_xor_sync(kFullMask, v, 16);   // gate lanes: silu(gate) * up
                if (real && (!a.swiglu || lane < 16)) y[n * a.y_ld] = from_float<T>(v);
            }
        }
    }
    if (warp >= kLoader && p.split > 1 && item0 < item1) {   // (as the warpgroups do)
        cluster_sync();
        cluster_sync();
    }
    __syncthreads();
    if (warp == kLoader) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kTmem) : "memory");
    }
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

// Bytes [w][z][y][x] (x: 16-byte multiples), read in boxes of 128 x box_y x box_z with the 128-byte swizzle; zeros past the ends.
cudaError_t byte_map(CUtensorMap* map, const void* base, int64_t x, int64_t y, int64_t z, int64_t w, int box_y, int box_z) {
    const EncodeFn encode = encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(x), static_cast<cuuint64_t>(y), static_cast<cuuint64_t>(z),
                                static_cast<cuuint64_t>(w)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(x), static_cast<cuuint64_t>(x * y), static_cast<cuuint64_t>(x * y * z)};
    const cuuint32_t box[4] = {128, static_cast<cuuint32_t>(box_y), static_cast<cuuint32_t>(box_z), 1}, step[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// A device's SMs, and how many clusters of 2, 4 and 8 CTAs of a kernel it holds at once.
struct Room {
    int sms, clusters[3];
};

// Of the current device, with the kernel's shared memory limit raised: looked up once per device (a race writes the
// same values, `ready` after them).
template <typename Kernel>
cudaError_t prepare_kernel(Kernel kernel, int smem, Room* known, int* ready, Room* room) {
    constexpr int kDevices = 64;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < kDevices && __atomic_load_n(&ready[dev], __ATOMIC_ACQUIRE)) {
        *room = known[dev];
        return cudaSuccess;
    }
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&room->sms, cudaDevAttrMultiProcessorCount, dev);
    for (int i = 0; i < 3 && err == cudaSuccess; ++i) {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2 << i;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(room->sms / (2 << i) * (2 << i));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        err = cudaOccupancyMaxActiveClusters(&room->clusters[i], kernel, &cfg);
    }
    if (err == cudaSuccess && dev < kDevices) {
        known[dev] = *room;
        __atomic_store_n(&ready[dev], 1, __ATOMIC_RELEASE);
    }
    return err;
}

int64_t split_bytes(int64_t rows, int I, int dtype) {
    return rows * I * (dtype == EP_DTYPE_FP16 ? kParts<__half> : kParts<__nv_bfloat16>);
}

template <typename T, int NR, int GROUP, bool ZEROS>
cudaError_t launch_shape(const W4Args& a, const unsigned char* x, const float2* stats, cudaStream_t stream) {
    using S = Shape<T, NR, GROUP>;
    static Room known[64];
    static int ready[64];
    constexpr int smem = S::kShared;
    Plan p{};
    Room room{};
    cudaError_t err = prepare_kernel(expert_w4_kernel<T, NR, GROUP, ZEROS>, smem, known, ready, &room);
    if (err != cudaSuccess) return err;
    const int cols = a.swiglu ? a.O / 2 : a.O, cta_cols = kGroupsOfWarps * (a.swiglu ? kTileRows / 2 : kTileRows);
    p.tiles = (cols + cta_cols - 1) / cta_cols;
    while (((a.E - 1) >> p.table_shift) + 1 > kTable) ++p.table_shift;
    p.stages = (a.I + kIn - 1) / kIn;
    p.groups = a.I / GROUP;
    p.stats = reinterpret_cast<const float*>(stats);
    p.slots = room.sms;
    // items at most: an expert of n rows has (n + NR - 1) / NR passes; with few, clusters share them, all at
    // once on the device (4096 x 4096, us: 64 rows, 32 items, 16.9 by clusters of 4, 22.7 of 2; 32 rows, 16 items, of
    // which not all fit as clusters of 8, 16.5 by 4, 23.8 by 8)
    const int64_t used = a.rows < a.E ? a.rows : a.E;
    const int64_t most = (a.rows + used * (NR - 1)) / NR * p.tiles;
    p.split = 1;
    for (int i = 0; p.split < kMostSplit && 2 * p.split <= p.stages && most <= room.clusters[i]; ++i) p.split *= 2;
    const int64_t clusters = most < p.slots / p.split ? most : p.slots / p.split;
    p.slots = static_cast<int>(clusters) * p.split;
    CUtensorMap weight_map, x_map;
    err = a.swiglu ? byte_map(&weight_map, a.w, a.I / 2, cols, 2, a.E, 16, 2) : byte_map(&weight_map, a.w, a.I / 2, a.O, 1, a.E, kTileRows, 1);
    if (err == cudaSuccess) err = byte_map(&x_map, x, a.I, a.rows, kParts<T>, 1, 8, kParts<T>);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.slots);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, expert_w4_kernel<T, NR, GROUP, ZEROS>, a, p, weight_map, x_map);
}

template <typename T, int GROUP>
cudaError_t launch_group(const W4Args& a, void* workspace, int dtype, cudaStream_t stream) {
    float2* stats = static_cast<float2*>(workspace);
    const int64_t stats_bytes = (static_cast<int64_t>(a.rows) * (a.I / GROUP) * 8 + 15) / 16 * 16;
    unsigned char* x = static_cast<unsigned char*>(workspace) + stats_bytes;
    const int64_t blocks = (static_cast<int64_t>(a.rows) * (a.I / 8) + kSplitThreads - 1) / kSplitThreads;
    const cudaError_t err = launch_dependent(split_kernel<T, GROUP>, dim3(static_cast<unsigned>(blocks < 8192 ? blocks : 8192)),
                                             dim3(kSplitThreads), 0, stream, a, x, stats);
    if (err != cudaSuccess) return err;
    // rows of an item: 8, or 16 where experts have more than 4 rows on average: a second pass over a tile costs more than
    // columns that stay empty (256 tokens, 8 rows an expert: 935 us with 8, 773 with 16 when that was measured)
    const int used = a.rows < a.E ? a.rows : a.E, mean = (a.rows - 1) / used + 1;
    if constexpr (kParts<T> == 2)
        if (mean <= 4 || a.rows <= 8)
            return a.zeros ? launch_shape<T, 8, GROUP, true>(a, x, stats, stream) : launch_shape<T, 8, GROUP, false>(a, x, stats, stream);
    return a.zeros ? launch_shape<T, 16, GROUP, true>(a, x, stats, stream) : launch_shape<T, 16, GROUP, false>(a, x, stats, stream);
}

template <typename T>
cudaError_t launch_type(const W4Args& a, void* workspace, int dtype, cudaStream_t stream) {
    return a.group == 32   ? launch_group<T, 32>(a, workspace, dtype, stream)
           : a.group == 64 ? launch_group<T, 64>(a, workspace, dtype, stream)
                           : launch_group<T, 128>(a, workspace, dtype, stream);
}

}  // namespace

int64_t expert_w4_workspace(int64_t rows, int I, int group, int dtype) {
    return (rows * (I / group) * 8 + 15) / 16 * 16 + split_bytes(rows, I, dtype);
}

cudaError_t launch_expert_w4(const W4Args& a, void* workspace, int dtype, cudaStream_t stream) {
    if (expert_w4_few(a)) return launch_expert_w4_few(a, dtype, stream);
    return dtype == EP_DTYPE_BF16 ? launch_type<__nv_bfloat16>(a, workspace, dtype, stream)
                                  : launch_type<__half>(a, workspace, dtype, stream);
}

}  // namespace ep
