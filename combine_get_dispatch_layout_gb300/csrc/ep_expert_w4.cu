// The experts' products on dispatched rows: 4-bit weights, group scales.
//
// Mathematics. y[n, o] = sum over groups g of s[g, o] * sum over i in g of
// (code[o, i] - zero[g, o]) x[n, i]. The inner sums run through the 5th-generation
// tensor cores on e4m3 operands with fp32 sums:
//  - a code 0 .. 15 in a byte IS the e4m3 number code * 2^-9 (subnormal up to 7,
//    the first binade from 8 on), so unpacking eight codes is two masks and one
//    shift. (As bf16 operands of mma.sync they take 11 instructions, and that
//    kernel ran at 37 % of the memory rate, bound by instruction issue; e4m3
//    operands of mma.sync are converted to fp16 by further instructions.)
//  - x is taken as a sum of e4m3 numbers, two for bf16 and three for fp16, after
//    a power of two has brought the largest input of the group to [128, 256).
//    Four significant bits each make up the 8 or 11 of x, exactly, down to
//    e4m3's smallest step: what is left off is below 2^-17 of the group's
//    largest. The product's narrow side is 16 wide at least: the parts of 8 rows
//    share it, those of more rows are added into the same sums.
//  - the zero point enters as zero * (sum of the group's inputs), in fp32.
// Scales multiply a group's sum in fp32. y is rounded once.
//
// What bounds it: with few rows per expert each weight is used a few times, so
// reading the codes (half a byte each) once is the floor. Instruction issue is
// next: about 6 instructions a word of 8 codes of the 22 clocks that DRAM takes
// for 128 bytes an SM quarter.
//
// Layout. A tile of 128 weight rows is the product's 128 lanes: thread = weight
// row = TMEM lane, for unpacking (shared memory to TMEM operand A), for the
// scales (one a thread) and for the sums (tcgen05.ld, one column a row of x). A
// persistent CTA walks its items (an expert, a tile, at most NR rows of x). One
// warp fills a ring of stages (256 inputs: 16 KB of codes by TMA) that runs on
// across items; two warpgroups take half a stage each: they unpack it, hand it
// to the warp that issues the products, and take in the sums of the half before
// meanwhile. The first weights are on their way while split_kernel still runs.
// Where there are few items, the CTAs of a cluster share an item's inputs and
// join through distributed shared memory.
#include <cuda.h>

#include <type_traits>

#include "ep_layer.cuh"

namespace ep {
namespace {

constexpr int kThreads = 320;          // two warpgroups, a warp that loads, a warp that issues products
constexpr int kConsumers = 256;
constexpr int kLoader = kConsumers / 32, kIssuer = kLoader + 1;   // warps
constexpr int kRows = 128;             // weight rows of a tile
constexpr int kIn = 256;               // inputs of a stage, 128 a warpgroup
constexpr int kWeightBytes = kRows * kIn / 2;
constexpr int kSplitThreads = 256;
constexpr int kMostSplit = 8;          // CTAs of a cluster that share an item

// Parts that x is split into.
template <typename T>
constexpr int kParts = std::is_same_v<T, __half> ? 3 : 2;

constexpr int power_of_two(int n) { return n <= 32 ? 32 : 2 * power_of_two((n + 1) / 2); }

// T: type of x, scales and y. NR: rows of x of an item. GROUP: inputs that share a scale.
template <typename T, int NR, int GROUP>
struct Shape {
    static constexpr bool kSideBySide = NR == 8;               // two parts of 8 rows in one product
    static_assert(NR % 16 == 0 || (kSideBySide && kParts<T> == 2), "");
    static constexpr int kN = kSideBySide ? 16 : NR;           // columns of the product
    static constexpr int kProducts = kSideBySide ? 1 : kParts<T>;
    static constexpr int kGroups = 128 / GROUP;                // of a warpgroup's half of a stage
    static constexpr int kXBytes = NR * kParts<T> * 128;       // x of half a stage
    static constexpr int kStats = 2 * kGroups * NR * 2;        // floats of a stage
    static constexpr int kSumCols = kN * kGroups;
    // columns of TMEM: operand A twice for both warpgroups, sums twice too where that leaves room for two CTAs a core
    static constexpr int kSumBuffers = 128 + 4 * kSumCols <= 256 ? 2 : 1;
    static constexpr int kTmem = power_of_two(128 + 2 * kSumBuffers * kSumCols);
    static constexpr int kStageBytes = kWeightBytes + 2 * kXBytes + kStats * 4;
    // two CTAs a core where TMEM (512 columns) allows it
    static constexpr int kResident = kTmem <= 256 ? 2 : 1;
    static constexpr int kFixed = NR * kRows * 4 + 2048;       // join buffer, barriers, alignment
    static constexpr int kTable = 4 * (EP_MAX_EXPERTS + 1) + 1024;   // first_pass, at most (two CTAs have room for a quarter)
    static constexpr int kFit = (227 * 1024 / kResident - 1024 - kFixed - kTable / (kResident * kResident)) / kStageBytes;
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static_assert(kStages >= 2 && kN % 16 == 0 && kN <= 256 && kTmem <= 512, "");
};

struct Plan {
    int tiles;       // of an expert
    int slots;       // CTAs of the grid
    int split;       // CTAs that share an item
    int stages;      // of an item
    int groups;      // of a weight row
    const float* stats;    // [rows][groups][2]: power of two, 2^-9 * sum, of a group's inputs
};

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

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
__device__ __forceinline__ void barrier_wait(uint32_t bar, uint32_t parity, volatile int* dead) {
    for (int i = 0; i < (1 << 22); ++i) {
        if (barrier_try(bar, parity)) return;
        if ((i & 1023) == 1023 && *dead) return;
    }
    *dead = 1;
}
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int real) {   // zeros where real is 0
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(128) : "memory"); }
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 3, %0;" ::"n"(kConsumers) : "memory"); }

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
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t (&u)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
                   "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
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
// Rows of 128 bytes along the inputs, 128-byte swizzle: 8 rows are 1024 bytes.
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3fff) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}

// ------------------------------------------------------------------ rows and items

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

struct Item {
    int expert, row, rows, col;   // col: first output column of the tile
};

// Four values as e4m3 codes in a word, each reduced by what its code stands for.
__device__ __forceinline__ uint32_t take_part(float (&v)[4]) {
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(make_float2(v[i], v[i + 1]), __NV_SATFINITE, __NV_E4M3);
        const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
        v[i] -= f.x;
        v[i + 1] -= f.y;
        word |= static_cast<uint32_t>(c) << (8 * i);
    }
    return word;
}

// x as sums of e4m3 numbers, a plane [rows][I] for each part; of 8 neighbouring inputs the even ones come first, as
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
            w.x = take_part(even);
            w.y = take_part(odd);
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

template <typename T, int NR, int GROUP>
__global__ void __launch_bounds__(kThreads, (Shape<T, NR, GROUP>::kResident))
    expert_w4_kernel(W4Args a, Plan p, const __grid_constant__ CUtensorMap weight_map, const __grid_constant__ CUtensorMap x_map) {
    using S = Shape<T, NR, GROUP>;
    constexpr int kStages = S::kStages, kGroups = S::kGroups;
    extern __shared__ unsigned char shared_bytes[];
    // [kStages] weights (rows of 128 bytes, 128-byte swizzle), [kStages] x (two halves [parts][NR][128 bytes]), stats, the
    // join buffer [NR][kRows], barriers, first_pass [E + 1]. stats: [kStages][2][kGroups] of NR / 2 pairs of rows, a pair's
    // two powers of two, then its two sums
    unsigned char* const weights = shared_bytes + (1024 - smem_addr(shared_bytes) % 1024) % 1024;
    unsigned char* const inputs = weights + kStages * kWeightBytes;
    float* const stats = reinterpret_cast<float*>(inputs + kStages * 2 * S::kXBytes);
    float* const join = reinterpret_cast<float*>(stats + kStages * S::kStats);
    uint64_t* const barriers = reinterpret_cast<uint64_t*>(join + NR * kRows);
    const uint32_t full = smem_addr(barriers), empty = full + 8 * kStages;
    const uint32_t ready = empty + 8 * kStages, done = ready + 32;   // [2 warpgroups][2 buffers]
    uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(barriers + 2 * kStages + 8);
    volatile int* const dead = reinterpret_cast<volatile int*>(tmem_at + 1);
    int* const first_pass = reinterpret_cast<int*>(tmem_at + 2);
    __shared__ int warp_sum[kThreads / 32];
    // Everything before split_kernel, which this kernel follows, is complete once this one runs: split_kernel lets it
    // start only after it has waited for that itself. So all but split_kernel's own outputs can be read at once, and
    // griddepcontrol.wait comes before those (in the loading warp; the others see them through its barriers).

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cols = a.swiglu ? a.O / 2 : a.O, tile_cols = a.swiglu ? kRows / 2 : kRows;
    const int rank = blockIdx.x % p.split;

    if (warp == kLoader) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_at)), "n"(S::kTmem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        if (lane == 0) {
            *dead = 0;
            for (int i = 0; i < kStages; ++i) {
                barrier_init(full + 8 * i, 33);                  // the TMA loads' thread and 32 lanes' copies
                barrier_init(empty + 8 * i, kConsumers / 32);
            }
            for (int i = 0; i < 4; ++i) {
                barrier_init(ready + 8 * i, 4);
                barrier_init(done + 8 * i, 1);
            }
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    }
    // ---- items: an expert's rows in passes of NR, each pass over all tiles; a tile's passes follow each other, so
    // the weights of the second come from L2
    {
        const int per = (a.E + kThreads - 1) / kThreads, lo = min(a.E, tid * per), hi = min(a.E, lo + per);
        int own = 0, first;
        for (int e = lo; e < hi; ++e) own += (expert_rows(a, e, first) + NR - 1) / NR;
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
        for (int e = lo; e < hi; ++e) {
            first_pass[e] = base;
            base += (expert_rows(a, e, first) + NR - 1) / NR;
        }
        if (hi == a.E && lo < hi) first_pass[a.E] = base;
        tmem_fence_before();
        __syncthreads();
        tmem_fence_after();
    }
    const uint32_t tmem = *tmem_at;
    const int64_t items = static_cast<int64_t>(first_pass[a.E]) * p.tiles;
    // as many clusters as share the items evenly: all of them wait on the same DRAM, so an SM with one CTA less costs nothing
    const int clusters = p.slots / p.split;
    const int64_t each = (items + clusters - 1) / clusters;
    const int64_t item0 = min(items, each * (blockIdx.x / p.split)), item1 = min(items, item0 + each);
    // this CTA's stages of every item
    const int stage0 = p.stages * rank / p.split, stage1 = p.stages * (rank + 1) / p.split;

    const auto decode = [&](int64_t it) {
        int lo = 0, hi = a.E - 1;   // the last expert whose first item is not behind `it`: it has passes of its own
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (static_cast<int64_t>(first_pass[mid]) * p.tiles <= it) lo = mid;
            else hi = mid - 1;
        }
        const int passes = first_pass[lo + 1] - first_pass[lo];
        const int in = static_cast<int>(it - static_cast<int64_t>(first_pass[lo]) * p.tiles);
        Item r;
        int first;
        const int n = expert_rows(a, lo, first), pass = in % passes;
        r.expert = lo;
        r.row = first + pass * NR;
        r.rows = min(NR, n - pass * NR);
        r.col = in / passes * tile_cols;
        return r;
    };

    const int64_t steps = (item1 - item0) * (stage1 - stage0);

    if (warp == kLoader) {
        const auto load_weights = [&](const Item& it, int stage, int slot) {
            if (lane != 0) return;
            const uint32_t bar = full + 8 * slot, to = smem_addr(weights) + slot * kWeightBytes;
            barrier_expect(bar, kWeightBytes + 2 * S::kXBytes);
            load_tile(to, &weight_map, stage * (kIn / 2), it.col, it.expert, bar);
            if (a.swiglu) load_tile(to + kWeightBytes / 2, &weight_map, stage * (kIn / 2), cols + it.col, it.expert, bar);
        };
        const auto load_inputs = [&](const Item& it, int stage, int slot) {
            const uint32_t bar = full + 8 * slot;
            if (lane == 0)
                for (int h = 0; h < 2; ++h)
                    load_tile(smem_addr(inputs) + (slot * 2 + h) * S::kXBytes, &x_map, stage * kIn + h * 128, it.row, 0, bar);
            for (int i = lane; i < S::kStats; i += 32) {
                const int n = i / 4 % (NR / 2) * 2 + (i & 1), which = (i >> 1) & 1, grp = stage * (kIn / GROUP) + i / (2 * NR);
                const bool in = n < it.rows && grp < p.groups;
                copy4(smem_addr(stats + slot * S::kStats + i),
                      p.stats + (in ? (static_cast<int64_t>(it.row + n) * p.groups + grp) * 2 + which : 0), in ? 4 : 0);
            }
            copies_arrive(bar);
        };
        const int first_steps = static_cast<int>(min(steps, static_cast<int64_t>(kStages)));
        int64_t item = item0;
        int stage = stage0;
        Item it{};
        const auto next = [&]() {
            if (++stage == stage1) stage = stage0, ++item;
        };
        for (int i = 0; i < first_steps; ++i, next()) {
            if (i == 0 || stage == stage0) it = decode(item);
            load_weights(it, stage, i);
        }
        dependent_entry();
        item = item0, stage = stage0;
        for (int64_t i = 0; i < steps; ++i, next()) {
            const int slot = static_cast<int>(i % kStages);
            if (i == 0 || stage == stage0) it = decode(item);
            if (i >= kStages) {
                barrier_wait(empty + 8 * slot, (i / kStages + 1) & 1, dead);
                load_weights(it, stage, slot);
            }
            load_inputs(it, stage, slot);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == kIssuer) {
        if (lane == 0) {
            constexpr uint32_t kShape = (1u << 4) | (static_cast<uint32_t>(S::kN / 8) << 17) | (static_cast<uint32_t>(kRows / 16) << 24);
            int slot = 0, buffer = 0;
            uint32_t full_parity = 0, ready_parity = 0;
            for (int64_t i = 0; i < steps; ++i) {
                barrier_wait(full + 8 * slot, full_parity, dead);
                for (int wg = 0; wg < 2; ++wg) {
                    barrier_wait(ready + 8 * (wg * 2 + buffer), ready_parity, dead);
                    tmem_fence_after();
                    const uint32_t a_at = tmem + wg * 64 + buffer * 32;
                    const uint32_t sums = tmem + 128 + (wg * S::kSumBuffers + (S::kSumBuffers == 2 ? buffer : 0)) * S::kSumCols;
                    const uint64_t b = operand(smem_addr(inputs) + (slot * 2 + wg) * S::kXBytes);
#pragma unroll
                    for (int grp = 0; grp < kGroups; ++grp)
#pragma unroll
                        for (int part = 0; part < S::kProducts; ++part)
#pragma unroll
                            for (int k = 0; k < GROUP / 32; ++k) {
                                const int step = grp * (GROUP / 32) + k;
                                multiply(sums + grp * S::kN, a_at + step * 8, b + step * 2 + part * (NR * 128 / 16), kShape, part > 0 || k > 0);
                            }
                    multiply_done(done + 8 * (wg * 2 + buffer));
                }
                buffer ^= 1;
                if (buffer == 0) ready_parity ^= 1;
                if (++slot == kStages) slot = 0, full_parity ^= 1;
            }
        }
        __syncwarp();
    } else {
        // ---- a warpgroup: unpack half a stage, take in the sums of the half before
        const int wg = warp >> 2, row = tid & 127;      // row: of the tile; its TMEM lane
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // lane 32 * (warp % 4) in an address's upper half
        const uint32_t operand_at = tmem + wg * 64 + lanes, sums_at = tmem + 128 + wg * S::kSumBuffers * S::kSumCols + lanes;
        int slot = 0, buffer = 0;
        uint32_t full_parity = 0, done_parity = 0;   // of done: a bit a buffer
        for (int64_t item = item0; item < item1; ++item) {
            const Item it = decode(item);
            int o;   // this thread's weight row; with an activation the tile's halves are gate and up rows
            if (a.swiglu) {
                const int j = it.col + (row & 63);
                o = j >= cols ? -1 : row < 64 ? j : cols + j;
            } else {
                o = it.col + row < cols ? it.col + row : -1;
            }
            const int64_t scale_base = static_cast<int64_t>(it.expert) * p.groups * a.O + max(o, 0);
            T scale[kGroups], scale_next[kGroups];
            uint8_t zero[kGroups], zero_next[kGroups];
            const auto load_scales = [&](int stage) {
#pragma unroll
                for (int i = 0; i < kGroups; ++i) {
                    const int grp = (stage * kIn + wg * 128) / GROUP + i;
                    scale_next[i] = from_float<T>(0.0f);
                    zero_next[i] = 8;
                    if (o >= 0 && grp < p.groups) {
                        scale_next[i] = static_cast<const T*>(a.scales)[scale_base + static_cast<int64_t>(grp) * a.O];
                        if (a.zeros) zero_next[i] = a.zeros[scale_base + static_cast<int64_t>(grp) * a.O];
                    }
                }
            };
            uint64_t acc2[NR / 2];   // rows 2 n, 2 n + 1
#pragma unroll
            for (int n = 0; n < NR / 2; ++n) acc2[n] = 0;
            // takes in the sums of the half stage that was multiplied into buffer b, its slot s
            const auto take_sums = [&](int b, int s) {
                barrier_wait(done + 8 * (wg * 2 + b), (done_parity >> b) & 1, dead);
                done_parity ^= 1u << b;
                tmem_fence_after();
#pragma unroll
                for (int i = 0; i < kGroups; ++i) {
                    const uint64_t sc = both(to_float(scale[i])), z = both(-static_cast<float>(zero[i]));
                    const float* st = stats + s * S::kStats + (wg * kGroups + i) * (NR * 2);
                    uint32_t v[S::kN / 16][16];
#pragma unroll
                    for (int k = 0; k < S::kN / 16; ++k)
                        tmem_load16(sums_at + (S::kSumBuffers == 2 ? b * S::kSumCols : 0) + i * S::kN + 16 * k, v[k]);
                    tmem_load_wait();
#pragma unroll
                    for (int n = 0; n < NR / 2; ++n) {
                        uint64_t sum = pair(v[n / 8][n % 8 * 2], v[n / 8][n % 8 * 2 + 1]);
                        if constexpr (S::kSideBySide) sum = add2(sum, pair(v[0][8 + 2 * n], v[0][8 + 2 * n + 1]));
                        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(st + 4 * n);
                        acc2[n] = fma2(mul2(sc, f.x), fma2(z, f.y, sum), acc2[n]);
                    }
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) barrier_arrive(empty + 8 * s);
            };
            load_scales(stage0);
            int before = -1;
            for (int stage = stage0; stage < stage1; ++stage) {
                barrier_wait(full + 8 * slot, full_parity, dead);
                const unsigned char* w = weights + slot * kWeightBytes + row * 128;
                uint32_t codes[32];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 v = *reinterpret_cast<const uint4*>(w + (((4 * wg + j) ^ (row & 7)) << 4));
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        codes[8 * j + 2 * k] = u[k] & 0x0f0f0f0fu;
                        codes[8 * j + 2 * k + 1] = (u[k] >> 4) & 0x0f0f0f0fu;
                    }
                }
                // (the products that read this operand buffer last have been waited for in take_sums)
                tmem_store32(operand_at + buffer * 32, codes);
                if (S::kSumBuffers == 1 && before >= 0) take_sums(buffer ^ 1, before);
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) barrier_arrive(ready + 8 * (wg * 2 + buffer));
                if (S::kSumBuffers == 2 && before >= 0) take_sums(buffer ^ 1, before);
#pragma unroll
                for (int i = 0; i < kGroups; ++i) scale[i] = scale_next[i], zero[i] = zero_next[i];
                if (stage + 1 < stage1) load_scales(stage + 1);
                before = slot;
                buffer ^= 1;
                if (++slot == kStages) slot = 0, full_parity ^= 1;
            }
            if (before >= 0) take_sums(buffer ^ 1, before);

            float acc[NR];
#pragma unroll
            for (int n = 0; n < NR / 2; ++n) {
                const float2 v = apart(acc2[n]);
                acc[2 * n] = v.x, acc[2 * n + 1] = v.y;
            }
            // ---- the item's end: the warpgroups join, then the cluster's CTAs, in their order; codes count as code * 2^-9
            if (wg == 1) {
#pragma unroll
                for (int n = 0; n < NR; ++n) join[n * kRows + row] = acc[n];
            }
            consumers_sync();
            if (wg == 0) {
#pragma unroll
                for (int n = 0; n < NR; ++n) acc[n] = 512.0f * (acc[n] + join[n * kRows + row]);
                if (*dead) {
#pragma unroll
                    for (int n = 0; n < NR; ++n) acc[n] = __int_as_float(0x7fffffff);
                }
            }
            if (p.split > 1) {
                if (wg == 0) {   // (its own entries of the join buffer: no one else reads them before the cluster's barrier)
#pragma unroll
                    for (int n = 0; n < NR; ++n) join[n * kRows + row] = acc[n];
                }
                asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
                if (wg == 0 && rank == 0) {
                    for (int r = 1; r < p.split; ++r) {
                        uint32_t from;
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(smem_addr(join)), "r"(r));
#pragma unroll
                        for (int n = 0; n < NR; ++n) {
                            float v;
                            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(from + (n * kRows + row) * 4) : "memory");
                            acc[n] += v;
                        }
                    }
                }
                asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
            }
            if (rank == 0) {
                T* y = static_cast<T*>(a.y) + static_cast<int64_t>(it.row) * a.y_ld + it.col;
                if (a.swiglu) {
                    if (wg == 0 && row >= 64) {
#pragma unroll
                        for (int n = 0; n < NR; ++n) join[n * kRows + row] = acc[n];
                    }
                    if (wg == 0) {
                        group_sync(1);
                        if (row < 64 && o >= 0) {
#pragma unroll
                            for (int n = 0; n < NR; ++n)
                                if (n < it.rows)
                                    y[n * a.y_ld + row] =
                                        from_float<T>(acc[n] / (1.0f + expf(-acc[n])) * join[n * kRows + 64 + row]);
                        }
                    }
                } else if (wg == 0 && o >= 0) {
#pragma unroll
                    for (int n = 0; n < NR; ++n)
                        if (n < it.rows) y[n * a.y_ld + row] = from_float<T>(acc[n]);
                }
            }
            consumers_sync();   // the join buffer is free again
        }
    }
    // (with clusters each has one item at most, so the other warps are through with it)
    if (warp >= kLoader && p.split > 1 && item0 < item1) {
        asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
        asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
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

// Bytes [z][y][x], read in boxes of 128 x box_y x box_z; zeros past the ends.
cudaError_t byte_map(CUtensorMap* map, const void* base, int64_t x, int64_t y, int64_t z, int box_y, int box_z) {
    const EncodeFn encode = encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(x), static_cast<cuuint64_t>(y), static_cast<cuuint64_t>(z)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(x), static_cast<cuuint64_t>(x * y)};
    const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(box_y), static_cast<cuuint32_t>(box_z)}, step[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// SMs of the current device, with the kernel's shared memory limit raised for at least this size: looked up when a
// larger size than before comes (a race writes the same values).
template <typename Kernel>
cudaError_t prepare_kernel(Kernel kernel, int smem, int* known_smem, int* known_sms, int* sms) {
    constexpr int kDevices = 64;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < kDevices && __atomic_load_n(&known_smem[dev], __ATOMIC_ACQUIRE) >= smem) {
        *sms = __atomic_load_n(&known_sms[dev], __ATOMIC_RELAXED);
        return cudaSuccess;
    }
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    if (dev < kDevices) {
        __atomic_store_n(&known_sms[dev], *sms, __ATOMIC_RELAXED);
        __atomic_store_n(&known_smem[dev], smem, __ATOMIC_RELEASE);
    }
    return cudaSuccess;
}

int64_t split_bytes(int64_t rows, int I, int dtype) {
    return rows * I * (dtype == EP_DTYPE_FP16 ? kParts<__half> : kParts<__nv_bfloat16>);
}

template <typename T, int NR, int GROUP>
cudaError_t launch_shape(const W4Args& a, const unsigned char* x, const float2* stats, cudaStream_t stream) {
    using S = Shape<T, NR, GROUP>;
    static int known_smem[64], known_sms[64];
    const int smem = S::kStages * S::kStageBytes + S::kFixed + (a.E + 1) * 4;
    Plan p{};
    int sms = 0;
    cudaError_t err = prepare_kernel(expert_w4_kernel<T, NR, GROUP>, smem, known_smem, known_sms, &sms);
    if (err != cudaSuccess) return err;
    const int tile_cols = a.swiglu ? kRows / 2 : kRows, cols = a.swiglu ? a.O / 2 : a.O;
    p.tiles = (cols + tile_cols - 1) / tile_cols;
    p.stages = (a.I + kIn - 1) / kIn;
    p.groups = a.I / GROUP;
    p.stats = reinterpret_cast<const float*>(stats);
    p.slots = sms * S::kResident;
    // items at most; with fewer than half the CTAs' number, clusters share them
    const int64_t most = (static_cast<int64_t>(a.rows) / NR + (a.rows < a.E ? a.rows : a.E)) * p.tiles;
    p.split = 1;
    while (p.split < kMostSplit && 2 * p.split <= p.stages && most * 2 * p.split <= p.slots) p.split *= 2;
    const int64_t clusters = most < p.slots / p.split ? most : p.slots / p.split;
    p.slots = static_cast<int>(clusters) * p.split;
    CUtensorMap weight_map, x_map;
    err = byte_map(&weight_map, a.w, a.I / 2, a.O, a.E, tile_cols, 1);
    if (err == cudaSuccess) err = byte_map(&x_map, x, a.I, a.rows, kParts<T>, NR, kParts<T>);
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
    return cudaLaunchKernelEx(&cfg, expert_w4_kernel<T, NR, GROUP>, a, p, weight_map, x_map);
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
    // rows of an item: 8, or 16 where experts have more than 4 rows on average (a second pass over a tile costs more)
    const int used = a.rows < a.E ? a.rows : a.E, mean = (a.rows + used - 1) / used;
    if constexpr (kParts<T> == 2)
        if (mean <= 4 || a.rows <= 8) return launch_shape<T, 8, GROUP>(a, x, stats, stream);
    return launch_shape<T, 16, GROUP>(a, x, stats, stream);
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
    return dtype == EP_DTYPE_BF16 ? launch_type<__nv_bfloat16>(a, workspace, dtype, stream)
                                  : launch_type<__half>(a, workspace, dtype, stream);
}

}  // namespace ep
