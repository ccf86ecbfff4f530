// The experts' products on dispatched rows: 4-bit weights, group scales.
//
// Mathematics. y[n, o] = sum over groups g of s[g, o] * sum over i in g of
// (code[o, i] - zero[g, o]) x[n, i]. code - zero is a whole number of at most five
// bits and exact in fp16; x is exact in fp16 once a power of two has brought the
// row's largest input to [2^14, 2^15) (down to 2^-28 of it, below that to
// 2^-39 of it). So the inner sums run through the fp16 matrix instruction with
// exact products and fp32 sums, and the scale multiplies a group's sum in fp32:
// no weight is rounded.
//
// What bounds it: with few rows per expert each weight is used a few times, so
// reading the codes (half a byte each) once is the floor: 22 clocks for 128 bytes
// an SM quarter. Next is instruction issue: a word of eight codes takes five
// logic instructions (two nibble pairs under an fp16 exponent, one shift, two
// more), four fp16 ones for the zero points, and a matrix instruction for each 8
// rows. Measured on the way, for 256 tokens: bf16 operands (three shifts, loads
// and copies by all warps) 1562 us, bound by issue; codes as e4m3 numbers
// through tcgen05.mma with the unpacked operand in TMEM 925 us, bound by TMEM,
// which takes the unpacked operand in and out (a product of 128 x 32 inputs 54
// clocks however narrow).
//
// Layout. Weight rows are the instruction's 16 rows, dispatched rows its 8
// columns. The order of a product's inputs is free: a thread takes neighbouring
// codes of a weight row, in the order in which masks leave them ((0, 4), (1, 5),
// (2, 6), (3, 7) of a word), and x is written in the order in which the threads
// ask for it (order_kernel), so the codes are used in the plain layout in which
// they are stored. One persistent CTA a core walks its items (an expert, 512
// weight rows, at most 8 NT rows of x). One warp fills the rings by TMA, straight on
// across items: stages of 256 inputs, 64 KB of codes; x, which comes from L2, is
// shared by all 512 rows (with 128 rows it was half as much traffic again as the
// codes, and the ring alone could not pass 77 % of the memory rate). Sixteen
// warps take 32 rows each and never wait for each other. The first weights are on
// their way while order_kernel still runs. Where there are few items, the CTAs of
// a cluster share an item's inputs and join through distributed shared memory.
#include <cuda.h>

#include <type_traits>

#include "ep_layer.cuh"

namespace ep {
namespace {

constexpr int kWarps = 16;                         // that multiply
constexpr int kConsumers = 32 * kWarps;
constexpr int kLoader = kWarps;                    // the warp that loads
constexpr int kThreads = kConsumers + 32;
constexpr int kWarpRows = 32;                      // weight rows of a warp: two of the instruction
constexpr int kIn = 256;                           // inputs of a stage
constexpr int kWarpBytes = kWarpRows * kIn / 2;
constexpr int kWeightBytes = kWarps * kWarpBytes;
constexpr int kWeightSlots = 3, kXSlots = 3;
constexpr int kOrderThreads = 256;
constexpr int kMostSplit = 8;                      // CTAs of a cluster that share an item
constexpr int kTable = 1024;                       // entries of the table of experts' passes

// NT: eights of rows of x of an item. GROUP: inputs that share a scale; a thread takes GROUP / 32 words of a row.
template <int NT, int GROUP>
struct Shape {
    static constexpr int kXBytes = NT * 8 * kIn * 2;           // x of a stage
    static constexpr int kShared = 1024 + kWeightSlots * kWeightBytes + kXSlots * kXBytes + 256 + (kTable + 1) * 4;
    static_assert(kShared <= 227 * 1024 - 256, "");
    // Row of the instruction g, of 8, is weight row place(g): loads of 16 (8) bytes by 8 (16) lanes then find 2 (4)
    // rows that the 128-byte swizzle, which exchanges 16-byte pieces by the row's number, keeps on different banks.
    static __device__ __forceinline__ int place(int g) {
        if constexpr (GROUP == 128) return x_place(g);
        return (g & 3) * 2 + (g >> 2);
    }
    // Column g is row x_place(g) of the eight, for the same reason (x is always loaded 16 bytes by 8 lanes).
    static __device__ __forceinline__ int x_place(int g) { return (g & 1) * 4 + (g >> 1); }
};

struct Plan {
    int tiles;       // of kConsumers weight rows, of an expert
    int table_shift; // an entry of the table stands for 2^table_shift experts
    int slots;       // CTAs of the grid
    int split;       // CTAs that share an item
    int stages;      // of an item
    int groups;      // of a weight row
    const float* factor;   // [rows]: what x was divided by
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
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); }
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void multiply(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bits(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }
__device__ __forceinline__ __half2 halves(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }

// Two codes of a word as fp16 numbers less the zero point: in the low mantissa bits under the exponent of 1024 they
// read 1024 + code, four bits further up 1024 + 16 code. low = -(1024 + zero), high = -(64 + zero), both exact.
__device__ __forceinline__ uint32_t low_pair(uint32_t w, __half2 low) {
    return bits(__hadd2(halves((w & 0x000f000fu) | 0x64006400u), low));
}
__device__ __forceinline__ uint32_t high_pair(uint32_t w, __half2 high) {
    return bits(__hfma2(halves((w & 0x00f000f0u) | 0x64006400u), halves(0x2c002c00u), high));   // * 1/16
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

// x as fp16, a row divided by a power of two (bf16 only), in the order in which the threads of expert_w4_kernel ask for
// it: the eights of a group of 128 (64, 32), thread by thread before word by word there, are written word by word. Of an
// eight the pairs (0, 4), (1, 5), (2, 6), (3, 7). One block a row.
template <typename T, int GROUP>
__global__ void __launch_bounds__(kOrderThreads) order_kernel(W4Args a, uint4* to, float* factor) {
    dependent_entry();
    constexpr bool kScaled = std::is_same_v<T, __nv_bfloat16>;
    constexpr int kWords = GROUP / 32, kEights = GROUP / 8;
    __shared__ float biggest[kOrderThreads / 32];
    const int last = a.offsets ? min(max(a.offsets[a.E], 0), a.rows) : a.rows;   // rows behind belong to nobody
    const int per_row = a.I / 8;
    for (int row = blockIdx.x; row < last; row += gridDim.x) {
        const T* from = static_cast<const T*>(a.x) + static_cast<int64_t>(row) * a.x_ld;
        float up = 1.0f;
        if constexpr (kScaled) {
            float big = 0.0f;
            for (int c = threadIdx.x; c < per_row; c += kOrderThreads) {
                Vec8<T> v;
                v.raw = *reinterpret_cast<const uint4*>(from + c * 8);
#pragma unroll
                for (int k = 0; k < 8; ++k) big = fmaxf(big, fabsf(to_float(v.v[k])));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(kFullMask, big, o));
            if (threadIdx.x % 32 == 0) biggest[threadIdx.x / 32] = big;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kOrderThreads / 32; ++w) big = fmaxf(big, biggest[w]);
            __syncthreads();
            const int e = big > 0.0f && big < INFINITY ? min(14 - ilogbf(big), 126) : 0;
            up = __int_as_float((e + 127) << 23);
            if (threadIdx.x == 0) factor[row] = __int_as_float((127 - e) << 23);
        }
        for (int c = threadIdx.x; c < per_row; c += kOrderThreads) {
            Vec8<T> v;
            v.raw = *reinterpret_cast<const uint4*>(from + c * 8);
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (kScaled) w[k] = bits(__floats2half2_rn(to_float(v.v[k]) * up, to_float(v.v[k + 4]) * up));
                else w[k] = bits(__halves2half2(v.v[k], v.v[k + 4]));
            }
            const int in = c % kEights;   // thread in / kWords, word in % kWords
            to[static_cast<int64_t>(row) * per_row + c - in + in % kWords * 4 + in / kWords] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

template <typename T, int NT, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kThreads, 1)
    expert_w4_kernel(W4Args a, Plan p, const __grid_constant__ CUtensorMap weight_map, const __grid_constant__ CUtensorMap x_map) {
    using S = Shape<NT, GROUP>;
    constexpr int kItemRows = 8 * NT;
    extern __shared__ unsigned char shared_bytes[];
    // weights: [kWeightSlots][warp][32 rows][128 bytes], 128-byte swizzle; inputs: [kXSlots][64 inputs][NT][8 rows][128 bytes],
    // likewise; barriers; the table of passes
    unsigned char* const weights = shared_bytes + (1024 - smem_addr(shared_bytes) % 1024) % 1024;
    unsigned char* const inputs = weights + kWeightSlots * kWeightBytes;
    uint64_t* const barriers = reinterpret_cast<uint64_t*>(inputs + kXSlots * S::kXBytes);
    const uint32_t w_full = smem_addr(barriers), w_empty = w_full + 8 * kWeightSlots;
    const uint32_t x_full = w_empty + 8 * kWeightSlots, x_empty = x_full + 8 * kXSlots;
    volatile int* const dead = reinterpret_cast<volatile int*>(barriers + 2 * (kWeightSlots + kXSlots));
    int* const table = reinterpret_cast<int*>(barriers + 32);
    static_assert(2 * (kWeightSlots + kXSlots) < 32, "");
    __shared__ int warp_sum[kThreads / 32];
    // Everything before order_kernel, which this kernel follows, is complete once this one runs: order_kernel lets it
    // start only after it has waited for that itself. So all but order_kernel's own outputs can be read at once, and
    // griddepcontrol.wait comes before those (in the loading warp; the others see them through its barriers).

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cols = a.swiglu ? a.O / 2 : a.O;
    const int warp_cols = a.swiglu ? kWarpRows / 2 : kWarpRows;   // output columns of a warp
    const int rank = blockIdx.x % p.split;

    if (tid == kConsumers) {
        *dead = 0;
        for (int i = 0; i < kWeightSlots; ++i) {
            barrier_init(w_full + 8 * i, 1);
            barrier_init(w_empty + 8 * i, kWarps);
        }
        for (int i = 0; i < kXSlots; ++i) {
            barrier_init(x_full + 8 * i, 1);
            barrier_init(x_empty + 8 * i, kWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // ---- items: an expert's rows in passes of 8 NT, each pass over all tiles; a tile's passes follow each other, so
    // the weights of the second come from L2
    const auto passes_of = [&](int e) {
        int first;
        return (expert_rows(a, e, first) + kItemRows - 1) / kItemRows;
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
        __syncthreads();
    }
    const int64_t items = static_cast<int64_t>(table[entries]) * p.tiles;
    // as many clusters as share the items evenly: all of them wait on the same DRAM, so an idle SM costs nothing
    const int clusters = p.slots / p.split;
    const int64_t each = (items + clusters - 1) / clusters;
    const int64_t item0 = min(items, each * (blockIdx.x / p.split)), item1 = min(items, item0 + each);
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
        while (in >= static_cast<int64_t>(passes) * p.tiles) {   // (an entry of several experts)
            in -= static_cast<int64_t>(passes) * p.tiles;
            passes = passes_of(++e);
        }
        Item r;
        int first;
        const int n = expert_rows(a, e, first), pass = static_cast<int>(in % passes);
        r.expert = e;
        r.row = first + pass * kItemRows;
        r.rows = min(kItemRows, n - pass * kItemRows);
        r.col = static_cast<int>(in / passes) * (kWarps * warp_cols);
        return r;
    };
    const int64_t steps = (item1 - item0) * (stage1 - stage0);

    if (warp == kLoader) {
        const auto load_weights = [&](const Item& it, int stage, int slot) {
            const uint32_t bar = w_full + 8 * slot, to = smem_addr(weights) + slot * kWeightBytes;
            if (lane == 0) barrier_expect(bar, kWeightBytes);
            __syncwarp();
            // a box: with an activation the 16 gate and the 16 up rows of a warp, else 128 rows
            if (a.swiglu) {
                if (lane < kWarps) load_box(to + lane * kWarpBytes, &weight_map, stage * (kIn / 2), it.col + lane * 16, 0, it.expert, bar);
            } else if (lane < kWarps / 4) {
                load_box(to + lane * 4 * kWarpBytes, &weight_map, stage * (kIn / 2), it.col + lane * 128, 0, it.expert, bar);
            }
        };
        const auto load_inputs = [&](const Item& it, int stage, int slot) {
            const uint32_t bar = x_full + 8 * slot;
            const int eights = (it.rows + 7) / 8;   // (rows that are not there leave garbage in columns that are not written)
            if (lane == 0) barrier_expect(bar, eights * 8 * kIn * 2);
            __syncwarp();
            if (lane < 4 * eights)
                load_box(smem_addr(inputs) + slot * S::kXBytes + (lane / eights * NT + lane % eights) * 1024, &x_map,
                         (stage * kIn + lane / eights * 64) * 2, it.row + lane % eights * 8, 0, 0, bar);
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
    } else {
        // ---- a warp: 32 weight rows, two of the instruction's 16 (with an activation gate and up rows)
        const int g = lane >> 2, t = lane & 3, row0 = S::place(g);   // weight rows row0, + 8, + 16, + 24
        constexpr int kWords = GROUP / 32;                           // of a row and group, a thread's
        int w_slot = 0, x_slot = 0;
        uint32_t w_parity = 0, x_parity = 0;
        for (int64_t item = item0; item < item1; ++item) {
            const Item it = decode(item);
            const int col0 = it.col + warp * warp_cols;
            // this lane's row for the scales; the lanes exchange them
            const int mine = a.swiglu ? col0 + (lane & 15) : col0 + lane;
            const bool real = mine < cols;
            const int o = a.swiglu && lane >= 16 ? cols + mine : mine;
            int grp_next = stage0 * (kIn / GROUP);
            const int64_t scale_base = (static_cast<int64_t>(it.expert) * p.groups + grp_next) * a.O + (real ? o : 0);
            const T* scale_at = static_cast<const T*>(a.scales) + scale_base;
            const uint8_t* zero_at = ZEROS ? a.zeros + scale_base : nullptr;
            T scale_next = from_float<T>(0.0f);
            uint8_t zero_next = 8;
            const auto load_scales = [&]() {   // of the next group
                if (real && grp_next < p.groups) {
                    scale_next = *scale_at;
                    if constexpr (ZEROS) zero_next = *zero_at;
                } else {
                    scale_next = from_float<T>(0.0f);
                }
                ++grp_next;
                scale_at += a.O;
                if constexpr (ZEROS) zero_at += a.O;
            };
            float acc[2][NT][4];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.0f;
            const bool both = NT == 1 || it.rows > 8;
            load_scales();
            for (int stage = stage0; stage < stage1; ++stage) {
                barrier_wait(w_full + 8 * w_slot, w_parity, dead);
                barrier_wait(x_full + 8 * x_slot, x_parity, dead);
                const unsigned char* w = weights + w_slot * kWeightBytes + warp * kWarpBytes + row0 * 128;
                const unsigned char* x = inputs + x_slot * S::kXBytes + S::x_place(g) * 128;
#pragma unroll
                for (int grp = 0; grp < kIn / GROUP; ++grp) {
                    // scales and zero points of this thread's rows
                    float scale[4];
                    __half2 low[4], high[4];
                    {
                        const uint32_t packed = *reinterpret_cast<const uint16_t*>(&scale_next) | static_cast<uint32_t>(zero_next) << 16;
                        load_scales();
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const uint32_t sz = __shfl_sync(kFullMask, packed, row0 + 8 * h);
                            const uint16_t s16 = static_cast<uint16_t>(sz);
                            scale[h] = to_float(*reinterpret_cast<const T*>(&s16));
                            if constexpr (ZEROS) {   // 1024 + zero and 64 + zero, by their bits, negative
                                const uint32_t z = sz >> 16, lo = 0xe400u | z, hi = 0xd400u | z << 4;
                                low[h] = halves(lo | lo << 16);
                                high[h] = halves(hi | hi << 16);
                            } else {
                                low[h] = halves(0xe408e408u);    // -1032
                                high[h] = halves(0xd480d480u);   // -72
                            }
                        }
                    }
                    // codes: kWords neighbouring words of each of the four rows
                    uint32_t word[4][kWords];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int byte = grp * (GROUP / 2) + t * 4 * kWords;
                        const unsigned char* from = w + h * 1024 + (((byte >> 4) ^ row0) << 4) + (byte & 15);
                        if constexpr (kWords == 4) {
                            const uint4 v = *reinterpret_cast<const uint4*>(from);
                            word[h][0] = v.x, word[h][1] = v.y, word[h][2] = v.z, word[h][3] = v.w;
                        } else if constexpr (kWords == 2) {
                            const uint2 v = *reinterpret_cast<const uint2*>(from);
                            word[h][0] = v.x, word[h][1] = v.y;
                        } else {
                            word[h][0] = *reinterpret_cast<const uint32_t*>(from);
                        }
                    }
                    float sum[2][NT][4];
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int n = 0; n < NT; ++n) sum[m][n][0] = sum[m][n][1] = sum[m][n][2] = sum[m][n][3] = 0.0f;
#pragma unroll
                    for (int k = 0; k < kWords; ++k) {
                        uint4 xf[NT];
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const int at = grp * (GROUP / 8) + k * 4 + t;   // piece of the row's 32
                            if (n == 0 || both)
                                xf[n] = *reinterpret_cast<const uint4*>(x + ((at >> 3) * NT + n) * 1024 + (((at & 7) ^ S::x_place(g)) << 4));
                        }
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint32_t u0 = word[2 * m][k], u1 = word[2 * m + 1][k];
                            const uint32_t a0[4] = {low_pair(u0, low[2 * m]), low_pair(u1, low[2 * m + 1]), high_pair(u0, high[2 * m]),
                                                    high_pair(u1, high[2 * m + 1])};
                            const uint32_t a1[4] = {low_pair(u0 >> 8, low[2 * m]), low_pair(u1 >> 8, low[2 * m + 1]),
                                                    high_pair(u0 >> 8, high[2 * m]), high_pair(u1 >> 8, high[2 * m + 1])};
                            multiply(sum[m][0], a0, xf[0].x, xf[0].y);
                            multiply(sum[m][0], a1, xf[0].z, xf[0].w);
                            if constexpr (NT == 2) {
                                if (both) {
                                    multiply(sum[m][1], a0, xf[1].x, xf[1].y);
                                    multiply(sum[m][1], a1, xf[1].z, xf[1].w);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[m][n][j] += scale[2 * m + (j >> 1)] * sum[m][n][j];
                }
                __syncwarp();
                if (lane == 0) {
                    barrier_arrive(w_empty + 8 * w_slot);
                    barrier_arrive(x_empty + 8 * x_slot);
                }
                if (++w_slot == kWeightSlots) w_slot = 0, w_parity ^= 1;
                if (++x_slot == kXSlots) x_slot = 0, x_parity ^= 1;
            }
            // ---- the item's end: a cluster's CTAs join, in their order
            if (*dead) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[m][n][j] = __int_as_float(0x7fffffff);
            }
            if (p.split > 1) {   // (each cluster has one item at most: the ring is used up and serves the join)
                float* const join = reinterpret_cast<float*>(weights);   // [8 NT][kConsumers]
                consumers_sync();
#pragma unroll
                for (int i = 0; i < 8 * NT; ++i) join[i * kConsumers + tid] = acc[i / (4 * NT)][i / 4 % NT][i & 3];
                cluster_sync();
                if (rank == 0) {
                    for (int r = 1; r < p.split; ++r) {
                        uint32_t from;
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(smem_addr(join)), "r"(r));
#pragma unroll
                        for (int i = 0; i < 8 * NT; ++i) {
                            float v;
                            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(from + (i * kConsumers + tid) * 4) : "memory");
                            acc[i / (4 * NT)][i / 4 % NT][i & 3] += v;
                        }
                    }
                }
                cluster_sync();
            }
            if (rank == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = 8 * n + S::x_place(2 * t + j);
                        if (r >= it.rows) continue;
                        float factor = 1.0f;
                        if constexpr (std::is_same_v<T, __nv_bfloat16>) factor = __ldcg(p.factor + it.row + r);
                        T* y = static_cast<T*>(a.y) + static_cast<int64_t>(it.row + r) * a.y_ld + col0;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int c = row0 + 8 * h;
                            const float v = acc[0][n][2 * h + j] * factor, u = acc[1][n][2 * h + j] * factor;
                            if (a.swiglu) {
                                if (col0 + c < cols) y[c] = from_float<T>(v / (1.0f + expf(-v)) * u);
                            } else {
                                if (col0 + c < cols) y[c] = from_float<T>(v);
                                if (col0 + 16 + c < cols) y[16 + c] = from_float<T>(u);
                            }
                        }
                    }
            }
        }
    }
    if (warp == kLoader && p.split > 1 && item0 < item1) {   // (as the other warps do)
        cluster_sync();
        cluster_sync();
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

// Bytes [w][z][y][x], read in boxes of 128 x box_y x box_z; zeros past the ends.
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

// SMs of the current device, with the kernel's shared memory limit raised: looked up once per device (a race writes
// the same values).
template <typename Kernel>
cudaError_t prepare_kernel(Kernel kernel, int smem, int* known, int* sms) {
    constexpr int kDevices = 64;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < kDevices && (*sms = __atomic_load_n(&known[dev], __ATOMIC_RELAXED)) > 0) return cudaSuccess;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (err == cudaSuccess && dev < kDevices) __atomic_store_n(&known[dev], *sms, __ATOMIC_RELAXED);
    return err;
}

template <typename T, int NT, int GROUP, bool ZEROS>
cudaError_t launch_shape(const W4Args& a, const uint4* x, const float* factor, cudaStream_t stream) {
    using S = Shape<NT, GROUP>;
    static int known[64];
    Plan p{};
    int sms = 0;
    cudaError_t err = prepare_kernel(expert_w4_kernel<T, NT, GROUP, ZEROS>, S::kShared, known, &sms);
    if (err != cudaSuccess) return err;
    const int cols = a.swiglu ? a.O / 2 : a.O, cta_cols = a.swiglu ? kConsumers / 2 : kConsumers;
    p.tiles = (cols + cta_cols - 1) / cta_cols;
    while (((a.E - 1) >> p.table_shift) + 1 > kTable) ++p.table_shift;
    p.stages = (a.I + kIn - 1) / kIn;
    p.groups = a.I / GROUP;
    p.factor = factor;
    p.slots = sms;
    // items at most; with fewer than half the CTAs' number, clusters share them
    const int64_t most = (static_cast<int64_t>(a.rows) / (8 * NT) + (a.rows < a.E ? a.rows : a.E)) * p.tiles;
    p.split = 1;
    while (p.split < kMostSplit && 2 * p.split <= p.stages && most * 2 * p.split <= p.slots) p.split *= 2;
    const int64_t clusters = most < p.slots / p.split ? most : p.slots / p.split;
    p.slots = static_cast<int>(clusters) * p.split;
    CUtensorMap weight_map, x_map;
    err = a.swiglu ? byte_map(&weight_map, a.w, a.I / 2, cols, 2, a.E, 16, 2) : byte_map(&weight_map, a.w, a.I / 2, a.O, 1, a.E, 128, 1);
    if (err == cudaSuccess) err = byte_map(&x_map, x, static_cast<int64_t>(a.I) * 2, a.rows, 1, 1, 8, 1);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.slots);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kShared;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, expert_w4_kernel<T, NT, GROUP, ZEROS>, a, p, weight_map, x_map);
}

template <typename T, int GROUP>
cudaError_t launch_group(const W4Args& a, void* workspace, cudaStream_t stream) {
    uint4* x = static_cast<uint4*>(workspace);
    float* factor = reinterpret_cast<float*>(x + static_cast<int64_t>(a.rows) * (a.I / 8));
    const cudaError_t err = launch_dependent(order_kernel<T, GROUP>, dim3(a.rows < 65536 ? a.rows : 65536), dim3(kOrderThreads), 0,
                                             stream, a, x, factor);
    if (err != cudaSuccess) return err;
    // rows of an item: 8, or 16 where experts have more than 4 rows on average (a second pass over a tile costs more)
    const int used = a.rows < a.E ? a.rows : a.E, mean = (a.rows + used - 1) / used;
    if (mean <= 4 || a.rows <= 8)
        return a.zeros ? launch_shape<T, 1, GROUP, true>(a, x, factor, stream) : launch_shape<T, 1, GROUP, false>(a, x, factor, stream);
    return a.zeros ? launch_shape<T, 2, GROUP, true>(a, x, factor, stream) : launch_shape<T, 2, GROUP, false>(a, x, factor, stream);
}

template <typename T>
cudaError_t launch_type(const W4Args& a, void* workspace, cudaStream_t stream) {
    return a.group == 32   ? launch_group<T, 32>(a, workspace, stream)
           : a.group == 64 ? launch_group<T, 64>(a, workspace, stream)
                           : launch_group<T, 128>(a, workspace, stream);
}

}  // namespace

// x in its order, and the power of two of each row.
int64_t expert_w4_workspace(int64_t rows, int I) { return rows * I * 2 + rows * 4; }

cudaError_t launch_expert_w4(const W4Args& a, void* workspace, int dtype, cudaStream_t stream) {
    return dtype == EP_DTYPE_BF16 ? launch_type<__nv_bfloat16>(a, workspace, stream) : launch_type<__half>(a, workspace, stream);
}

}  // namespace ep
