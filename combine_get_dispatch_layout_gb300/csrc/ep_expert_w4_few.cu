// The experts' products with 4-bit weights for few rows in all: one kernel,
// weights straight from memory into registers.
//
// Mathematics: y[n, o] = sum over groups of s[g, o] * sum (code - zero) * x, as
// mma.sync on fp16 operands with fp32 sums, 16 weight rows by 8 rows of x. A code
// in the low bits of a half word is the fp16 number code * 2^-24 (subnormal), and
// so four bits further up 16 times that: four masks and one shift part eight
// codes, and four fused multiply-adds of two halves make (code - zero) * 2^-10 of
// them, exactly. (The subnormal numbers themselves would do as operands, but the
// tensor cores add products in 25 bits or so below the largest, and there a
// subnormal operand counts as 2^-14 whatever its value: beside an input much
// larger than the others, what falls off the others' products shows.) fp16 inputs
// enter as they are; bf16 inputs after a power of two has brought the largest of the
// group to [2^14, 2^15), so that fp16's 10 bits and its subnormals hold every
// input down to 2^-39 of the largest.
//
// What bounds it: each weight is used once or a few times, so DRAM, and below
// some megabytes the chain launch, offsets, first weights, join. So there is one
// launch, no operand passes through shared memory but x (read from L2 by every
// CTA), and a warp has five steps of 16 rows x 128 inputs in flight. A CTA takes
// whole tiles of 16 rows; its warps share their inputs evenly, end to end over
// the tiles, and join once for a batch of tiles, in the warps' order.
// Measured, launches in a graph: 4096 x 4096, 4 rows of fp16: 7.8 us (1.1 TB/s);
// 8 experts of 4096 x 7168, a row each, with the activation: 29.9 us (4.1 TB/s),
// of which about 7 are start and join. The rest runs at 5.1 TB/s with 55 % of
// the issue slots used; the five steps in flight, 80 KB a core, would cover 1.7 us of
// latency at the memory's rate. Codes as subnormal operands from bits 0 and 4, with
// the loss above: 28.9 us; from bits 6 to 9, by one more shift for each mask: 31.3.
// Of earlier forms: two steps of 256 inputs in flight: 31.3 us where six of 128
// took 29.0, prefetches of 128 bytes to L2 instead of 256: 30.4; 8, 12, 24 and 32
// warps a block instead of 16: 38.6, 34.2, 32.2, 38.8 where 16 took 32.0; the codes
// by TMA into a ring of each warp: 32.1.
#include <math.h>
#include <string.h>

#include <type_traits>

#include "ep_w4.cuh"

namespace ep {
namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kTile = 16;                // weight rows
constexpr int kBlock = 128;              // inputs of a step
constexpr int kBatch = 32;               // tiles of a batch at most
constexpr int kEntries = kFewRows;       // experts with rows: no more than there are rows
constexpr int kJoinBytes = (kBatch + kWarps - 1) * kTile * 8 * 4;

// Codes in fp16: bits 0 to 3 alone are the subnormal number code * 2^-24, bits 4 to 7 alone 16 times that; two of them
// brought to code * 2^-kCodeBits.
constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u, kLowUp = 0x74007400u, kHighUp = 0x64006400u;
constexpr int kCodeBits = 10;

struct Entry {
    int expert, row, rows, local;   // local: rows of the entries before
};

__device__ __forceinline__ void load_codes(uint32_t (&r)[4], const uint8_t* p) {
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "l"(p));
}
__device__ __forceinline__ void load_codes(uint32_t (&r)[2], const uint8_t* p) {
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v2.u32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "l"(p));
}
__device__ __forceinline__ void load_codes(uint32_t (&r)[1], const uint8_t* p) {
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.u32 %0, [%1];" : "=r"(r[0]) : "l"(p));
}
__device__ __forceinline__ void multiply(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(d[0]), "f"(d[1]), "f"(d[2]), "f"(d[3]));
}

__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// T: type of x, scales and y. GROUP: inputs that share a scale.
template <typename T, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kThreads, 1) expert_w4_few_kernel(W4Args a, int tiles, int x_stride) {
    constexpr int kGroups = kBlock / GROUP;   // of a step
    constexpr int kWords = GROUP / 32;        // words of 8 codes: a lane's of a row, of a group
    constexpr int kAhead = GROUP == 32 ? 2 : GROUP == 64 ? 4 - ZEROS : 5 - ZEROS;   // steps, as the registers allow
    extern __shared__ __align__(16) unsigned char shared_bytes[];
    __shared__ int2 found[kEntries];          // expert whose rows begin in this row, and their number
    __shared__ Entry entry[kEntries];
    __shared__ int row_of[kEntries], entries_found;
    // x: [rows] rows of x_stride bytes, the inputs of a step in the order in which lanes take them; back: [rows][groups],
    // what a group's sum of products is multiplied with; join: [slots][16][8]
    unsigned char* const inputs = shared_bytes;
    const int groups = a.I / GROUP, blocks = (a.I + kBlock - 1) / kBlock;
    float* const back = reinterpret_cast<float*>(inputs + a.rows * x_stride);
    float* const join = back + (a.rows * groups + 3) / 4 * 4;
    dependent_entry();

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int cols = a.swiglu ? a.O / 2 : a.O, tile_cols = a.swiglu ? kTile / 2 : kTile;

    // ---- entries: the experts with rows, in the order of their rows
    if (tid < kEntries) found[tid] = make_int2(0, 0);
    __syncthreads();
    for (int e = tid; e < a.E; e += kThreads) {
        int first;
        const int n = expert_rows(a, e, first);
        if (n > 0) found[first] = make_int2(e, n);
    }
    __syncthreads();
    if (warp == 0) {
        const int2 f = lane < kEntries ? found[lane] : make_int2(0, 0);
        int scan = f.y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFullMask, scan, o);
            if (lane >= o) scan += v;
        }
        const unsigned real = __ballot_sync(kFullMask, f.y > 0);
        if (f.y > 0 && scan <= a.rows) {   // (more only where offsets contradict one another)
            entry[__popc(real & ((1u << lane) - 1))] = {f.x, lane, f.y, scan - f.y};
            for (int r = 0; r < f.y; ++r) row_of[scan - f.y + r] = lane + r;
        }
        const unsigned kept = __ballot_sync(kFullMask, f.y > 0 && scan <= a.rows);
        if (lane == 0) entries_found = __popc(kept);
    }
    __syncthreads();
    const int64_t all = static_cast<int64_t>(entries_found) * tiles;
    const int64_t share0 = all * blockIdx.x / gridDim.x, share1 = all * (blockIdx.x + 1) / gridDim.x;

    int have0 = 0, have1 = 0;   // rows of x in shared memory
    for (int64_t t0 = share0, t1; t0 < share1; t0 = t1) {
        // ---- a batch: as many tiles as there is room for their sums
        t1 = min(share1, t0 + kBatch);
        const int first = static_cast<int>(t0 / tiles), last = static_cast<int>((t1 - 1) / tiles);   // entries
        const int row0 = entry[first].local, row1 = entry[last].local + entry[last].rows;
        const int count = static_cast<int>(t1 - t0);
        const int steps = count * blocks, step0 = static_cast<int>(static_cast<int64_t>(steps) * warp / kWarps);
        const int step1 = static_cast<int>(static_cast<int64_t>(steps) * (warp + 1) / kWarps);

        // where this lane's weight rows g and g + 8 of a tile are read next; past the end the last one's, not written
        struct Rows {
            const uint8_t *codes[2], *zeros[2];
            const T* scales[2];
        };
        const auto rows_of = [&](int i, int tile, int block) {
            const int o0 = min(tile * tile_cols + g, cols - 1), o1 = a.swiglu ? cols + o0 : min(tile * tile_cols + g + 8, cols - 1);
            const int64_t e = entry[i].expert, first_group = (e * groups + block * kGroups) * a.O;
            Rows r{};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                r.codes[k] = a.w + (e * a.O + (k ? o1 : o0)) * (a.I / 2) + block * (kBlock / 2) + t * (GROUP / 8);
                r.scales[k] = static_cast<const T*>(a.scales) + first_group + (k ? o1 : o0);
                if constexpr (ZEROS) r.zeros[k] = a.zeros + first_group + (k ? o1 : o0);
            }
            return r;
        };
        uint32_t codes[kAhead][kGroups][2][kWords];
        T scale[kAhead][kGroups][2];
        uint8_t zero[kAhead][kGroups][2];
        const int k0 = step0 / blocks, entry0 = min(last, static_cast<int>((t0 + k0) / tiles));
        const int tile0 = static_cast<int>(t0 + k0 - static_cast<int64_t>(entry0) * tiles);
        int load_step = step0, load_entry = entry0, load_tile = tile0, load_block = step0 - k0 * blocks;
        Rows at{};
        if (step0 < step1) at = rows_of(load_entry, load_tile, load_block);
        const auto load = [&](int slot) {
            if (load_step >= step1) return;
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                if (j > 0 && load_block * kGroups + j >= groups) break;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    load_codes(codes[slot][j][k], at.codes[k] + j * (GROUP / 2));
                    scale[slot][j][k] = *at.scales[k];
                    at.scales[k] += a.O;
                    if constexpr (ZEROS) {
                        zero[slot][j][k] = *at.zeros[k];
                        at.zeros[k] += a.O;
                    }
                }
            }
            at.codes[0] += kBlock / 2;
            at.codes[1] += kBlock / 2;
            ++load_step;
            if (++load_block == blocks) {
                load_block = 0;
                if (++load_tile == tiles) load_tile = 0, ++load_entry;
                if (load_step < step1) at = rows_of(load_entry, load_tile, 0);
            }
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load(i);

        // ---- x to shared memory, while the first weights come
        if (row0 != have0 || row1 > have1) {
            const int per_row = a.I / 8, work = (row1 - row0) * per_row;
            constexpr int kLoads = 4;   // under way at a time
            for (int i0 = tid; i0 - lane < work; i0 += kLoads * kThreads) {   // (a group's threads are of one warp)
                Vec8<T> v[kLoads];
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    const int i = i0 + u * kThreads, r = i / per_row, c = i - r * per_row;
                    v[u].raw = make_uint4(0, 0, 0, 0);
                    if (i < work) v[u].raw = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + row_of[row0 + r] * a.x_ld + c * 8);
                }
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    const int i = i0 + u * kThreads, r = i / per_row, c = i - r * per_row;
                    if (i - lane >= work) break;
                    float f[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = to_float(v[u].v[k]);
                    // (magnitudes in the order of their bits, two to a word; NaN lies above infinity)
                    const uint4 raw = v[u].raw;
                    uint32_t big = __vmaxu2(__vmaxu2(raw.x & 0x7fff7fffu, raw.y & 0x7fff7fffu), __vmaxu2(raw.z & 0x7fff7fffu, raw.w & 0x7fff7fffu));
#pragma unroll
                    for (int o = 1; o < GROUP / 8; o <<= 1) big = __vmaxu2(big, __shfl_xor_sync(kFullMask, big, o));
                    big = max(big & 0xffffu, big >> 16);
                    int e = 0;
                    bool finite = big < 0x7c00u;   // fp16
                    if constexpr (!std::is_same_v<T, __half>) {
                        const int exponent = static_cast<int>(big >> 7);   // + 127; subnormal numbers have 0
                        finite = exponent < 255;
                        e = finite ? min(14 + 127 - exponent, 126) : 0;
                    }
                    const float up = __int_as_float((e + 127) << 23);
                    __half2 h[4];   // (0, 4) (2, 6) (1, 5) (3, 7)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int from = (k & 1) * 2 + (k >> 1);
                        h[k] = __floats2half2_rn(f[from] * up, f[from + 4] * up);
                    }
                    if (i >= work) continue;
                    const int grp = c / (GROUP / 8), inside = c - grp * (GROUP / 8);
                    uint4 packed;
                    memcpy(&packed, h, 16);
                    *reinterpret_cast<uint4*>(inputs + r * x_stride + (grp * kWords + inside % kWords) * 64 + inside / kWords * 16) = packed;
                    if (inside == 0) back[r * groups + grp] = __int_as_float(finite ? (127 + kCodeBits - e) << 23 : 0x7fffffff);
                }
            }
            have0 = row0, have1 = row1;
        }
        __syncthreads();

        // ---- this warp's steps
        int k = k0, in_entry = entry0, in_tile = tile0, block = step0 - k0 * blocks;
        float total[4] = {};
        const unsigned char* x_at = nullptr;
        const float* back_at[2] = {};
        const auto begin = [&]() {
            const Entry it = entry[in_entry];
            const int local = it.local - row0;
            // (columns past the rows take another's: they are not written)
            x_at = inputs + (local + min(g, it.rows - 1)) * x_stride + t * 16 + block * (kBlock * 2);
            back_at[0] = back + (local + min(2 * t, it.rows - 1)) * groups + block * kGroups;
            back_at[1] = back + (local + min(2 * t + 1, it.rows - 1)) * groups + block * kGroups;
        };
        if (step0 < step1) begin();
        for (int step = step0; step < step1; step += kAhead) {
#pragma unroll
            for (int slot = 0; slot < kAhead; ++slot) {
                if (step + slot >= step1) break;
#pragma unroll
                for (int j = 0; j < kGroups; ++j) {
                    if (j > 0 && block * kGroups + j >= groups) break;
                    float sum[4] = {};
                    // -zero * 2^-kCodeBits, twice, of the two weight rows
                    uint32_t nz[2] = {0xa000a000u, 0xa000a000u};
                    if constexpr (ZEROS) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) nz[k] = fma2(zero[slot][j][k] * 0x00010001u, kLowUp ^ 0x80008000u, 0);
                    }
#pragma unroll
                    for (int w = 0; w < kWords; ++w) {
                        const uint4 b = *reinterpret_cast<const uint4*>(x_at + (j * kWords + w) * 64);
                        const uint32_t u0 = codes[slot][j][0][w], u1 = codes[slot][j][1][w];
                        const uint32_t v0 = u0 >> 8, v1 = u1 >> 8;
                        multiply(sum, fma2(u0 & kLow, kLowUp, nz[0]), fma2(u1 & kLow, kLowUp, nz[1]), fma2(v0 & kLow, kLowUp, nz[0]),
                                 fma2(v1 & kLow, kLowUp, nz[1]), b.x, b.y);
                        multiply(sum, fma2(u0 & kHigh, kHighUp, nz[0]), fma2(u1 & kHigh, kHighUp, nz[1]), fma2(v0 & kHigh, kHighUp, nz[0]),
                                 fma2(v1 & kHigh, kHighUp, nz[1]), b.z, b.w);
                    }
                    const float bk[2] = {back_at[0][j], back_at[1][j]};
#pragma unroll
                    for (int i = 0; i < 4; ++i)   // (the scale first: a group's sum by itself may pass fp32's range)
                        total[i] = fmaf(to_float(scale[slot][j][i >> 1]) * bk[i & 1], sum[i], total[i]);
                }
                x_at += kBlock * 2;
                back_at[0] += kGroups;
                back_at[1] += kGroups;
                load(slot);
                if (++block == blocks || step + slot + 1 == step1) {
                    // slot k + warp: warps with later tiles are later ones
                    float* to = join + (k + warp) * (kTile * 8) + g * 8 + 2 * t;
                    *reinterpret_cast<float2*>(to) = make_float2(total[0], total[1]);
                    *reinterpret_cast<float2*>(to + 64) = make_float2(total[2], total[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) total[i] = 0.0f;
                    block = 0;
                    ++k;
                    if (++in_tile == tiles) in_tile = 0, ++in_entry;
                    if (step + slot + 1 < step1) begin();
                }
            }
        }
        __syncthreads();

        // ---- join, in the order of the warps, and write
        for (int i = tid; i < count * 64; i += kThreads) {
            const int tile = i >> 6, n = (i >> 3) & 7, r = i & 7;
            const int en = static_cast<int>((t0 + tile) / tiles);
            const Entry it = entry[en];
            if (n >= it.rows) continue;
            const auto owner = [&](int step) { return static_cast<int>((static_cast<int64_t>(kWarps) * (step + 1) - 1) / steps); };
            const int last = owner((tile + 1) * blocks - 1);
            float v0 = 0.0f, v1 = 0.0f;
            for (int w = owner(tile * blocks); w <= last; ++w) {
                if (static_cast<int64_t>(steps) * w / kWarps == static_cast<int64_t>(steps) * (w + 1) / kWarps) continue;   // (without steps)
                const float* from = join + (tile + w) * (kTile * 8) + r * 8 + n;
                v0 += from[0];
                v1 += from[64];
            }
            const int col = static_cast<int>((t0 + tile) - static_cast<int64_t>(en) * tiles) * tile_cols + r;
            T* y = static_cast<T*>(a.y) + (it.row + n) * a.y_ld + col;
            if (a.swiglu) {
                if (col < cols) *y = from_float<T>(v0 / (1.0f + expf(-v0)) * v1);
            } else {
                if (col < cols) y[0] = from_float<T>(v0);
                if (col + 8 < cols) y[8] = from_float<T>(v1);
            }
        }
    }
}

// x of a row in bytes, 64 more than a multiple of 128: the lanes of two rows then read from different banks.
int row_stride(int I) { return (2 * I + 63) / 128 * 128 + 64; }
constexpr int kShared = 224 * 1024;
int64_t shared_bytes_of(const W4Args& a) {
    return static_cast<int64_t>(a.rows) * (row_stride(a.I) + a.I / a.group * 4) + 16 + kJoinBytes;
}

template <typename T, int GROUP, bool ZEROS>
cudaError_t launch_few(const W4Args& a, cudaStream_t stream) {
    constexpr int kDevices = 64;
    static int known[kDevices];   // SMs, with the kernel's shared memory limit raised; a race writes the same values
    auto* kernel = expert_w4_few_kernel<T, GROUP, ZEROS>;
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < kDevices) sms = __atomic_load_n(&known[dev], __ATOMIC_RELAXED);
    if (sms <= 0) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared);
        if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (err != cudaSuccess) return err;
        if (dev < kDevices) __atomic_store_n(&known[dev], sms, __ATOMIC_RELAXED);
    }
    const int cols = a.swiglu ? a.O / 2 : a.O, tile_cols = a.swiglu ? kTile / 2 : kTile;
    const int tiles = (cols + tile_cols - 1) / tile_cols;
    const int64_t most = static_cast<int64_t>(a.rows < a.E ? a.rows : a.E) * tiles;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(most < sms ? most : sms)), dim3(kThreads),
                            static_cast<size_t>(shared_bytes_of(a)), stream, a, tiles, row_stride(a.I));
}

template <typename T>
cudaError_t launch_type(const W4Args& a, cudaStream_t stream) {
    if (a.zeros)
        return a.group == 32   ? launch_few<T, 32, true>(a, stream)
               : a.group == 64 ? launch_few<T, 64, true>(a, stream)
                               : launch_few<T, 128, true>(a, stream);
    return a.group == 32   ? launch_few<T, 32, false>(a, stream)
           : a.group == 64 ? launch_few<T, 64, false>(a, stream)
                           : launch_few<T, 128, false>(a, stream);
}

}  // namespace

// Up to 8 rows, and codes of less than 1 MiB times the group's size. Beyond, the other kernel's higher rate makes up for
// its second launch and its longer start. This one / the other, us: groups of 128: 4096 x 4096, 4 rows of fp16: 7.8 / 12.4;
// 8 experts of 4096 x 7168 (117 MB), a bf16 row each: 29.9 / 34.1; one of 65536 x 4096 (134 MB), 4 bf16 rows: 33.6 / 32.5.
// Groups of 64: 4096 x 4096, 8 rows: 9.8 / 11.4, 4 experts (59 MB) 21.3 / 21.9, 117 MB: 37.0 / 35.8. Groups of 32: 2 experts
// (29 MB): 19.1 / 23.7, 4 experts: 28.4 / 26.6, 8 experts: 55.8 / 43.8.
bool expert_w4_few(const W4Args& a) {
    if (a.rows > kFewRows || shared_bytes_of(a) > kShared) return false;
    const int64_t bytes = static_cast<int64_t>(a.rows < a.E ? a.rows : a.E) * a.O * (a.I / 2);
    return bytes < static_cast<int64_t>(a.group) << 20;
}

cudaError_t launch_expert_w4_few(const W4Args& a, int dtype, cudaStream_t stream) {
    return dtype == EP_DTYPE_BF16 ? launch_type<__nv_bfloat16>(a, stream) : launch_type<__half>(a, stream);
}

}  // namespace ep
