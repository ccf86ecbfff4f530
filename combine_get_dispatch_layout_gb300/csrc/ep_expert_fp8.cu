// The experts' products in 8-bit floating point: rows with a scale per 128 inputs
// (as the fp8 dispatch writes them), weights with a scale per block of 128 x 128.
//
// Mathematics. y[n, o] = sum over blocks b of sx[n, b] sw[o / 128, b] * sum over i in b of cx[n, i] cw[o, i]. The inner
// sums, 128 products of two codes, run through the tensor cores with fp32 sums; each is then scaled and added in fp32
// registers, so no scale is rounded and the sums of blocks are plain fp32. With the activation: silu(gate) * up. An fp8
// output is quantised as the dispatch quantises: amax of 128 channels / 448, codes by IEEE division.
#include "ep_expert_tiles.cuh"

namespace ep {
namespace {

constexpr int kBlock = 128;                     // inputs of a stage: 128 bytes, one scale
constexpr int kTileRows = 256;                  // weight rows of an item: 128 in each CTA of the pair
constexpr int kParts = 4;                       // warps over a CTA's weight rows: 32 lanes each
constexpr int kABytes = kTileRows / 2 * kBlock;
constexpr int kGroups = 2;                      // groups of kParts warps: they take blocks, columns or channels in turn
constexpr int kConsumers = 32 * kParts * kGroups;
constexpr int kLoader = kConsumers / 32, kIssuer = kLoader + 1, kScaler = kLoader + 2;   // warps; two scalers
constexpr int kThreads = kConsumers + 128;
constexpr int kBuffers = 4;                     // of sums in TMEM, 64 or 128 columns apart
constexpr int kScaleSlots = 4;                  // of the ring of scales
constexpr int kScaleSets = 3;                   // weight scales that a CTA's 128 weight rows have at most in a block
constexpr int kOut = 32;                        // columns that a group has in the end
constexpr int kMostStages = 10;

// COLS: rows of x that are columns of a product, at most. LANES: tiles of more rows have them as lanes.
template <int COLS, bool LANES>
struct Shape {
    static_assert(COLS == 32 || COLS == 64, "");
    static constexpr int kStride = LANES ? 128 : 64;             // columns of a buffer; rows as lanes take two buffers
    static constexpr int kRows = LANES ? 128 : COLS;             // rows of x whose scales a CTA needs
    static constexpr int kScaleBlocks = LANES ? 2 : 4;           // blocks of a slot of the ring of scales
    static constexpr int kScaleStep = kScaleSets * COLS;         // floats of a block in the ring of scales
    static_assert(!LANES || kScaleStep >= 128 + 4, "");
    static constexpr int kBox = COLS / 2;
    static constexpr int kStageBytes = kABytes + (LANES ? 128 : COLS / 2) * kBlock;
    static constexpr int kStages = 192 * 1024 / kStageBytes < kMostStages ? 192 * 1024 / kStageBytes : kMostStages;
    static constexpr int kScales = kScaleSlots * kScaleBlocks * kScaleStep;   // floats
    static constexpr int kJoin = kOut * 128;
    static constexpr int kMost = kParts * 128 + 3 * COLS;
    static constexpr int kShared = 1024 + kStages * kStageBytes + (kScales + kJoin + kMost) * 4 + 512 + (kTileTable + 1) * 4;
    static_assert(kShared <= 227 * 1024 - 256, "");
};

__device__ __forceinline__ float ue8m0(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fffffffu : byte << 23);
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); }

// Smallest power of two >= s (s > 0), as the dispatch's scales.
__device__ __forceinline__ float power_of_two(float s) {
    const uint32_t u = __float_as_uint(s), e = u >> 23, f = u & 0x7fffffu;
    if (e == 0) return __uint_as_float((f & (f - 1u)) == 0u ? f : (1u << (32 - __clz(f))));
    return f == 0u || e == 255 ? s : __uint_as_float((e + 1u) << 23);
}

// SWIGLU: y = silu(gate) * up.
template <int COLS, bool LANES, bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1)
    expert_fp8_kernel(Fp8Args a, TilePlan plan, const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap w_half_map,
                      const __grid_constant__ CUtensorMap x_map) {
    using S = Shape<COLS, LANES>;
    constexpr int kScaleBlocks = S::kScaleBlocks;
    extern __shared__ unsigned char shared_bytes[];
    unsigned char* const ring = shared_bytes + (1024 - smem_addr(shared_bytes) % 1024) % 1024;
    float* const scales = reinterpret_cast<float*>(ring + S::kStages * S::kStageBytes);   // [kScaleSlots][kScaleBlocks][kScaleStep]
    float* const join = scales + S::kScales;                                              // [kOut][128]
    float* const most = join + S::kJoin;                                                  // [kParts][128]: largest by part
    float* const found = most + kParts * 128;                                             // [COLS]: the output's scales
    float* const other_most = found + COLS;                                               // [2][COLS]: the other CTA's largest
    uint64_t* const barriers = reinterpret_cast<uint64_t*>(other_most + 2 * COLS);
    const uint32_t full = smem_addr(barriers), empty = full + 8 * kMostStages;
    const uint32_t sums_full = empty + 8 * kMostStages, sums_empty = sums_full + 32;
    const uint32_t scales_full = sums_empty + 32, scales_empty = scales_full + 8 * kScaleSlots;
    const uint32_t most_full = scales_empty + 8 * kScaleSlots;
    uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(barriers) + 120;
    volatile int* const dead = reinterpret_cast<volatile int*>(tmem_at + 1);
    int* const table = reinterpret_cast<int*>(barriers) + 128;
    static_assert((2 * kMostStages + 9 + 2 * kScaleSlots) * 2 <= 120, "");
    __shared__ int warp_sum[kThreads / 32];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = pair_rank();
    if (warp == kLoader) {
        tmem_alloc_all(smem_addr(tmem_at));
        if (lane == 0) {
            *dead = 0;
            for (int i = 0; i < S::kStages; ++i) {
                barrier_init(full + 8 * i, 1);
                barrier_init(empty + 8 * i, 1);
            }
            for (int i = 0; i < kBuffers; ++i) {
                barrier_init(sums_full + 8 * i, 1);
                barrier_init(sums_empty + 8 * i, 2 * kParts);   // a group of each CTA
            }
            barrier_init(most_full, kConsumers / 32);
            for (int i = 0; i < kScaleSlots; ++i) {
                barrier_init(scales_full + 8 * i, 1);
                barrier_init(scales_empty + 8 * i, kConsumers / 32);
            }
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    }
    dependent_entry();
    fill_table<kThreads>(a.g, plan, table, warp_sum);
    tmem_fence_before();
    __syncthreads();
    cluster_sync();   // (both CTAs' barriers are ready)
    tmem_fence_after();
    const uint32_t tmem = __shfl_sync(kFullMask, *tmem_at, 0);
    const bool leader = elected();
    const int blocks = a.I / kBlock, cols = SWIGLU ? a.O / 2 : a.O;
    const int64_t items = tile_count(a.g, plan, table);
    const int pair_id = blockIdx.x / 2, pairs = gridDim.x / 2;

    // Weight scales of a block that this CTA's rows of tile m have: those of the gate rows (or all), then of the up rows.
    const auto scale_row = [&](int m, int set) {
        const int row0 = m * kTileRows + rank * (kTileRows / 2);
        if (!SWIGLU) return row0 / kBlock;
        return set == 0 ? row0 / 2 / kBlock : (cols + row0 / 2) / kBlock + set - 1;
    };
    // What an e4m3 output needs: the scale of a block whose largest value is `big`, its place, two values' codes.
    const auto larger = [](float x, float y) { return x > y || x != x ? x : y; };   // (NaN stays)
    const auto output_scale = [&](float big) {
        if (big == 0.0f) return 0.0f;
        float s = __fdiv_rn(big, 448.0f);
        if (a.y_scale_mode != EP_SCALE_FP32 && s > 0.0f) s = power_of_two(s);
        if (a.y_scale_mode == EP_SCALE_UE8M0 && s < __uint_as_float(0x00400000u)) s = __uint_as_float(0x00400000u);   // 2^-127
        return s;
    };
    const auto write_scale = [&](int64_t row, int block, float s) {
        const int64_t to = row * a.y_scale_row + block * a.y_scale_block;
        if (a.y_scale_mode == EP_SCALE_UE8M0) static_cast<uint8_t*>(a.y_scales)[to] = static_cast<uint8_t>(__float_as_uint(s) >> 23);
        else static_cast<float*>(a.y_scales)[to] = s;
    };
    const auto codes = [](float2 v, float s) -> uint32_t {
        return s == 0.0f ? 0u : __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(v.x, s), __fdiv_rn(v.y, s)), __NV_SATFINITE, __NV_E4M3);
    };
    const int scale_rows = ceil_div(a.O, kBlock), sets = !SWIGLU ? 1 : cols % 64 == 0 ? 2 : 3;

    // (registers: 256 x 216 + 128 x 72 of the launch's 384 x 168)
    if (warp < kLoader) {
        if constexpr (LANES) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // 32 of the CTA's 128 lanes
        const int part = warp % kParts, group = warp / kParts;
        const uint32_t mine = tmem + (static_cast<uint32_t>(part) << 21);
        int buffer = 0, slot = 0;
        uint32_t parities = 0, scales_parity = 0, most_parity = 0;   // parities: a bit for each buffer
        // A tile whose rows of x are the lanes: a thread has one of them and 64 columns of each half of the 256 weight rows (gate
        // and up of the same 64 channels). Its scales are two numbers a block.
        const auto rows_as_lanes = [&](const Tile& it) {
            const int r = rank * 128 + part * 32 + lane, h = group;
            const bool real = r < it.rows;
            const int64_t row = it.row + static_cast<int64_t>(real ? r : 0);
            const int first = SWIGLU ? it.m * 128 + h * 64 : it.m * kTileRows + h * 64;   // channel of column 0 of the first half
            const int second = SWIGLU ? first : first + 128;
            uint64_t acc[2][32];
#pragma unroll
            for (int n = 0; n < 32; ++n) acc[0][n] = acc[1][n] = 0;
            const uint32_t from = mine + h * 64;
            for (int b = 0; b < blocks; ++b) {
                if (b % kScaleBlocks == 0) barrier_wait_inline(scales_full + 8 * slot, scales_parity, dead);
                const float* sx = scales + (slot * kScaleBlocks + b % kScaleBlocks) * S::kScaleStep;
                const float x_scale = sx[part * 32 + lane];
                const uint64_t s0 = both(x_scale * sx[128 + h]), s1 = both(x_scale * sx[128 + 2 + h]);
                buffer = (buffer + 1) & 2;   // an even one
                barrier_wait_inline(sums_full + 8 * buffer, (parities >> buffer) & 1, dead);
                tmem_fence_after();
                const uint32_t at = from + buffer * S::kStride;
                uint32_t raw[2][16];
                tmem_load16(at, raw[0]);
#pragma unroll
                for (int c = 0; c < 8; ++c) {   // a chunk of sums is on its way while the one before is added
                    tmem_loaded(raw[c & 1]);
                    if (c < 7) {
                        tmem_load16(at + (c + 1) / 4 * 128 + (c + 1) % 4 * 16, raw[(c + 1) & 1]);
                    } else {
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0) barrier_arrive_pair(in_first(sums_empty + 8 * (buffer + h)));   // (the issuer waits for both)
                    }
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        uint64_t& to = acc[c / 4][c % 4 * 8 + n];
                        to = fma2(pair(raw[c & 1][2 * n], raw[c & 1][2 * n + 1]), c < 4 ? s0 : s1, to);
                    }
                }
                if (b % kScaleBlocks == kScaleBlocks - 1 || b + 1 == blocks) {
                    if (lane == 0) barrier_arrive(scales_empty + 8 * slot);
                    if (++slot == kScaleSlots) slot = 0, scales_parity ^= 1;
                }
                parities ^= 1u << buffer;
                buffer = (buffer + 2) & 3;
            }
            if (*dead) {
#pragma unroll
                for (int n = 0; n < 32; ++n) acc[0][n] = acc[1][n] = both(__int_as_float(0x7fffffff));
            }
            if constexpr (SWIGLU) {
#pragma unroll
                for (int n = 0; n < 32; ++n) {
                    const float2 g = apart(acc[0][n]), u = apart(acc[1][n]);
                    acc[0][n] = pair(__float_as_uint(silu(g.x) * u.x), __float_as_uint(silu(g.y) * u.y));
                }
            }
            constexpr int kHalves = SWIGLU ? 1 : 2;
            if (a.y_dtype != EP_DTYPE_FP8_E4M3) {
                const bool bf16 = a.y_dtype == EP_DTYPE_BF16, wide = a.y_ld % 8 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
                if (!real) return;
#pragma unroll
                for (int half = 0; half < kHalves; ++half) {
                    const int chan = half == 0 ? first : second;
                    uint16_t* to = static_cast<uint16_t*>(a.y) + row * a.y_ld + chan;
#pragma unroll
                    for (int n = 0; n < 32; n += 4) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 v = apart(acc[half][n + k]);
                            const __nv_bfloat162 vb = __floats2bfloat162_rn(v.x, v.y);
                            const __half2 vh = __floats2half2_rn(v.x, v.y);
                            w[k] = bf16 ? *reinterpret_cast<const uint32_t*>(&vb) : *reinterpret_cast<const uint32_t*>(&vh);
                        }
                        if (wide && chan + 2 * n + 8 <= cols) {
                            *reinterpret_cast<uint4*>(to + 2 * n) = make_uint4(w[0], w[1], w[2], w[3]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (chan + 2 * n + k < cols) to[2 * n + k] = static_cast<uint16_t>(w[k / 2] >> (k % 2 * 16));
                        }
                    }
                }
                return;
            }
            // e4m3: the largest of 128 channels, of which another warp's thread has the other 64
            float big[kHalves];
#pragma unroll
            for (int half = 0; half < kHalves; ++half) {
                big[half] = 0.0f;
#pragma unroll
                for (int n = 0; n < 32; ++n) {
                    const float2 v = apart(acc[half][n]);
                    big[half] = larger(fabsf(v.x), larger(fabsf(v.y), big[half]));
                }
                most[(half * 2 + h) * 128 + part * 32 + lane] = big[half];
            }
            consumers_sync();
            const bool wide = a.y_ld % 16 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
#pragma unroll
            for (int half = 0; half < kHalves; ++half) {
                const int chan = half == 0 ? first : second;
                const float s = output_scale(larger(most[(half * 2 + (h ^ 1)) * 128 + part * 32 + lane], big[half]));
                if (!real || chan >= cols) continue;   // (columns are a multiple of 128)
                if (h == 0) write_scale(row, chan / kBlock, s);
                uint8_t* to = static_cast<uint8_t*>(a.y) + row * a.y_ld + chan;
#pragma unroll
                for (int n = 0; n < 32; n += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 v = apart(acc[half][n + 2 * k]), u = apart(acc[half][n + 2 * k + 1]);
                        w[k] = codes(v, s) | codes(u, s) << 16;
                    }
                    if (wide) {
                        *reinterpret_cast<uint4*>(to + 2 * n) = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k) to[2 * n + k] = static_cast<uint8_t>(w[k / 4] >> (k % 4 * 8));
                    }
                }
            }
            consumers_sync();   // (`most` is written again)
        };
        for (int64_t i = pair_id; i < items; i += pairs) {
            const Tile it = tile_at(a.g, plan, table, i);
            if constexpr (LANES) {
                if (it.rows > COLS) {
                    rows_as_lanes(it);
                    continue;
                }
            }
            // this thread's output channel and weight row; with the activation a warp's lanes are 16 gate and 16 up rows
            const int row0 = it.m * kTileRows + rank * (kTileRows / 2) + part * 32;
            const int chan = SWIGLU ? row0 / 2 + (lane & 15) : row0 + lane;
            const bool real = chan < cols;
            const int set = SWIGLU && lane >= 16 && real ? (cols + chan) / kBlock - scale_row(it.m, 1) + 1 : 0;
            const int there = max(it.rows, 1);   // (a tile without rows has a product all the same)
            uint64_t acc[COLS / 2];   // columns 2 n, 2 n + 1; the groups take every other block each
#pragma unroll
            for (int n = 0; n < COLS / 2; ++n) acc[n] = 0;
            for (int b = 0; b < blocks; ++b) {
                if (b % kScaleBlocks == 0) barrier_wait_inline(scales_full + 8 * slot, scales_parity, dead);
                if (b % kGroups == group) {
                    const float* sx = scales + (slot * kScaleBlocks + b % kScaleBlocks) * S::kScaleStep + set * COLS;
                    barrier_wait_inline(sums_full + 8 * buffer, (parities >> buffer) & 1, dead);
                    tmem_fence_after();
#pragma unroll
                    for (int c0 = 0; c0 < COLS; c0 += 32) {
                        if (c0 >= there) continue;
                        uint32_t raw[32];
                        tmem_load16(mine + buffer * S::kStride + c0, raw);
                        if (c0 + 16 < there) tmem_load16(mine + buffer * S::kStride + c0 + 16, raw + 16);
                        tmem_loaded(raw);
                        if (c0 + 32 >= there) {   // (all that there are)
                            tmem_fence_before();
                            __syncwarp();
                            if (lane == 0) barrier_arrive_pair(in_first(sums_empty + 8 * buffer));
                        }
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            if (c0 + c / 16 * 16 >= there) continue;
                            const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(sx + c0 + c);
                            uint64_t *to = acc + (c0 + c) / 2;
                            to[0] = fma2(pair(raw[c], raw[c + 1]), s.x, to[0]);
                            to[1] = fma2(pair(raw[c + 2], raw[c + 3]), s.y, to[1]);
                        }
                    }
                    __syncwarp();
                }
                if (b % kScaleBlocks == kScaleBlocks - 1 || b + 1 == blocks) {
                    if (lane == 0) barrier_arrive(scales_empty + 8 * slot);
                    if (++slot == kScaleSlots) slot = 0, scales_parity ^= 1;
                }
                parities ^= 1u << buffer;
                buffer = (buffer + 1) % kBuffers;
            }
            // The groups' sums meet: columns 0 .. 31 in the first, the others in the second.
            float* const meet = join + part * 32 + lane;
            float sums[kOut];
#pragma unroll
            for (int g = 0; g < COLS / kOut; ++g) {
                if (g > 0 && it.rows <= kOut) continue;
                if (group != g) {
#pragma unroll
                    for (int n = 0; n < kOut / 2; ++n) {
                        const float2 v = apart(acc[g * (kOut / 2) + n]);
                        meet[2 * n * 128] = v.x, meet[(2 * n + 1) * 128] = v.y;
                    }
                }
                consumers_sync();
                if (group == g) {
#pragma unroll
                    for (int n = 0; n < kOut / 2; ++n) {   // (the first group's plus the second's, whichever adds)
                        const float2 v = apart(acc[g * (kOut / 2) + n]);
                        sums[2 * n] = v.x + meet[2 * n * 128], sums[2 * n + 1] = v.y + meet[(2 * n + 1) * 128];
                    }
                }
                consumers_sync();
            }
            const int c0 = group * kOut, many = it.rows - c0;   // of this warp's columns, those with a row
            if (*dead) {
#pragma unroll
                for (int n = 0; n < kOut; ++n) sums[n] = __int_as_float(0x7fffffff);
            }
            // Results: column n, or with the activation column 2 n + odd: gate lanes take the even one of two, up lanes the odd one.
            constexpr int kResults = SWIGLU ? kOut / 2 : kOut;
            const int odd = SWIGLU ? lane >> 4 : 0;
            float v[kResults];
#pragma unroll
            for (int n = 0; n < kResults; ++n) {
                if constexpr (SWIGLU) {
                    const float own = lane < 16 ? sums[2 * n] : sums[2 * n + 1];
                    const float got = __shfl_xor_sync(kFullMask, lane < 16 ? sums[2 * n + 1] : sums[2 * n], 16);
                    v[n] = lane < 16 ? silu(own) * got : silu(got) * own;
                } else {
                    v[n] = sums[n];
                }
            }
            constexpr int kStep = SWIGLU ? 2 : 1;   // columns from one result to the next
            const int64_t row = static_cast<int64_t>(it.row) + c0 + odd;
            const int left = many - odd;
            if (a.y_dtype != EP_DTYPE_FP8_E4M3) {
                if (!real) continue;
                uint16_t* to = static_cast<uint16_t*>(a.y) + row * a.y_ld + chan;
                const int64_t step = kStep * a.y_ld;
                const bool bf16 = a.y_dtype == EP_DTYPE_BF16;
#pragma unroll
                for (int n = 0; n < kResults; ++n, to += step)
                    if (n * kStep < left)
                        *to = bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v[n])) : __half_as_ushort(__float2half_rn(v[n]));
                continue;
            }
            // ---- e4m3: the largest of each column's 128 channels (with the activation half of them in the other CTA), its
            // scale, codes
            const auto largest = [&](uint32_t mask, float v) {   // (of numbers that are not negative the bits compare as they do)
                return __uint_as_float(__reduce_max_sync(mask, real ? __float_as_uint(fabsf(v)) : 0u));
            };
#pragma unroll
            for (int n = 0; n < kResults; ++n) {
                if (n * kStep >= many) continue;
                const float big = largest(!SWIGLU ? kFullMask : lane < 16 ? 0x0000ffffu : 0xffff0000u, v[n]);
                if ((lane & (SWIGLU ? 15 : 31)) == 0) most[part * 128 + c0 + n * kStep + odd] = big;
            }
            consumers_sync();
            float big[COLS / kConsumers + 1];
#pragma unroll
            for (int k = 0, n = tid; n < COLS; ++k, n += kConsumers) {
                big[k] = 0.0f;
                for (int w = 0; w < kParts; ++w) big[k] = larger(most[w * 128 + n], big[k]);
                if (SWIGLU) store_other(smem_addr(other_most + most_parity * COLS + n), rank ^ 1, big[k]);
            }
            if (SWIGLU) {   // (two buffers: the other CTA waits for this item's before it is done with the next one's)
                __syncwarp();
                if (lane == 0) barrier_arrive_cluster(in_cta(most_full, rank ^ 1));
                barrier_wait_cluster(most_full, most_parity, dead);
            }
#pragma unroll
            for (int k = 0, n = tid; n < COLS; ++k, n += kConsumers) {
                if (n >= it.rows) continue;
                if (SWIGLU) big[k] = larger(other_most[most_parity * COLS + n], big[k]);
                const float s = output_scale(big[k]);
                found[n] = s;
                const int block = SWIGLU ? it.m : it.m * 2 + rank;   // of 128 channels
                if (block * kBlock < cols && (!SWIGLU || rank == 0)) write_scale(static_cast<int64_t>(it.row) + n, block, s);
            }
            most_parity ^= 1;
            consumers_sync();
            if (real) {
                const float* my = found + c0 + odd;
                uint8_t* to = static_cast<uint8_t*>(a.y) + row * a.y_ld + chan;
                const int64_t step = kStep * a.y_ld;
#pragma unroll
                for (int n = 0; n < kResults; ++n, to += step)
                    if (n * kStep < left)
                        *to = static_cast<uint8_t>(codes(make_float2(v[n], 0.0f), my[n * kStep]));
            }
        }
    } else {
        if constexpr (LANES) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == kLoader) {
            int slot = 0;
            uint32_t parity = 1;
            for (int64_t i = pair_id; i < items; i += pairs) {
                const Tile it = tile_at(a.g, plan, table, i);
                const int half = columns_of(it.rows) / 2, a_boxes = SWIGLU ? 4 : 1, x_boxes = (half + S::kBox - 1) / S::kBox;
                const int row0 = it.m * kTileRows + rank * (kTileRows / 2);
                const bool lanes = LANES && it.rows > COLS;
                // with rows as lanes: boxes of this CTA's 128 rows (none of those behind the tile's), and of both
                const int own = lanes ? (min(max(it.rows - rank * 128, 0), 128) + S::kBox - 1) / S::kBox : 0;
                const int both_bytes = lanes ? 2 * kABytes + (it.rows + S::kBox - 1) / S::kBox * S::kBox * kBlock
                                             : 2 * (kABytes + x_boxes * S::kBox * kBlock);
                for (int b = 0; b < blocks; ++b) {
                    // both CTAs' boxes count on the first one's barrier
                    const uint32_t bar = in_first(full + 8 * slot), at_a = smem_addr(ring) + slot * S::kStageBytes, at_x = at_a + kABytes;
                    barrier_wait_inline(empty + 8 * slot, parity, dead);
                    if (lane == 0 && rank == 0) barrier_expect(full + 8 * slot, both_bytes);
                    __syncwarp();
                    if (lanes) {
                        if (lane < own) {
                            load_box_pair(at_a + lane * S::kBox * kBlock, &x_map, b * kBlock, it.row + rank * 128 + lane * S::kBox, 0, 0, bar);
                        } else if (lane == 31) {   // the first CTA has the gate rows or the first half, the second the others
                            if (SWIGLU) load_box_pair(at_x, &w_half_map, b * kBlock, it.m * (kTileRows / 2), rank, it.expert, bar);
                            else load_box_pair(at_x, &w_map, b * kBlock, row0, 0, it.expert, bar);
                        }
                    } else if (lane < a_boxes) {
                        if (SWIGLU) load_box_pair(at_a + lane * 4096, &w_map, b * kBlock, row0 / 2 + lane * 16, 0, it.expert, bar);
                        else load_box_pair(at_a, &w_map, b * kBlock, row0, 0, it.expert, bar);
                    } else if (lane - a_boxes < x_boxes) {
                        const int j = lane - a_boxes;
                        load_box_pair(at_x + j * S::kBox * kBlock, &x_map, b * kBlock, it.row + rank * half + j * S::kBox, 0, 0, bar);
                    }
                    if (++slot == S::kStages) slot = 0, parity ^= 1;
                }
            }
        } else if (warp == kIssuer && rank == 1) {   // (the first CTA's issues for both)
        } else if (warp == kIssuer) {
            const uint32_t base = (1u << 4) | (static_cast<uint32_t>(kTileRows / 16) << 24), e5m2 = a.x_dtype == EP_DTYPE_FP8_E5M2 ? 1u : 0u;
            int slot = 0, buffer = 0;
            uint32_t parity = 0, parities = 15;   // parities: a bit for each buffer of sums
            for (int64_t i = pair_id; i < items; i += pairs) {
                const Tile it = tile_at(a.g, plan, table, i);
                const bool lanes = LANES && it.rows > COLS;
                const uint32_t shape = base | (lanes ? e5m2 << 7 : e5m2 << 10) | static_cast<uint32_t>((lanes ? 256 : columns_of(it.rows)) / 8) << 17;
                for (int b = 0; b < blocks; ++b) {
                    barrier_wait_inline(full + 8 * slot, parity, dead);
                    if (lanes) {
                        buffer = (buffer + 1) & 2;   // an even one and the next
                        barrier_wait_inline(sums_empty + 8 * buffer + 8, (parities >> (buffer + 1)) & 1, dead);
                        parities ^= 2u << buffer;
                    }
                    barrier_wait_inline(sums_empty + 8 * buffer, (parities >> buffer) & 1, dead);
                    parities ^= 1u << buffer;
                    tmem_fence_after();
                    if (leader) {
                        const uint32_t at_a = smem_addr(ring) + slot * S::kStageBytes;
                        const uint64_t dw = operand(at_a, 1024), dx = operand(at_a + kABytes, 1024);
    #pragma unroll
                        for (int k = 0; k < kBlock / 32; ++k) multiply_pair<true>(tmem + buffer * S::kStride, dw + k * 2, dx + k * 2, shape, k > 0);
                        pair_done(empty + 8 * slot);
                        pair_done(sums_full + 8 * buffer);
                    }
                    __syncwarp();
                    if (++slot == S::kStages) slot = 0, parity ^= 1;
                    buffer = (buffer + (lanes ? 2 : 1)) % kBuffers;
                }
            }
        } else if (warp >= kScaler) {
            // Scales for two blocks at a time, the two warps in turn: products of the rows' and the weights' for rows as columns;
            // for rows as lanes the CTA's rows', and behind them the weights' of the first and second half's 64-row quarters.
            // Lanes run along what is dense in memory.
            int turn = warp - kScaler, slot = 0;
            uint32_t parity = 1;
            const bool by_rows = a.x_scale_block == 1;
            constexpr int kEach = kScaleBlocks * S::kRows / 32;
            const int wk = lane / 4 % kScaleBlocks, wj = lane % 4;   // lanes 0 .. 15 load the weights' scales: block, which one
            const auto row_of = [&](int j) { return by_rows ? j * (32 / kScaleBlocks) + lane / kScaleBlocks : j * 32 % S::kRows + lane; };
            const auto block_of = [&](int j) { return by_rows ? lane % kScaleBlocks : j * 32 / S::kRows; };
            for (int64_t i = pair_id; i < items; i += pairs) {
                const Tile it = tile_at(a.g, plan, table, i);
                const bool lanes = LANES && it.rows > COLS;
                const int skip = lanes ? rank * 128 : 0, rows = it.rows - skip;
                int o;
                if (!lanes) o = scale_row(it.m, min(wj, kScaleSets - 1));
                else if (SWIGLU) o = ((wj < 2 ? 0 : cols) + it.m * 128 + wj % 2 * 64) / kBlock;
                else o = it.m * 2 + wj / 2;
                const float* w_scales = a.w_scales + (static_cast<int64_t>(it.expert) * scale_rows + min(o, scale_rows - 1)) * blocks;
                for (int b = 0; b < blocks; b += kScaleBlocks) {
                    if (turn == 0) {
                        float v[kEach];
#pragma unroll
                        for (int j = 0; j < kEach; ++j) {
                            const int n = row_of(j), k = block_of(j);
                            v[j] = 0.0f;
                            if (n < rows && b + k < blocks) {
                                const int64_t from = (static_cast<int64_t>(it.row) + skip + n) * a.x_scale_row + (b + k) * a.x_scale_block;
                                v[j] = a.x_ue8m0 ? ue8m0(static_cast<const uint8_t*>(a.x_scales)[from]) : static_cast<const float*>(a.x_scales)[from];
                            }
                        }
                        const float w = w_scales[min(b + wk, blocks - 1)];
                        barrier_wait_inline(scales_empty + 8 * slot, parity, dead);
                        float* to = scales + slot * (kScaleBlocks * S::kScaleStep);
                        if (lanes && lane < 4 * kScaleBlocks) to[wk * S::kScaleStep + 128 + wj] = w;
#pragma unroll
                        for (int s = 0; s < kScaleSets; ++s) {
                            if (s >= (lanes ? 1 : sets)) continue;
#pragma unroll
                            for (int j = 0; j < kEach; ++j) {
                                const int n = row_of(j), k = block_of(j);
                                const float factor = __shfl_sync(kFullMask, w, k * 4 + s);
                                if (lanes || n < COLS) to[k * S::kScaleStep + s * COLS + n] = lanes ? v[j] : v[j] * factor;
                            }
                        }
                        __syncwarp();
                        if (lane == 0) barrier_arrive(scales_full + 8 * slot);
                    }
                    turn ^= 1;
                    if (++slot == kScaleSlots) slot = 0, parity ^= 1;
                }
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    cluster_sync();   // (neither CTA leaves while the other may arrive on its barriers)
    if (warp == kLoader) {
        tmem_fence_after();
        tmem_free_all(tmem);
    }
}

template <int COLS, bool LANES, bool SWIGLU>
cudaError_t launch_shape(const Fp8Args& a, cudaStream_t stream) {
    using S = Shape<COLS, LANES>;
    static int known[64];
    int pairs = 0;
    cudaError_t err = pairs_at_once(expert_fp8_kernel<COLS, LANES, SWIGLU>, kThreads, S::kShared, known, &pairs);
    if (err != cudaSuccess) return err;
    const int64_t I = a.I, O = a.O, E = a.g.E;
    const int cols = SWIGLU ? a.O / 2 : a.O;
    TilePlan p{};
    p.cap = LANES ? 256 : COLS;
    p.whole = LANES;
    p.chunk = 16;
    p.m_tiles = ceil_div(cols, SWIGLU ? kTileRows / 2 : kTileRows);
    while (((a.g.E - 1) >> p.shift) + 1 > kTileTable) ++p.shift;
    CUtensorMap w_map, w_half_map, x_map;
    err = SWIGLU ? box_map(&w_map, a.w, EP_DTYPE_FP8_E4M3, I, cols, 2, E, I, I * cols, I * O, 16, 2)
                 : box_map(&w_map, a.w, EP_DTYPE_FP8_E4M3, I, O, 1, E, I, I * O, I * O, 128, 1);
    w_half_map = w_map;
    if (SWIGLU && LANES && err == cudaSuccess) err = box_map(&w_half_map, a.w, EP_DTYPE_FP8_E4M3, I, cols, 2, E, I, I * cols, I * O, 128, 1);
    if (err == cudaSuccess) err = box_map(&x_map, a.x, EP_DTYPE_FP8_E4M3, I, a.g.rows, 1, 1, a.x_ld, a.x_ld, a.x_ld, S::kBox, 1);
    if (err != cudaSuccess) return err;
    const int64_t used = a.g.rows < a.g.E ? a.g.rows : a.g.E;
    const int64_t most = (a.g.rows + used * (p.cap - 1)) / p.cap * p.m_tiles;
    return launch_pairs(expert_fp8_kernel<COLS, LANES, SWIGLU>, static_cast<int>(most < pairs ? most : pairs), kThreads, S::kShared,
                        stream, a, p, w_map, w_half_map, x_map);
}

template <bool SWIGLU>
cudaError_t launch_activation(const Fp8Args& a, cudaStream_t stream) {
    const int used = a.g.rows < a.g.E ? a.g.rows : a.g.E, mean = (a.g.rows - 1) / used + 1;
    if (mean <= 24) return launch_shape<32, false, SWIGLU>(a, stream);
    // (64 neighbouring up rows have one scale)
    if (mean <= 48 || (SWIGLU && a.O / 2 % 64 != 0)) return launch_shape<64, false, SWIGLU>(a, stream);
    return launch_shape<64, true, SWIGLU>(a, stream);
}

}  // namespace

cudaError_t launch_expert_fp8(const Fp8Args& a, cudaStream_t stream) {
    return a.swiglu ? launch_activation<true>(a, stream) : launch_activation<false>(a, stream);
}

}  // namespace ep
