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

constexpr int kParts = 8;                       // warps over an item's weight rows: 32 lanes each
constexpr int kBlock = 128;                     // inputs of a stage: 128 bytes, one scale
constexpr int kTileRows = 256;                  // weight rows of an item: 128 a warpgroup
constexpr int kABytes = kTileRows * kBlock;
constexpr int kScaleBlocks = 4, kScaleSlots = 4;
constexpr int kMostStages = 6;

template <int COLS>
struct Shape {
    static constexpr int kCols = COLS < 64 ? COLS : 64;      // columns of a consuming warp
    static constexpr int kConsumers = 32 * kParts * (COLS / kCols);
    static constexpr int kLoader = kConsumers / 32, kIssuer = kLoader + 1, kScaler = kLoader + 2;   // warps
    static constexpr int kThreads = kConsumers + 96;
    static constexpr int kStageBytes = kABytes + COLS * kBlock;
    static constexpr int kStages = 196 * 1024 / kStageBytes < kMostStages ? 196 * 1024 / kStageBytes : kMostStages;
    static constexpr int kBox = COLS < 32 ? 16 : 32;
    static constexpr int kScaleBytes = kScaleSlots * kScaleBlocks * COLS * 4;
    static constexpr int kMostBytes = (kParts + 2) * COLS * 4;   // amax by part and column, then scales by column
    static constexpr int kShared = 1024 + kStages * kStageBytes + kScaleBytes + kMostBytes + 512 + (kTileTable + 1) * 4;
    static_assert(kShared <= 227 * 1024 - 256, "");
};

__device__ __forceinline__ float ue8m0(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fffffffu : byte << 23);
}
template <int THREADS>
__device__ __forceinline__ void consumers_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// Smallest power of two >= s (s > 0), as the dispatch's scales.
__device__ __forceinline__ float power_of_two(float s) {
    const uint32_t u = __float_as_uint(s), e = u >> 23, f = u & 0x7fffffu;
    if (e == 0) return __uint_as_float((f & (f - 1u)) == 0u ? f : (1u << (32 - __clz(f))));
    return f == 0u || e == 255 ? s : __uint_as_float((e + 1u) << 23);
}

// COLS: rows of x of an item at most.
template <int COLS>
__global__ void __launch_bounds__(Shape<COLS>::kThreads, 1)
    expert_fp8_kernel(Fp8Args a, TilePlan plan, const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map) {
    using S = Shape<COLS>;
    constexpr int kConsumers = S::kConsumers, kLoader = S::kLoader, kIssuer = S::kIssuer, kScaler = S::kScaler, kThreads = S::kThreads;
    extern __shared__ unsigned char shared_bytes[];
    unsigned char* const ring = shared_bytes + (1024 - smem_addr(shared_bytes) % 1024) % 1024;
    float* const scales = reinterpret_cast<float*>(ring + S::kStages * S::kStageBytes);   // [kScaleSlots][kScaleBlocks][COLS]
    float* const most = scales + kScaleSlots * kScaleBlocks * COLS;                       // [kParts][COLS]
    float* const found = most + kParts * COLS;                                            // [2][COLS]
    uint64_t* const barriers = reinterpret_cast<uint64_t*>(found + 2 * COLS);
    const uint32_t full = smem_addr(barriers), empty = full + 8 * kMostStages;
    const uint32_t sums_full = empty + 8 * kMostStages, sums_empty = sums_full + 16;
    const uint32_t scales_full = sums_empty + 16, scales_empty = scales_full + 8 * kScaleSlots;
    uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(barriers) + 120;
    volatile int* const dead = reinterpret_cast<volatile int*>(tmem_at + 1);
    int* const table = reinterpret_cast<int*>(barriers) + 128;
    static_assert((2 * kMostStages + 4 + 2 * kScaleSlots) * 2 <= 120, "");
    __shared__ int warp_sum[kThreads / 32];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (warp == kLoader) {
        tmem_alloc_all(smem_addr(tmem_at));
        if (lane == 0) {
            *dead = 0;
            for (int i = 0; i < S::kStages; ++i) {
                barrier_init(full + 8 * i, 1);
                barrier_init(empty + 8 * i, 1);
            }
            for (int i = 0; i < 2; ++i) {
                barrier_init(sums_full + 8 * i, 1);
                barrier_init(sums_empty + 8 * i, kConsumers / 32);
            }
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
    tmem_fence_after();
    const uint32_t tmem = __shfl_sync(kFullMask, *tmem_at, 0);
    const bool leader = elected();
    const int blocks = a.I / kBlock, cols = a.swiglu ? a.O / 2 : a.O;
    const int64_t items = tile_count(a.g, plan, table);

    if (warp == kLoader) {
        int slot = 0;
        uint32_t parity = 1;
        for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
            const Tile it = tile_at(a.g, plan, table, i);
            const int a_boxes = a.swiglu ? 8 : 2, x_boxes = (max(it.rows, 1) + S::kBox - 1) / S::kBox;
            for (int b = 0; b < blocks; ++b) {
                const uint32_t bar = full + 8 * slot, at_a = smem_addr(ring) + slot * S::kStageBytes, at_x = at_a + kABytes;
                barrier_wait(empty + 8 * slot, parity, dead);
                if (lane == 0) barrier_expect(bar, kABytes + x_boxes * S::kBox * kBlock);
                __syncwarp();
                if (lane < a_boxes) {
                    if (a.swiglu) load_box(at_a + lane * 4096, &w_map, b * kBlock, it.m * (kTileRows / 2) + lane * 16, 0, it.expert, bar);
                    else load_box(at_a + lane * 16384, &w_map, b * kBlock, it.m * kTileRows + lane * 128, 0, it.expert, bar);
                } else if (lane - a_boxes < x_boxes) {
                    const int j = lane - a_boxes;
                    load_box(at_x + j * S::kBox * kBlock, &x_map, b * kBlock, it.row + j * S::kBox, 0, 0, bar);
                }
                if (++slot == S::kStages) slot = 0, parity ^= 1;
            }
        }
    } else if (warp == kIssuer) {
        const uint32_t base = (1u << 4) | (a.x_dtype == EP_DTYPE_FP8_E5M2 ? 1u << 10 : 0u) | (128u / 16 << 24);
        int slot = 0, buffer = 0;
        uint32_t parity = 0, sums_parity = 1;
        for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
            const Tile it = tile_at(a.g, plan, table, i);
            const uint32_t shape = base | static_cast<uint32_t>(columns_of(it.rows) / 8) << 17;
            for (int b = 0; b < blocks; ++b) {
                barrier_wait(full + 8 * slot, parity, dead);
                barrier_wait(sums_empty + 8 * buffer, sums_parity, dead);
                tmem_fence_after();
                if (leader) {
                    const uint32_t at_a = smem_addr(ring) + slot * S::kStageBytes;
                    const uint64_t dx = operand(at_a + kABytes, 1024);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const uint64_t dw = operand(at_a + g * 16384, 1024);
#pragma unroll
                        for (int k = 0; k < kBlock / 32; ++k)
                            multiply_shared<true>(tmem + buffer * 256 + g * 128, dw + k * 2, dx + k * 2, shape, k > 0);
                    }
                    multiply_done(empty + 8 * slot);
                    multiply_done(sums_full + 8 * buffer);
                }
                __syncwarp();
                if (++slot == S::kStages) slot = 0, parity ^= 1;
                buffer ^= 1;
                if (buffer == 0) sums_parity ^= 1;
            }
        }
    } else if (warp == kScaler) {
        // scales of x, four blocks ahead of their use or more; lanes run along what is dense in memory
        int slot = 0;
        uint32_t parity = 1;
        const bool by_rows = a.x_scale_block == 1;
        for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
            const Tile it = tile_at(a.g, plan, table, i);
            for (int b = 0; b < blocks; b += kScaleBlocks) {
                constexpr int kEach = kScaleBlocks * COLS / 32;
                float v[kEach];
#pragma unroll
                for (int j = 0; j < kEach; ++j) {
                    const int at = j * 32 + lane, k = by_rows ? at % kScaleBlocks : at / COLS, n = by_rows ? at / kScaleBlocks : at % COLS;
                    v[j] = 0.0f;
                    if (n < it.rows && b + k < blocks) {
                        const int64_t from = (static_cast<int64_t>(it.row) + n) * a.x_scale_row + (b + k) * a.x_scale_block;
                        v[j] = a.x_ue8m0 ? ue8m0(static_cast<const uint8_t*>(a.x_scales)[from]) : static_cast<const float*>(a.x_scales)[from];
                    }
                }
                barrier_wait(scales_empty + 8 * slot, parity, dead);
#pragma unroll
                for (int j = 0; j < kEach; ++j) {
                    const int at = j * 32 + lane, k = by_rows ? at % kScaleBlocks : at / COLS, n = by_rows ? at / kScaleBlocks : at % COLS;
                    scales[(slot * kScaleBlocks + k) * COLS + n] = v[j];
                }
                __syncwarp();
                if (lane == 0) barrier_arrive(scales_full + 8 * slot);
                if (++slot == kScaleSlots) slot = 0, parity ^= 1;
            }
        }
    } else {
        // 32 weight rows (the product's lanes) of one of the two tiles, columns c0 .. c0 + kCols
        constexpr int kCols = S::kCols;
        const int part = warp % kParts, wg = part >> 2, c0 = warp / kParts * kCols;
        const uint32_t mine = tmem + wg * 128 + c0 + (static_cast<uint32_t>(part & 3) << 21);
        int buffer = 0, slot = 0;
        uint32_t parity = 0, scales_parity = 0;
        for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
            const Tile it = tile_at(a.g, plan, table, i);
            const int many = it.rows - c0;   // of this warp's columns, those with a row
            // this thread's output channel and weight row; with the activation a warp's lanes are 16 gate and 16 up rows
            const int chan = a.swiglu ? it.m * (kTileRows / 2) + part * 16 + (lane & 15) : it.m * kTileRows + part * 32 + lane;
            const bool real = chan < cols;
            const int o = real ? (a.swiglu && lane >= 16 ? cols + chan : chan) : 0;
            const float* w_scale = a.w_scales + (static_cast<int64_t>(it.expert) * ceil_div(a.O, kBlock) + o / kBlock) * blocks;
            uint64_t acc[kCols / 2];   // columns 2 n, 2 n + 1
#pragma unroll
            for (int n = 0; n < kCols / 2; ++n) acc[n] = 0;
            float sw = *w_scale;
            for (int b = 0; b < blocks; ++b) {
                if (b % kScaleBlocks == 0) barrier_wait(scales_full + 8 * slot, scales_parity, dead);
                const float* sx = scales + (slot * kScaleBlocks + b % kScaleBlocks) * COLS + c0;
                const uint64_t sw2 = both(sw);
                sw = w_scale[min(b + 1, blocks - 1)];
                barrier_wait(sums_full + 8 * buffer, parity, dead);
                tmem_fence_after();
#pragma unroll
                for (int c = 0; c < kCols; c += 8) {
                    if (c >= many) continue;
                    uint32_t raw[8];
                    tmem_load8(mine + buffer * 256 + c, raw);
                    tmem_load_wait();
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(sx + c + j);
                        acc[(c + j) / 2] = fma2(mul2(pair(raw[j], raw[j + 1]), s.x), sw2, acc[(c + j) / 2]);
                        acc[(c + j) / 2 + 1] = fma2(mul2(pair(raw[j + 2], raw[j + 3]), s.y), sw2, acc[(c + j) / 2 + 1]);
                    }
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) barrier_arrive(sums_empty + 8 * buffer);
                if (b % kScaleBlocks == kScaleBlocks - 1 || b + 1 == blocks) {
                    if (lane == 0) barrier_arrive(scales_empty + 8 * slot);
                    if (++slot == kScaleSlots) slot = 0, scales_parity ^= 1;
                }
                buffer ^= 1;
                if (buffer == 0) parity ^= 1;
            }

            if (*dead) {
#pragma unroll
                for (int n = 0; n < kCols / 2; ++n) acc[n] = both(__int_as_float(0x7fffffff));
            }
            // The epilogue takes column pairs; with the activation each thread has one result a pair: gate lanes the even
            // column's, up lanes the odd one's.
            const int odd = lane >> 4;
            if (a.swiglu) {
#pragma unroll
                for (int n = 0; n < kCols / 2; ++n) {
                    const float2 v = apart(acc[n]);
                    const float own = lane < 16 ? v.x : v.y, got = __shfl_xor_sync(kFullMask, lane < 16 ? v.y : v.x, 16);
                    acc[n] = both(lane < 16 ? silu(own) * got : silu(got) * own);
                }
            }
            const int64_t row = static_cast<int64_t>(it.row) + c0;
            if (a.y_dtype != EP_DTYPE_FP8_E4M3) {
                if (!real) continue;
                const auto store = [&](int c, float v) {
                    const int64_t to = (row + c) * a.y_ld + chan;
                    if (c >= many) return;
                    if (a.y_dtype == EP_DTYPE_BF16) static_cast<__nv_bfloat16*>(a.y)[to] = __float2bfloat16_rn(v);
                    else static_cast<__half*>(a.y)[to] = __float2half_rn(v);
                };
#pragma unroll
                for (int n = 0; n < kCols / 2; ++n) {
                    const float2 v = apart(acc[n]);
                    if (a.swiglu) store(2 * n + odd, v.x);
                    else store(2 * n, v.x), store(2 * n + 1, v.y);
                }
                continue;
            }
            // ---- e4m3: the largest of each column's 128 channels (4 parts, with the activation 8), its scale, codes
            const auto largest = [&](uint32_t mask, float v) {   // (of numbers that are not negative the bits compare as they do)
                return __uint_as_float(__reduce_max_sync(mask, real ? __float_as_uint(fabsf(v)) : 0u));
            };
#pragma unroll
            for (int n = 0; n < kCols / 2; ++n) {
                if (2 * n >= many) continue;
                const float2 v = apart(acc[n]);
                float* to = most + part * COLS + c0 + 2 * n;
                if (a.swiglu) {
                    const float big = largest(lane < 16 ? 0x0000ffffu : 0xffff0000u, v.x);
                    if ((lane & 15) == 0) to[odd] = big;
                } else {
                    const float2 big = make_float2(largest(kFullMask, v.x), largest(kFullMask, v.y));
                    if (lane == 0) to[0] = big.x, to[1] = big.y;
                }
            }
            consumers_sync<kConsumers>();
            const int each = a.swiglu ? 8 : 4;   // parts of a block of 128 channels
            for (int t = tid; t < COLS * (8 / each); t += kConsumers) {
                const int n = t % COLS, first = t / COLS * each, block = it.m * (8 / each) + t / COLS;
                if (n >= it.rows) continue;
                float big = 0.0f;
                for (int w = first; w < first + each; ++w) {
                    const float m = most[w * COLS + n];
                    big = m > big || m != m ? m : big;   // (NaN stays)
                }
                float s = 0.0f;
                if (big != 0.0f) {
                    s = __fdiv_rn(big, 448.0f);
                    if (a.y_scale_mode != EP_SCALE_FP32 && s > 0.0f) s = power_of_two(s);
                    if (a.y_scale_mode == EP_SCALE_UE8M0) s = s < __uint_as_float(0x00400000u) ? __uint_as_float(0x00400000u) : s;
                }
                found[t] = s;
                if (block * kBlock < cols) {
                    const int64_t to = (static_cast<int64_t>(it.row) + n) * a.y_scale_row + block * a.y_scale_block;
                    if (a.y_scale_mode == EP_SCALE_UE8M0) static_cast<uint8_t*>(a.y_scales)[to] = static_cast<uint8_t>(__float_as_uint(s) >> 23);
                    else static_cast<float*>(a.y_scales)[to] = s;
                }
            }
            consumers_sync<kConsumers>();
            if (real) {
                const float* my = found + (a.swiglu ? 0 : wg * COLS) + c0;
                const auto store = [&](int c, float v) {
                    if (c >= many) return;
                    const float s = my[c];
                    static_cast<uint8_t*>(a.y)[(row + c) * a.y_ld + chan] =
                        s == 0.0f ? 0 : __nv_cvt_float_to_fp8(__fdiv_rn(v, s), __NV_SATFINITE, __NV_E4M3);
                };
#pragma unroll
                for (int n = 0; n < kCols / 2; ++n) {
                    const float2 v = apart(acc[n]);
                    if (a.swiglu) store(2 * n + odd, v.x);
                    else store(2 * n, v.x), store(2 * n + 1, v.y);
                }
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == kLoader) {
        tmem_fence_after();
        tmem_free_all(tmem);
    }
}

template <int COLS>
cudaError_t launch_columns(const Fp8Args& a, cudaStream_t stream) {
    using S = Shape<COLS>;
    static int known[64];
    int sms = 0;
    cudaError_t err = prepare_persistent(expert_fp8_kernel<COLS>, S::kShared, known, &sms);
    if (err != cudaSuccess) return err;
    const int64_t I = a.I, O = a.O, E = a.g.E;
    const int cols = a.swiglu ? a.O / 2 : a.O;
    TilePlan p{};
    p.cap = COLS;
    p.chunk = 16;
    p.m_tiles = ceil_div(cols, a.swiglu ? kTileRows / 2 : kTileRows);
    while (((a.g.E - 1) >> p.shift) + 1 > kTileTable) ++p.shift;
    CUtensorMap w_map, x_map;
    err = a.swiglu ? box_map(&w_map, a.w, EP_DTYPE_FP8_E4M3, I, cols, 2, E, I, I * cols, I * O, 16, 2)
                   : box_map(&w_map, a.w, EP_DTYPE_FP8_E4M3, I, O, 1, E, I, I * O, I * O, 128, 1);
    if (err == cudaSuccess)
        err = box_map(&x_map, a.x, EP_DTYPE_FP8_E4M3, I, a.g.rows, 1, 1, a.x_ld, a.x_ld, a.x_ld, S::kBox, 1);
    if (err != cudaSuccess) return err;
    const int64_t used = a.g.rows < a.g.E ? a.g.rows : a.g.E;
    const int64_t most = (a.g.rows + used * (COLS - 1)) / COLS * p.m_tiles;
    return launch_dependent(expert_fp8_kernel<COLS>, dim3(static_cast<unsigned>(most < sms ? most : sms)), dim3(S::kThreads), S::kShared,
                            stream, a, p, w_map, x_map);
}

}  // namespace

cudaError_t launch_expert_fp8(const Fp8Args& a, cudaStream_t stream) {
    const int used = a.g.rows < a.g.E ? a.g.rows : a.g.E, mean = (a.g.rows - 1) / used + 1;
    return mean <= 12 ? launch_columns<16>(a, stream) : mean <= 48 ? launch_columns<64>(a, stream) : launch_columns<128>(a, stream);
}

}  // namespace ep
