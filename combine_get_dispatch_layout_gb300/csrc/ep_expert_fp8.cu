// The experts' products in 8-bit floating point: rows with a scale per 128 inputs
// (as the fp8 dispatch writes them), weights with a scale per block of 128 x 128.
//
// Mathematics. y[n, o] = sum over blocks b of sx[n, b] sw[o / 128, b] * sum over i in b of cx[n, i] cw[o, i]. The inner
// sums, 128 products of two codes, run through the tensor cores with fp32 sums; each is then scaled and added in fp32
// registers, because the scales change from block to block and so cannot stay behind in the tensor cores' sums. The two
// scales are multiplied first. With the activation: silu(gate) * up of the fp32 sums. An fp8 output is quantised as the
// dispatch quantises: amax of 128 channels / 448, codes by IEEE division; that is the format that the next call reads.
//
// Kernel. An item is 256 weight rows (gate and up of the same 128 channels with the activation) times a tile of rows of one
// expert, on one CTA: a loader thread (TMA ring, 128 inputs a stage), an issuer thread (four buffers of sums in TMEM), two
// warps that bring scales, and eight warps that take each block's sums from TMEM and add them. Two layouts:
//   rows as columns (up to 64 rows): a thread has a channel of each half and all rows; two groups of four warps take every other
//     block and join at the end. Few rows cost few columns. The rows' scales are read from shared memory, four clocks for
//     four of them a warp, which is what bounds tiles of many rows.
//   rows as lanes (65 to 128 rows): a thread has a row and 64 channels of each half; its scales are two numbers a block.
// The sums of the next chunk, and at a block's end of the next block, are on their way while a chunk is added (16 columns;
// without the block's end: 8192 x 4096 x 8192 386 us, with it 352).
//
// What bounds it (one GB300). Decode, 256 tokens of top 8 of 256 experts, 7168 x 2048, both products: 1590 to 1640 us, 6.9 to 7.1 TB/s of
// weights: memory. One token of the same, gate and up: 41 us, 5.7 TB/s after 6 us of start. 4 rows of one 4096 x 4096 matrix:
// 8.2 us, start and latency. Prompt of 8192 tokens, 7168 x 4096: 2.6 to 2.8 ms, 1360 to 1470 TFLOP/s (256 rows of each of 128 experts:
// 1800): a block of a full tile takes an SM 710 ns; without the additions 577, which is 48 KB at the 83 GB/s that come into
// an SM; the products are 210 of them. Twice the warps for the additions: no less. As CTA pairs (32 KB a block) it took as long
// for prompts and 1.85 ms instead of 1.62 for the decode step, because the two CTAs wait for one another's consumers; with the
// weights sent to two CTAs by multicast full tiles took as long too (as much comes into each SM), and experts of 138 rows 1227
// us instead of 980. Rows as lanes leave through shared memory, four lanes a row's 64 bytes: prompt 2.87 to 2.70 ms.
#include "ep_expert_tiles.cuh"
#include "ep_sums_turn.cuh"

namespace ep {
namespace {

constexpr int kBlock = 128;                     // inputs of a stage: 128 bytes, one scale
constexpr int kTileRows = 256;                  // weight rows of an item: two halves of 128, gate and up with the activation
constexpr int kParts = 4;                       // warps over 128 lanes
constexpr int kGroups = 2;                      // groups of kParts warps: they take blocks or columns in turn
constexpr int kConsumers = 32 * kParts * kGroups;
constexpr int kLoader = kConsumers / 32, kIssuer = kLoader + 1, kScaler = kLoader + 2;   // warps; two scalers
constexpr int kThreads = kConsumers + 128;
constexpr int kWBytes = kTileRows * kBlock;
constexpr int kScaleSlots = 4;                  // of the ring of scales
constexpr int kMostStages = 6;
constexpr int kMostSplit = 8;                   // CTAs of a cluster that share an item (the largest portable cluster)

// COLS: rows of x that are columns of a product, at most. LANES: tiles of more rows have them as lanes.
template <int COLS, bool LANES>
struct Shape {
    static_assert(COLS == 32 || COLS == 64, "");
    static constexpr bool kMoved = COLS == 64;                   // up to 128 sums a thread: registers move to the consumers
    static constexpr int kRows = LANES ? 128 : COLS;             // rows of x of an item
    static constexpr int kScaleBlocks = LANES ? 2 : 4;           // blocks of a slot of the ring of scales
    static constexpr int kScaleStep = kRows + 4;                 // floats of a block: the rows' scales, up to four of the weights'
    static constexpr int kBox = COLS / 2;
    static constexpr int kStageBytes = kWBytes + kRows * kBlock;
    static constexpr int kStages = 192 * 1024 / kStageBytes < kMostStages ? 192 * 1024 / kStageBytes : kMostStages;
    static constexpr int kScales = kScaleSlots * kScaleBlocks * kScaleStep;   // floats
    static constexpr int kChunk = LANES ? 8 : 16;                // columns whose sums meet at a time
    static constexpr int kJoin = kGroups * 2 * kChunk * 128;
    static constexpr int kMost = 4 * 128;
    static constexpr int kShared = 1024 + kStages * kStageBytes + (kScales + kJoin + kMost) * 4 + 512 + static_cast<int>(sizeof(Tables));
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
    expert_fp8_kernel(Fp8Args a, TilePlan plan, int split, const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map) {
    using S = Shape<COLS, LANES>;
    constexpr int kScaleBlocks = S::kScaleBlocks, kChunk = S::kChunk;
    extern __shared__ unsigned char shared_bytes[];
    unsigned char* const ring = shared_bytes + (1024 - smem_addr(shared_bytes) % 1024) % 1024;
    float* const scales = reinterpret_cast<float*>(ring + S::kStages * S::kStageBytes);   // [kScaleSlots][kScaleBlocks][kScaleStep]
    float* const join = scales + S::kScales;                                              // [kGroups][2 halves][kChunk][128]
    // the largest: [2][2][128] of rows as lanes; [kGroups][2][2 halves][kParts] of rows as columns
    float* const most = join + S::kJoin;
    uint64_t* const barriers = reinterpret_cast<uint64_t*>(most + S::kMost);
    const uint32_t full = smem_addr(barriers), empty = full + 8 * kMostStages;
    const uint32_t sums_full = empty + 8 * kMostStages, sums_empty = sums_full + 8 * kBuffers;
    const uint32_t scales_full = sums_empty + 8 * kBuffers, scales_empty = scales_full + 8 * kScaleSlots;
    uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(barriers) + 120;
    volatile int* const dead = reinterpret_cast<volatile int*>(tmem_at + 1);
    Tables* const table = reinterpret_cast<Tables*>(barriers + 64);
    static_assert((2 * kMostStages + 2 * kBuffers + 2 * kScaleSlots) * 2 <= 120, "");
    __shared__ int warp_sum[kThreads / 32];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (warp == kScaler && elected()) {
        prefetch_map(&w_map);
        prefetch_map(&x_map);
    }
    if (warp == kLoader) {
        tmem_alloc_one(smem_addr(tmem_at));
        if (lane == 0) {
            *dead = 0;
            for (int i = 0; i < S::kStages; ++i) {
                barrier_init(full + 8 * i, 1);
                barrier_init(empty + 8 * i, 1);
            }
            for (int i = 0; i < kBuffers; ++i) {
                barrier_init(sums_full + 8 * i, 1);
                barrier_init(sums_empty + 8 * i, kParts);   // a group
            }
            for (int i = 0; i < kScaleSlots; ++i) {
                barrier_init(scales_full + 8 * i, 1);
                barrier_init(scales_empty + 8 * i, kConsumers / 32);
            }
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    }
    dependent_entry();
    fill_tables<kThreads>(a.g, plan, table, warp_sum);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = __shfl_sync(kFullMask, *tmem_at, 0);
    const bool leader = elected();
    const int blocks = a.I / kBlock, cols = SWIGLU ? a.O / 2 : a.O;
    const int64_t items = tile_count(a.g, plan, table);
    // CTAs of a cluster that share items have one each at most, of which each takes some of the blocks.
    const int sharer = split > 1 ? cluster_rank() : 0;
    const int block0 = static_cast<int>(static_cast<int64_t>(blocks) * sharer / split);
    const int block1 = static_cast<int>(static_cast<int64_t>(blocks) * (sharer + 1) / split);
    const int64_t item0 = blockIdx.x / split, item_step = split > 1 ? items : gridDim.x;

    // First channel of an item's halves (of gate and up they are the same ones), and their first weight rows.
    const auto channel = [&](int m, int half) { return SWIGLU ? m * 128 : m * kTileRows + half * 128; };
    const auto weight_row = [&](int m, int half) { return SWIGLU ? half * cols + m * 128 : m * kTileRows + half * 128; };

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
    const auto code8 = [](float v, float s) -> uint8_t { return s == 0.0f ? 0 : __nv_cvt_float_to_fp8(__fdiv_rn(v, s), __NV_SATFINITE, __NV_E4M3); };
    const auto codes = [](float2 v, float s) -> uint32_t {
        return s == 0.0f ? 0u : __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(v.x, s), __fdiv_rn(v.y, s)), __NV_SATFINITE, __NV_E4M3);
    };

    // (registers: 256 x 216 + 128 x 72 of the launch's 384 x 168)
    if (warp < kLoader) {
        if constexpr (S::kMoved) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int part = warp % kParts, group = warp / kParts;
        const uint32_t mine = tmem + (static_cast<uint32_t>(part) << 21);   // lanes 32 * part, upper half
        int buffer = 0, slot = 0;
        uint32_t parities = 0, scales_parity = 0;   // parities: a bit for each buffer
        // A tile whose rows of x are the lanes: a thread has one of them and 64 columns of each half of the 256 weight rows (gate
        // and up of the same 64 channels). Its scales are two numbers a block.
        const auto rows_as_lanes = [&](const Tile& it) {
            const int r = part * 32 + lane, h = group;
            const bool real = r < it.rows;
            const int64_t row = it.row + static_cast<int64_t>(real ? r : 0);
            const int first = channel(it.m, 0) + h * 64, second = channel(it.m, 1) + h * 64;
            uint64_t acc[2][32];
#pragma unroll
            for (int n = 0; n < 32; ++n) acc[0][n] = acc[1][n] = 0;
            // the scales of a block are fetched while the sums of the one before are on their way
            float s0, s1;
            const auto fetch = [&](int b) {
                if (b % kScaleBlocks == 0) barrier_wait_inline(scales_full + 8 * slot, scales_parity, dead);
                const float* sx = scales + (slot * kScaleBlocks + b % kScaleBlocks) * S::kScaleStep;
                const float x_scale = sx[r];
                s0 = x_scale * sx[S::kRows + h], s1 = x_scale * sx[S::kRows + 2 + h];
                if (b % kScaleBlocks == kScaleBlocks - 1 || b + 1 == blocks) {
                    __syncwarp();
                    if (lane == 0) barrier_arrive(scales_empty + 8 * slot);
                    if (++slot == kScaleSlots) slot = 0, scales_parity ^= 1;
                }
            };
            fetch(0);
            buffer = (buffer + 1) & 2;   // an even one and the next

            uint32_t raw[2][16];
            const auto begin = [&] {
                barrier_wait_inline(sums_full + 8 * buffer, (parities >> buffer) & 1, dead);
                tmem_fence_after();
                tmem_load16(mine + buffer * 128 + h * 64, raw[0]);
            };
            begin();
            for (int b = 0; b < blocks; ++b) {
                const uint32_t at = mine + buffer * 128 + h * 64;
                const uint64_t f0 = both(s0), f1 = both(s1);
                if (b + 1 < blocks) fetch(b + 1);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    tmem_loaded(raw[c & 1]);
                    if (c < 7) {
                        tmem_load16(at + (c + 1) / 4 * 128 + (c + 1) % 4 * 16, raw[(c + 1) & 1]);
                    } else {
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0) barrier_arrive(sums_empty + 8 * (buffer + h));
                        parities ^= 1u << buffer;
                        buffer ^= 2;
                        if (b + 1 < blocks) begin();
                    }
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        uint64_t& to = acc[c / 4][c % 4 * 8 + n];
                        to = fma2(pair(raw[c & 1][2 * n], raw[c & 1][2 * n + 1]), c < 4 ? f0 : f1, to);
                    }
                }
            }
            if (*dead) {
#pragma unroll
                for (int n = 0; n < 32; ++n) acc[0][n] = acc[1][n] = both(__int_as_float(0x7fffffff));
            }
            if constexpr (SWIGLU) {
#pragma unroll
                for (int n = 0; n < 32; ++n) {
                    const float2 g = apart(acc[0][n]), u = apart(acc[1][n]);
                    acc[0][n] = pair(__float_as_uint(gated(g.x, u.x)), __float_as_uint(gated(g.y, u.y)));
                }
            }
            constexpr int kHalves = SWIGLU ? 1 : 2;
            // 64 bytes of each of the warp's rows (at the rows' end `bytes`), through the warp's part of `join` (16-byte pieces
            // swapped by row against bank conflicts): four lanes write a row's
            static_assert(!LANES || S::kJoin >= kConsumers * 16, "");
            uint32_t* const turn = reinterpret_cast<uint32_t*>(join) + warp * (32 * 16);
            const int most_rows = min(it.rows - part * 32, 32);
            const int64_t row0 = static_cast<int64_t>(it.row) + part * 32;
            const auto leave = [&](const uint32_t (&w)[16], char* to, int64_t pitch, int bytes) {
                uint4* const lines = reinterpret_cast<uint4*>(turn);
#pragma unroll
                for (int q = 0; q < 4; ++q) lines[lane * 4 + (q ^ (lane >> 1 & 3))] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
                __syncwarp();
                const int at = lane % 4 * 16;
                to += lane / 4 * pitch + at;
#pragma unroll
                for (int k = 0; k < 32; k += 8, to += 8 * pitch) {
                    if (k + lane / 4 >= most_rows || at >= bytes) continue;
                    const uint4 v = lines[(k + lane / 4) * 4 + (lane % 4 ^ lane / 8)];
                    if (at + 16 <= bytes) {
                        *reinterpret_cast<uint4*>(to) = v;
                    } else {
                        const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (at + 2 * j < bytes) reinterpret_cast<uint16_t*>(to)[j] = static_cast<uint16_t>(word[j / 2] >> (j % 2 * 16));
                    }
                }
                __syncwarp();
            };
            if (a.y_dtype != EP_DTYPE_FP8_E4M3) {
                const bool bf16 = a.y_dtype == EP_DTYPE_BF16, wide = a.y_ld % 8 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
                if (!wide) {   // rows that start anywhere: 32 rows x 32 channels at a time through shared memory, a row a warp's store
#pragma unroll
                    for (int half = 0; half < kHalves; ++half)
#pragma unroll
                        for (int n0 = 0; n0 < 32; n0 += 16) {
                            const int chan = (half == 0 ? first : second) + 2 * n0;
#pragma unroll
                            for (int n = 0; n < 16; ++n) {
                                const float2 v = apart(acc[half][n0 + n]);
                                const __nv_bfloat162 vb = __floats2bfloat162_rn(v.x, v.y);
                                const __half2 vh = __floats2half2_rn(v.x, v.y);
                                turn[lane * 16 + ((n + lane / 2) & 15)] = bf16 ? *reinterpret_cast<const uint32_t*>(&vb) : *reinterpret_cast<const uint32_t*>(&vh);
                            }
                            __syncwarp();
                            uint16_t* to = static_cast<uint16_t*>(a.y) + row0 * a.y_ld + chan + lane;
                            for (int k = 0; k < most_rows; ++k, to += a.y_ld)
                                if (chan + lane < cols) *to = reinterpret_cast<const uint16_t*>(turn + k * 16)[(2 * ((lane / 2 + k / 2) & 15)) + (lane & 1)];
                            __syncwarp();
                        }
                    consumers_sync();   // (a tile with rows as columns uses `join` otherwise)
                    return;
                }
#pragma unroll
                for (int half = 0; half < kHalves; ++half) {
#pragma unroll
                    for (int n0 = 0; n0 < 32; n0 += 16) {
                        const int chan = (half == 0 ? first : second) + 2 * n0;
                        uint32_t w[16];
#pragma unroll
                        for (int n = 0; n < 16; ++n) {
                            const float2 v = apart(acc[half][n0 + n]);
                            const __nv_bfloat162 vb = __floats2bfloat162_rn(v.x, v.y);
                            const __half2 vh = __floats2half2_rn(v.x, v.y);
                            w[n] = bf16 ? *reinterpret_cast<const uint32_t*>(&vb) : *reinterpret_cast<const uint32_t*>(&vh);
                        }
                        leave(w, reinterpret_cast<char*>(static_cast<uint16_t*>(a.y) + row0 * a.y_ld + chan), a.y_ld * 2, min(cols - chan, 32) * 2);
                    }
                }
                consumers_sync();
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
                if (chan >= cols) continue;   // (columns are a multiple of 128)
                if (h == 0 && real) write_scale(row, chan / kBlock, s);
                uint32_t w[16];
#pragma unroll
                for (int n = 0; n < 16; ++n) w[n] = codes(apart(acc[half][2 * n]), s) | codes(apart(acc[half][2 * n + 1]), s) << 16;
                if (wide) {
                    leave(w, static_cast<char*>(a.y) + row0 * a.y_ld + chan, a.y_ld, 64);
                } else if (real) {
                    uint8_t* to = static_cast<uint8_t*>(a.y) + row * a.y_ld + chan;
#pragma unroll
                    for (int k = 0; k < 64; ++k) to[k] = static_cast<uint8_t>(w[k / 4] >> (k % 4 * 8));
                }
            }
            consumers_sync();   // (`most` and `join` are written again)
        };
        for (int64_t i = item0; i < items; i += item_step) {
            const Tile it = tile_at(a.g, plan, table, i);
            if constexpr (LANES) {
                if (it.rows > COLS) {
                    rows_as_lanes(it);
                    continue;
                }
            }
            // A tile whose rows of x are columns: a thread has a channel of each half (gate and up of one).
            const int there = max(it.rows, 1);   // (a tile without rows has a product all the same)
            const int first = channel(it.m, 0) + part * 32 + lane, second = channel(it.m, 1) + part * 32 + lane;
            // its second weight scale is the third of the ring where up rows of a tile lie in two blocks
            const int w_second = SWIGLU && second < cols ? 1 + (cols + second) / kBlock - weight_row(it.m, 1) / kBlock : 1;
            uint64_t acc[2][COLS / 2];   // columns 2 n, 2 n + 1; the groups take every other block each
#pragma unroll
            for (int n = 0; n < COLS / 2; ++n) acc[0][n] = acc[1][n] = 0;
            for (int b = 0; b < block1 - block0; ++b) {
                if (b % kScaleBlocks == 0) barrier_wait_inline(scales_full + 8 * slot, scales_parity, dead);
                if (b % kGroups == group) {
                    const float* sx = scales + (slot * kScaleBlocks + b % kScaleBlocks) * S::kScaleStep;
                    const uint64_t w[2] = {both(sx[S::kRows]), both(sx[S::kRows + w_second])};
                    barrier_wait_inline(sums_full + 8 * buffer, (parities >> buffer) & 1, dead);
                    tmem_fence_after();
#pragma unroll
                    for (int c0 = 0; c0 < COLS; c0 += 16) {
                        if (c0 >= there) continue;
                        uint32_t raw[2][16];
                        tmem_load16(mine + buffer * 128 + c0, raw[0]);
                        tmem_load16(mine + buffer * 128 + 64 + c0, raw[1]);
                        tmem_loaded(raw[0]);
                        tmem_loaded(raw[1]);
                        if (c0 + 16 >= there) {   // (all that there are)
                            tmem_fence_before();
                            __syncwarp();
                            if (lane == 0) barrier_arrive(sums_empty + 8 * buffer);
                        }
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(sx + c0 + c);
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                uint64_t* to = acc[half] + (c0 + c) / 2;
                                to[0] = fma2(pair(raw[half][c], raw[half][c + 1]), mul2(s.x, w[half]), to[0]);
                                to[1] = fma2(pair(raw[half][c + 2], raw[half][c + 3]), mul2(s.y, w[half]), to[1]);
                            }
                        }
                    }
                    __syncwarp();
                }
                if (b % kScaleBlocks == kScaleBlocks - 1 || b + 1 == block1 - block0) {
                    if (lane == 0) barrier_arrive(scales_empty + 8 * slot);
                    if (++slot == kScaleSlots) slot = 0, scales_parity ^= 1;
                }
                parities ^= 1u << buffer;
                buffer = (buffer + 1) % kBuffers;
            }
            // The groups' sums meet in shared memory, kChunk columns at a time; then a group finishes every other column. (Loops
            // that are not unrolled: of a small call most of the time would go into fetching the code.)
            const int chan = part * 32 + lane;
            int turn = 0;
            const auto finish = [&](int column, float one, float two) {   // the two halves' sums of this thread's channels
                if (SWIGLU) one = gated(one, two);
                const int64_t row = static_cast<int64_t>(it.row) + column;
                if (a.y_dtype != EP_DTYPE_FP8_E4M3) {
                    uint16_t* to = static_cast<uint16_t*>(a.y) + row * a.y_ld;
                    const auto code = [&](float v) {
                        return a.y_dtype == EP_DTYPE_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
                    };
                    if (first < cols) to[first] = code(one);
                    if (!SWIGLU && second < cols) to[second] = code(two);
                    return;
                }
                // e4m3: the largest of 128 channels (of numbers that are not negative the bits compare as they do)
                float* const big = most + (group * 2 + turn) * 2 * kParts;
                turn ^= 1;
                const uint32_t of_one = __reduce_max_sync(kFullMask, __float_as_uint(fabsf(one)));
                const uint32_t of_two = SWIGLU ? 0u : __reduce_max_sync(kFullMask, __float_as_uint(fabsf(two)));
                if (lane == 0) big[part] = __uint_as_float(of_one), big[kParts + part] = __uint_as_float(of_two);
                asm volatile("bar.sync %0, 128;" ::"r"(2 + group) : "memory");
                for (int half = 0; half < (SWIGLU ? 1 : 2); ++half) {
                    const float* b = big + half * kParts;
                    const float s = output_scale(larger(larger(b[0], b[1]), larger(b[2], b[3])));
                    const int to = half == 0 ? first : second;   // (columns are a multiple of 128)
                    if (to >= cols) continue;
                    if (chan == 0) write_scale(row, to / kBlock, s);
                    static_cast<uint8_t*>(a.y)[row * a.y_ld + to] = code8(half == 0 ? one : two, s);
                }
            };
            float* const meet = reinterpret_cast<float*>(ring) + chan;   // [2 halves][COLS][128], of a shared item
#pragma unroll 1
            for (int k = 0; k * kChunk < there; ++k) {
#pragma unroll
                for (int c = 0; c < COLS; c += kChunk) {   // (constant places in registers)
                    if (c != k * kChunk) continue;
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int n = 0; n < kChunk; n += 2) {
                            const float2 v = apart(acc[half][(c + n) / 2]);
                            float* to = join + ((group * 2 + half) * kChunk + n) * 128 + chan;
                            to[0] = v.x, to[128] = v.y;
                        }
                }
                consumers_sync();
#pragma unroll 1
                for (int n = group; n < kChunk && k * kChunk + n < it.rows; n += kGroups) {
                    const float* from = join + n * 128 + chan;
                    float one = from[0] + from[2 * kChunk * 128], two = from[kChunk * 128] + from[3 * kChunk * 128];
                    if (*dead) one = two = __int_as_float(0x7fffffff);
                    if (split == 1) {
                        finish(k * kChunk + n, one, two);
                    } else {
                        meet[(k * kChunk + n) * 128] = one;
                        meet[(COLS + k * kChunk + n) * 128] = two;
                    }
                }
                consumers_sync();
            }
            if (!LANES && split > 1) {   // each CTA has every split-th column (the ring is used up: the cluster has one item)
                __syncwarp();
                cluster_sync();
#pragma unroll 1
                for (int column = sharer + split * group; column < it.rows; column += split * kGroups) {
                    float one[kMostSplit], two[kMostSplit], sum[2] = {0.0f, 0.0f};   // (all on their way before the first is needed)
#pragma unroll
                    for (int q = 0; q < kMostSplit; ++q) {
                        const uint32_t from = in_cta(smem_addr(meet + column * 128), min(q, split - 1));
                        one[q] = q < split ? load_cluster(from) : 0.0f;
                        two[q] = q < split ? load_cluster(from + COLS * 512) : 0.0f;
                    }
#pragma unroll
                    for (int q = 0; q < kMostSplit; ++q) sum[0] += one[q], sum[1] += two[q];
                    finish(column, sum[0], sum[1]);
                }
                __syncwarp();
                cluster_sync();
            }
        }
    } else {
        if constexpr (S::kMoved) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        // (the loader and the issuer are one thread each: the compiler knows it behind elect.sync, and waits cost it less)
        if (warp == kLoader) {
            if (leader) {
                int slot = 0;
                uint32_t parity = 1;   // (the first round of the ring waits for nothing)
                for (int64_t i = item0; i < items; i += item_step) {
                    const Tile it = tile_at(a.g, plan, table, i);
                    const int x_boxes = (max(it.rows, 1) + S::kBox - 1) / S::kBox;
                    for (int b = block0; b < block1; ++b) {
                        const uint32_t bar = full + 8 * slot, at_w = smem_addr(ring) + slot * S::kStageBytes, at_x = at_w + kWBytes;
                        barrier_wait_inline(empty + 8 * slot, parity, dead);
                        barrier_expect(bar, kWBytes + x_boxes * S::kBox * kBlock);
                        load_box(at_w, &w_map, b * kBlock, SWIGLU ? it.m * 128 : it.m * kTileRows, 0, it.expert, bar);
                        for (int j = 0; j < x_boxes; ++j)
                            load_box(at_x + j * S::kBox * kBlock, &x_map, b * kBlock, it.row + j * S::kBox, 0, 0, bar);
                        if (++slot == S::kStages) slot = 0, parity ^= 1;
                    }
                }
            }
            __syncwarp();
        } else if (warp == kIssuer) {
            if (leader) {
                const uint32_t e5m2 = a.x_dtype == EP_DTYPE_FP8_E5M2 ? 1u : 0u;
                const uint32_t base = (1u << 4) | (128u / 16 << 24);   // fp32 sums, 128 lanes
                SumsTurn turn;
                int slot = 0;
                uint32_t parity = 0;
                for (int64_t i = item0; i < items; i += item_step) {
                    const Tile it = tile_at(a.g, plan, table, i);
                    const bool lanes = LANES && it.rows > COLS;
                    const uint32_t columns = lanes ? 256 : columns_of(it.rows);
                    const uint32_t shape = base | (lanes ? e5m2 << 7 : e5m2 << 10) | columns / 8 << 17;
                    for (int b = block0; b < block1; ++b) {
                        barrier_wait_inline(full + 8 * slot, parity, dead);
                        const int buffer = turn.next(lanes, [&](int which, uint32_t phase) { barrier_wait_inline(sums_empty + 8 * which, phase, dead); });
                        tmem_fence_after();
                        const uint32_t at_w = smem_addr(ring) + slot * S::kStageBytes;
                        const uint64_t dw = operand(at_w, 1024), dx = operand(at_w + kWBytes, 1024);
                        const uint32_t sums = tmem + buffer * 128;
                        if (lanes) {
#pragma unroll
                            for (int k = 0; k < kBlock / 32; ++k) multiply_one(sums, dx + k * 2, dw + k * 2, shape, k > 0);
                        } else {
#pragma unroll
                            for (int half = 0; half < 2; ++half)
#pragma unroll
                                for (int k = 0; k < kBlock / 32; ++k)
                                    multiply_one(sums + half * 64, dw + half * (128 * kBlock / 16) + k * 2, dx + k * 2, shape, k > 0);
                        }
                        multiply_done(sums_full + 8 * buffer);
                        multiply_done(empty + 8 * slot);
                        if (++slot == S::kStages) slot = 0, parity ^= 1;
                    }
                }
            }
            __syncwarp();
        } else if (warp >= kScaler) {
            // The rows' scales for some blocks at a time, the two warps in turn, and behind them the weights' (rows as columns:
            // the first half's, the second half's one or two; rows as lanes: of 64 weight rows each). Lanes run along what is
            // dense in memory.
            int turn = warp - kScaler, slot = 0;
            uint32_t parity = 1;
            const bool by_rows = a.x_scale_block == 1;
            const int scale_rows = ceil_div(a.O, kBlock);
            constexpr int kEach = kScaleBlocks * S::kRows / 32;
            const int wk = lane / 4 % kScaleBlocks, wj = lane % 4;   // the first lanes load the weights' scales: block, which one
            const auto row_of = [&](int j) { return by_rows ? j * (32 / kScaleBlocks) + lane / kScaleBlocks : j * 32 % S::kRows + lane; };
            const auto block_of = [&](int j) { return by_rows ? lane % kScaleBlocks : j * 32 / S::kRows; };
            for (int64_t i = item0; i < items; i += item_step) {
                const Tile it = tile_at(a.g, plan, table, i);
                const bool lanes = LANES && it.rows > COLS;
                const int o = lanes ? weight_row(it.m, wj / 2) + wj % 2 * 64 : wj == 0 ? weight_row(it.m, 0) : weight_row(it.m, 1) + (wj - 1) * 128;
                const float* w_scales = a.w_scales + (static_cast<int64_t>(it.expert) * scale_rows + min(o / kBlock, scale_rows - 1)) * blocks;
                for (int b = block0; b < block1; b += kScaleBlocks) {
                    if (turn == 0) {
                        float v[kEach];
#pragma unroll
                        for (int j = 0; j < kEach; ++j) {
                            const int n = row_of(j), k = block_of(j);
                            v[j] = 0.0f;
                            if (n < it.rows && b + k < block1) {
                                const int64_t from = (static_cast<int64_t>(it.row) + n) * a.x_scale_row + (b + k) * a.x_scale_block;
                                v[j] = a.x_ue8m0 ? ue8m0(static_cast<const uint8_t*>(a.x_scales)[from]) : static_cast<const float*>(a.x_scales)[from];
                            }
                        }
                        const float w = w_scales[min(b + wk, blocks - 1)];
                        barrier_wait_inline(scales_empty + 8 * slot, parity, dead);
                        float* to = scales + slot * (kScaleBlocks * S::kScaleStep);
                        if (lane < 4 * kScaleBlocks) to[wk * S::kScaleStep + S::kRows + wj] = w;
#pragma unroll
                        for (int j = 0; j < kEach; ++j) to[block_of(j) * S::kScaleStep + row_of(j)] = v[j];
                        __syncwarp();
                        if (lane == 0) barrier_arrive(scales_full + 8 * slot);
                    }
                    turn ^= 1;
                    if (++slot == kScaleSlots) slot = 0, parity ^= 1;
                }
            }
        }
    }
    if (warp >= kLoader && split > 1 && item0 < items) {   // (as the consumers do)
        __syncwarp();
        cluster_sync();
        cluster_sync();
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == kLoader) {
        tmem_fence_after();
        tmem_free_one(tmem);
    }
}

template <int COLS, bool LANES, bool SWIGLU>
cudaError_t launch_shape(const Fp8Args& a, cudaStream_t stream) {
    using S = Shape<COLS, LANES>;
    static ClusterRoom known[64];
    static int ready[64];
    ClusterRoom room{};
    cudaError_t err = cluster_room(expert_fp8_kernel<COLS, LANES, SWIGLU>, kThreads, S::kShared, known, ready, &room);
    if (err != cudaSuccess) return err;
    const int64_t I = a.I, O = a.O, E = a.g.E;
    const int cols = SWIGLU ? a.O / 2 : a.O;
    TilePlan p{};
    p.cap = S::kRows;
    while (1 << p.cap_shift < p.cap) ++p.cap_shift;
    p.whole = LANES;
    p.chunk = 16;   // (of no weight: 1, 16 and 64 within 1 % on prompts)
    p.m_tiles = ceil_div(cols, SWIGLU ? kTileRows / 2 : kTileRows);
    while (((a.g.E - 1) >> p.shift) + 1 > kTileTable) ++p.shift;
    CUtensorMap w_map, x_map;
    err = SWIGLU ? box_map(&w_map, a.w, EP_DTYPE_FP8_E4M3, I, cols, 2, E, I, I * cols, I * O, 128, 2)
                 : box_map(&w_map, a.w, EP_DTYPE_FP8_E4M3, I, O, 1, E, I, I * O, I * O, kTileRows, 1);
    if (err == cudaSuccess) err = box_map(&x_map, a.x, EP_DTYPE_FP8_E4M3, I, a.g.rows, 1, 1, a.x_ld, a.x_ld, a.x_ld, S::kBox, 1);
    if (err != cudaSuccess) return err;
    const int64_t most = most_tiles(a.g, p.cap) * p.m_tiles;
    // Few items are shared by the CTAs of clusters, each with some of the blocks, whose sums meet in shared memory: where all
    // items are on the device at once with that many CTAs each (4096 x 4096, one row: 16.5 to 8.5 us; 64 rows 19.6 to 12.1).
    int split = 1;
    for (int i = 1; !LANES && split < kMostSplit && 2 * split <= a.I / kBlock && most <= room.clusters[i]; ++i) split *= 2;
    p.flip = room.clusters[0];
    const int64_t clusters = most < room.clusters[0] / split ? most : room.clusters[0] / split;
    return launch_clusters(expert_fp8_kernel<COLS, LANES, SWIGLU>, static_cast<int>(clusters), split, kThreads, S::kShared, stream, a, p, split,
                           w_map, x_map);
}

template <bool SWIGLU>
cudaError_t launch_activation(const Fp8Args& a, cudaStream_t stream) {
    const int used = a.g.rows < a.g.E ? a.g.rows : a.g.E, mean = (a.g.rows - 1) / used + 1;
    // Tiles of 32, 64 or (rows as lanes) 128 rows, the smallest that hold most experts' rows in one tile. 32 experts of 4096 x 2048 with
    // the activation, us at mean rows
    //   24: 52.0 (32), 54.6 (64), 56.1 (128)   32: 61.0, 58.3, 60.5   48: 72.8, 64.5, 67.5   64: 88.5, 83.0, 69.2   112: 121, 111, 63
    // Shorter ones where at most half of the SMs, or a third, would have work (4096 x 4096: 64 rows 31.2 us as 128, 12.1 as 32; 256 rows
    // 29.2 as 128, 24.4 as 64, 20.7 as 32; 512 rows 29.7, 30.8, 36.7).
    const int cols = SWIGLU ? a.O / 2 : a.O, m_tiles = ceil_div(cols, SWIGLU ? kTileRows / 2 : kTileRows);
    const auto few = [&](int cap, int times) { return times * most_tiles(a.g, cap) * m_tiles <= sm_count(); };
    if (mean <= 24 || few(64, 2)) return launch_shape<32, false, SWIGLU>(a, stream);
    // (rows as lanes need one scale for 64 neighbouring up rows)
    if (mean <= 48 || few(128, 3) || (SWIGLU && a.O / 2 % 64 != 0)) return launch_shape<64, false, SWIGLU>(a, stream);
    return launch_shape<64, true, SWIGLU>(a, stream);
}

}  // namespace

cudaError_t launch_expert_fp8(const Fp8Args& a, cudaStream_t stream) {
    return a.swiglu ? launch_activation<true>(a, stream) : launch_activation<false>(a, stream);
}

}  // namespace ep
