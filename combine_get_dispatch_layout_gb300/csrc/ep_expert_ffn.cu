// The experts' gated feed-forward block in 16 bits and its gradients: grouped
// products on the 5th-generation tensor cores, fp32 sums in TMEM.
//
// Mathematics, for an expert's rows (x [n, H], W1 [2F, H] gate above up, W2 [H, F]):
//   gate_up = x W1^T,  act = silu(gate) * up,  y = act W2^T
//   dact = dy W2,  dgate = dact up s (1 + gate (1 - s)),  dup = dact gate s,  s = 1 / (1 + exp(-gate))
//   dx = [dgate dup] W1,  dW1 = [dgate dup]^T x,  dW2 = dy^T act
// Each is one product D [lanes][columns] of a tile: the lanes are the output's channels (the dimension that is contiguous
// in it; of the weights' gradients its rows), the columns its rows, so that few rows cost few columns. Operands come as
// they lie in memory, contraction inward (K-major) or outward (MN-major): no transposed copies.
//
// Roundings. act and grad_gate_up are rounded to the tensors' type because they are operands of the next product, whose
// tensor core takes 16-bit operands, and outputs of the call; all sums, gate, up and the sigmoid are fp32 until then.
//
// Kernel. A pair of CTAs on two SMs multiplies as one: 256 lanes, up to 256 columns, of which each CTA loads half, so that
// an SM reads 32 KB for 4.2 M products (alone with a tile of 128 x 256 it would be 48 KB: training step 3.85 ms, with pairs 3.5).
// Persistent: a loader thread fills a ring by TMA, an issuer thread multiplies, eight warps empty one of two buffers of
// sums in TMEM while the other fills. Rows go out through shared memory in 16-byte pieces (2-byte stores of a channel a
// thread: training step 3.43 ms, through shared memory 3.26).
// Two launches forward; backward two of two products each that do not depend on one another, so that the second fills what
// the first leaves idle (small block's gradients 46 to 37 us against four launches).
//
// What bounds it (one GB300). 16384 tokens of top 6 of 64 experts, 4096 x 2048: 3.2 to 3.4 ms by the card, 1470 to 1540 TFLOP/s, gradients 6.9 to
// 7.1 ms, 1390 to 1440 TFLOP/s (of one dense 8192-row block 1820 to 1900): the power limit, at which a plain library product holds 1731, and the
// partly filled last tiles. 16 tokens of top 6 of 64 experts, 4096 x 2048: 350 to 375 us, 6.8 to 7.3 TB/s of weights: memory. 2048 tokens
// of top 4 of 60 uneven experts, 2056 x 1368: 203 to 226 us, 5.1 to 5.6 TB/s; its gradients 518 to 549: tiles of 137 rows on average use half
// the columns of a stage, so the bytes that come into the SMs count (9.9 TB/s of at most 12.6), and of the weights'
// gradients, with two or three stages an item, the epilogue. One row of 64 x 64: 8.5 us for two launches, the latency of
// start, tables, first load, product and store.
#include "ep_expert_tiles.cuh"

namespace ep {
namespace {

constexpr int kEpilogueWarps = 8;
constexpr int kLoader = kEpilogueWarps, kIssuer = kLoader + 1, kCleaner = kLoader + 2;   // warps
constexpr int kCleaners = 3;                    // each has its slots of the ring
constexpr int kThreads = 32 * (kEpilogueWarps + 2 + kCleaners);
constexpr int kLanes = 256;                     // of a pair: 128 in each CTA's TMEM
constexpr int kStep = 64;                       // contraction of a stage: 128 bytes
constexpr int kABytes = kLanes / 2 * kStep * 2;
constexpr int kMostStages = 6;                  // of 32 KB; those of two parts are larger
constexpr int kRing = 192 * 1024;
// Outputs leave through shared memory: chunks of kChunk rows of 128 channels (gate and up of 64), of which two fit for each
// half of the epilogue's warps, and for the activation rows of 64 channels, apart so that two rows lie in other banks.
constexpr int kChunk = 16;
constexpr int kRowBytes = 256, kActBytes = 160;
constexpr int kOutBytes = 2 * kChunk * kRowBytes, kHalfBytes = kOutBytes + 2 * kChunk * kActBytes;
constexpr int kShared = 1024 + kRing + 2 * kHalfBytes + 512 + static_cast<int>(sizeof(Tables));
static_assert(kShared <= 227 * 1024 - 256, "");

enum Product { kNone = -1, kGateUp, kDown, kGradAct, kGradX, kGradW };
template <int WHAT>
struct Kind {
    static constexpr int value = WHAT;
};

struct Gemm {
    ExpertRows g;
    TilePlan plan;
    int lanes;           // channels of the output
    int inner;           // contraction (of kGradW: the expert's rows instead)
    int columns;         // kGradW: length of the output's rows, which are the lanes
    int n_tiles;         // kGradW: tiles of them
    int atoms;           // kStep deep parts of a stage (kGradW: 1)
    int stages, stage_bytes, atom_bytes, box;   // box: rows of a box of operand B (kGradW: of both)
    void* out;
    void* out2;          // kGateUp: gate and up, or NULL
    const void* in;      // kGradAct: gate and up
    int64_t out_ld, out2_ld, in_ld;
    int out_fp32, accumulate;       // kGradW
    int follows;         // the kernel before is one of the same call
};

// An item: `cols` columns (rows of the output; of kGradW places in its rows) from `col` on, lanes from m * kLanes on,
// `steps` stages; of kGradW the contraction is over rows [row, row + rows).
struct Item {
    int expert, m, col, cols, row, rows, steps;
};

template <int WHAT>
__device__ __forceinline__ int64_t items_of(const Gemm& a, const Tables* table) {
    if constexpr (WHAT == kGradW) return static_cast<int64_t>(a.g.E) * a.plan.m_tiles * a.n_tiles;
    else return a.plan.m_tiles > 0 ? tile_count(a.g, a.plan, table) : 0;
}

template <int WHAT>
__device__ __forceinline__ Item item_at(const Gemm& a, const Tables* table, int64_t it, int64_t items) {
    Item r;
    if constexpr (WHAT == kGradW) {
        const int64_t per = static_cast<int64_t>(a.plan.m_tiles) * a.n_tiles;
        r.expert = items < INT32_MAX ? static_cast<int>(it) / static_cast<int>(per) : static_cast<int>(it / per);
        const int64_t in = it - r.expert * per;
        r.m = items < INT32_MAX ? static_cast<int>(in) / a.n_tiles : static_cast<int>(in / a.n_tiles);
        r.col = static_cast<int>(in - static_cast<int64_t>(r.m) * a.n_tiles) * a.plan.cap;
        r.cols = min(a.plan.cap, a.columns - r.col);
        r.rows = rows_of(a.g, table, r.expert, r.row);
        r.steps = (r.rows + kStep - 1) / kStep;
    } else {
        const Tile t = tile_at(a.g, a.plan, table, it);
        r.expert = t.expert;
        r.m = t.m;
        r.col = r.row = t.row;
        r.cols = r.rows = t.rows;
        r.steps = (a.inner + kStep * a.atoms - 1) / (kStep * a.atoms);
    }
    return r;
}

// kGradW: whether a stage has rows of others among the 16 of a product behind the expert's last, and zeros are wanted there.
template <int WHAT>
__device__ __forceinline__ bool unclean(const Item& it, int s) {
    return WHAT == kGradW && it.rows - s * kStep < kStep && it.rows % 16 != 0;
}

// One product, or two that do not depend on each other, the second's items after the first's (kNone: no second).
template <typename T, int FIRST, int SECOND>
__global__ void __launch_bounds__(kThreads, 1)
    expert_gemm_kernel(const __grid_constant__ Gemm first, const __grid_constant__ Gemm second, const __grid_constant__ CUtensorMap first_a_map,
                       const __grid_constant__ CUtensorMap first_b_map, const __grid_constant__ CUtensorMap second_a_map,
                       const __grid_constant__ CUtensorMap second_b_map) {
    extern __shared__ unsigned char shared_bytes[];
    unsigned char* const ring = shared_bytes + (1024 - smem_addr(shared_bytes) % 1024) % 1024;
    uint64_t* const barriers = reinterpret_cast<uint64_t*>(ring + kRing + 2 * kHalfBytes);
    const uint32_t full = smem_addr(barriers), empty = full + 8 * kMostStages;
    // kGradW, an expert's last rows: a CTA's half is there, both are clean
    const uint32_t part_full = empty + 8 * kMostStages, clean = part_full + 8 * kMostStages;
    const uint32_t sums_full = clean + 8 * kMostStages, sums_empty = sums_full + 16;
    uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(barriers) + 120;
    volatile int* const dead = reinterpret_cast<volatile int*>(tmem_at + 1);
    Tables* const table = reinterpret_cast<Tables*>(barriers + 64);
    static_assert((4 * kMostStages + 4) * 2 <= 120, "");
    __shared__ int warp_sum[kThreads / 32];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = cluster_rank();
    if (warp == kCleaner && elected()) {   // (a product without an output has no maps)
        if (first.out) {
            prefetch_map(&first_a_map);
            prefetch_map(&first_b_map);
        }
        if (SECOND != kNone && second.out) {
            prefetch_map(&second_a_map);
            prefetch_map(&second_b_map);
        }
    }
    if (warp == kLoader) {
        tmem_alloc_all(smem_addr(tmem_at));
        if (lane == 0) {
            *dead = 0;
            for (int i = 0; i < first.stages; ++i) {
                barrier_init(full + 8 * i, 1);
                barrier_init(empty + 8 * i, 1);
                barrier_init(part_full + 8 * i, 1);
                barrier_init(clean + 8 * i, 2);
            }
            for (int i = 0; i < 2; ++i) {
                barrier_init(sums_full + 8 * i, 1);
                barrier_init(sums_empty + 8 * i, 2 * kEpilogueWarps);
            }
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    }
    // Behind a kernel of the same call, which lets this one start only after its own wait, all that came before the call is
    // complete, so the tables need not wait for that kernel (a block of one token 11.9 to 10.6 us; the first weights as well: no
    // further gain).
    const bool follows = (FIRST == kDown || FIRST == kGradX) && first.follows;
    if (!follows) dependent_entry();
    fill_tables<kThreads>(first.g, first.plan, table, warp_sum);
    tmem_fence_before();
    __syncthreads();
    cluster_sync();   // (both CTAs' barriers are ready)
    if (follows) dependent_entry();
    tmem_fence_after();
    const uint32_t tmem = __shfl_sync(kFullMask, *tmem_at, 0);
    const bool leader = elected();

    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;

    // A role over all items of this pair; what it keeps (places in rings, parities) goes on from the first product to the second.
    const auto walk = [&](auto role) {
        const int64_t n = items_of<FIRST>(first, table);
        role(Kind<FIRST>{}, first, first_a_map, first_b_map, static_cast<int64_t>(pair), n);
        if constexpr (SECOND != kNone) {
            const int64_t start = (pair - n % pairs + pairs) % pairs;   // (the turn of the pairs goes on)
            role(Kind<SECOND>{}, second, second_a_map, second_b_map, start, items_of<SECOND>(second, table));
        }
    };

    // (the loader and the issuer are one thread each: the compiler knows it behind elect.sync, and waits cost it less)
    if (warp == kLoader) {
        if (leader) {
            int slot = 0;
            uint32_t parity = 1;   // (the first round of the ring waits for nothing)
            walk([&](auto kind, const Gemm& a, const CUtensorMap& a_map, const CUtensorMap& b_map, int64_t start, int64_t items) {
                constexpr int WHAT = decltype(kind)::value;
                for (int64_t i = start; i < items; i += pairs) {
                    const Item it = item_at<WHAT>(a, table, i, items);
                    const int half = columns_of(it.cols) / 2;   // columns of each CTA
                    const int b_boxes = WHAT == kGradW ? (half + 63) / 64 : (half + a.box - 1) / a.box;
                    const int lane0 = it.m * kLanes + rank * (kLanes / 2), col0 = it.col + rank * half;
                    for (int s = 0; s < it.steps; ++s) {
                        // both CTAs' boxes count on the first one's barrier
                        const uint32_t mine = full + 8 * slot, at_a = smem_addr(ring) + slot * a.stage_bytes, at_b = at_a + kABytes;
                        const uint32_t bar = in_first(mine);
                        barrier_wait_inline(empty + 8 * slot, parity, dead);
                        if constexpr (WHAT == kGradW) {
                            // [64 channels] x [box rows] of both operands, boxes with real rows only
                            // (a stage that has to be cleaned first counts on a barrier of each CTA's own)
                            const bool own = unclean<WHAT>(it, s);
                            const uint32_t to = own ? part_full + 8 * slot : bar;
                            const int down = (min(kStep, it.rows - s * kStep) + a.box - 1) / a.box, all = (2 + b_boxes) * down;
                            if (rank == 0 || own) barrier_expect(own ? to : mine, all * a.box * 128 * (own ? 1 : 2));
                            for (int k = 0; k < down; ++k) {
                                const int row = it.row + s * kStep + k * a.box, at = k * a.box * 128;
                                for (int j = 0; j < 2; ++j) load_box_pair(at_a + j * 8192 + at, &a_map, lane0 + j * 64, row, 0, 0, to);
                                for (int j = 0; j < b_boxes; ++j) load_box_pair(at_b + j * 8192 + at, &b_map, col0 + j * 64, row, 0, 0, to);
                            }
                        } else {
                            if (rank == 0) barrier_expect(mine, 2 * a.atoms * (kABytes + b_boxes * a.box * 128));
                            for (int part = 0; part < a.atoms; ++part) {   // (zeros behind the contraction's end)
                                const int k = (s * a.atoms + part) * kStep;
                                const uint32_t to_a = at_a + part * a.atom_bytes, to_b = to_a + kABytes;
                                if constexpr (WHAT == kGateUp) {   // the 16 gate and the 16 up rows of each warp
                                    for (int j = 0; j < 4; ++j) load_box_pair(to_a + j * 4096, &a_map, k, lane0 / 2 + j * 16, 0, it.expert, bar);
                                } else if constexpr (WHAT == kDown) {
                                    load_box_pair(to_a, &a_map, k, lane0, 0, it.expert, bar);
                                } else {
                                    for (int j = 0; j < 2; ++j) load_box_pair(to_a + j * 8192, &a_map, lane0 + j * 64, k, 0, it.expert, bar);
                                }
                                for (int j = 0; j < b_boxes; ++j) load_box_pair(to_b + j * a.box * 128, &b_map, k, col0 + j * a.box, 0, 0, bar);
                            }
                        }
                        if (++slot == a.stages) slot = 0, parity ^= 1;
                    }
                }
            });
        }
        __syncwarp();
    } else if (warp == kIssuer) {
        if (leader && rank == 0) {   // (it issues for both CTAs)
            int slot = 0, buffer = 0;
            uint32_t parities = 0, sums_parity = 1, clean_parity = 0;   // parities, clean_parity: a bit for each slot
            walk([&](auto kind, const Gemm& a, const CUtensorMap&, const CUtensorMap&, int64_t start, int64_t items) {
                constexpr int WHAT = decltype(kind)::value;
                // fp32 sums; operands' type; A outward, B outward; 256 lanes
                constexpr uint32_t kType = std::is_same_v<T, __nv_bfloat16> ? 1u : 0u;
                constexpr bool kAOut = WHAT >= kGradAct, kBOut = WHAT == kGradW;
                constexpr uint32_t kShape = (1u << 4) | (kType << 7) | (kType << 10) | (kAOut ? 1u << 15 : 0u) | (kBOut ? 1u << 16 : 0u) |
                                                  (static_cast<uint32_t>(kLanes / 16) << 24);
                for (int64_t i = start; i < items; i += pairs) {
                    const Item it = item_at<WHAT>(a, table, i, items);
                    if (it.steps == 0) continue;
                    const uint32_t shape = kShape | static_cast<uint32_t>(columns_of(it.cols) / 8) << 17;
                    const uint32_t sums = tmem + buffer * 256;
                    barrier_wait_inline(sums_empty + 8 * buffer, sums_parity, dead);
                    for (int s = 0; s < it.steps; ++s) {
                        const uint32_t at_a = smem_addr(ring) + slot * a.stage_bytes, at_b = at_a + kABytes;
                        const uint64_t da = kAOut ? operand_outward(at_a, 8192) : operand(at_a, 1024);
                        const uint64_t db = kBOut ? operand_outward(at_b, 8192) : operand(at_b, 1024);
                        if (unclean<WHAT>(it, s)) {
                            barrier_wait_cluster(clean + 8 * slot, (clean_parity >> slot) & 1, dead);
                            clean_parity ^= 1u << slot;
                        } else {
                            barrier_wait_inline(full + 8 * slot, (parities >> slot) & 1, dead);
                            parities ^= 1u << slot;
                        }
                        tmem_fence_after();
                        const int depth = WHAT == kGradW ? min((it.rows - s * kStep + 15) / 16, kStep / 16) : kStep / 16;   // products of 16
                        if (WHAT != kGradW || depth == kStep / 16) {
                            for (int part = 0; part < (WHAT == kGradW ? 1 : a.atoms); ++part) {
                                const uint64_t on = part * (a.atom_bytes / 16);
#pragma unroll
                                for (int k = 0; k < kStep / 16; ++k)
                                    multiply_pair(sums, da + on + k * (kAOut ? 128 : 2), db + on + k * (kBOut ? 128 : 2), shape,
                                                  s > 0 || part > 0 || k > 0);
                            }
                        } else {
                            for (int k = 0; k < depth; ++k) multiply_pair(sums, da + k * 128, db + k * 128, shape, s > 0 || k > 0);
                        }
                        pair_done(empty + 8 * slot);
                        if (s + 1 == it.steps) pair_done(sums_full + 8 * buffer);
                        if (++slot == a.stages) slot = 0;
                    }
                    buffer ^= 1;
                    if (buffer == 0) sums_parity ^= 1;
                }
            });
        }
        __syncwarp();
    } else if (warp >= kCleaner) {
        // Rows behind an expert's last belong to others, NaN perhaps: zeros instead, in both operands, some stages before their
        // product. Each warp has its slots of the ring (a barrier's phase must not pass it by), next to one another, so that
        // stages that come every second or third slot are spread: the release of its arrival takes a warp 2000 clocks (60 experts
        // of 136 rows, 2056 x 1368, all gradients: one warp 572 us, slots in turn 600, these 520).
        if constexpr (FIRST == kGradW || SECOND == kGradW) {
            int slot = 0;
            uint32_t parities = 0;   // a bit for each slot
            walk([&](auto kind, const Gemm& a, const CUtensorMap&, const CUtensorMap&, int64_t start, int64_t items) {
                constexpr int WHAT = decltype(kind)::value;
                for (int64_t i = start; i < items; i += pairs) {
                    const Item it = item_at<WHAT>(a, table, i, items);
                    if constexpr (WHAT != kGradW) {
                        slot = (slot + it.steps) % a.stages;
                    } else {
                        for (int s = 0; s < it.steps; ++s) {
                            if (unclean<WHAT>(it, s) && slot * kCleaners / a.stages == warp - kCleaner) {
                                barrier_wait_inline(part_full + 8 * slot, (parities >> slot) & 1, dead);
                                parities ^= 1u << slot;
                                const int left = it.rows - s * kStep, end = (left + 15) / 16 * 16, lines = 2 + (columns_of(it.cols) / 2 + 63) / 64;
                                for (int j = lane; j < (end - left) * lines * 8; j += 32) {
                                    const int line = j / 8, row = left + line / lines;
                                    *reinterpret_cast<uint4*>(ring + slot * a.stage_bytes + line % lines * 8192 + row * 128 + j % 8 * 16) =
                                        make_uint4(0, 0, 0, 0);
                                }
                                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                                __syncwarp();
                                if (lane == 0) barrier_arrive_cluster(in_first(clean + 8 * slot));
                            }
                            if (++slot == a.stages) slot = 0;
                        }
                    }
                }
            });
        }
    } else {   // (the first kEpilogueWarps)
        const int half = warp >> 2, part = warp & 3;   // of the chunks of columns; of the lanes
        unsigned char* const out = ring + kRing + half * kHalfBytes;
        unsigned char* const act_out = out + kOutBytes;
        const auto half_sync = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory"); };
        int buffer = 0, chunk = 0;
        uint32_t parity = 0;
        const auto release = [&] {   // the buffer of sums
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) barrier_arrive_pair(in_first(sums_empty + 8 * buffer));
            buffer ^= 1;
            if (buffer == 0) parity ^= 1;
        };
        // Weight gradients: written once, summed over the expert's rows in one item, in order, so that the same inputs give the
        // same bits. (Two pairs on one item of many rows would have to join in memory; there are E m_tiles n_tiles items.)
        // A thread has a row of the output and 32 neighbouring places of it at a time. They leave through the
        // warp's own part of the shared memory, 64 bytes of its 32 rows at a time, so that four lanes write 64 bytes of one; the
        // 16-byte pieces are swapped by row against bank conflicts.
        const auto weight_gradients = [&](const Gemm& a, const Item& it, uint32_t mine, int tile) {
            constexpr int kWide = 32;
            static_assert(32 * 64 <= kHalfBytes / 4 && kHalfBytes % 64 == 0, "");
            if (it.steps == 0) {   // no rows: zeros, a row a warp's store
                const int bytes = it.cols * (a.out_fp32 ? 4 : 2), some = min(a.lanes - tile - part * 32, 32);
                if (a.accumulate) return;
                for (int row = half; row < some; row += 2) {
                    const int64_t at = (static_cast<int64_t>(it.expert) * a.lanes + tile + part * 32 + row) * a.columns + it.col;
                    char* const to = static_cast<char*>(a.out) + at * (a.out_fp32 ? 4 : 2);
                    for (int b = lane * 16; b < bytes; b += 512) *reinterpret_cast<uint4*>(to + b) = make_uint4(0, 0, 0, 0);
                }
                return;
            }
            barrier_wait(sums_full + 8 * buffer, parity, dead);
            tmem_fence_after();
            unsigned char* const own = out + part * (kHalfBytes / 4);
            const int64_t first = static_cast<int64_t>(it.expert) * a.lanes + tile + part * 32;   // the warp's first row
            const int rows = a.lanes - tile - part * 32, size = a.out_fp32 ? 4 : 2;
            const int64_t pitch = static_cast<int64_t>(a.columns) * size;
            // this thread's pieces are of rows lane / 4 and every eighth after that
            char* const to = static_cast<char*>(a.out) + (first + lane / 4) * pitch + lane % 4 * 16;
            // the pieces of the place from `at` bytes on, of which `bytes` are real
            const auto leave = [&](const uint4 (&piece)[4], int64_t at, int bytes, bool add) {
#pragma unroll
                for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(own + lane * 64 + (q ^ (lane >> 1 & 3)) * 16) = piece[q];
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int row = k * 8 + lane / 4;
                    if (row >= rows || lane % 4 * 16 >= bytes) continue;
                    uint4 v = *reinterpret_cast<const uint4*>(own + row * 64 + (lane % 4 ^ (row >> 1 & 3)) * 16);
                    uint4* const place = reinterpret_cast<uint4*>(to + 8 * k * pitch + at);
                    if (add) {
                        const float4 old = *reinterpret_cast<const float4*>(place);
                        v = make_uint4(__float_as_uint(old.x + __uint_as_float(v.x)), __float_as_uint(old.y + __uint_as_float(v.y)),
                                       __float_as_uint(old.z + __uint_as_float(v.z)), __float_as_uint(old.w + __uint_as_float(v.w)));
                    }
                    *place = v;
                }
                __syncwarp();
            };
            for (int c0 = half * kWide; c0 < it.cols; c0 += 2 * kWide) {
                uint32_t raw[kWide];
                tmem_load32(mine + c0, raw);
                tmem_loaded(raw);
                if (*dead) {
#pragma unroll
                    for (int j = 0; j < kWide; ++j) raw[j] = 0x7fffffff;
                }
                const int many = min(kWide, it.cols - c0);   // (a multiple of 8)
                const int64_t at = static_cast<int64_t>(it.col + c0) * size;
                uint4 piece[4];
                if (a.out_fp32) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            piece[q] = make_uint4(raw[16 * h + 4 * q], raw[16 * h + 4 * q + 1], raw[16 * h + 4 * q + 2], raw[16 * h + 4 * q + 3]);
                        leave(piece, at + h * 64, many * 4 - h * 64, a.accumulate);
                    }
                    continue;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    Vec8<T> v;
                    if (a.accumulate && lane < rows && 8 * q < many) {
                        Vec8<T> old;
                        old.raw = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.out) + (first + lane) * pitch + at + 16 * q);
#pragma unroll
                        for (int j = 0; j < 8; ++j) raw[8 * q + j] = __float_as_uint(to_float(old.v[j]) + __uint_as_float(raw[8 * q + j]));
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) v.v[j] = from_float<T>(__uint_as_float(raw[8 * q + j]));
                    piece[q] = v.raw;
                }
                leave(piece, at, many * 2, false);
            }
        };
        walk([&](auto kind, const Gemm& a, const CUtensorMap&, const CUtensorMap&, int64_t start, int64_t items) {
            constexpr int WHAT = decltype(kind)::value;
            if constexpr (WHAT == kGradW) half_sync();   // (the product before may still be read from where rows go)
            // kGradAct: this thread's pieces of gate's and up's rows of a chunk of columns
            uint4 ahead[4] = {};
            const auto fetch = [&](const Item& it, int c0, int chan0, int bytes) {
                const int piece_at = tid % 16 * 16;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = (tid & 127) / 16 + k % 2 * 8;
                    const T* row = static_cast<const T*>(a.in) + (static_cast<int64_t>(it.row) + c0 + j) * a.in_ld + chan0 + (k < 2 ? 0 : a.lanes);
                    if (c0 + j < it.cols && piece_at < bytes)
                        ahead[k] = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(row) + piece_at);
                }
            };
            for (int64_t i = start; i < items; i += pairs) {
                const Item it = item_at<WHAT>(a, table, i, items);
                const uint32_t mine = tmem + buffer * 256 + (static_cast<uint32_t>(part) << 21);   // lane 32 * part, upper half
                // the CTA's first channel (of gate and up a warp's lanes are 16 gate and 16 up rows)
                const int tile = it.m * kLanes + rank * (kLanes / 2), chan0 = WHAT == kGateUp ? tile / 2 : tile;
                const int bytes = min(WHAT == kGateUp ? 64 : 128, a.lanes - chan0) * 2;   // of a row of this CTA (a multiple of 16)
                if (WHAT == kGradAct && half * kChunk < it.cols) fetch(it, half * kChunk, chan0, bytes);
                if constexpr (WHAT == kGradW) {
                    weight_gradients(a, it, mine, tile);
                    if (it.steps > 0) release();
                    continue;
                }
                barrier_wait(sums_full + 8 * buffer, parity, dead);
                tmem_fence_after();
                for (int c0 = half * kChunk; c0 < it.cols; c0 += 2 * kChunk, ++chunk) {
                    uint32_t raw[kChunk];
                    tmem_load16(mine + c0, raw);
                    tmem_loaded(raw);
                    if (*dead) {
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) raw[j] = 0x7fffffff;
                    }
                    const int many = min(kChunk, it.cols - c0);
                    const int64_t row0 = static_cast<int64_t>(it.row) + c0;
                    const int place = WHAT == kGradAct ? 0 : chunk & 1;   // (kGradAct has both places: gate and up, or their gradients)
                    unsigned char* const to = out + place * (kChunk * kRowBytes);
                    unsigned char* const act_to = act_out + place * (kChunk * kActBytes);
                    // 16-byte pieces of the rows: this thread's are of rows `piece / 16` and that plus 8
                    const int piece_row = (tid & 127) / 16, piece_at = tid % 16 * 16;
                    if constexpr (WHAT == kGateUp) {
                        if (a.out2) {
                            T* at = reinterpret_cast<T*>(to + (lane < 16 ? 0 : 128)) + part * 16 + (lane & 15);
#pragma unroll
                            for (int j = 0; j < kChunk; ++j) at[j * (kRowBytes / 2)] = from_float<T>(__uint_as_float(raw[j]));
                        }
                        T* at = reinterpret_cast<T*>(act_to + (lane >> 4) * kActBytes) + part * 16 + (lane & 15);
#pragma unroll
                        for (int j = 0; j < kChunk; j += 2) {   // gate lanes take the even columns, up lanes the odd ones
                            const float own = __uint_as_float(lane < 16 ? raw[j] : raw[j + 1]);
                            const float got = __uint_as_float(__shfl_xor_sync(kFullMask, lane < 16 ? raw[j + 1] : raw[j], 16));
                            const float gate = lane < 16 ? own : got, up = lane < 16 ? got : own;
                            at[j * (kActBytes / 2)] = from_float<T>(gated(gate, up));
                        }
                        half_sync();
                        const int row = (tid & 127) / 8, byte = tid % 8 * 16;
                        if (row < many && byte < bytes)
                            *reinterpret_cast<uint4*>(reinterpret_cast<char*>(static_cast<T*>(a.out) + (row0 + row) * a.out_ld + chan0) + byte) =
                                *reinterpret_cast<const uint4*>(act_to + row * kActBytes + byte);
                        if (a.out2) {
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int j = piece_row + 8 * k, at_byte = piece_at & 127;
                                T* both = static_cast<T*>(a.out2) + (row0 + j) * a.out2_ld + chan0 + (piece_at < 128 ? 0 : a.lanes);
                                if (j < many && at_byte < bytes)
                                    *reinterpret_cast<uint4*>(reinterpret_cast<char*>(both) + at_byte) =
                                        *reinterpret_cast<const uint4*>(to + j * kRowBytes + piece_at);
                            }
                        }
                    } else {
                        T* at = reinterpret_cast<T*>(to) + part * 32 + lane;
                        if constexpr (WHAT == kGradAct) {
                            // gate and up come as the gradients leave, a chunk ahead
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                *reinterpret_cast<uint4*>(to + (k / 2 * kChunk + piece_row + k % 2 * 8) * kRowBytes + piece_at) = ahead[k];
                            half_sync();
                            if (c0 + 2 * kChunk < it.cols) fetch(it, c0 + 2 * kChunk, chan0, bytes);
#pragma unroll
                            for (int j = 0; j < kChunk; ++j) {
                                const float d = __uint_as_float(raw[j]);
                                T &g = at[j * (kRowBytes / 2)], &u = at[(kChunk + j) * (kRowBytes / 2)];
                                const float gate = to_float(g), up = to_float(u);
                                // (the sigmoid first: what it is multiplied with may pass fp32's range before it, and where it is 0 give
                                // NaN; its small factor in two parts, which loses bits only where the slope times up is below 2^-188)
                                const Sigmoid s = sigmoid_of(gate);
                                const float f = s.far ? 0x1p-62f : 1.0f, not_s = s.far ? 1.0f : 1.0f - s.r;
                                g = from_float<T>(s.r * (1.0f + gate * not_s) * (up * f) * (d * f));
                                u = from_float<T>(gate * s.r * (d * f * f));
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < kChunk; ++j) at[j * (kRowBytes / 2)] = from_float<T>(__uint_as_float(raw[j]));
                        }
                        half_sync();
#pragma unroll
                        for (int k = 0; k < (WHAT == kGradAct ? 4 : 2); ++k) {
                            const int j = piece_row + k % 2 * 8;
                            T* row = static_cast<T*>(a.out) + (row0 + j) * a.out_ld + chan0 + (k < 2 ? 0 : a.lanes);
                            if (j < many && piece_at < bytes)
                                *reinterpret_cast<uint4*>(reinterpret_cast<char*>(row) + piece_at) =
                                    *reinterpret_cast<const uint4*>(to + (k / 2 * kChunk + j) * kRowBytes + piece_at);
                        }
                        if constexpr (WHAT == kGradAct) half_sync();   // (there is no second place)
                    }
                }
                release();
            }
        });
    }
    tmem_fence_before();
    __syncthreads();
    cluster_sync();   // (neither CTA leaves while the other may arrive on its barriers)
    if (warp == kLoader) {
        tmem_fence_after();
        tmem_free_all(tmem);
    }
}

// ------------------------------------------------------------------ host

// A product with its operands' maps.
struct Operands {
    Gemm gemm{};
    CUtensorMap a_map, b_map;
};

template <typename T, int FIRST, int SECOND>
cudaError_t launch_gemms(Operands& first, Operands& second, bool* launched, cudaStream_t stream) {
    static ClusterRoom known[64];
    static int ready[64];
    ClusterRoom room{};
    cudaError_t err = cluster_room(expert_gemm_kernel<T, FIRST, SECOND>, kThreads, kShared, known, ready, &room);
    if (err != cudaSuccess) return err;
    const int pairs = room.clusters[1];
    // Two 64-deep parts a stage where both fit four times into the ring: the issuer spends 0.2 us a stage whatever its size (32
    // experts of 2048 x 1024: mean 16 rows 81.0 to 77.9 us, mean 80 90.7 to 87.4; one expert of 4096 x 2048, 512 rows: 44.8 to 38.6).
    first.gemm.atoms = first.gemm.plan.cap <= 128 ? 2 : 1;
    second.gemm.atoms = 1;
    int bytes = 0;   // one ring serves both
    for (Gemm* a : {&first.gemm, &second.gemm}) {
        a->atom_bytes = kABytes + a->plan.cap / 2 * kStep * 2;
        if (a->atoms * a->atom_bytes > bytes) bytes = a->atoms * a->atom_bytes;
    }
    int64_t items = 0;
    for (Gemm* a : {&first.gemm, &second.gemm}) {
        a->stage_bytes = bytes;
        a->stages = kRing / bytes < kMostStages ? kRing / bytes : kMostStages;   // (4 to 6)
        if (a->columns > 0) items += static_cast<int64_t>(a->g.E) * a->plan.m_tiles * a->n_tiles;
        else if (a->plan.m_tiles > 0) items += most_tiles(a->g, a->plan.cap) * a->plan.m_tiles;
    }
    if (items == 0) return cudaSuccess;
    first.gemm.follows = *launched;
    *launched = true;
    return launch_clusters(expert_gemm_kernel<T, FIRST, SECOND>, static_cast<int>(items < pairs ? items : pairs), 2, kThreads, kShared, stream,
                           first.gemm, second.gemm, first.a_map, first.b_map, second.a_map, second.b_map);
}

// A product whose output has `lanes` channels, `of_tile` of them a tile; none without an output.
Gemm gemm_of(const FfnArgs& f, void* out, int64_t out_ld, int lanes, int of_tile, int inner) {
    Gemm a{};
    a.g = f.g;
    a.lanes = lanes;
    a.inner = inner;
    a.plan.m_tiles = out ? ceil_div(lanes, of_tile) : 0;
    // (the pairs at work together share 16 tiles of rows and some of the weights: dense 8192-row block 902 us; 4: 915, 64: 937, 1: 994)
    a.plan.chunk = 16;
    while (((f.g.E - 1) >> a.plan.shift) + 1 > kTileTable) ++a.plan.shift;
    const int64_t used = f.g.rows < f.g.E ? f.g.rows : f.g.E, mean = (f.g.rows - 1) / used + 1;
    // Rows of a tile at most: the smallest that holds most experts' rows in one tile. Smaller ones leave room for more stages and
    // cost fewer columns of zeros, larger ones read the weights less often. 32 experts of 2048 x 1024, us forward at mean rows
    //   24: 77.8 (32), 79.1 (64)     48: 90 (32), 83.1 (64), 86.9 (128)     112: 105 (64), 92.3 (128), 97.0 (256)
    //   128: 96.8 (128), 99.1 (256), but gradients 217.7 and 210.3          200: 122.8 (128), 110.7 (256)
    a.plan.cap = mean <= 24 ? 32 : mean <= 48 ? 64 : mean <= 112 ? 128 : 256;
    // Smaller ones where at most half the pairs would have work: a stage of few rows takes little less than one of many, so more
    // pairs with shorter tiles end sooner (one expert of 4096 x 2048: 64 rows 39.0 to 29.9 us, 256 rows 51.6 to 35.2).
    while (a.plan.cap > 32 && a.plan.m_tiles > 0 && 4 * most_tiles(f.g, a.plan.cap) * a.plan.m_tiles <= sm_count()) a.plan.cap /= 2;
    while (1 << a.plan.cap_shift < a.plan.cap) ++a.plan.cap_shift;
    a.box = a.plan.cap <= 64 ? 16 : 64;   // (each CTA loads half of a tile's rows, rounded up to boxes: small ones for small tiles)
    a.out = out;
    a.out_ld = out_ld;
    return a;
}

// Rows [rows][width] as operand B, contraction inward.
cudaError_t rows_map(CUtensorMap* map, const FfnArgs& f, const void* x, int64_t width, int64_t ld, int box) {
    return box_map(map, x, f.dtype, width, f.g.rows, 1, 1, ld * 2, ld * 2, ld * 2, box, 1);
}
// Weights [E][rows][width] in boxes of 64 x box.
cudaError_t weights_map(CUtensorMap* map, const FfnArgs& f, const void* w, int64_t rows, int64_t width, int box) {
    return box_map(map, w, f.dtype, width, rows, 1, f.g.E, width * 2, rows * width * 2, rows * width * 2, box, 1);
}

template <typename T>
cudaError_t forward(const FfnArgs& f, cudaStream_t stream) {
    const int64_t H = f.H, F = f.F;
    Operands p{}, none{};
    bool launched = false;
    p.gemm = gemm_of(f, f.act, f.act_ld, f.F, kLanes / 2, f.H);
    p.gemm.out2 = f.gate_up, p.gemm.out2_ld = f.gate_up_ld;
    cudaError_t err = box_map(&p.a_map, f.w_gate_up, f.dtype, H, F, 2, f.g.E, H * 2, F * H * 2, 2 * F * H * 2, 16, 2);
    if (err == cudaSuccess) err = rows_map(&p.b_map, f, f.x, H, f.x_ld, p.gemm.box);
    if (err == cudaSuccess) err = launch_gemms<T, kGateUp, kNone>(p, none, &launched, stream);
    if (err != cudaSuccess || !f.y) return err;
    p.gemm = gemm_of(f, f.y, f.y_ld, f.H, kLanes, f.F);
    err = weights_map(&p.a_map, f, f.w_down, H, F, kLanes / 2);
    if (err == cudaSuccess) err = rows_map(&p.b_map, f, f.act, F, f.act_ld, p.gemm.box);
    return err == cudaSuccess ? launch_gemms<T, kDown, kNone>(p, none, &launched, stream) : err;
}

// dW [E][outputs][inputs] = (by [rows][outputs])^T x [rows][inputs]: the outputs are the lanes
cudaError_t weight_gradient(Operands* p, const FfnArgs& f, void* out, const void* x, int inputs, int64_t x_ld, const void* by, int outputs,
                            int64_t by_ld) {
    Gemm& a = p->gemm = gemm_of(f, out, inputs, outputs, kLanes, 0);
    if (!out) return cudaSuccess;
    a.box = 32;   // (rows of a stage come by 32: 32 experts of 200 rows 226 us, by 16 234, by 64 226.5; of 8 rows 187.5, 187.2, 188.1)
    a.plan.cap = 256;
    a.columns = inputs;
    a.n_tiles = ceil_div(inputs, a.plan.cap);
    a.out_fp32 = f.grad_w_fp32, a.accumulate = f.accumulate;
    const cudaError_t err = rows_map(&p->a_map, f, by, outputs, by_ld, a.box);
    return err == cudaSuccess ? rows_map(&p->b_map, f, x, inputs, x_ld, a.box) : err;
}

// Two launches of two products each that do not depend on each other: their ends and starts cost once.
template <typename T>
cudaError_t backward(const FfnArgs& f, cudaStream_t stream) {
    const int64_t H = f.H, F = f.F;
    Operands p{}, w{};
    bool launched = false;
    p.gemm = gemm_of(f, f.grad_gate_up, f.grad_gate_up_ld, f.F, kLanes, f.H);
    p.gemm.in = f.gate_up, p.gemm.in_ld = f.gate_up_ld;
    cudaError_t err = weights_map(&p.a_map, f, f.w_down, H, F, kStep);
    if (err == cudaSuccess) err = rows_map(&p.b_map, f, f.grad_y, H, f.grad_y_ld, p.gemm.box);
    if (err == cudaSuccess) err = weight_gradient(&w, f, f.grad_w_down, f.act, f.F, f.act_ld, f.grad_y, f.H, f.grad_y_ld);
    if (err == cudaSuccess) err = launch_gemms<T, kGradAct, kGradW>(p, w, &launched, stream);
    if (err != cudaSuccess || (!f.grad_x && !f.grad_w_gate_up)) return err;
    p.gemm = gemm_of(f, f.grad_x, f.grad_x_ld, f.H, kLanes, 2 * f.F);
    if (f.grad_x) {
        err = weights_map(&p.a_map, f, f.w_gate_up, 2 * F, H, kStep);
        if (err == cudaSuccess) err = rows_map(&p.b_map, f, f.grad_gate_up, 2 * F, f.grad_gate_up_ld, p.gemm.box);
    }
    if (err == cudaSuccess)
        err = weight_gradient(&w, f, f.grad_w_gate_up, f.x, f.H, f.x_ld, f.grad_gate_up, 2 * f.F, f.grad_gate_up_ld);
    return err == cudaSuccess ? launch_gemms<T, kGradX, kGradW>(p, w, &launched, stream) : err;
}

}  // namespace

cudaError_t launch_expert_ffn(const FfnArgs& f, cudaStream_t stream) {
    return f.dtype == EP_DTYPE_BF16 ? forward<__nv_bfloat16>(f, stream) : forward<__half>(f, stream);
}

cudaError_t launch_expert_ffn_backward(const FfnArgs& f, cudaStream_t stream) {
    return f.dtype == EP_DTYPE_BF16 ? backward<__nv_bfloat16>(f, stream) : backward<__half>(f, stream);
}

}  // namespace ep
