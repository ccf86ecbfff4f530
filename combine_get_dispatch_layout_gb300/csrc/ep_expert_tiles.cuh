// What the kernels of the experts' products share: whose rows are whose, and
// the walk of persistent CTAs over tiles of them.
#pragma once

#include "ep_tensor.cuh"

namespace ep {
namespace {

constexpr int kTileTable = 1024;   // entries of the table of experts' tiles
constexpr int kRowTable = 256;     // experts whose rows are kept in shared memory, if there are no more

// In shared memory: tiles before an expert, and the experts' first rows and numbers of rows.
struct Tables {
    int tiles[kTileTable + 1];
    int2 rows[kRowTable];
};

// First row and number of real rows of expert e, within [0, rows).
__device__ __forceinline__ int rows_of(const ExpertRows& g, int e, int& first) {
    if (!g.offsets) {
        first = 0;
        return g.rows;
    }
    first = min(max(g.offsets[e], 0), g.rows);
    int n = min(max(g.offsets[e + 1], 0), g.rows) - first;
    if (g.counts) n = min(n, g.counts[e]);
    return max(n, 0);
}

// The same from the table.
__device__ __forceinline__ int rows_of(const ExpertRows& g, const Tables* t, int e, int& first) {
    if (g.E > kRowTable) return rows_of(g, e, first);
    const int2 r = t->rows[e];
    first = r.x;
    return r.y;
}

// Tiles of an expert's product: m_tiles along the weights' rows, and along its own rows as many as `cap` rows a tile
// make, of nearly equal width. All weight tiles are passed over for `chunk` tiles of rows at a time, so that the CTAs
// at work together share the weights of few tiles and the inputs of few.
struct TilePlan {
    int m_tiles, cap, cap_shift, chunk;   // cap = 2^cap_shift
    int whole;   // tiles of `cap` rows and a rest, instead of equal ones
    int shift;   // an entry of the table stands for 2^shift experts
    // Items after which the order of an expert's tiles turns about, or 0: with a full and a short tile each and an even number of
    // CTAs some would have only full ones (fp8, 128 experts of 138 rows, 7168 x 4096: 1265 to 980 us).
    int flip;
};
struct Tile {
    int expert, m;     // m: tile of weight rows
    int row, rows;     // the expert's rows of this tile
};

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a - 1) / b + 1; }   // a >= 1

__device__ __forceinline__ int tiles_of(const TilePlan& p, int n) { return static_cast<int>((static_cast<uint32_t>(n) + p.cap - 1) >> p.cap_shift); }

// Fills the tables, by all threads of the CTA (THREADS of them); they are there after the next barrier.
template <int THREADS>
__device__ __forceinline__ void fill_tables(const ExpertRows& g, const TilePlan& p, Tables* t, int* warp_sum) {
    static_assert(kRowTable < THREADS, "");
    int* const table = t->tiles;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const auto tiles_at = [&](int e) {
        int first;
        return tiles_of(p, rows_of(g, e, first));
    };
    const int entries = ((g.E - 1) >> p.shift) + 1;
    const int per = (entries + THREADS - 1) / THREADS, lo = min(entries, tid * per), hi = min(entries, lo + per);
    const int e0 = lo << p.shift, e1 = min(g.E, hi << p.shift);
    int own = 0;
    if (g.E <= kRowTable) {   // an expert a thread
        if (tid < g.E) {
            int first;
            const int n = rows_of(g, tid, first);
            t->rows[tid] = make_int2(first, n);
            own = tiles_of(p, n);
        }
    } else {
        for (int e = e0; e < e1; ++e) own += tiles_at(e);
    }
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
    for (int w = 0; w < THREADS / 32; ++w)
        if (w < warp) base += warp_sum[w];
    if (g.E <= kRowTable) {
        if (tid <= g.E) table[tid] = base;   // (the thread behind the last has all of them)
        return;
    }
    for (int e = e0; e < e1; ++e) {
        if ((e & ((1 << p.shift) - 1)) == 0) table[e >> p.shift] = base;
        base += tiles_at(e);
    }
    if (hi == entries && lo < hi) table[entries] = base;
}

__device__ __forceinline__ int64_t tile_count(const ExpertRows& g, const TilePlan& p, const Tables* t) {
    return static_cast<int64_t>(t->tiles[((g.E - 1) >> p.shift) + 1]) * p.m_tiles;
}

// (Offsets that contradict one another can make tiles without rows, never one outside [0, rows). Items are fewer than 2^31:
// each has 32 rows x 128 channels of a buffer or is an expert's last along its rows; every role looks each item up, so the
// common cases go without divisions: 1500 to 1000 clocks.)
__device__ __forceinline__ Tile tile_at(const ExpertRows& g, const TilePlan& p, const Tables* tables, int64_t item) {
    const int* const table = tables->tiles;
    const uint32_t it = static_cast<uint32_t>(item), m_tiles = p.m_tiles;
    const int unit = static_cast<int>(it / m_tiles);   // tiles of rows before it, if all weight tiles of one came together
    int lo = 0, hi = (g.E - 1) >> p.shift;   // the last entry whose first tile is not behind `it`
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (table[mid] <= unit) lo = mid;
        else hi = mid - 1;
    }
    uint32_t in = it - table[lo] * m_tiles;
    int first, e = lo << p.shift, n = rows_of(g, tables, e, first), tiles = tiles_of(p, n);
    while (in >= tiles * m_tiles && e + 1 < g.E) {   // (an entry of several experts)
        in -= tiles * m_tiles;
        n = rows_of(g, tables, ++e, first);
        tiles = tiles_of(p, n);
    }
    Tile t;
    t.expert = e;
    int place = 0, width = p.cap;
    if (tiles <= 1) {
        t.m = static_cast<int>(min(in, m_tiles - 1));
    } else {
        const uint32_t per_chunk = p.chunk * m_tiles;
        const int c = in < per_chunk ? 0 : static_cast<int>(in / per_chunk);
        const uint32_t r = in - c * per_chunk, wide = max(min(p.chunk, tiles - c * p.chunk), 1);
        t.m = static_cast<int>(r / wide);
        place = static_cast<int>(r - t.m * wide);
        if (p.flip > 0 && ((it - place) / p.flip & 1)) place = static_cast<int>(wide) - 1 - place;   // (all of these tiles or none, so that each has its turn)
        place += c * p.chunk;
        if (!p.whole && 16 * tiles < p.cap) width = (ceil_div(n, tiles) + 15) / 16 * 16;   // nearly equal, none left without rows by the rounding
    }
    const int64_t at = static_cast<int64_t>(place) * width;
    t.row = first + static_cast<int>(min(at, static_cast<int64_t>(n)));
    t.rows = static_cast<int>(max(min(static_cast<int64_t>(width), n - at), static_cast<int64_t>(0)));
    return t;
}

// Columns of the product for n rows of a tile.
__device__ __forceinline__ int columns_of(int n) { return max((n + 15) / 16 * 16, 16); }

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tmem_alloc_one(uint32_t to) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(to) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_one(uint32_t tmem) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}
// sums [128 lanes][N] (+)= A [128 lanes] * B [N columns]^T, 8-bit operands in shared memory.
__device__ __forceinline__ void multiply_one(uint32_t sums, uint64_t a, uint64_t b, uint32_t shape, bool add) {
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(sums),
                 "l"(a), "l"(b), "r"(shape), "r"(static_cast<uint32_t>(add))
                 : "memory");
}

// ---- pairs: two CTAs of a cluster multiply as one, operand A's 256 rows and operand B's columns half in each. The first
// issues for both; each has the sums of its own 128 rows in its TMEM.

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Address, for the cluster, of the same place in a CTA's shared memory.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t in_first(uint32_t addr) { return in_cta(addr, 0); }
__device__ __forceinline__ float load_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
// On a barrier of either CTA. (It orders no memory but, behind the tcgen05 fence, the tensor memory that has been read:
// as a release for the CTA it held the thread for 1000 clocks, for the cluster for 2000.)
__device__ __forceinline__ void barrier_arrive_pair(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same, ordering what this thread has written, for barrier_wait_cluster.
__device__ __forceinline__ void barrier_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool barrier_try_cluster(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}
// As barrier_wait, for a barrier that the other CTA arrives on.
__device__ __forceinline__ void barrier_wait_cluster(uint32_t bar, uint32_t parity, volatile int* dead) {
    for (int i = 0; i < (1 << 22); ++i) {
        if (barrier_try_cluster(bar, parity)) return;
        if ((i & 1023) == 1023 && *dead) return;
    }
    *dead = 1;
}
// A box into this CTA's shared memory that counts on a barrier of either CTA.
__device__ __forceinline__ void load_box_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tmem_alloc_all(uint32_t to) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(to) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_all(uint32_t tmem) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}
// The loads into these registers are complete. (It orders nothing else, so loads from shared memory pass it.)
template <int N>
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::);
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
}
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
        "%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}
// sums [2 x 128 lanes][N] (+)= A [2 x 128 lanes] * B [2 x N / 2 columns]^T, all in the pair's shared memory.
__device__ __forceinline__ void multiply_pair(uint32_t sums, uint64_t a, uint64_t b, uint32_t shape, bool add) {
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(sums), "l"(a),
                 "l"(b), "r"(shape), "r"(static_cast<uint32_t>(add))
                 : "memory");
}
// Arrives on both CTAs' barriers at this place once the products so far are done.
__device__ __forceinline__ void pair_done(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"(static_cast<uint16_t>(3))
                 : "memory");
}

// 1 / (1 + exp(-v)) = r, or r 2^-124 if it is `far` below 1, so that it keeps its bits where exp(-v) is past fp32's range and the
// sigmoid below its normal numbers (it is 0 below 2^-250; NaN stays). exp is 2^t for t = -v log2(e) in two parts, so that large |v| lose
// nothing. Every number that the instructions see is normal, or nothing beside the 1 that it is added to: those that flush
// subnormals do (those that do not take several times as many). Within 5 * 2^-23 of itself (2^-22 of the exponential, 2^-23 of the
// reciprocal, four roundings); over all fp32 numbers the largest error is 2.52 * 2^-23, silu's 2.76 * 2^-23.
struct Sigmoid {
    float r;
    bool far;
};
__device__ __forceinline__ Sigmoid sigmoid_of(float v) {
    float x, e;
    Sigmoid s;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(-v), "f"(-104.0f));   // (t stays finite; 0 beside 1, and 2^-250, lie within)
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(176.0f));
    const float t = x * 1.44269504f;
    const float rest = fmaf(x, 1.44269504f, -t) + x * 1.92596299e-8f;
    s.far = t > 124.0f;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t - (s.far ? 124.0f : 0.0f)));   // (an exact difference)
    e *= fmaf(rest, 0.69314718f, 1.0f);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.r) : "f"((s.far ? 0x1p-124f : 1.0f) + e));
    return s;
}
// silu(gate) * up = gate * sigmoid * up, without an overflow or underflow on the way that the result has not.
__device__ __forceinline__ float gated(float gate, float up) {
    const Sigmoid s = sigmoid_of(gate);
    return gate * s.r * (up * (s.far ? 0x1p-124f : 1.0f));
}

// ------------------------------------------------------------------ host

// [w][z][y][x] with x dense and y, z, w `stride` bytes apart (multiples of 16), read in boxes of 128 bytes x box_y x
// box_z with the 128-byte swizzle; zeros past the ends.
cudaError_t box_map(CUtensorMap* map, const void* base, int dtype, int64_t x, int64_t y, int64_t z, int64_t w, int64_t stride_y,
                    int64_t stride_z, int64_t stride_w, int box_y, int box_z) {
    const EncodeFn encode = encoder();
    if (!encode) return cudaErrorNotSupported;
    const CUtensorMapDataType type = dtype == EP_DTYPE_BF16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                     : dtype == EP_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                              : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const int box_x = type == CU_TENSOR_MAP_DATA_TYPE_UINT8 ? 128 : 64;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(x), static_cast<cuuint64_t>(y), static_cast<cuuint64_t>(z),
                                static_cast<cuuint64_t>(w)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(stride_y), static_cast<cuuint64_t>(stride_z),
                                   static_cast<cuuint64_t>(stride_w)};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(box_x), static_cast<cuuint32_t>(box_y), static_cast<cuuint32_t>(box_z), 1},
                     step[4] = {1, 1, 1, 1};
    return encode(map, type, 4, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// SMs of the current device, 0 on an error: looked up once per device (a race writes the same value).
int sm_count() {
    static int known[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 64 && (sms = __atomic_load_n(&known[dev], __ATOMIC_RELAXED)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) __atomic_store_n(&known[dev], sms, __ATOMIC_RELAXED);
    return sms;
}

// Tiles of rows at most, of `cap` rows each.
int64_t most_tiles(const ExpertRows& g, int cap) {
    const int64_t used = g.rows < g.E ? g.rows : g.E;
    return (g.rows + used * (cap - 1)) / cap;
}

// Clusters of 1, 2, 4 and 8 CTAs of a kernel that a device holds at once.
struct ClusterRoom {
    int clusters[4];
};

// Of the current device, with the kernel's shared memory limit raised: looked up once per device (a race writes the same
// values, `ready` after them).
template <typename Kernel>
cudaError_t cluster_room(Kernel kernel, int threads, int smem, ClusterRoom* known, int* ready, ClusterRoom* room) {
    constexpr int kDevices = 64;
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < kDevices && __atomic_load_n(&ready[dev], __ATOMIC_ACQUIRE)) {
        *room = known[dev];
        return cudaSuccess;
    }
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    room->clusters[0] = sms;
    for (int i = 1; i < 4 && err == cudaSuccess; ++i) {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 1 << i;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(sms >> i << i);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        err = cudaOccupancyMaxActiveClusters(&room->clusters[i], kernel, &cfg);
    }
    if (err == cudaSuccess && room->clusters[1] < 1) err = cudaErrorInvalidConfiguration;
    if (err == cudaSuccess && dev < kDevices) {
        known[dev] = *room;
        __atomic_store_n(&ready[dev], 1, __ATOMIC_RELEASE);
    }
    return err;
}

// Launches clusters of `size` CTAs as a programmatic dependent of the work before.
template <typename... Params, typename... Args>
cudaError_t launch_clusters(void (*kernel)(Params...), int clusters, int size, int threads, int smem, cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * size);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = size > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
}  // namespace ep
