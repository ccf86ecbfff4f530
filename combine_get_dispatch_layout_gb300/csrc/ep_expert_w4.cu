// The experts' products on dispatched rows: 4-bit weights, group scales.
//
// Mathematics. y[n, o] = sum over groups g of s[g, o] * sum over i in g of
// (code[o, i] - zero[g, o]) x[n, i]. code - zero is a whole number of at most
// five bits, exact in bf16 and fp16, so the inner sums run through the matrix
// instructions with exact products and fp32 sums, and the scale multiplies a
// group's sum in fp32: no weight is rounded.
//
// What bounds it: with few rows per expert each weight is used a few times, so
// reading the codes (half a byte each) once is the floor. Next to that come the
// integer instructions that unpack them (seven a word of eight codes, 2 clocks
// each a warp and SM quarter: 14 of the 22 clocks that DRAM takes for 128
// bytes a quarter), so the unpacking is kept to a mask, a shift and one
// subtraction per pair, and every unpacked fragment serves all rows at once.
//
// Layout. Weight rows are the instruction's 16 rows, dispatched rows its 8
// columns. The order of a product's inputs is free: a thread takes 8
// neighbouring codes of a weight row and the same 8 inputs of x, in the order
// in which masks leave the codes ((0, 4), (1, 5), (2, 6), (3, 7)), so the codes
// are used in the plain layout in which they are stored. A persistent CTA
// walks its items (an expert, a tile of weight rows, at most 8 NT rows of x)
// through one ring of asynchronous copies that runs on across items; its warps
// split tile rows and inputs, 64 inputs each a stage, and join at an item's end.
#include <type_traits>

#include "ep_layer.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kStages = 4;
constexpr int kSlice = 64;   // inputs of a warp per stage

// Tile shapes. Large: 128 weight rows, warps 2 (rows) x 4 (inputs), 256 inputs a stage: x is read once for
// 128 rows. Small: 32 rows, 8 warps over 512 inputs: four times as many items where there are few.
template <bool SMALL>
struct Tile {
    static constexpr int kMTiles = SMALL ? 2 : 4;          // 16-row tiles of a warp
    static constexpr int kRowWarps = SMALL ? 1 : 2;
    static constexpr int kInWarps = 8 / kRowWarps;
    static constexpr int kRows = 16 * kMTiles * kRowWarps;
    static constexpr int kIn = kSlice * kInWarps;          // inputs of a stage
    static constexpr int kRowBytes = kIn / 2;
    static constexpr int kPieces = kRowBytes / 16;         // 16-byte pieces of a weight row
    static constexpr int kCopies = kRows * kPieces / kThreads;
    static constexpr int kXPieces = kIn * 2 / 16;
    static constexpr int kXRows = kThreads / kXPieces;     // rows of x that one pass of the threads copies
};

template <bool SMALL, int NT>
struct Stage {
    using L = Tile<SMALL>;
    static constexpr int kWeights = L::kRows * L::kRowBytes;
    static constexpr int kX = 8 * NT * L::kIn * 2;
    // scale (16 bits) and zero point (as the unpacked pairs hold it) of each row and group
    static constexpr int kScales = L::kRows * (L::kIn / 32) * 4;
    // the weights of a used-up stage also hold a quarter of the partial sums at an item's end
    static_assert((L::kInWarps + 3) / 4 * 8 * NT * L::kRows * 4 <= kWeights, "");
};

struct Plan {
    int tiles;      // of an expert
    int slots;      // CTAs that the device holds at once (the grid)
    int stages;     // of an item
    int groups;     // of a weight row
    int log_group;
};

template <typename T>
__device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t b) {
    if constexpr (std::is_same_v<T, __half>) {
        const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    } else {
        const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
}

// A code in the low mantissa bits under this exponent is 128 + code (bf16), 1024 + code (fp16).
template <typename T>
constexpr uint32_t kBias = std::is_same_v<T, __half> ? 0x6400u : 0x4300u;

// Pair k of a word's codes, (k, k + 4), minus the zero point: exact.
template <typename T>
__device__ __forceinline__ uint32_t unpack(uint32_t word, int k, uint32_t zero) {
    return minus<T>(((word >> (4 * k)) & 0x000f000fu) | (kBias<T> * 0x10001u), zero);
}

template <typename T>
__device__ __forceinline__ void multiply(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same_v<T, __half>)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
// 16 bytes to shared memory, of which the first `real` (16 or 0) are read and the rest are zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real) : "memory");
}

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

// T: type of x, scales and y. NT: eights of x rows of an item. SLICES: a warp's 64 inputs of a stage are one slice of
// a group (1), or two groups of 32 (2).
template <typename T, bool SMALL, int NT, int SLICES>
__global__ void __launch_bounds__(kThreads, NT <= 2 ? 2 : 1) expert_w4_kernel(W4Args a, Plan p) {
    using L = Tile<SMALL>;
    using S = Stage<SMALL, NT>;
    constexpr int kSpan = kSlice / SLICES;          // inputs that share a thread's scale
    constexpr int kWords = kSpan / 32;              // words of codes a thread takes of them
    constexpr int kItemRows = 8 * NT;
    extern __shared__ __align__(128) unsigned char shared_bytes[];
    unsigned char* const weights = shared_bytes;                               // [kStages][kWeights]
    unsigned char* const inputs = weights + kStages * S::kWeights;             // [kStages][kX]
    uint32_t* const scales = reinterpret_cast<uint32_t*>(inputs + kStages * S::kX);   // [kStages][groups of a stage][kRows]
    int* const first_pass = reinterpret_cast<int*>(scales + kStages * (S::kScales / 4 / (SLICES == 2 ? 1 : 2)));  // [E + 1]
    constexpr int kScaleWords = S::kScales / 4 / (SLICES == 2 ? 1 : 2);   // a group has 64 inputs at least with one slice
    __shared__ int warp_sum[kThreads / 32];
    dependent_entry();

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int row_warp = warp % L::kRowWarps, in_warp = warp / L::kRowWarps;
    const int cols = a.swiglu ? a.O / 2 : a.O, tile_cols = a.swiglu ? L::kRows / 2 : L::kRows;

    // ---- items: an expert's rows in passes of kItemRows, each pass over all tiles; a tile's passes follow each
    // other, so the weights of the second come from L2
    {
        const int per = (a.E + kThreads - 1) / kThreads, lo = min(a.E, tid * per), hi = min(a.E, lo + per);
        int own = 0, first;
        for (int e = lo; e < hi; ++e) own += (expert_rows(a, e, first) + kItemRows - 1) / kItemRows;
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
            base += (expert_rows(a, e, first) + kItemRows - 1) / kItemRows;
        }
        if (hi == a.E && lo < hi) first_pass[a.E] = base;
        __syncthreads();
    }
    const int64_t items = static_cast<int64_t>(first_pass[a.E]) * p.tiles;
    // as many CTAs as share the items evenly: all of them wait on the same DRAM, so an SM with one CTA less costs nothing
    const int64_t each = (items + p.slots - 1) / p.slots;
    const int64_t item0 = each * blockIdx.x, item1 = min(items, item0 + each);
    if (item0 >= item1) return;
    const int64_t steps = (item1 - item0) * p.stages;

    const auto decode = [&](int64_t it) {
        int lo = 0, hi = a.E - 1;   // the last expert whose first item is not behind `it`, with passes of its own
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
        r.row = first + pass * kItemRows;
        r.rows = min(kItemRows, n - pass * kItemRows);
        r.col = in / passes * tile_cols;
        return r;
    };
    // weight row of the tile's row r, or -1 past the end: with an activation the tile's halves are gate and up rows
    const auto weight_row = [&](int col, int r) {
        if (!a.swiglu) return col + r < a.O ? col + r : -1;
        const int j = col + (r < L::kRows / 2 ? r : r - L::kRows / 2);
        return j >= cols ? -1 : r < L::kRows / 2 ? j : cols + j;
    };

    // ---- the copies of a stage. Thread's pieces of the weights: rows tid / kPieces + k * kThreads / kPieces, of x
    // likewise. Pieces of a row are exchanged so that fragment loads meet no bank twice: of the weights by
    // ((row & 3) << 1 | row >> 2 & 1) (a load takes 4 rows x 32 bytes or 8 x 16), of x by 5 for odd rows.
    int64_t load_item = item0;
    int load_stage = 0, load_slot = 0;
    const unsigned char* weight_at[L::kCopies];
    bool weight_real[L::kCopies];
    const unsigned char* x_at = nullptr;
    Item li{};
    const int piece = tid % L::kPieces, piece_row = tid / L::kPieces;
    const int x_piece = tid % L::kXPieces, x_row = tid / L::kXPieces;
    constexpr int kXCopies = kItemRows / L::kXRows;
    // scales of a stage: entries tid + k * kThreads of [groups][rows], held in registers while they load
    const int stage_groups = L::kIn >> p.log_group;   // 2 .. 16
    constexpr int kScaleLoads = (kScaleWords + kThreads - 1) / kThreads;
    uint16_t scale_in[kScaleLoads];
    uint8_t zero_in[kScaleLoads];
    int scale_row[kScaleLoads];
    const uint16_t* scale_at = nullptr;
    const uint8_t* zero_at = nullptr;

    const auto load = [&](int64_t step) {   // issues the copies and the scale loads of the next stage
        if (step >= steps) return;
        if (load_stage == 0) {
            li = decode(load_item);
#pragma unroll
            for (int k = 0; k < L::kCopies; ++k) {
                const int o = weight_row(li.col, piece_row + k * (kThreads / L::kPieces));
                weight_real[k] = o >= 0;
                weight_at[k] = a.w + (static_cast<int64_t>(li.expert) * a.O + max(o, 0)) * (a.I / 2) + piece * 16;
            }
            x_at = static_cast<const unsigned char*>(a.x) + (static_cast<int64_t>(li.row + x_row) * a.x_ld + x_piece * 8) * 2;
#pragma unroll
            for (int k = 0; k < kScaleLoads; ++k) scale_row[k] = weight_row(li.col, (tid + k * kThreads) % L::kRows);
            const int64_t at = static_cast<int64_t>(li.expert) * p.groups * a.O;
            scale_at = static_cast<const uint16_t*>(a.scales) + at;
            zero_at = a.zeros ? a.zeros + at : nullptr;
        }
        const uint32_t to = smem_addr(weights + load_slot * S::kWeights);
        const bool piece_in = load_stage * L::kRowBytes + piece * 16 < a.I / 2;
#pragma unroll
        for (int k = 0; k < L::kCopies; ++k) {
            const int r = piece_row + k * (kThreads / L::kPieces);
            copy16(to + r * L::kRowBytes + ((piece ^ ((r & 3) << 1 | ((r >> 2) & 1))) << 4),
                   piece_in ? weight_at[k] + load_stage * L::kRowBytes : a.w, piece_in && weight_real[k] ? 16 : 0);
        }
        const uint32_t xto = smem_addr(inputs + load_slot * S::kX);
        const bool x_in = load_stage * L::kIn + x_piece * 8 < a.I;
#pragma unroll
        for (int k = 0; k < kXCopies; ++k) {
            const int r = x_row + k * L::kXRows;
            if (r < li.rows)   // (rows that are not there leave garbage in columns that are not written)
                copy16(xto + r * (L::kIn * 2) + ((x_piece ^ ((r & 1) * 5)) << 4),
                       x_in ? x_at + (static_cast<int64_t>(k) * L::kXRows * a.x_ld + load_stage * L::kIn) * 2 : a.x, x_in ? 16 : 0);
        }
#pragma unroll
        for (int k = 0; k < kScaleLoads; ++k) {
            const int i = tid + k * kThreads, grp = load_stage * stage_groups + i / L::kRows;
            scale_in[k] = 0;
            zero_in[k] = 8;
            if (i < stage_groups * L::kRows && grp < p.groups && scale_row[k] >= 0) {
                const int64_t at = static_cast<int64_t>(grp) * a.O + scale_row[k];
                scale_in[k] = scale_at[at];
                if (zero_at) zero_in[k] = zero_at[at];
            }
        }
    };
    const auto loaded = [&](int64_t step) {   // the scales to their slot, once here
        if (step < steps) {
            uint32_t* to = scales + load_slot * kScaleWords;
#pragma unroll
            for (int k = 0; k < kScaleLoads; ++k) {
                const int i = tid + k * kThreads;
                if (i < stage_groups * L::kRows) to[i] = scale_in[k] | (kBias<T> + zero_in[k]) << 16;
            }
            if (++load_stage == p.stages) load_stage = 0, ++load_item;
        }
        load_slot = (load_slot + 1) % kStages;
    };

#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) {
        load(i);
        asm volatile("cp.async.commit_group;" ::: "memory");
        loaded(i);
    }

    float acc[L::kMTiles][NT][4];
    Item ci{};
    int64_t item = item0;
    int stage = 0, slot = 0, eights = 0;
    for (int64_t step = 0; step < steps; ++step) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncthreads();
        load(step + kStages - 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (stage == 0) {
            ci = decode(item);
            eights = (ci.rows + 7) / 8;
#pragma unroll
            for (int m = 0; m < L::kMTiles; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.0f;
        }
        const unsigned char* ws = weights + slot * S::kWeights;
        const unsigned char* xs = inputs + slot * S::kX;
        const uint32_t* ss = scales + slot * kScaleWords;
#pragma unroll
        for (int sub = 0; sub < SLICES; ++sub) {
            const int in0 = in_warp * kSlice + sub * kSpan;   // inputs [in0, in0 + kSpan) of the stage
            // x: 8 kWords neighbouring inputs of row 8 n + g, in the order of the unpacked codes
            uint32_t xf[NT][kWords][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n > 0 && n >= eights) break;
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    const int r = 8 * n + g, pc = in0 / 8 + t * kWords + w;
                    const uint4 v = *reinterpret_cast<const uint4*>(xs + r * (L::kIn * 2) + ((pc ^ ((r & 1) * 5)) << 4));
                    xf[n][w][0] = __byte_perm(v.x, v.z, 0x5410);   // (0, 4)
                    xf[n][w][1] = __byte_perm(v.x, v.z, 0x7632);   // (1, 5)
                    xf[n][w][2] = __byte_perm(v.y, v.w, 0x5410);   // (2, 6)
                    xf[n][w][3] = __byte_perm(v.y, v.w, 0x7632);   // (3, 7)
                }
            }
            const uint32_t* sg = ss + (in0 >> p.log_group) * L::kRows;
#pragma unroll
            for (int m = 0; m < L::kMTiles; ++m) {
                const int r0 = (row_warp * L::kMTiles + m) * 16 + g;
                uint32_t word[2][kWords];
                uint32_t zero[2];
                float scale[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = r0 + 8 * h;
                    const int byte = in0 / 2 + t * 4 * kWords;
                    const unsigned char* from = ws + r * L::kRowBytes + (((byte >> 4) ^ ((r & 3) << 1 | ((r >> 2) & 1))) << 4) + (byte & 15);
                    if constexpr (kWords == 2) {
                        const uint2 v = *reinterpret_cast<const uint2*>(from);
                        word[h][0] = v.x, word[h][1] = v.y;
                    } else {
                        word[h][0] = *reinterpret_cast<const uint32_t*>(from);
                    }
                    const uint32_t sz = sg[r];
                    zero[h] = __byte_perm(sz, sz, 0x3232);
                    if constexpr (std::is_same_v<T, __half>) scale[h] = __half2float(__ushort_as_half(static_cast<unsigned short>(sz)));
                    else scale[h] = __uint_as_float(sz << 16);
                }
                float sum[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) sum[n][0] = sum[n][1] = sum[n][2] = sum[n][3] = 0.0f;
#pragma unroll
                for (int w = 0; w < kWords; ++w)
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const uint32_t af[4] = {unpack<T>(word[0][w], k, zero[0]), unpack<T>(word[1][w], k, zero[1]),
                                                unpack<T>(word[0][w], k + 1, zero[0]), unpack<T>(word[1][w], k + 1, zero[1])};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (n > 0 && n >= eights) break;
                            multiply<T>(sum[n], af, xf[n][w][k], xf[n][w][k + 1]);
                        }
                    }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[m][n][0] += scale[0] * sum[n][0];
                    acc[m][n][1] += scale[0] * sum[n][1];
                    acc[m][n][2] += scale[1] * sum[n][2];
                    acc[m][n][3] += scale[1] * sum[n][3];
                }
            }
        }
        if (++stage == p.stages) {
            // ---- the item's end: the warps' partial sums join by halves, through the weights of the stage just
            // used up, in a fixed order; sums[x row][weight row], weight rows exchanged by 8 t to keep off one bank
            stage = 0;
            ++item;
            constexpr int kStride = L::kRows;
            float* sums = reinterpret_cast<float*>(weights + slot * S::kWeights);
            const auto place = [&](int m, int n, int j) {
                return (8 * n + 2 * t + (j & 1)) * kStride + (((row_warp * L::kMTiles + m) * 16 + g + 8 * (j >> 1)) ^ (t << 3));
            };
            __syncthreads();
#pragma unroll
            for (int half = L::kInWarps / 2; half >= 1; half /= 2) {
                for (int turn = 0; turn < (half > 1 ? 2 : 1); ++turn) {
                    // at most kInWarps / 4 partial sums at a time fit the area
                    const int part = half > 1 ? half / 2 : 1;
                    const int from = half + turn * part;
                    if (in_warp >= from && in_warp < from + part) {
#pragma unroll
                        for (int m = 0; m < L::kMTiles; ++m)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int j = 0; j < 4; ++j) sums[(in_warp - from) * kItemRows * kStride + place(m, n, j)] = acc[m][n][j];
                    }
                    __syncthreads();
                    const int to = from - half;
                    if (in_warp >= to && in_warp < to + part) {
#pragma unroll
                        for (int m = 0; m < L::kMTiles; ++m)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int j = 0; j < 4; ++j) acc[m][n][j] += sums[(in_warp - to) * kItemRows * kStride + place(m, n, j)];
                    }
                    __syncthreads();
                }
            }
            if (in_warp == 0) {
#pragma unroll
                for (int m = 0; m < L::kMTiles; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) sums[place(m, n, j)] = acc[m][n][j];
            }
            __syncthreads();
            T* y = static_cast<T*>(a.y) + static_cast<int64_t>(ci.row) * a.y_ld + ci.col;
            const int wide = min(tile_cols, cols - ci.col);
            for (int i = tid; i < ci.rows * tile_cols; i += kThreads) {
                const int n = i / tile_cols, c = i % tile_cols;
                if (c >= wide) continue;
                const int x = ((n >> 1) & 3) << 3;
                float v = sums[n * kStride + (c ^ x)];
                if (a.swiglu) v = v / (1.0f + expf(-v)) * sums[n * kStride + ((L::kRows / 2 + c) ^ x)];
                y[n * a.y_ld + c] = from_float<T>(v);
            }
            // (the area is written again only behind the next step's barrier)
        }
        slot = (slot + 1) % kStages;
        loaded(step + kStages - 1);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Resident CTAs per device of one kernel, with its shared memory limit raised: fixed for a size of shared
// memory, looked up when a larger one than before comes (a race writes the same values).
template <typename Kernel>
cudaError_t prepare_kernel(Kernel kernel, int smem, int* known_smem, int* known_ctas, int* ctas) {
    constexpr int kDevices = 64;
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < kDevices && __atomic_load_n(&known_smem[dev], __ATOMIC_ACQUIRE) >= smem) {
        *ctas = __atomic_load_n(&known_ctas[dev], __ATOMIC_RELAXED);
        return cudaSuccess;
    }
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err == cudaSuccess) err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, smem);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    *ctas = per_sm * sms;
    if (dev < kDevices) {
        __atomic_store_n(&known_ctas[dev], *ctas, __ATOMIC_RELAXED);
        __atomic_store_n(&known_smem[dev], smem, __ATOMIC_RELEASE);
    }
    return cudaSuccess;
}

template <typename T, bool SMALL, int NT, int SLICES>
cudaError_t launch_shape(const W4Args& a, cudaStream_t stream) {
    using L = Tile<SMALL>;
    using S = Stage<SMALL, NT>;
    static int known_smem[64], known_ctas[64];
    const int smem = kStages * (S::kWeights + S::kX + S::kScales / (SLICES == 2 ? 1 : 2)) + (a.E + 1) * 4;
    Plan p{};
    cudaError_t err = prepare_kernel(expert_w4_kernel<T, SMALL, NT, SLICES>, smem, known_smem, known_ctas, &p.slots);
    if (err != cudaSuccess) return err;
    const int tile_cols = a.swiglu ? L::kRows / 2 : L::kRows, cols = a.swiglu ? a.O / 2 : a.O;
    p.tiles = (cols + tile_cols - 1) / tile_cols;
    p.stages = (a.I + L::kIn - 1) / L::kIn;
    p.groups = a.I / a.group;
    p.log_group = a.group == 32 ? 5 : a.group == 64 ? 6 : 7;
    const int64_t most = (static_cast<int64_t>(a.rows) / (8 * NT) + (a.rows < a.E ? a.rows : a.E)) * p.tiles;   // items at most
    const int grid = static_cast<int>(most < p.slots ? (most > 0 ? most : 1) : p.slots);
    p.slots = grid;
    return launch_dependent(expert_w4_kernel<T, SMALL, NT, SLICES>, dim3(grid), dim3(kThreads), smem, stream, a, p);
}

template <typename T, bool SMALL, int NT>
cudaError_t launch_slices(const W4Args& a, cudaStream_t stream) {
    return a.group == 32 ? launch_shape<T, SMALL, NT, 2>(a, stream) : launch_shape<T, SMALL, NT, 1>(a, stream);
}

template <typename T>
cudaError_t launch_type(const W4Args& a, cudaStream_t stream) {
    // experts that may have rows, and the rows one of them has on average
    const int used = a.rows < a.E ? a.rows : a.E, mean = (a.rows + used - 1) / used;
    const bool small = static_cast<int64_t>(used) * ((a.O + 127) / 128) < 1024;
    if (small) return mean <= 2 || a.rows <= 8 ? launch_slices<T, true, 1>(a, stream) : launch_slices<T, true, 2>(a, stream);
    if (mean <= 2 || a.rows <= 8) return launch_slices<T, false, 1>(a, stream);
    return mean <= 12 ? launch_slices<T, false, 2>(a, stream) : launch_slices<T, false, 4>(a, stream);
}

}  // namespace

cudaError_t launch_expert_w4(const W4Args& a, int dtype, cudaStream_t stream) {
    return dtype == EP_DTYPE_BF16 ? launch_type<__nv_bfloat16>(a, stream) : launch_type<__half>(a, stream);
}

}  // namespace ep
