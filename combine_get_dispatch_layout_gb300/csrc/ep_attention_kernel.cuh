// Paged attention of one new token: the kernels' template, instantiated per
// element type by ep_attention_*.cu.
//
// Mathematics. For one cache head and the `heads` query heads that share it,
// with scores s_i = c q.k_i (c = scale * log2 e): the running maximum m, the sum
// l = sum 2^(s_i - m) and O = sum 2^(s_i - m) v_i, one pass over the keys; a
// larger m rescales l and O by 2^(m_old - m). Parts of the key range join by
// the same rule, so the range can be cut anywhere.
//
// What bounds it: each key and value is read once for all its query heads, so
// DRAM (4 * heads / 2 operations per cache byte is far below the tensor rate).
// The layout serves that: a persistent grid whose CTAs take equal shares of
// all sequences' keys, laid end to end in chunks of 64 to 256, so no CTA waits for
// another's longer sequence; a ring of chunks in shared memory, filled by
// 16-byte asynchronous copies that run several chunks ahead and straight on
// into the next sequence.
//
// The products run transposed, keys as the matrix instruction's 16 rows and
// query heads as its 8 columns: S^T = K Q^T, O^T = V^T P^T. One cache head is
// shared by few query heads (8 is common); as the 16-row operand they would
// leave half the instruction empty. A warp takes its share of each chunk with
// statistics of its own; the warps join when a segment (a CTA's part of one
// sequence and head) ends.
//
// Measured, launches in a graph, join kernel included, heads of 128: one
// sequence of 131071 keys, 8 cache heads, bf16: 86.9 us (6.2 TB/s); 64 of up to
// 4096 keys, 64 query heads: 89.1 us (5.7 TB/s), fp16 the same; 128 of up to 8192
// over an e4m3 cache: 173 us (5.9 TB/s), all of 8192: 337 us (6.4 TB/s); one of 129
// keys: 6.4 us. What is over the time at the full rate is start, join and each
// segment's end: 15 us (20 with e4m3) where a CTA has 3 or 4 segments.
#pragma once

#include <math.h>

#include <type_traits>

#include "ep_layer.cuh"

namespace ep {
namespace attn {

constexpr int kJoinThreads = 256;
constexpr int kMaxResident = 4; // CTAs a core, at most (the workspace is sized for this)
constexpr int kMaxGrid = 1024;  // CTAs of the main kernel, and so parts of one sequence

struct Plan {
    int grid;        // CTAs of the main kernel
    int split;       // 1: CTAs take equal shares of chunks and the join kernel runs; 0: whole (sequence, head) units
    int units;       // units of one sequence: cache heads * head blocks
    int blocks;      // head blocks per cache head
    unsigned page_mul, page_shift;  // i / page_size = (umulhi(i, page_mul) + ...) as page_of
    float out_scale; // of O / l
    float lift;      // the parts' sums are 2^lift times as large
    int by_unit;     // join blocks belong to units (else to the CTAs a unit began in)
};

// Quotient by the page size for 0 <= i < 2^31: with L = ceil(log2 d) and
// mul = ceil(2^(31 + L) / d), floor(i * mul / 2^(31 + L)) is exact (the error
// of mul, below 1, times i / 2^(31 + L) stays below 1 / d).
__device__ __forceinline__ int page_of(const Plan& p, int i) {
    return static_cast<int>((static_cast<uint64_t>(static_cast<unsigned>(i)) * p.page_mul) >> p.page_shift);
}

// Keys [low, end) of sequence b count; returns their number of chunks.
template <int CHUNK>
__device__ __forceinline__ int sequence(const AttentionArgs& a, int b, int& low, int& end) {
    const int most = a.max_pages * a.page_size;   // < 2^31, checked on the host
    end = min(max(a.lens[b], 0), most);
    low = a.window > 0 && end > a.window ? end - a.window : 0;
    return (end - low) / CHUNK + ((end - low) % CHUNK != 0);
}

// CTAs that share a work of W, and the first place of CTA i.
__device__ __forceinline__ int sharers(const Plan& p, int64_t W) {
    return static_cast<int>(min(static_cast<int64_t>(p.grid), W));
}
__device__ __forceinline__ int64_t share_start(int64_t W, int ctas, int i) { return W * i / ctas; }

// All sequences' units laid end to end, a unit of n chunks as kBegin + n places: to begin and to end one takes a CTA as
// long as kBegin chunks, and with sequences of very different lengths equal shares of the chunks alone let those with
// many short ones wait. (128 sequences of up to 8192 e4m3 keys, 8 heads: kBegin of 0, 1, 2, 3, 4:
// 187, 175, 173, 174, 176 us; 64 of up to 4096 bf16 keys: 98.1, 88.7, 89.1, 89.1, 89.8 us.)
constexpr int kBegin = 2;

struct Share {
    int64_t all;               // places in all (W)
    int64_t start, end;        // this CTA's
    int ctas;                  // CTAs that have one
    int seq[2];                // the sequences of its first and its last place
    int64_t before[2];         // places before those sequences
    int64_t chunks_before[2];  // chunks before them
};

// Computed by a prefix sum over the sequences; every thread gets the same result.
template <int THREADS, int CHUNK>
__device__ Share find_share(const AttentionArgs& a, const Plan& p) {
    __shared__ int64_t warp_sum[THREADS / 32], warp_chunks[THREADS / 32];
    __shared__ int64_t found_before[2], found_chunks[2];
    __shared__ int found[2];
    const int tid = threadIdx.x, lane = tid & 31;
    // (a.B may be 2^31 - 1: no sum here passes it)
    const int per = (a.B - 1) / THREADS + 1, first = min(a.B, tid * per), last = first + min(per, a.B - first);
    const auto places = [](int n) { return n > 0 ? n + kBegin : 0; };
    int64_t own = 0, own_chunks = 0;
    int low, end;
    for (int b = first; b < last; ++b) {
        const int n = sequence<CHUNK>(a, b, low, end);
        own += places(n);
        own_chunks += n;
    }
    int64_t scan = own, scan_chunks = own_chunks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(kFullMask, scan, o), c = __shfl_up_sync(kFullMask, scan_chunks, o);
        if (lane >= o) scan += v, scan_chunks += c;
    }
    if (lane == 31) warp_sum[tid >> 5] = scan, warp_chunks[tid >> 5] = scan_chunks;
    __syncthreads();
    int64_t total = 0, base = scan - own, chunks = scan_chunks - own_chunks;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < (tid >> 5)) base += warp_sum[w], chunks += warp_chunks[w];
        total += warp_sum[w];
    }
    Share s{};
    s.all = total * p.units;
    s.ctas = sharers(p, s.all);
    if (static_cast<int>(blockIdx.x) >= s.ctas) return s;   // the whole block
    s.start = share_start(s.all, s.ctas, blockIdx.x);
    s.end = share_start(s.all, s.ctas, blockIdx.x + 1);
    base *= p.units;
    chunks *= p.units;
    const int64_t ends[2] = {s.start, s.end - 1};
    if (ends[1] >= base && ends[0] < base + own * p.units) {
        for (int b = first; b < last; ++b) {
            const int n = sequence<CHUNK>(a, b, low, end);
            const int64_t behind = base + static_cast<int64_t>(places(n)) * p.units;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (ends[i] >= base && ends[i] < behind) found[i] = b, found_before[i] = base, found_chunks[i] = chunks;
            base = behind;
            chunks += static_cast<int64_t>(n) * p.units;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) s.seq[i] = found[i], s.before[i] = found_before[i], s.chunks_before[i] = found_chunks[i];
    return s;
}

// 16 bytes to shared memory, of which the first `real` (16 or 0) are read and the rest are zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int real) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void load_matrices_transposed(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void load_words(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
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
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Four e4m3 codes as two pairs of fp16 values, exactly. The instruction issues at the rate of the integer ones (2 clocks
// per warp and SM quarter), which would take seven for four codes.
__device__ __forceinline__ void e4m3_values(uint32_t codes, uint32_t& first, uint32_t& second) {
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.rn.f16x2.e4m3x2 %0, lo; cvt.rn.f16x2.e4m3x2 %1, hi; }"
        : "=r"(first), "=r"(second)
        : "r"(codes));
}
template <typename M>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    if constexpr (std::is_same_v<M, __half>) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// Weights that enter the products as M are 2^lift times as large.
template <typename M>
__host__ __device__ constexpr float lift() { return std::is_same_v<M, __half> ? 11.0f : 0.0f; }
template <typename M>
__device__ __forceinline__ float2 apart(uint32_t w) {
    if constexpr (std::is_same_v<M, __half>) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Left by each CTA of a split launch for the join kernel: the unit that began in it and goes on in later
// CTAs, if there is one (seq -1 otherwise).
struct Cut {
    int seq, unit, last;   // last CTA that holds a part
    int pad;
};

// What a ring slot holds, beside its keys and values.
struct SlotInfo {
    int unit;    // of its sequence; -1: no more chunks
    int seq;
    int chunk;   // index within (sequence, head)
    int chunks;  // of that sequence
};

// Byte offsets of a key's and a value's row.
struct alignas(16) RowAt {
    int64_t key, value;
};

// T: type of q and out. FP8: the cache is e4m3, else T. DP: head_dim rounded up
// to 64, 128 or 256 (the rest zeros). NT: eights of query heads per unit.
template <typename T, bool FP8, int DP, int NT>
struct Shape {
    using M = std::conditional_t<FP8, __half, T>;   // type of the products' operands
    static constexpr int kHeads = 8 * NT;
    // Warps: kKeyWarps shares of a chunk's keys times NT eights of heads. Codes have to be unpacked for half the
    // bytes, so an e4m3 cache gets more warps (8: 172.6 us, 4: 173.9 us for 128 sequences of up to 8192).
    static constexpr int kKeyWarps = FP8 && NT == 1 && DP <= 128 ? 8 : 4;
    static constexpr int kThreads = 32 * kKeyWarps * NT;
    static constexpr int kCacheBytes = FP8 ? 1 : 2;
    static constexpr int kRowBytes = DP * kCacheBytes;
    static constexpr int kPieces = kRowBytes / 16;          // 16-byte pieces of a row
    // Keys per chunk: 32 KB of keys and values (64 KB for 512-byte rows), 16 kTiles keys a warp.
    static constexpr int kChunk = kRowBytes <= 64 ? 256 : kRowBytes <= 128 ? 128 : 64;
    static constexpr int kTiles = kChunk / (16 * kKeyWarps);
    static constexpr int kTile = kChunk * kRowBytes;        // bytes of a chunk's keys, or values
    // Three slots: two CTAs a core keep 128 KB on the way, above what DRAM's latency needs at full rate.
    static constexpr int kSlots = 3;
    // An e4m3 kernel has no registers for the next segment's queries: they come to shared memory with its first chunk.
    // (Where that room would cost the second CTA a core, they are loaded when the segment begins.)
    static constexpr bool kQueriesShared = FP8 && NT == 1 && DP <= 128;
    static constexpr int kQueryWords = DP / 2 + 4;   // of a head

    struct Shared {
        alignas(128) unsigned char ring[kSlots][2][kTile];  // a used-up slot also serves the join of the warps
        RowAt at[kSlots + 1][kChunk];
        unsigned real[kSlots + 1][kChunk / 32];             // bit per key: it exists
        SlotInfo info[kSlots + 1];
        alignas(16) float top[kHeads][kKeyWarps], sum[kHeads][kKeyWarps];
        alignas(16) uint32_t q[kQueriesShared ? kSlots : 1][kQueriesShared ? kHeads : 1][kQueryWords];
    };
    static_assert(kKeyWarps * kHeads * DP * 4 <= 2 * kTile, "the join of the warps fits a slot");

    // Byte offset of 16-byte piece c of row r: pieces are exchanged within 8 (4) so that the 8
    // rows of a matrix load, and the 2 rows x 4 pieces of the e4m3 key loads, lie in different banks.
    static __device__ __forceinline__ int place(int r, int c) {
        if constexpr (kPieces >= 8) return r * kRowBytes + ((c ^ (((r & 1) << 2) | ((r >> 1) & 3))) << 4);
        return r * kRowBytes + ((c ^ ((r >> 1) & 3)) << 4);
    }
};

template <typename T, bool FP8, int DP, int NT>
__global__ void __launch_bounds__((Shape<T, FP8, DP, NT>::kThreads)) attention_kernel(AttentionArgs a, Plan p) {
    using S = Shape<T, FP8, DP, NT>;
    using M = typename S::M;
    extern __shared__ __align__(128) unsigned char shared_bytes[];
    typename S::Shared& sh = *reinterpret_cast<typename S::Shared*>(shared_bytes);
    constexpr int kSlots = S::kSlots, kInfos = kSlots + 1, kChunk = S::kChunk, kTiles = S::kTiles;
    constexpr int kWarps = S::kKeyWarps, kThreads = S::kThreads;
    dependent_entry();

    const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int warp = (tid >> 5) % kWarps, eight = (tid >> 5) / kWarps;   // share of the keys, of the heads
    const int D = a.head_dim, group = a.num_heads / a.num_kv_heads;
    Cut* cuts = static_cast<Cut*>(a.workspace);   // [grid], then the parts
    float* part = reinterpret_cast<float*>(cuts + p.grid);

    // ---- this CTA's chunks: `left` of them from (seq, unit, chunk) on
    int seq, unit, chunk, chunks, low, end;
    int left;   // (a share stays below 2^31 chunks: 2^31 keys a sequence and head at most, 64 a chunk)
    if (p.split) {
        const Share share = find_share<kThreads, kChunk>(a, p);
        // sequences without keys: zeros
        for (unsigned b = blockIdx.x; b < static_cast<unsigned>(a.B); b += gridDim.x) {
            if (sequence<kChunk>(a, b, low, end) > 0) continue;
            for (int i = tid; i < a.num_heads * D; i += kThreads)
                static_cast<T*>(a.out)[b * a.out_ld + i] = from_float<T>(0.0f);
            if (a.lse)
                for (int h = tid; h < a.num_heads; h += kThreads) a.lse[static_cast<int64_t>(b) * a.num_heads + h] = -INFINITY;
        }
        if (static_cast<int>(blockIdx.x) >= share.ctas) {
            if (tid == 0) cuts[blockIdx.x].seq = -1;
            return;
        }
        // its first chunk, the one behind its last, and the unit that holds the last place
        int64_t at[2], unit_at[2], chunk_at[2];
        int n[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            n[i] = sequence<kChunk>(a, share.seq[i], low, end);
            const int64_t in = (i == 0 ? share.start : share.end - 1) - share.before[i];
            unit_at[i] = in / (n[i] + kBegin);
            chunk_at[i] = max(in - unit_at[i] * (n[i] + kBegin) - kBegin + i, static_cast<int64_t>(0));
            at[i] = share.chunks_before[i] + unit_at[i] * n[i] + chunk_at[i];
        }
        left = static_cast<int>(at[1] - at[0]);
        if (tid == 0) {
            // the unit that holds this share's last chunk, if it began here and goes on behind it
            Cut cut{-1, 0, 0, 0};
            if (chunk_at[1] > 0 && chunk_at[1] < n[1] && at[1] - chunk_at[1] >= at[0]) {
                // the CTA whose share holds place x is the largest i with all i / ctas (rounded down) <= x
                const int64_t behind = share.before[1] + (unit_at[1] + 1) * (n[1] + kBegin);
                cut = {share.seq[1], static_cast<int>(unit_at[1]), static_cast<int>((behind * share.ctas - 1) / share.all), 0};
            }
            cuts[blockIdx.x] = cut;
        }
        if (left <= 0) return;   // (nothing but a unit's begin)
        seq = share.seq[0];
        chunks = sequence<kChunk>(a, seq, low, end);
        unit = static_cast<int>(unit_at[0]);
        chunk = static_cast<int>(chunk_at[0]);
    } else {
        const int64_t all = static_cast<int64_t>(a.B) * p.units;
        int64_t u = share_start(all, gridDim.x, blockIdx.x);
        const int64_t stop = share_start(all, gridDim.x, blockIdx.x + 1);
        seq = -1;
        left = 0;
        unit = chunk = chunks = low = end = 0;
        for (; u < stop; ++u) {
            const int b = static_cast<int>(u / p.units), w = static_cast<int>(u % p.units);
            int lo, en;
            const int n = sequence<kChunk>(a, b, lo, en);
            left += n;
            if (n > 0) {
                if (seq < 0) seq = b, unit = w, chunks = n, low = lo, end = en;
                continue;
            }
            // no keys: zeros
            const int h0 = w / p.blocks * group + w % p.blocks * S::kHeads, heads = min(S::kHeads, group - w % p.blocks * S::kHeads);
            for (int i = tid; i < heads * D; i += kThreads)
                static_cast<T*>(a.out)[b * a.out_ld + static_cast<int64_t>(h0) * D + i] = from_float<T>(0.0f);
            if (a.lse && tid < heads) a.lse[static_cast<int64_t>(b) * a.num_heads + h0 + tid] = -INFINITY;
        }
    }

    // ---- ring. A chunk's rows are looked up in the block table (look_up, which only issues the loads, and
    // note, which writes the rows' places) one chunk before copies() starts their way to the ring slot.
    // Rows by thread; with fewer rows than threads, other warps for every chunk.
    constexpr int kLookups = (kChunk + kThreads - 1) / kThreads;
    int located = 0;
    int note_slot = 0;
    int32_t page_id[kLookups];
    int page_place[kLookups];
    const auto look_row = [&](int k) {
        if constexpr (kChunk >= kThreads) return tid + k * kThreads;
        return (tid + located * kChunk) & (kThreads - 1);
    };
    const auto look_up = [&]() {
        if (located >= left) return;
        const int first = low + chunk * kChunk, here = min(kChunk, end - first);   // (first + kChunk may pass 2^31)
#pragma unroll
        for (int k = 0; k < kLookups; ++k) {
            page_id[k] = -1;
            const int r = look_row(k);
            if (r < here) {
                const int i = first + r, pg = page_of(p, i);
                page_id[k] = a.table[seq * a.table_ld + pg];
                page_place[k] = i - pg * a.page_size;
            }
        }
    };
    const bool alike = a.k_page == a.v_page && a.k_slot == a.v_slot && a.k_head == a.v_head;
    const auto note = [&]() {
        if (located < left) {
            const int h = unit / p.blocks;
#pragma unroll
            for (int k = 0; k < kLookups; ++k) {
                const int r = look_row(k);
                const bool real = page_id[k] >= 0 && page_id[k] < a.num_pages;
                if (r < kChunk) {   // (whole warps)
                    RowAt at{0, 0};
                    if (real) {
                        at.key = (page_id[k] * a.k_page + page_place[k] * a.k_slot + h * a.k_head) * S::kCacheBytes;
                        at.value = alike ? at.key : (page_id[k] * a.v_page + page_place[k] * a.v_slot + h * a.v_head) * S::kCacheBytes;
                    }
                    sh.at[note_slot][r] = at;
                    const unsigned mask = __ballot_sync(kFullMask, real);
                    if (lane == 0) sh.real[note_slot][r >> 5] = mask;
                }
            }
            if (tid == 0) sh.info[note_slot] = {unit, seq, chunk, chunks};
            if (++chunk == chunks) {
                chunk = 0;
                if (++unit == p.units && located + 1 < left) {
                    unit = 0;
                    do chunks = sequence<kChunk>(a, ++seq, low, end);
                    while (chunks == 0);
                }
            }
        } else if (tid == 0) {
            sh.info[note_slot].unit = -1;
        }
        ++located;
        note_slot = note_slot + 1 == kInfos ? 0 : note_slot + 1;
    };
    const auto all_real = [&](int slot) {
        unsigned m = ~0u;
#pragma unroll
        for (int i = 0; i < kChunk / 32; ++i) m &= sh.real[slot][i];
        return m == ~0u;
    };

    const int piece = tid % S::kPieces, piece_bytes = piece * 16 < D * S::kCacheBytes ? 16 : 0;   // a piece past head_dim: zeros
    // (a cache without pages may be NULL: then nothing is read, at any valid address)
    const unsigned char* key_base = static_cast<const unsigned char*>(a.k ? a.k : a.q) + (piece_bytes ? piece * 16 : 0);
    const unsigned char* value_base = static_cast<const unsigned char*>(a.v ? a.v : a.q) + (piece_bytes ? piece * 16 : 0);
    int copy_slot = 0, copy_info = 0;
    bool copied = false;
    const auto copies = [&]() {
        const SlotInfo in = sh.info[copy_info];
        if (in.unit >= 0) {
            if constexpr (S::kQueriesShared) {
                if (in.chunk == 0 || !copied) {
                    const int first_head = in.unit % p.blocks * S::kHeads;   // within the group
                    const T* q = static_cast<const T*>(a.q) + in.seq * a.q_ld + static_cast<int64_t>(in.unit / p.blocks * group + first_head) * D;
#pragma unroll
                    for (int i = tid; i < S::kHeads * DP / 2; i += kThreads) {
                        const int h = i / (DP / 2), d = i % (DP / 2) * 2;
                        const bool real = first_head + h < group && d < D;
                        copy4(smem_addr(&sh.q[copy_slot][h][d / 2]), real ? q + h * D + d : q, real ? 4 : 0);
                    }
                }
                copied = true;
            }
            constexpr int kRows = kThreads / S::kPieces;
            const int row = tid / S::kPieces;
            const uint32_t slot_addr = smem_addr(sh.ring[copy_slot][0]), first = slot_addr + S::place(row, piece);
            const auto to = [&](int r) {   // 8 rows on, the exchange of pieces is the same
                return kRows % 8 == 0 ? first + r * S::kRowBytes : slot_addr + S::place(r + row, piece);
            };
            if (all_real(copy_info)) {
#pragma unroll
                for (int r = 0; r < kChunk; r += kRows) {
                    const RowAt at = sh.at[copy_info][r + row];
                    copy16(to(r), key_base + at.key, piece_bytes);
                    copy16(to(r) + S::kTile, value_base + at.value, piece_bytes);
                }
            } else {
#pragma unroll 2
                for (int r = 0; r < kChunk; r += kRows) {
                    const RowAt at = sh.at[copy_info][r + row];
                    const int bytes = (sh.real[copy_info][(r + row) >> 5] >> ((r + row) & 31)) & 1 ? piece_bytes : 0;
                    copy16(to(r), key_base + at.key, bytes);
                    copy16(to(r) + S::kTile, value_base + at.value, bytes);
                }
            }
        }
        copy_commit();
        copy_slot = copy_slot + 1 == kSlots ? 0 : copy_slot + 1;
        copy_info = copy_info + 1 == kInfos ? 0 : copy_info + 1;
    };

#pragma unroll 1
    for (int i = 0; i < kSlots; ++i) {
        look_up();
        note();
    }
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < kSlots - 1; ++i) copies();

    // ---- the pass over the chunks
    // This thread's places in a slot's keys and values; the exchange of pieces repeats every 8 of them (128 bytes).
    constexpr int kPlaces = S::kPieces >= 8 ? 4 : 2;
    const uint32_t ring_at = smem_addr(sh.ring[0][0]);
    const int r0 = warp * 16 * kTiles;
    uint32_t key_place[kPlaces], value_place[kPlaces];
#pragma unroll
    for (int i = 0; i < kPlaces; ++i) {
        key_place[i] = FP8 ? S::place(r0 + g, (4 * i + t) % S::kPieces) : S::place(r0 + (lane & 15), 2 * i + (lane >> 4));
        value_place[i] = S::kTile + (FP8 ? S::place(r0 + (lane & 15), 2 * i + (lane >> 4))
                                         : S::place(r0 + (lane & 7) + ((lane >> 4) << 3), 2 * i + ((lane >> 3) & 1)));
    }
    float o[DP / 16][4];             // O^T: rows d, columns heads
    float top[2], sum[2], c2[2];     // of the warp's heads 2 t, 2 t + 1
    constexpr bool kQueriesAhead = !FP8 && DP <= 128;   // (an e4m3 kernel has no registers left for them)
    uint32_t qf[DP / 16][2], q_next[kQueriesAhead ? DP / 16 : 1][2];
    // Queries as the products' column operand: value pairs of step k for head g. An e4m3 key load brings 16
    // neighbouring values a lane, so its steps run through the head in that order.
    const auto load_queries = [&](const SlotInfo& in, uint32_t (&to)[DP / 16][2]) {
        const int in_group = in.unit % p.blocks * S::kHeads + 8 * eight + g;
        const T* q = static_cast<const T*>(a.q) + in.seq * a.q_ld + static_cast<int64_t>(in.unit / p.blocks * group + in_group) * D;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int d = FP8 ? (k / 4) * 64 + 16 * t + (k % 4) * 4 + 2 * j : 16 * k + 2 * t + 8 * j;
                to[k][j] = in_group < group && d < D ? *reinterpret_cast<const uint32_t*>(q + d) : 0u;
            }
    };
    int slot = 0, info = 0, first_chunk = 0;
    bool fresh = true;
    if constexpr (kQueriesAhead) {
        if (left > 0) load_queries(sh.info[0], q_next);
    }
    for (int n = 0; n < left; ++n) {
        copy_wait<kSlots - 2>();
        __syncthreads();
        const SlotInfo in = sh.info[info];
        copies();
        look_up();
        if (fresh || in.chunk == 0) {
            // a segment starts: its queries, fresh statistics
            fresh = false;
            first_chunk = in.chunk;
            if constexpr (kQueriesAhead) {
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) qf[k][0] = q_next[k][0], qf[k][1] = q_next[k][1];
            } else if constexpr (S::kQueriesShared) {
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    const uint2 w = *reinterpret_cast<const uint2*>(&sh.q[slot][g][(k / 4) * 32 + 8 * t + (k % 4) * 2]);
                    qf[k][0] = w.x, qf[k][1] = w.y;
                }
            } else {
                load_queries(in, qf);
            }
            float scale[2] = {1.0f, 1.0f};
            if constexpr (FP8) {
                // a power of two brings the head's largest query to [2^14, 2^15): fp16 then holds every one of
                // them to 2^-11, or to 2^-39 of the largest, whatever its type's range
                const auto value = [](uint32_t pair, int j) {
                    const uint16_t half = static_cast<uint16_t>(j ? pair >> 16 : pair);
                    return to_float(*reinterpret_cast<const T*>(&half));
                };
                float big = 0.0f;
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) big = fmaxf(big, fabsf(value(qf[k][j >> 1], j & 1)));
                big = fmaxf(big, __shfl_xor_sync(kFullMask, big, 1));
                big = fmaxf(big, __shfl_xor_sync(kFullMask, big, 2));
                const int e = big > 0.0f && big < INFINITY ? min(14 - ilogbf(big), 126) : 0;
                const float up = __int_as_float((e + 127) << 23), down = __int_as_float((127 - e) << 23);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                    for (int j = 0; j < 2; ++j) qf[k][j] = pack<M>(value(qf[k][j], 0) * up, value(qf[k][j], 1) * up);
                scale[0] = __shfl_sync(kFullMask, down, 8 * t);      // of heads 2 t and 2 t + 1
                scale[1] = __shfl_sync(kFullMask, down, 8 * t + 4);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                top[j] = -INFINITY;
                sum[j] = 0.0f;
                c2[j] = a.score_scale * scale[j] * 1.4426950408889634f;
            }
#pragma unroll
            for (int m = 0; m < DP / 16; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[m][j] = 0.0f;
        }
        if constexpr (kQueriesAhead) {
            // the next segment's queries, a chunk ahead: with short sequences each would wait for memory
            if (n + 1 < left) {
                const SlotInfo next = sh.info[info + 1 == kInfos ? 0 : info + 1];
                if (next.chunk == 0) load_queries(next, q_next);
            }
        }
        // S^T = K Q^T for this warp's keys r0 .. r0 + 16 kTiles - 1
        const uint32_t slot_at = ring_at + slot * (2 * S::kTile);
        float s[kTiles][4];
#pragma unroll
        for (int kt = 0; kt < kTiles; ++kt) s[kt][0] = s[kt][1] = s[kt][2] = s[kt][3] = 0.0f;
        if constexpr (FP8) {
#pragma unroll
            for (int j = 0; j < DP / 64; ++j)
#pragma unroll
                for (int kt = 0; kt < kTiles; ++kt) {
                    const uint32_t at = slot_at + key_place[j % 2] + j / 2 * 128 + kt * 16 * S::kRowBytes;
                    uint32_t xs[4], ys[4];
                    load_words(xs, at);
                    load_words(ys, at + 8 * S::kRowBytes);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t af[4];
                        e4m3_values(xs[i], af[0], af[2]);
                        e4m3_values(ys[i], af[1], af[3]);
                        multiply<M>(s[kt], af, qf[4 * j + i][0], qf[4 * j + i][1]);
                    }
                }
        } else {
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int kt = 0; kt < kTiles; ++kt) {
                    uint32_t af[4];
                    load_matrices(af, slot_at + key_place[k % kPlaces] + k / 4 * 128 + kt * 16 * S::kRowBytes);
                    multiply<M>(s[kt], af, qf[k][0], qf[k][1]);
                }
        }
        // softmax: this lane's keys r0 + 16 kt + g and + 8 (s[kt][0, 1] and [2, 3]) for two heads. The maximum that
        // the weights refer to follows the running one only when a score passes it by more than kSlack: most chunks
        // need no exchange between lanes. An fp16 weight is 2^kLift times as large, below 2^15 then, so that fp16 has
        // its full precision down to 2^-25 of the largest weight: many keys far below one of them still add up.
        constexpr float kSlack = std::is_same_v<M, __half> ? 4.0f : 8.0f, kLift = lift<M>();
#pragma unroll
        for (int kt = 0; kt < kTiles; ++kt)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[kt][j] *= c2[j & 1];
        if (!all_real(info)) {
#pragma unroll
            for (int kt = 0; kt < kTiles; ++kt) {
                const unsigned mask = sh.real[info][(r0 + 16 * kt) >> 5] >> ((r0 + 16 * kt) & 31);
                if (!((mask >> g) & 1)) s[kt][0] = s[kt][1] = -INFINITY;
                if (!((mask >> (g + 8)) & 1)) s[kt][2] = s[kt][3] = -INFINITY;
            }
        }
        bool over = false;
#pragma unroll
        for (int kt = 0; kt < kTiles; ++kt)
#pragma unroll
            for (int j = 0; j < 4; ++j) over |= s[kt][j] > top[j & 1] + kSlack;
        if (__any_sync(kFullMask, over)) {
            float fade[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float m = top[j];
#pragma unroll
                for (int kt = 0; kt < kTiles; ++kt) m = fmaxf(m, fmaxf(s[kt][j], s[kt][2 + j]));
                m = fmaxf(m, __shfl_xor_sync(kFullMask, m, 4));
                m = fmaxf(m, __shfl_xor_sync(kFullMask, m, 8));
                m = fmaxf(m, __shfl_xor_sync(kFullMask, m, 16));
                fade[j] = exp2_fast(top[j] - (m == -INFINITY ? 0.0f : m));
                top[j] = m;
                sum[j] *= fade[j];
            }
#pragma unroll
            for (int m = 0; m < DP / 16; ++m) o[m][0] *= fade[0], o[m][1] *= fade[1], o[m][2] *= fade[0], o[m][3] *= fade[1];
        }
        // A weight is taken as the sum of two: rounded once, its 8 or 11 bits would add as much error as the output's.
        // (Over an e4m3 cache the second product costs 3 %: 167.3 us with one, 172.6 with both, 128 sequences of up to 8192;
        // over a 16-bit one nothing.)
        constexpr int kWeightParts = 2;
        uint32_t pf[kTiles][kWeightParts][2];
        // (nothing seen yet: all weights 0)
        const float base[2] = {top[0] == -INFINITY ? 0.0f : top[0], top[1] == -INFINITY ? 0.0f : top[1]};
#pragma unroll
        for (int kt = 0; kt < kTiles; ++kt) {
            float pr[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) pr[j] = exp2_fast((s[kt][j] - base[j & 1]) + kLift);   // (in this order: at most kSlack + kLift)
            sum[0] += pr[0] + pr[2];
            sum[1] += pr[1] + pr[3];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t w = pack<M>(pr[2 * j], pr[2 * j + 1]);
                pf[kt][0][j] = transpose8x8(w);
                const float2 taken = apart<M>(w);
                pf[kt][1][j] = transpose8x8(pack<M>(pr[2 * j] - taken.x, pr[2 * j + 1] - taken.y));
            }
        }
        // O^T += V^T P^T
        if constexpr (FP8) {
#pragma unroll
            for (int m = 0; m < DP / 16; m += 2)
#pragma unroll
                for (int kt = 0; kt < kTiles; ++kt) {
                    // four 8 x 8 matrices of value pairs: keys 0-7 and 8-15 of 16 values, then of the next 16
                    uint32_t v[4];
                    load_matrices_transposed(v, slot_at + value_place[m / 2 % kPlaces] + m / 8 * 128 + kt * 16 * S::kRowBytes);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // bytes (key, value): (0,0) (0,1) (1,0) (1,1); row g of the tile is value 2 g, row g + 8 value 2 g + 1
                        const uint32_t u0 = __byte_perm(v[2 * i], 0, 0x3120), u1 = __byte_perm(v[2 * i + 1], 0, 0x3120);
                        uint32_t af[4];
                        e4m3_values(u0, af[0], af[1]);
                        e4m3_values(u1, af[2], af[3]);
#pragma unroll
                        for (int k = 0; k < kWeightParts; ++k) multiply<M>(o[m + i], af, pf[kt][k][0], pf[kt][k][1]);
                    }
                }
        } else {
#pragma unroll
            for (int m = 0; m < DP / 16; ++m)
#pragma unroll
                for (int kt = 0; kt < kTiles; ++kt) {
                    uint32_t af[4];
                    load_matrices_transposed(af, slot_at + value_place[m % kPlaces] + m / 4 * 128 + kt * 16 * S::kRowBytes);
#pragma unroll
                    for (int k = 0; k < kWeightParts; ++k) multiply<M>(o[m], af, pf[kt][k][0], pf[kt][k][1]);
                }
        }

        if (n + 1 == left || in.chunk + 1 == in.chunks) {
            // ---- the segment ends: join the warps, in their order, through the slot just used up, and write
            const int head0 = 8 * eight + 2 * t;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                sum[j] += __shfl_xor_sync(kFullMask, sum[j], 4);
                sum[j] += __shfl_xor_sync(kFullMask, sum[j], 8);
                sum[j] += __shfl_xor_sync(kFullMask, sum[j], 16);
                if (g == 0) sh.top[head0 + j][warp] = top[j];
            }
            __syncthreads();
            float* stage = reinterpret_cast<float*>(sh.ring[slot][0]);   // [kWarps][kHeads][DP]
            float fade[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float m = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sh.top[head0 + j][w]);
                fade[j] = exp2_fast(top[j] - (m == -INFINITY ? 0.0f : m));
                if (g == 0) sh.sum[head0 + j][warp] = sum[j] * fade[j];
            }
            // heads 2 t apart by a multiple of 32 words: value index exchanged by t * 8 to keep off one bank
#pragma unroll
            for (int m = 0; m < DP / 16; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int d = 16 * m + (FP8 ? 2 * g + (j >> 1) : g + 8 * (j >> 1));
                    stage[(warp * S::kHeads + head0 + (j & 1)) * DP + (d ^ (t << 3))] = o[m][j] * fade[j & 1];
                }
            __syncthreads();
            const int hb = in.unit % p.blocks;
            const int h0 = in.unit / p.blocks * group + hb * S::kHeads, heads = min(S::kHeads, group - hb * S::kHeads);
            const bool whole = first_chunk == 0 && in.chunk + 1 == in.chunks;
            // a part goes to this CTA's place 0 if the unit began in an earlier CTA, else to place 1
            float* to = part + (static_cast<int64_t>(blockIdx.x) * 2 + (first_chunk > 0 ? 0 : 1)) * S::kHeads * (DP + 2);
            for (int i = tid; i < heads * (DP / 4); i += kThreads) {
                const int h = i / (DP / 4), d = i % (DP / 4) * 4;
                const float* from = stage + h * DP + (d ^ (((h >> 1) & 3) << 3));
                float4 x = *reinterpret_cast<const float4*>(from);
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    const float4 y = *reinterpret_cast<const float4*>(from + w * S::kHeads * DP);
                    x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
                }
                float l = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) l += sh.sum[h][w];
                const auto largest = [&]() {
                    float m = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sh.top[h][w]);
                    return m;
                };
                if (whole) {
                    if (d < D) {
                        const float r = l == 0.0f ? 0.0f : p.out_scale / l;
                        T* out = static_cast<T*>(a.out) + in.seq * a.out_ld + static_cast<int64_t>(h0 + h) * D + d;
                        *reinterpret_cast<uint2*>(out) = make_uint2(pack<T>(x.x * r, x.y * r), pack<T>(x.z * r, x.w * r));
                    }
                    if (d == 0 && a.lse)
                        a.lse[static_cast<int64_t>(in.seq) * a.num_heads + h0 + h] =
                            l == 0.0f ? -INFINITY : 0.6931471805599453f * (largest() + (log2f(l) - lift<M>()));
                } else {
                    *reinterpret_cast<float4*>(to + h * DP + d) = x;
                    if (d == 0) to[S::kHeads * DP + 2 * h] = largest(), to[S::kHeads * DP + 2 * h + 1] = l;
                }
            }
            // (the slot and the statistics are written again only behind the next chunk's barrier)
        }
        slot = slot + 1 == kSlots ? 0 : slot + 1;
        info = info + 1 == kInfos ? 0 : info + 1;
        note();
    }
    copy_wait<0>();
}

// Joins the parts of the units that several CTAs shared, in the CTAs' order. With many sequences most units
// have few parts, and waves of blocks would cost more than the loads: blocks (i, *) serve the unit that
// began in CTA i and went on behind it, if there is one, the first of them all of its heads (another block
// each if the parts are many: up to kFew are joined from registers, which takes 64 sequences of up to 4096
// keys from 92.9 to 88.9 us). With few long sequences (by_unit) the parts are many: blocks (u, *) serve
// unit u, each 32 values of one head, its threads over values and parts.
template <typename T, int DP, int NT>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttentionArgs a, Plan p) {
    constexpr int kHeads = 8 * NT, kVecs = DP / 4, kLanes = kJoinThreads / kVecs, kPart = kHeads * (DP + 2), kFew = 8;
    __shared__ float weight[kMaxGrid];
    __shared__ float red[kJoinThreads / 32];
    __shared__ float4 acc[kJoinThreads];
    __shared__ float lsum[kJoinThreads / 8];
    __shared__ int found;
    dependent_entry();
    const int tid = threadIdx.x, D = a.head_dim;
    int i0 = blockIdx.x;
    if (p.by_unit) {
        if (tid == 0) found = -1;
        __syncthreads();
        for (int i = tid; i < p.grid; i += kJoinThreads) {
            const Cut c = static_cast<const Cut*>(a.workspace)[i];
            if (c.seq >= 0 && static_cast<int64_t>(c.seq) * p.units + c.unit == blockIdx.x) found = i;
        }
        __syncthreads();
        i0 = found;
        if (i0 < 0) return;
    }
    const Cut cut = static_cast<const Cut*>(a.workspace)[i0];
    if (cut.seq < 0) return;
    const int group = a.num_heads / a.num_kv_heads, first_head = cut.unit % p.blocks * kHeads;   // within the group
    const int parts = cut.last - i0 + 1;
    // CTA i0's place 1, the later ones' place 0
    const float* base = reinterpret_cast<const float*>(static_cast<const Cut*>(a.workspace) + p.grid) +
                        static_cast<int64_t>(i0) * 2 * kPart;
    const auto part = [&](int i) { return base + (i == 0 ? kPart : i * 2 * kPart); };
    const int vecs = p.by_unit ? 8 : kVecs, lanes = kJoinThreads / vecs, lane = tid / vecs;
    const int v = tid % vecs + (p.by_unit ? blockIdx.y % (DP / 32) * 8 : 0);
    const auto write = [&](int h, const float4& x, float m, float l) {
        const int head = cut.unit / p.blocks * group + first_head + h;
        if (4 * v < D) {
            const float r = l == 0.0f ? 0.0f : p.out_scale / l;
            T* out = static_cast<T*>(a.out) + cut.seq * a.out_ld + static_cast<int64_t>(head) * D + 4 * v;
            *reinterpret_cast<uint2*>(out) = make_uint2(pack<T>(x.x * r, x.y * r), pack<T>(x.z * r, x.w * r));
        }
        if (v == 0 && a.lse)
            a.lse[static_cast<int64_t>(cut.seq) * a.num_heads + head] = l == 0.0f ? -INFINITY : 0.6931471805599453f * (m + (log2f(l) - p.lift));
    };
    if (!p.by_unit && parts <= kFew) {
        if (blockIdx.y != 0) return;
        for (int h = lane; h < kHeads && first_head + h < group; h += kLanes) {
            float m = -INFINITY, tops[kFew], l = 0.0f;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f), y[kFew];
#pragma unroll
            for (int i = 0; i < kFew; ++i)
                if (i < parts) {
                    y[i] = *reinterpret_cast<const float4*>(part(i) + h * DP + 4 * v);
                    m = fmaxf(m, tops[i] = part(i)[kHeads * DP + 2 * h]);
                }
#pragma unroll
            for (int i = 0; i < kFew; ++i)
                if (i < parts) {
                    const float w = exp2_fast(tops[i] - (m == -INFINITY ? 0.0f : m));
                    x.x += w * y[i].x, x.y += w * y[i].y, x.z += w * y[i].z, x.w += w * y[i].w;
                    l += w * part(i)[kHeads * DP + 2 * h + 1];
                }
            write(h, x, m, l);
        }
        return;
    }
    const int h = p.by_unit ? blockIdx.y / (DP / 32) : blockIdx.y;
    if (first_head + h >= group) return;
    float m = -INFINITY;
    for (int i = tid; i < parts; i += kJoinThreads) {
        weight[i] = part(i)[kHeads * DP + 2 * h];
        m = fmaxf(m, weight[i]);
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, s));
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) m = fmaxf(m, red[w]);
    for (int i = tid; i < parts; i += kJoinThreads) weight[i] = exp2_fast(weight[i] - (m == -INFINITY ? 0.0f : m));
    __syncthreads();
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
#pragma unroll 8
    for (int i = lane; i < parts; i += lanes) {
        const float4 y = *reinterpret_cast<const float4*>(part(i) + h * DP + 4 * v);
        const float w = weight[i];
        x.x += w * y.x, x.y += w * y.y, x.z += w * y.z, x.w += w * y.w;
        l += w * part(i)[kHeads * DP + 2 * h + 1];
    }
    acc[tid] = x;
    if (tid % vecs == 0) lsum[lane] = l;
    __syncthreads();
    if (lane != 0) return;
    l = 0.0f;
    x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = 0; i < lanes; ++i) {
        l += lsum[i];
        const float4 y = acc[i * vecs + tid];
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    write(h, x, m, l);
}

// CTAs of the kernel that the current device holds at once; its shared memory limit is raised on the way.
// Fixed properties, looked up once per device (a race writes the same value twice).
template <typename Kernel>
cudaError_t resident_ctas(Kernel kernel, int threads, int smem, int sms, int* known, int* ctas) {
    constexpr int kDevices = 64;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < kDevices && (*ctas = __atomic_load_n(&known[dev], __ATOMIC_RELAXED)) > 0) return cudaSuccess;
    int per_sm = 0;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err == cudaSuccess) err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
    if (err != cudaSuccess) return err;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    *ctas = (per_sm < kMaxResident ? per_sm : kMaxResident) * sms;
    if (*ctas > kMaxGrid) *ctas = kMaxGrid;
    if (dev < kDevices) __atomic_store_n(&known[dev], *ctas, __ATOMIC_RELAXED);
    return cudaSuccess;
}

template <typename T, bool FP8, int DP, int NT>
cudaError_t launch_shape(const AttentionArgs& a, Plan p, int sms, cudaStream_t stream) {
    using S = Shape<T, FP8, DP, NT>;
    constexpr int smem = static_cast<int>(sizeof(typename S::Shared));
    static int known[64];
    cudaError_t err = resident_ctas(attention_kernel<T, FP8, DP, NT>, S::kThreads, smem, sms, known, &p.grid);
    if (err != cudaSuccess) return err;
    const int64_t all = static_cast<int64_t>(a.B) * p.units;
    const int64_t most = (static_cast<int64_t>(a.max_pages) * a.page_size + S::kChunk - 1) / S::kChunk;
    // More units than CTAs: equal shares of their chunks, unless all have one; whole units / shares, us: 1000 sequences of up
    // to 100 bf16 keys, 8 heads: 119 / 105, of up to 200: 159 / 128. Fewer units: shares, whose join is another launch, only
    // where units have many chunks; 16 sequences of up to 300 keys: 8.9 / 11.7, one of 450: 11.6 / 10.1.
    p.split = most > (all > p.grid ? 1 : 6);
    const int64_t useful = p.split ? all * (most + kBegin) : all;
    if (useful < p.grid) p.grid = static_cast<int>(useful > 0 ? useful : 1);
    err = launch_dependent(attention_kernel<T, FP8, DP, NT>, dim3(p.grid), dim3(S::kThreads), smem, stream, a, p);
    if (err != cudaSuccess || !p.split) return err;
    // (by CTA / by unit, us: 8 units of 131071 keys 87.4 / 86.6, one unit 28.6 / 24.3, 32 units of 8000 keys 31.8 / 34.3)
    p.by_unit = all * 16 <= p.grid;
    const dim3 join_grid = p.by_unit ? dim3(static_cast<unsigned>(all), 8 * NT * (DP / 32)) : dim3(p.grid, 8 * NT);
    return launch_dependent(join_kernel<T, DP, NT>, join_grid, dim3(kJoinThreads), 0, stream, a, p);
}

// Eights of query heads per unit: all of a cache head's, as far as the accumulators and the query
// fragments (3/8 dp registers a thread for each eight) fit the register file. More heads make several
// units, which read the keys and values again, mostly from L2.
inline int eights(int group, int dp) {
    const int nt = group <= 8 ? 1 : group <= 16 ? 2 : 4;
    return nt * dp <= 256 ? nt : 256 / dp;
}

template <typename T, bool FP8>
cudaError_t launch_type(const AttentionArgs& a, int sms, cudaStream_t stream) {
    const int dp = a.head_dim <= 64 ? 64 : a.head_dim <= 128 ? 128 : 256;
    const int group = a.num_heads / a.num_kv_heads, nt = eights(group, dp);
    Plan p{};
    p.blocks = (group + 8 * nt - 1) / (8 * nt);
    p.units = a.num_kv_heads * p.blocks;
    p.out_scale = FP8 ? a.v_scale : 1.0f;
    p.lift = lift<std::conditional_t<FP8, __half, T>>();
    int log = 0;
    while ((int64_t{1} << log) < a.page_size) ++log;
    p.page_shift = 31 + log;
    p.page_mul = static_cast<unsigned>(((uint64_t{1} << p.page_shift) + a.page_size - 1) / a.page_size);
    if (dp == 64)
        return nt == 1   ? launch_shape<T, FP8, 64, 1>(a, p, sms, stream)
               : nt == 2 ? launch_shape<T, FP8, 64, 2>(a, p, sms, stream)
                         : launch_shape<T, FP8, 64, 4>(a, p, sms, stream);
    if (dp == 128)
        return nt == 1 ? launch_shape<T, FP8, 128, 1>(a, p, sms, stream) : launch_shape<T, FP8, 128, 2>(a, p, sms, stream);
    return launch_shape<T, FP8, 256, 1>(a, p, sms, stream);
}

// One per (type, cache type), each in a translation unit of its own.
cudaError_t launch_bf16(const AttentionArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_bf16_e4m3(const AttentionArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_fp16(const AttentionArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_fp16_e4m3(const AttentionArgs& a, int sms, cudaStream_t stream);

}  // namespace attn
}  // namespace ep
