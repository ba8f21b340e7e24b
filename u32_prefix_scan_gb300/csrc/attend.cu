// attend.cu -- attention over a paged cache of 8-bit keys and values.
//
// With every query head of one key head beside each other (n tokens times the
// group), a row's scores are S^T = K Q^T and its results O^T = V^T P^T: the
// cache's codes are the A operand of mma.sync m16n8k16 and become f16 in
// registers (every code is an f16 number), eight query rows are its B.
//
// Every warp has a ring of stages in shared memory, each 16 tokens' keys and
// values: one TMA box each where 16 tokens lie in one page, else 16 bytes a lane
// and copy (cp.async), in the same swizzled places. The k axis of a product may
// be taken in any order, so a lane's 16 adjacent elements of a key serve four
// k-steps of S; the order of dimensions in O and of tokens in both is chosen so
// that no two lanes of an access meet in a bank.
//
// The softmax in one pass: per query a reference m for the sum l of
// p = 2^(s - m), and a second one, c, for what the values are weighted by,
// w = p * (scale of the value's block) * c, so that f16 holds the weights of
// blocks whose scales lie far apart. The heaviest w of the tile that sets c
// is 2^7; both stay until one exceeds 2^15 (p: 2^32), and only then the warp
// takes new maxima and rescales its sums. w is rounded to f16 (products and
// sums are f32): to 2^-11 of itself, or below f16's normal range by 2^-25, so by
// 2^-32 of the query's heaviest (p in l is not rounded, so what is lost here is
// lost from the result). The codes it meets have 4 bits, and the result's type 8
// or 11. (With a heaviest of 1 and a limit of 2^8, which take the same time, tokens
// below 2^-25 of it were lost, by the thousand beside one that takes all.)
//
// The work of all rows is one line of units (a tile of 16 tokens for each of a
// block's eight warps: of up to four heads beside each other, so that a page's
// memory is read 512 bytes at a time), cut into equal pieces for the blocks,
// however ragged the rows are. Where a tile of queries falls to several blocks,
// the one that comes last joins their partial sums, in order.
//
// Measured on GB300s, launches back to back: 64 ragged rows of up to 8192
// tokens of 8 heads of 128, groups of eight, 108 to 111 us (540 MB, 4.9 TB/s);
// heads of 64, 80, 96 71, 103, 95 us, 4 heads of 256 101 us, groups of sixteen
// 152 us (4 heads of 256: 163, read twice). 16384 tokens each 374 us (5.8 TB/s),
// two rows of 200000 tokens 153 to 167 us, 33 rows of drafts (up to five tokens,
// groups of seven, heads of 64, pages of 20) 32 us, one row of 4000 tokens 14 us.
// Bound by the reading of the cache, unevenly: some groups of SMs read 18 %
// slower than the rest and end last; the same grid with its copies alone takes
// 100 of the 111 us. A block's fixed part (queries, page numbers, the first
// copies, the join) is some 10 us of latency, which is what one row takes. Many
// queries a row are not what it is for: each 16 of a key head read the cache
// again, and 5 rows of 8192 tokens with 256 new ones in the mean take 2.8 ms.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvcache.cuh"
#include "launch.cuh"

namespace u32scan {

constexpr int kTile = 16;                 // tokens of a warp at a time
constexpr int kMaxDim = 256;
constexpr unsigned int kMaxBlocks = 304;  // two on each of a GB300's 152 SMs; bounds the workspace
constexpr int kWarps = 8, kThreads = 32 * kWarps;
// What a tile of queries takes beside its units, in units (with 2, 4, 5, 6, 8: 64 ragged rows of up to 8192 tokens 114,
// 107, 108, 107, 106 us, drafts 33.4, 32.3, 31.9, 31.8, 32.9, two rows of 200000 156, 155, 154, 152, 154), and the least
// piece (with 2, 3, 4 units: one row of 4000 tokens 13.7, 14.5, 15.0 us, drafts 31.9; parts to join are the more of, the less).
constexpr uint32_t kTileCost = 5;
constexpr uint64_t kLeastUnits = 3;
constexpr int kMaxElements = 4096;        // heads x queries x dimensions of a tile of queries
constexpr int kMaxPairs = 64;             // its heads x queries
constexpr float kNoMax = -0x1.fffffep127f;  // the least f32: every finite score takes its place
constexpr float kHeaviest = 0x1p7f, kMaxWeight = 0x1p15f, kMaxAbove = 32.0f;

struct AttendArgs {
    RowsView v;
    const uint8_t *keys, *values;
    const float *key_scales, *value_scales;
    uint64_t page_stride, token_stride, head_stride, scale_stride;
    Divisor block_tokens, group;
    uint32_t heads, dim;
    const void *queries;
    void *out;
    uint64_t q_token_stride, q_head_stride, out_token_stride, out_head_stride;
    uint32_t pair_heads;  // log2 of the key heads that a block's warps have beside each other: 0, 1 or 2
    float scale;  // times log2(e)
    bool wide_blocks;  // a scale's block is a multiple of 16 tokens: 16 in one page have one scale
    WsHeader *hdr;
    float4 *partial;     // [2 blocks][heads][sums of a tile of queries, as the lanes hold them]
    float2 *partial_ml;  // [2 blocks][heads][queries of a tile]: reference and sum
    unsigned long long *arrived, clear_words;  // the workspace's tile words
};

template <typename T>
struct QType;
template <>
struct QType<__half> {
    static __device__ __forceinline__ float2 two(uint32_t x) { return __half22float2(*reinterpret_cast<__half2 *>(&x)); }
    static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <>
struct QType<__nv_bfloat16> {
    static __device__ __forceinline__ float2 two(uint32_t x) {
        return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    }
    static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Two codes to f16.
__device__ __forceinline__ uint32_t codes_lo(uint32_t x) {
    uint32_t y;
    asm("{.reg .b16 a, b; mov.b32 {a, b}, %1; cvt.rn.f16x2.e4m3x2 %0, a;}" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t x) {
    uint32_t y;
    asm("{.reg .b16 a, b; mov.b32 {a, b}, %1; cvt.rn.f16x2.e4m3x2 %0, b;}" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void *from, bool real) {
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(real ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(BYTES),
                     "r"(real ? BYTES : 0)
                     : "memory");
}

// 16 tokens of one head of one page, up to 128 dimensions; what lies past the
// dimensions or is no page's arrives as zeros.
__device__ __forceinline__ void copy_box(uint32_t to, const CUtensorMap *map, uint32_t bar, int d, int head, int slot,
                                         int page) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::
            "r"(to), "l"(map), "r"(bar), "r"(d), "r"(head), "r"(slot), "r"(page)
        : "memory");
}

template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A row's share of the line of units.
struct RowUnits {
    int64_t begin, n;   // its tokens of the call
    int64_t len;        // lens[s], not below 0
    uint32_t limit;     // tokens that the table can place
    uint32_t units, tiles;
};

// A unit is a tile of 16 tokens for each warp: the warps take 1, 2 or 4 heads, and of each as many tiles beside each
// other as there are warps left.
__device__ __forceinline__ uint32_t unit_of(const AttendArgs &a) { return (uint32_t)(kTile * kWarps) >> a.pair_heads; }

__device__ __forceinline__ RowUnits row_units(const AttendArgs &a, uint64_t s, uint32_t tile_rows) {
    RowUnits r;
    tokens_of(a.v, s, &r.begin, &r.n);
    const int32_t len = a.v.lens[s];
    r.len = len;
    const uint64_t placed = a.v.pages == 0 ? 0 : a.v.width * a.v.page_tokens.d;
    r.limit = (uint32_t)(len <= 0 ? 0 : (uint64_t)len < placed ? (uint64_t)len : placed);
    const uint32_t unit_tokens = unit_of(a);
    r.units = r.n == 0 ? 0u : r.limit <= unit_tokens ? 1u : (r.limit - 1) / unit_tokens + 1;
    r.tiles = (uint32_t)((r.n * a.group.d + tile_rows - 1) / tile_rows);
    return r;
}

// The sizes of one kernel: DP dimensions (dim, up to it), 8 * NT queries. A
// stage holds 16 rows of keys, then of values, of 128 bytes (dimensions past
// 128 in 16 rows more) or 64, 16-byte chunks swizzled as TMA does it.
template <int DP, int NT>
struct Shape {
    static constexpr int kRows = 8 * NT;
    static constexpr bool kSmall = DP * NT <= 128;  // 128 registers a thread do, else 255
    static constexpr uint32_t kMostPaired = kSmall ? 2 : 1;  // log2 of the heads beside each other
    static constexpr int kVectors = NT * (DP / 16) * 32;     // a tile's sums, four at a time
    static constexpr int kPitch = DP >= 128 ? 128 : 64;
    static constexpr int kHalves = DP / kPitch;
    static constexpr int kHalfBytes = kTile * kPitch;
    static constexpr int kKeyChunks = DP / 64;                    // of 16 bytes, for each of a lane's two keys
    static constexpr int kValueBytes = DP >= 128 ? 16 : 8;        // for each of a lane's four values and each half
    static constexpr int kBlocks = kSmall ? 2 : 1;                // an SM
    static constexpr int kStageBytes = DP * 2 * kTile;            // of a warp
    static constexpr int kStages = (228 * 1024 / kBlocks - 4096) / (kWarps * (kStageBytes + 128));
    static constexpr int kRing = kStages * kWarps * kStageBytes;
    static constexpr int kShared = kRing + kStages * kWarps * (128 + 8) + 1024;  // scales, barriers, alignment
    static_assert(kWarps * (kRows * DP + 2 * kRows) * 4 <= kRing, "the warps' sums take the ring's place");
    static_assert((kRows * DP << kMostPaired) <= kMaxElements && (kRows << kMostPaired) <= kMaxPairs, "the workspace's slots");
    static_assert(kBlocks * (kShared + 1024 + 256) <= 228 * 1024, "blocks of an SM");

    // Where 16-byte chunk c of row r lies in a half.
    static __device__ __forceinline__ uint32_t chunk(uint32_t r, uint32_t c) {
        return r * kPitch + ((DP >= 128 ? c ^ (r & 7) : c ^ (r >> 1 & 3)) << 4);
    }
    // The row of token k < 8 of a product's order (k + 8: that row + 8). Keys are read by rows 2 i, 2 i + 1 of
    // the order at a time, values by rows 0, 2, 4, 6 or 1, 3, 5, 7: either way all 32 banks serve.
    static __device__ __forceinline__ uint32_t token(uint32_t k) {
        return DP >= 128 ? k >> 1 | (k & 1) << 2 : 0x65742130u >> 4 * k & 7;
    }
};

// The line of all rows' units, and its equal pieces, one for each block.
struct Line {
    uint64_t total, per;
    uint64_t share, until;  // of row threadIdx.x: its units, and those up to its end

    __device__ static uint64_t share_of(const AttendArgs &a, uint64_t s, uint32_t tile_rows) {
        if (s >= a.v.rows) return 0;
        const RowUnits r = row_units(a, s, tile_rows);
        return r.units ? ((uint64_t)r.units + kTileCost) * r.tiles * (a.heads >> a.pair_heads) : 0;
    }

    // The sum of x up to this thread's, and (into *all) over the block.
    __device__ static uint64_t scan(uint64_t x, uint64_t *sums, uint64_t *all) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        for (int d = 1; d < 32; d <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        __syncthreads();  // the sums were read
        if (lane == 31) sums[warp] = x;
        __syncthreads();
        *all = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) x += sums[w];
            *all += sums[w];
        }
        return x;
    }

    __device__ void measure(const AttendArgs &a, uint32_t tile_rows, uint64_t *sums) {
        share = share_of(a, threadIdx.x, tile_rows);
        uint64_t mine = share;
        for (uint64_t s = threadIdx.x + kThreads; s < a.v.rows; s += kThreads) mine += share_of(a, s, tile_rows);
        until = scan(mine, sums, &total);  // (a row's, where there is one for each thread)
        per = (total + gridDim.x - 1) / gridDim.x;
        if (per < kLeastUnits) per = kLeastUnits;
    }

    // The row that holds place `at` of the line, and which of its units that is.
    __device__ void locate(const AttendArgs &a, uint32_t tile_rows, uint64_t at, uint64_t *sums, uint64_t *found) const {
        if (a.v.rows <= kThreads) {
            if (at < until && at >= until - share) found[0] = threadIdx.x, found[1] = at - (until - share);
        } else {
            uint64_t before = 0, all;
            for (uint64_t base = 0; base < a.v.rows && before <= at; base += kThreads, before += all) {
                const uint64_t x = share_of(a, base + threadIdx.x, tile_rows), end = before + scan(x, sums, &all);
                if (at < end && at >= end - x) found[0] = base + threadIdx.x, found[1] = at - (end - x);
            }
        }
        __syncthreads();
    }
};

// Counts a block in at a word of the workspace: tags grow from launch to launch (and the words are cleared before they
// start again), so the larger of the word and this launch's tag is a count of this launch. (Of 63 blocks at a time
// each takes its turn once; by compare-and-swap, where one of all that try succeeds, they took 50 us.)
__device__ __forceinline__ uint32_t count_arrival(unsigned long long *word, unsigned long long tag) {
    atomicMax(word, tag);
    return (uint32_t)atomicAdd(word, 1ull) + 1u;
}

// Row r of a tile of queries: its token of the row and query head of the key head.
__device__ __forceinline__ bool query_of(const AttendArgs &a, int64_t n, uint32_t tile, uint32_t tile_rows,
                                         uint32_t r, uint32_t *token, uint32_t *j) {
    const uint32_t f = tile * tile_rows + r;  // (tokens times the group stay below 2^31)
    if (f >= (uint64_t)n * a.group.d) return false;
    *token = divide(f, a.group);
    *j = f - *token * a.group.d;
    return true;
}

// Writes vector v of head h's sums of a tile of queries: x[2 k + j] is dimension d + k of query 2 t + j.
template <typename T, int DP, int NT>
__device__ __forceinline__ void write_out(const AttendArgs &a, const RowUnits &row, uint32_t head, uint32_t tile, uint32_t v,
                                          const float4 &x, const float (&sum)[2]) {
    using S = Shape<DP, NT>;
    const uint32_t lane = v % 32, i = v / 32 % (DP / 16), nt = v / 32 / (DP / 16), g = lane >> 2, t = lane & 3;
    constexpr uint32_t kPer = S::kValueBytes / 2;  // vectors of a half
    const uint32_t d = S::kPitch * (i / kPer) + S::kValueBytes * (DP >= 128 ? g >> 1 | (g & 1) << 2 : g) + 2 * (i % kPer);
    if (d >= a.dim) return;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t token, q;
        if (!query_of(a, row.n, tile, S::kRows, nt * 8 + 2 * t + j, &token, &q)) continue;
        T *to = static_cast<T *>(a.out) + (uint64_t)(row.begin + token) * a.out_token_stride +
                ((uint64_t)head * a.group.d + q) * a.out_head_stride + d;
        const float y[2] = {j ? x.y : x.x, j ? x.w : x.z};
        to[0] = QType<T>::put(sum[j] == 0.0f ? 0.0f : y[0] / sum[j]);
        to[1] = QType<T>::put(sum[j] == 0.0f ? 0.0f : y[1] / sum[j]);
    }
}

// Joins the parts of a tile of queries that blocks first .. first + parts - 1 left, in order: each part's reference and
// sum into shared memory, their maxima, sums and weights, then the parts, weighted, a vector of four a thread.
template <typename T, int DP, int NT>
__device__ void join_parts(const AttendArgs &a, uint8_t *shared, uint64_t first, uint32_t parts, const RowUnits &row,
                           uint32_t group, uint32_t tile) {
    using S = Shape<DP, NT>;
    const uint32_t pairs = S::kRows << a.pair_heads;  // of a head and a query
    float2 *const total = reinterpret_cast<float2 *>(shared), *const each = total + kMaxPairs;
    const uint32_t room = (S::kRing / sizeof(float2) - kMaxPairs) / pairs;  // parts at a time
    auto from = [&](uint32_t part) { return (2 * (first + part) + (part == 0 ? 1 : 0)) << a.pair_heads; };
    auto fetch = [&](uint32_t p0, uint32_t n) {
        __syncthreads();
#pragma unroll 4
        for (uint32_t e = threadIdx.x; e < n * pairs; e += kThreads)
            each[e] = __ldcg(a.partial_ml + from(p0 + e / pairs) * S::kRows + e % pairs);
        __syncthreads();
    };
    auto weigh = [&](uint32_t n) {
        for (uint32_t i = threadIdx.x; i < pairs; i += kThreads) {
            const float top = total[i].x;
#pragma unroll 4
            for (uint32_t k = 0; k < n; ++k) each[k * pairs + i].x = exp2_approx(each[k * pairs + i].x - top);
        }
        __syncthreads();
    };
    for (uint32_t p0 = 0; p0 < parts; p0 += room) {
        const uint32_t n = parts - p0 < room ? parts - p0 : room;
        fetch(p0, n);
        for (uint32_t i = threadIdx.x; i < pairs; i += kThreads) {
            const float2 was = p0 ? total[i] : make_float2(kNoMax, 0.0f);
            float top = was.x;
#pragma unroll 4
            for (uint32_t k = 0; k < n; ++k) top = fmaxf(top, each[k * pairs + i].x);
            float sum = was.y * exp2_approx(was.x - top);
#pragma unroll 4
            for (uint32_t k = 0; k < n; ++k) sum += each[k * pairs + i].y * exp2_approx(each[k * pairs + i].x - top);
            total[i] = make_float2(top, sum);
        }
    }
    if (parts <= room) weigh(parts);
    // 16 parts' loads under way at a time: with the cache's copies in the same memory a load takes some 1.4 us
    constexpr uint32_t kAtOnce = 16;
    const uint32_t vectors = S::kVectors << a.pair_heads;  // (a multiple of the threads or, of few, of a warp)
    for (uint32_t e0 = 0; e0 < vectors; e0 += kThreads) {
        const uint32_t e = e0 + threadIdx.x, in = e % S::kVectors;
        const uint32_t pair = e / S::kVectors * S::kRows + in / (DP / 16 * 32) * 8 + 2 * (e & 3);
        float4 x = {0.0f, 0.0f, 0.0f, 0.0f};
        for (uint32_t p0 = 0; p0 < parts; p0 += room) {
            const uint32_t n = parts - p0 < room ? parts - p0 : room;
            if (parts > room) {
                fetch(p0, n);
                weigh(n);
            }
            if (e >= vectors) continue;
            for (uint32_t k0 = 0; k0 < n; k0 += kAtOnce) {
                float4 y[kAtOnce];
#pragma unroll
                for (uint32_t k = 0; k < kAtOnce; ++k)
                    y[k] = k0 + k < n ? __ldcg(a.partial + from(p0 + k0 + k) * S::kVectors + e) : float4{0, 0, 0, 0};
#pragma unroll
                for (uint32_t k = 0; k < kAtOnce; ++k) {
                    if (k0 + k >= n) break;
                    const float b0 = each[(k0 + k) * pairs + pair].x, b1 = each[(k0 + k) * pairs + pair + 1].x;
                    x.x += y[k].x * b0;
                    x.y += y[k].y * b1;
                    x.z += y[k].z * b0;
                    x.w += y[k].w * b1;
                }
            }
        }
        if (e >= vectors) continue;
        const float sum[2] = {total[pair].y, total[pair + 1].y};
        write_out<T, DP, NT>(a, row, (group << a.pair_heads) + e / S::kVectors, tile, in, x, sum);
    }
}

// BOX: 16 tokens from a multiple of 16 on lie in one page.
template <typename T, int DP, int NT, bool BOX>
__global__ void __launch_bounds__(kThreads, Shape<DP, NT>::kBlocks)
attend_kernel(const AttendArgs a, const __grid_constant__ CUtensorMap key_map,
              const __grid_constant__ CUtensorMap value_map) {
    using S = Shape<DP, NT>;
    extern __shared__ uint8_t unaligned[];
    const uint32_t ring_at = (smem_u32(unaligned) + 1023u) & ~1023u;
    uint8_t *const ring = unaligned + (ring_at - smem_u32(unaligned));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t g = lane >> 2, t = lane & 3;
    // stage i of this warp: codes at codes_at + i * kNextStage, scales (16 of keys, 16 of values) and barrier behind the ring
    constexpr uint32_t kNextStage = kWarps * S::kStageBytes, kValuesAt = DP * kTile;
    const uint32_t codes_at = ring_at + warp * S::kStageBytes;
    const uint32_t scales_at = ring_at + S::kRing + warp * S::kStages * 128 + lane * 4;
    const uint32_t bars_at = ring_at + S::kRing + S::kStages * kWarps * 128 + warp * S::kStages * 8;
    if (BOX && lane < S::kStages) mbar_init(bars_at + lane * 8, 1);
    fence_mbar_init();
    __shared__ uint64_t sums64[kWarps], found[2];
    __shared__ uint32_t last_here;
    uint32_t epoch, nth_block = 0;
    if (threadIdx.x == 0) last_here = ld_relaxed_u32(&a.hdr->epoch);
    Line line;
    line.measure(a, S::kRows, sums64);  // (block barriers within)
    epoch = last_here;
    // (every block has read the epoch when it counts itself; what the count was is looked at in the end)
    if (threadIdx.x == 0) nth_block = atom_add_acq_rel(&a.hdr->counter, 1u);
    const uint32_t unit_tokens = unit_of(a), warp_head = warp & ((1u << a.pair_heads) - 1), warp_tile = warp >> a.pair_heads;
    // what the lane reads of a stage: its first key and two values
    uint32_t key_at = S::chunk(S::token(g), t), value_at[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t r = S::token(2 * t + k);
        value_at[k] = kValuesAt + (DP >= 128 ? S::chunk(r, g >> 1 | (g & 1) << 2) : S::chunk(r, g >> 1) + 8 * (g & 1));
    }
    asm volatile("" : "+r"(key_at), "+r"(value_at[0]), "+r"(value_at[1]));  // kept, not computed in every turn
    uint32_t stage = 0, parity = 0;  // of the tile that is consumed next
    uint32_t in_flight = 0;
    bool gave_up = false;
    uint64_t at_line = blockIdx.x * line.per, left = at_line < line.total ? min(line.per, line.total - at_line) : 0;
    uint64_t row_at = 0;
    RowUnits row = {};
    uint32_t skip = 0, tile = 0, group = 0;  // group: of heads; skip: what of the tile of queries lies before this piece
    if (left > 0) {
        line.locate(a, S::kRows, at_line, sums64, found);
        row_at = found[0];
        row = row_units(a, row_at, S::kRows);
        const uint32_t width = row.units + kTileCost;  // of a tile of queries on the line
        skip = (uint32_t)(found[1] % width);
        tile = (uint32_t)(found[1] / width % row.tiles);
        group = (uint32_t)(found[1] / width / row.tiles);
    }
    while (left > 0) {
        // units [unit, unit + n_units) of the tile
        const uint64_t here = (uint64_t)row.units + kTileCost - skip;
        const uint32_t taken = (uint32_t)(left < here ? left : here);
        const uint32_t unit = skip > kTileCost ? skip - kTileCost : 0u;
        const uint32_t n_units = skip + taken > kTileCost ? skip + taken - kTileCost - unit : 0u;
        if (n_units > 0) {
            const uint32_t head = (group << a.pair_heads) + warp_head;
            // queries: lane (g, t) holds elements 64 c + 16 t .. + 15 of row g of each eight
            uint32_t q[NT][S::kKeyChunks * 8];
            float factor[NT][2];  // of the queries 2 t, 2 t + 1: what makes a product a score
            int32_t last[NT][2];  // and the last position they see
            int64_t first_last, last_last;
            {
                const int64_t before = row.len - row.n;
                const uint32_t f0 = tile * S::kRows, f1 = f0 + S::kRows - 1, all = (uint32_t)row.n * a.group.d;
                first_last = before + (int64_t)divide(f0, a.group);
                last_last = before + (int64_t)divide(f1 < all ? f1 : all - 1, a.group);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t token = 0, j = 0;
                    const bool real = query_of(a, row.n, tile, S::kRows, nt * 8 + g, &token, &j);
                    const T *x = static_cast<const T *>(a.queries) + (uint64_t)(row.begin + token) * a.q_token_stride +
                                 ((uint64_t)head * a.group.d + j) * a.q_head_stride;
                    uint4 raw[S::kKeyChunks][2];
                    float top = 0.0f;
#pragma unroll
                    for (int c = 0; c < S::kKeyChunks; ++c)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t d = 64 * c + 16 * t + 8 * h;
                            raw[c][h] = real && d < a.dim ? __ldg(reinterpret_cast<const uint4 *>(x + d)) : uint4{0, 0, 0, 0};
                            const uint32_t w[4] = {raw[c][h].x, raw[c][h].y, raw[c][h].z, raw[c][h].w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 v = QType<T>::two(w[i]);
                                top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
                            }
                        }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // the largest to 2^8 .. 2^9: f16 then holds what is 2^-22 of it in full
                    int up = 8 - ((int)(__float_as_uint(top) >> 23) - 127);
                    up = up > 110 ? 110 : up;
                    const float by = __uint_as_float((uint32_t)(up + 127) << 23);
                    const float back = __uint_as_float((uint32_t)(127 - up) << 23) * a.scale;
#pragma unroll
                    for (int c = 0; c < S::kKeyChunks; ++c)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t w[4] = {raw[c][h].x, raw[c][h].y, raw[c][h].z, raw[c][h].w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 v = QType<T>::two(w[i]);
                                q[nt][c * 8 + h * 4 + i] = pack_half(v.x * by, v.y * by);
                            }
                        }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        factor[nt][k] = __shfl_sync(0xffffffffu, back, 8 * t + 4 * k);
                        last[nt][k] = (int32_t)before + (int32_t)__shfl_sync(0xffffffffu, token, 8 * t + 4 * k);
                    }
                }
            }
            const uint32_t limit = last_last + 1 < (int64_t)row.limit ? (uint32_t)(last_last + 1 > 0 ? last_last + 1 : 0)
                                                                      : row.limit;
            const int32_t whole_until = (int32_t)(first_last - (kTile - 1) < -1 ? -1 : first_last - (kTile - 1));
            const int32_t *table = a.v.table + row_at * a.v.table_stride;

            float o[DP / 16][NT][4], m[NT][2], l[NT][2], c_ref[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < DP / 16; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[i][nt][k] = 0.0f;
#pragma unroll
                for (int k = 0; k < 2; ++k) m[nt][k] = kNoMax, l[nt][k] = 0.0f, c_ref[nt][k] = 1.0f;
            }

            // the warp's tiles: 16 tokens from (unit + i) * unit_tokens + warp_tile * 16 on
            const uint64_t start = (uint64_t)unit * unit_tokens + warp_tile * kTile;
            const uint32_t most = start < limit ? (uint32_t)(limit - start - 1) / unit_tokens + 1 : 0u;
            const uint32_t n_tiles = n_units < most ? n_units : most;
            // Starts the copies of tile i into a stage. BOX: lane j knows the pages of tile 32 n + j; else lane j (and
            // 16 + j) those of token j of the next tile.
            int32_t page = -1;
            uint32_t slot = 0;
            uint64_t scale_from = 0;
            uint32_t absent = 0;  // bit i: the tile in stage i has no page
            auto look_up = [&](uint32_t i) {
                const uint64_t at = start + (BOX ? 0 : lane & 15) + (uint64_t)(BOX ? i + lane : i) * unit_tokens;
                const uint32_t nth = divide((uint32_t)at, a.v.page_tokens);
                const int32_t p = (BOX ? i + lane : i) < n_tiles && at < limit ? __ldg(table + nth) : -1;
                slot = (uint32_t)at - nth * a.v.page_tokens.d;
                page = p >= 0 && (uint64_t)p < a.v.pages ? p : -1;
                if (BOX) scale_from = (uint64_t)(uint32_t)page * a.scale_stride +
                                      (a.wide_blocks ? (uint64_t)divide(slot, a.block_tokens) * a.heads : 0) + head;
            };
            auto issue = [&](uint32_t i, uint32_t to_stage) {
                const uint32_t to = codes_at + to_stage * kNextStage;
                if (BOX) {
                    if (i % 32 == 0) look_up(i);
                    const int32_t its_page = __shfl_sync(0xffffffffu, page, i % 32);
                    const uint32_t its_slot = __shfl_sync(0xffffffffu, slot, i % 32);
                    uint64_t from = __shfl_sync(0xffffffffu, scale_from, i % 32);
                    absent = its_page < 0 ? absent | 1u << to_stage : absent & ~(1u << to_stage);
                    if (lane == 0 && !gave_up) {
                        const uint32_t bar = bars_at + to_stage * 8;
                        if (its_page < 0) {
                            mbar_arrive(bar);
                        } else {
                            mbar_arrive_expect_tx(bar, S::kStageBytes);
#pragma unroll
                            for (int h = 0; h < S::kHalves; ++h) {
                                copy_box(to + h * S::kHalfBytes, &key_map, bar, S::kPitch * h, (int)head, (int)its_slot, its_page);
                                copy_box(to + kValuesAt + h * S::kHalfBytes, &value_map, bar, S::kPitch * h, (int)head, (int)its_slot,
                                         its_page);
                            }
                        }
                    }
                    in_flight += gave_up ? 0 : 1;
                    if (its_page >= 0) {
                        if (!a.wide_blocks) from += (uint64_t)divide(its_slot + (lane & 15), a.block_tokens) * a.heads;
                        copy_async<4>(scales_at + to_stage * 128, (lane < 16 ? a.key_scales : a.value_scales) + from, true);
                    }
                } else {
                    uint64_t off = ~0ull;
                    if (page >= 0) {
                        off = (uint64_t)page * a.page_stride + (uint64_t)slot * a.token_stride + (uint64_t)head * a.head_stride;
                        const uint64_t block = (uint64_t)page * a.scale_stride +
                                               (uint64_t)divide(slot, a.block_tokens) * a.heads + head;
                        copy_async<4>(scales_at + to_stage * 128, (lane < 16 ? a.key_scales : a.value_scales) + block, true);
                    } else {
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(scales_at + to_stage * 128), "f"(lane < 16 ? -1.0f : 0.0f)
                                     : "memory");
                    }
                    look_up(i + 1);
                    constexpr uint32_t kChunks = S::kPitch / 16, kRowsAtOnce = 32 / kChunks;
                    const uint32_t c = lane % kChunks;
#pragma unroll
                    for (uint32_t r0 = 0; r0 < kTile; r0 += kRowsAtOnce) {
                        const uint32_t r = r0 + lane / kChunks;
                        const uint64_t from = __shfl_sync(0xffffffffu, off, r);
#pragma unroll
                        for (int h = 0; h < S::kHalves; ++h) {
                            const uint32_t d = S::kPitch * h + 16 * c, dst = to + h * S::kHalfBytes + S::chunk(r, c);
                            const bool real = from != ~0ull && d < a.dim;
                            copy_async<16>(dst, a.keys + (real ? from + d : 0), real);
                            copy_async<16>(dst + kValuesAt, a.values + (real ? from + d : 0), real);
                        }
                    }
                }
            };

            if (!BOX) look_up(0);
            uint32_t ahead = stage;  // the stage that is filled next
#pragma unroll
            for (int i = 0; i < S::kStages - 1; ++i) {
                if ((uint32_t)i < n_tiles) {
                    issue(i, ahead);
                    ahead = ahead + 1 == S::kStages ? 0 : ahead + 1;
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
            for (uint32_t i = 0; i < n_tiles; ++i) {
                __syncwarp();  // every lane has read the stage that is filled now
                if (i + S::kStages - 1 < n_tiles) {
                    issue(i + S::kStages - 1, ahead);
                    ahead = ahead + 1 == S::kStages ? 0 : ahead + 1;
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                wait_copies<S::kStages - 1>();
                if (BOX) {
                    // (having given up, a warp starts no more copies, and waits for those in flight alone)
                    if (in_flight > 0) {
                        --in_flight;
                        const uint32_t bar = bars_at + stage * 8;
                        if (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)) &&
                            !__all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, kDefaultLimitNs))) {
                            if (lane == 0) report_timeout(a.hdr, blockIdx.x);
                            gave_up = true;
                        }
                    }
                } else {
                    __syncwarp();
                }
                const uint8_t *at = ring + warp * S::kStageBytes + stage * kNextStage;
                float own;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(own) : "r"(scales_at + stage * 128) : "memory");
                const bool none = BOX && (absent >> stage & 1u);
                if (++stage == S::kStages) stage = 0, parity ^= 1;
                if (none) continue;
                const uint32_t base = (uint32_t)start + i * unit_tokens;

                float s[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[nt][k] = 0.0f;
#pragma unroll
                for (int c = 0; c < S::kKeyChunks; ++c) {
                    const uint8_t *from = at + (DP >= 128 ? c / 2 * S::kHalfBytes : 0) + (key_at ^ (c & 1) << 6);
                    const uint4 x = *reinterpret_cast<const uint4 *>(from);
                    const uint4 y = *reinterpret_cast<const uint4 *>(from + 8 * S::kPitch);
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t a0 = codes_lo(xs[w]), a1 = codes_lo(ys[w]), a2 = codes_hi(xs[w]), a3 = codes_hi(ys[w]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma(s[nt], a0, a1, a2, a3, q[nt][c * 8 + 2 * w], q[nt][c * 8 + 2 * w + 1]);
                    }
                }
                // element 2 k + j of s, p and w: token(g) + 8 k, query 2 t + j
                float ks[2], vs[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    ks[k] = __shfl_sync(0xffffffffu, own, S::token(g) + 8 * k);
                    vs[k] = __shfl_sync(0xffffffffu, own, 16 + S::token(g) + 8 * k);
                }
                const bool partly = (int32_t)base > whole_until;  // some query does not see some token
                float p[NT][4], w[NT][4], top_w = 0.0f, top_x = 0.0f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            // (the product rounded alone, as where m is taken: equal scores are equal, however large)
                            float x = __fsub_rn(__fmul_rn(s[nt][2 * k + j], ks[k] * factor[nt][j]), m[nt][j]);
                            if (!BOX && ks[k] < 0.0f) x = -INFINITY;
                            const bool hidden = partly && (int32_t)(base + S::token(g) + 8 * k) > last[nt][j];
                            if (hidden) x = -INFINITY;
                            p[nt][2 * k + j] = exp2_approx(x);
                            // (of a hidden token the scale may be anybody's; and p first: its product with a seen token's
                            // scale is finite, or past kMaxWeight, where scale times reference may be infinite beside p = 0)
                            w[nt][2 * k + j] = hidden ? 0.0f : p[nt][2 * k + j] * vs[k] * c_ref[nt][j];
                            top_w = fmaxf(top_w, w[nt][2 * k + j]);
                            top_x = fmaxf(top_x, x);
                        }
                if (__any_sync(0xffffffffu, top_w > kMaxWeight || top_x > kMaxAbove)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float by[2];
                        bool hidden[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            hidden[k] = (!BOX && ks[k >> 1] < 0.0f) ||
                                        (partly && (int32_t)(base + S::token(g) + 8 * (k >> 1)) > last[nt][k & 1]);
                            s[nt][k] = hidden[k] ? -INFINITY : s[nt][k] * (ks[k >> 1] * factor[nt][k & 1]);
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float top = fmaxf(s[nt][j], s[nt][2 + j]);
                            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                            top = fmaxf(top, m[nt][j]);
                            const float less = exp2_approx(m[nt][j] - top), more = exp2_approx(top - m[nt][j]);
                            float heavy = 0.0f;
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                p[nt][2 * k + j] = exp2_approx(s[nt][2 * k + j] - top);
                                heavy = fmaxf(heavy, hidden[2 * k + j] ? 0.0f : p[nt][2 * k + j] * vs[k]);
                            }
                            for (int d = 4; d < 32; d <<= 1) heavy = fmaxf(heavy, __shfl_xor_sync(0xffffffffu, heavy, d));
                            const float fit = heavy > 0.0f ? fminf(kHeaviest / heavy, 0x1p100f) : 0x1p100f;
                            const float c_new = fminf(c_ref[nt][j] * more, fit);
                            by[j] = less > 0.0f ? c_new / c_ref[nt][j] * less : 0.0f;
                            l[nt][j] *= less;
                            m[nt][j] = top;
                            c_ref[nt][j] = c_new;
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                w[nt][2 * k + j] = hidden[2 * k + j] ? 0.0f : p[nt][2 * k + j] * vs[k] * c_new;
                        }
#pragma unroll
                        for (int i2 = 0; i2 < DP / 16; ++i2)
#pragma unroll
                            for (int k = 0; k < 4; ++k) o[i2][nt][k] *= by[k & 1];
                    }
                }
                uint32_t b[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    l[nt][0] += p[nt][0] + p[nt][2];
                    l[nt][1] += p[nt][1] + p[nt][3];
                    b[nt][0] = transposed(pack_half(w[nt][0], w[nt][1]));
                    b[nt][1] = transposed(pack_half(w[nt][2], w[nt][3]));
                }
                // A weight of 0 does not take a NaN away: a query must not meet one that it does not see.
                uint32_t sees[NT][2];
                bool guard = false;
                if (partly) {
                    uint32_t nan = 0;
#pragma unroll
                    for (int x = 0; x < S::kStageBytes / 2 / 32 / 4; ++x) {
                        const uint32_t v = *reinterpret_cast<const uint32_t *>(at + kValuesAt + (x * 32 + lane) * 4);
                        nan |= ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                    }
                    guard = __any_sync(0xffffffffu, nan != 0);
                    if (guard) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                {
                                const int32_t its = (int32_t)(base + S::token(g) + 8 * k);
                                sees[nt][k] = transposed(pack_half(its > last[nt][0] ? 0.0f : 1.0f, its > last[nt][1] ? 0.0f : 1.0f));
                            }
                    }
                }
                // values: lane (g, t) has tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of the order, and of each half's
                // dimensions chunk g / 2 + 4 (g mod 2) (or 8 bytes from 8 g on)
                constexpr int kWords = S::kValueBytes / 4;
#pragma unroll
                for (int h = 0; h < S::kHalves; ++h) {
                    uint32_t v[4][kWords];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint8_t *from = at + h * S::kHalfBytes + 8 * (k >> 1) * S::kPitch + value_at[k & 1];
                        if (S::kValueBytes == 16) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(from);
                            v[k][0] = x.x, v[k][1] = x.y, v[k][kWords - 2] = x.z, v[k][kWords - 1] = x.w;
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2 *>(from);
                            v[k][0] = x.x, v[k][1] = x.y;
                        }
                    }
#pragma unroll
                    for (int x = 0; x < kWords; ++x) {
                        if (guard) {
                            uint32_t is[4];  // 0x38 (the code of 1) where the code is NaN
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t f = ((v[k][x] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                                is[k] = (f >> 2) | (f >> 3) | (f >> 4);
                                v[k][x] &= ~((f >> 7) * 0xffu);
                            }
#pragma unroll
                            for (int i2 = 0; i2 < 2; ++i2) {
                                const uint32_t x0 = __byte_perm(is[0], is[1], i2 ? 0x7362 : 0x5140);
                                const uint32_t x1 = __byte_perm(is[2], is[3], i2 ? 0x7362 : 0x5140);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    float seen[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                    mma(seen, codes_lo(x0), codes_hi(x0), codes_lo(x1), codes_hi(x1), sees[nt][0], sees[nt][1]);
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        if (seen[k] > 0.0f) o[(h * kWords + x) * 2 + i2][nt][k] = NAN;
                                }
                            }
                        }
#pragma unroll
                        for (int i2 = 0; i2 < 2; ++i2) {
                            const uint32_t x0 = __byte_perm(v[0][x], v[1][x], i2 ? 0x7362 : 0x5140);
                            const uint32_t x1 = __byte_perm(v[2][x], v[3][x], i2 ? 0x7362 : 0x5140);
                            const uint32_t a0 = codes_lo(x0), a1 = codes_hi(x0), a2 = codes_lo(x1), a3 = codes_hi(x1);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma(o[(h * kWords + x) * 2 + i2][nt], a0, a1, a2, a3, b[nt][0], b[nt][1]);
                        }
                    }
                }
            }

            // Joins the warps' sums, as the lanes hold them.
            wait_copies<0>();
            __syncthreads();
            float4 *const sums = reinterpret_cast<float4 *>(ring);
            float2 *const refs = reinterpret_cast<float2 *>(sums + kWarps * S::kVectors);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float out_of[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = l[nt][j];
                    for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                    if (g == 0) refs[warp * S::kRows + nt * 8 + 2 * t + j] = make_float2(m[nt][j], x);
                    out_of[j] = 1.0f / c_ref[nt][j];
                }
#pragma unroll
                for (int i = 0; i < DP / 16; ++i)
                    sums[warp * S::kVectors + (nt * (DP / 16) + i) * 32 + lane] =
                        make_float4(o[i][nt][0] * out_of[0], o[i][nt][1] * out_of[1], o[i][nt][2] * out_of[0],
                                    o[i][nt][3] * out_of[1]);
            }
            __syncthreads();
            const bool whole = unit == 0 && n_units == row.units;
            const uint64_t place = (2ull * blockIdx.x + (unit == 0 ? 1 : 0)) << a.pair_heads;
            const uint32_t heads = 1u << a.pair_heads;
            for (uint32_t e = threadIdx.x; e < (uint32_t)S::kVectors << a.pair_heads; e += kThreads) {
                const uint32_t h = e / S::kVectors, v = e % S::kVectors, r = v / (DP / 16 * 32) * 8 + 2 * (v & 3);
                float top[2] = {kNoMax, kNoMax}, sum[2] = {0.0f, 0.0f};
                for (uint32_t w = h; w < kWarps; w += heads) {
                    top[0] = fmaxf(top[0], refs[w * S::kRows + r].x);
                    top[1] = fmaxf(top[1], refs[w * S::kRows + r + 1].x);
                }
                float4 x = {0.0f, 0.0f, 0.0f, 0.0f};
                for (uint32_t w = h; w < kWarps; w += heads) {
                    const float2 m0 = refs[w * S::kRows + r], m1 = refs[w * S::kRows + r + 1];
                    const float b0 = exp2_approx(m0.x - top[0]), b1 = exp2_approx(m1.x - top[1]);
                    const float4 y = sums[w * S::kVectors + v];
                    x.x += y.x * b0;
                    x.y += y.y * b1;
                    x.z += y.z * b0;
                    x.w += y.w * b1;
                    sum[0] += m0.y * b0;
                    sum[1] += m1.y * b1;
                }
                if (whole) {
                    write_out<T, DP, NT>(a, row, (group << a.pair_heads) + h, tile, v, x, sum);
                } else {
                    a.partial[(place + h) * S::kVectors + v] = x;
                    if (v % (DP / 16 * 32) < 4) {  // a lane for every two queries
                        a.partial_ml[(place + h) * S::kRows + r] = make_float2(top[0], sum[0]);
                        a.partial_ml[(place + h) * S::kRows + r + 1] = make_float2(top[1], sum[1]);
                    }
                }
            }
            if (!whole) {
                // Blocks first .. have this tile of queries; the block that comes last joins their sums, in order.
                const uint64_t units_at = at_line - skip + kTileCost;
                const uint64_t first = units_at / line.per;
                const uint32_t parts = (uint32_t)((units_at + row.units - 1) / line.per - first) + 1;
                __threadfence();
                __syncthreads();
                if (threadIdx.x == 0) last_here = count_arrival(a.arrived + first, tag_of(epoch)) == parts;
                __syncthreads();
                if (last_here) {
                    __threadfence();
                    join_parts<T, DP, NT>(a, ring, first, parts, row, group, tile);
                }
            }
            fence_proxy_async_smem();  // the sums' place becomes the ring again
            __syncthreads();
        }
        left -= taken;
        at_line += taken;
        if (left == 0) break;
        skip = 0;
        if (++tile == row.tiles) {
            tile = 0;
            if (++group == a.heads >> a.pair_heads) {
                group = 0;
                do {
                    if (++row_at >= a.v.rows) break;  // (lens that change meanwhile)
                    row = row_units(a, row_at, S::kRows);
                } while (row.units == 0);
                if (row_at >= a.v.rows) break;
            }
        }
    }
    if (threadIdx.x == 0 && nth_block == gridDim.x - 1) {  // the last to count itself re-arms the header
        st_relaxed_u32(&a.hdr->counter, 0u);
        st_relaxed_u32(&a.hdr->epoch, epoch + 1u);
    }
    finish_period(a.hdr, epoch, a.arrived, a.clear_words);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr size_t kPartialBytes = 2ull * kMaxBlocks * kMaxElements * sizeof(float);
constexpr size_t kPartialMlBytes = 2ull * kMaxBlocks * kMaxPairs * sizeof(float2);

size_t attend_workspace_bytes() {
    return round_up(round_up(tile_word_reach(), 256) + kPartialBytes + kPartialMlBytes, 256);
}

// The cache's codes as a tensor of dimensions, heads, slots and pages.
static bool box_map(CUtensorMap *map, const uint8_t *codes, const AttendArgs &a, bool wide) {
    typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                               const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (encode == nullptr) return false;
    const cuuint64_t sizes[4] = {a.dim, a.heads, a.v.page_tokens.d, a.v.pages};
    const cuuint64_t strides[3] = {a.head_stride ? a.head_stride : 16, a.token_stride ? a.token_stride : 16,
                                   a.page_stride ? a.page_stride : 16};  // (0 where there is one)
    const cuuint32_t box[4] = {wide ? 128u : 64u, 1, kTile, 1}, steps[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t *>(codes), sizes, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DP, int NT>
static int attend_launch(AttendArgs a, cudaStream_t s) {
    using S = Shape<DP, NT>;
    int sms = 0;
    const int rc = sm_count(&sms);
    if (rc != U32SCAN_OK) return rc;
    uint64_t blocks = (uint64_t)sms * S::kBlocks;
    if (blocks > kMaxBlocks) blocks = kMaxBlocks;
    // Tiles of queries, and units if every row is as long as its table: at most these. Several heads beside each other read
    // a page's memory together, but leave fewer and larger parts, which one block each joins. With 1, 2, 4 heads, us: 256
    // rows of up to 2048 tokens 124, 109, 106, of 500 61, 50, 48, 200 of 1500 of 16 heads 149, 128, 121, heads of 64: 77, 71, 71
    // and, of 16 heads, 105, 75, 73; but 64 rows of 8192 100 to 110, 100 to 102, 108 to 111 and 32 of them 62, 63, 72; two
    // rows of 200000 154 each. (As many as there are: long rows of 128 dimensions would go 8 to 13 % faster with two,
    // short ones 2 to 9 % slower.)
    const uint64_t tiles = a.v.tokens * a.group.d / S::kRows + a.v.rows;
    a.pair_heads = a.heads % 4 == 0 ? 2 : a.heads % 2 == 0 ? 1 : 0;
    if (a.pair_heads > S::kMostPaired) a.pair_heads = S::kMostPaired;
    while (a.pair_heads > 0 && tiles * (a.heads >> a.pair_heads) * 8 < blocks) --a.pair_heads;
    const uint64_t placed = a.v.width * a.v.page_tokens.d, length = placed < (1ull << 31) ? placed : (1ull << 31);
    const double units = (double)tiles * (a.heads >> a.pair_heads) *
                         (double)(length / ((kTile * kWarps) >> a.pair_heads) + 1 + kTileCost);
    if (units < (double)(blocks * kLeastUnits)) blocks = (uint64_t)units / kLeastUnits + 1;
    const bool box = a.v.page_tokens.d % kTile == 0 && a.v.pages > 0;
    const auto kernel = box ? attend_kernel<T, DP, NT, true> : attend_kernel<T, DP, NT, false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kShared) != cudaSuccess)
        return U32SCAN_ECUDA;
    CUtensorMap maps[2] = {};
    if (box && (!box_map(&maps[0], a.keys, a, DP >= 128) || !box_map(&maps[1], a.values, a, DP >= 128)))
        return U32SCAN_ECUDA;
    kernel<<<(unsigned int)blocks, kThreads, S::kShared, s>>>(a, maps[0], maps[1]);
    return cudaGetLastError() == cudaSuccess ? U32SCAN_OK : U32SCAN_ECUDA;
}

// Eight queries at a time, or sixteen where the mean row has nearly that many for each key head: the codes are then read and
// converted once for both, in twice the registers. 64 rows of up to 8192 tokens, 8 heads of 128, with 8 and 16 at a time:
// groups of 16 173 and 152 us, of 8 with one or two tokens (12 queries in the mean) 111 and 145, with one to five
// (24) 225 and 219, these with heads of 64 155 and 133; 33 short rows of drafts, heads of 64 (21), 28 and 32, 200 of them
// 96 and 92. (32 at a time, 33 rows: 42.)
template <typename T>
static int attend_dispatch(const AttendArgs &a, cudaStream_t s) {
    const bool many = a.v.tokens * a.group.d >= 14 * a.v.rows;
    if (a.dim <= 64) return many ? attend_launch<T, 64, 2>(a, s) : attend_launch<T, 64, 1>(a, s);
    if (a.dim <= 128) return many ? attend_launch<T, 128, 2>(a, s) : attend_launch<T, 128, 1>(a, s);
    return attend_launch<T, 256, 1>(a, s);
}

}  // namespace u32scan

using namespace u32scan;

extern "C" int pages_attend(const u32scan_kv_cache *cache, const int32_t *table, size_t table_stride, size_t rows,
                            size_t width, const int32_t *lens, const int32_t *starts, size_t tokens,
                            const void *queries, int type, size_t q_heads, size_t query_token_stride,
                            size_t query_head_stride, void *out, size_t out_token_stride, size_t out_head_stride,
                            float scale, void *ws, size_t ws_bytes, u32scan_stream_t stream) {
    if (!cache_ok(cache) || cache->type != U32SCAN_E4M3 || (type != U32SCAN_F16 && type != U32SCAN_BF16))
        return U32SCAN_EINVAL;
    if (!rows_ok(table, table_stride, rows, width, lens, starts, tokens)) return U32SCAN_EINVAL;
    if (cache->dim % 16 != 0 || cache->dim > kMaxDim || q_heads == 0 || q_heads >= (1ull << 16) ||
        q_heads % cache->heads != 0)
        return U32SCAN_EINVAL;
    if (!strides_ok(query_token_stride, query_head_stride) || !strides_ok(out_token_stride, out_head_stride))
        return U32SCAN_EINVAL;
    // 16 bytes at a time: 16 codes, 8 queries
    if (misaligned(cache->keys, 16) || misaligned(cache->values, 16) || misaligned(queries, 16) || misaligned(out, 2) ||
        ((cache->page_stride | cache->token_stride | cache->head_stride) & 15) != 0 ||
        ((query_token_stride | query_head_stride) & 7) != 0)
        return U32SCAN_EINVAL;
    if (tokens * (q_heads / cache->heads) >= (1ull << 31)) return U32SCAN_EINVAL;
    if (tokens == 0 || rows == 0) return U32SCAN_OK;
    if (queries == nullptr || out == nullptr) return U32SCAN_EINVAL;
    const size_t run = 2 * cache->dim;
    if (share_memory(Strided{queries, run, {tokens, q_heads, 1}, {2 * query_token_stride, 2 * query_head_stride, 0}},
                     Strided{out, run, {tokens, q_heads, 1}, {2 * out_token_stride, 2 * out_head_stride, 0}}))
        return U32SCAN_EINVAL;
    if (ws == nullptr || misaligned(ws, 256) || ws_bytes < attend_workspace_bytes()) return U32SCAN_EWORKSPACE;
    AttendArgs a{};
    a.v = RowsView{table, lens, starts, table_stride, rows, width, tokens, cache->pages,
                   divisor((uint32_t)cache->page_tokens)};
    a.keys = static_cast<const uint8_t *>(cache->keys);
    a.values = static_cast<const uint8_t *>(cache->values);
    a.key_scales = cache->key_scales;
    a.value_scales = cache->value_scales;
    a.page_stride = cache->page_stride;
    a.token_stride = cache->token_stride;
    a.head_stride = cache->head_stride;
    a.scale_stride = cache->scale_stride;
    a.block_tokens = divisor((uint32_t)(cache->page_tokens / cache->blocks));
    a.heads = (uint32_t)cache->heads;
    a.group = divisor((uint32_t)(q_heads / cache->heads));
    a.dim = (uint32_t)cache->dim;
    a.queries = queries;
    a.out = out;
    a.q_token_stride = query_token_stride;
    a.q_head_stride = query_head_stride;
    a.out_token_stride = out_token_stride;
    a.out_head_stride = out_head_stride;
    a.scale = scale * 1.4426950408889634f;
    a.wide_blocks = cache->page_tokens / cache->blocks % kTile == 0;
    a.hdr = static_cast<WsHeader *>(ws);
    char *w = static_cast<char *>(ws) + round_up(tile_word_reach(), 256);  // past every operation's tile words
    a.partial = reinterpret_cast<float4 *>(w);
    a.partial_ml = reinterpret_cast<float2 *>(w + kPartialBytes);
    a.arrived = reinterpret_cast<unsigned long long *>(static_cast<char *>(ws) + kHeaderBytes);
    a.clear_words = tile_words_to_clear(ws_bytes);
    const cudaStream_t s = (cudaStream_t)stream;
    if (type == U32SCAN_F16) return attend_dispatch<__half>(a, s);
    return attend_dispatch<__nv_bfloat16>(a, s);
}
