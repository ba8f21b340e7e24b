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
// blocks whose scales lie far apart. Both stay until a weight exceeds 2^8
// (p: 2^32); only then the warp takes new maxima and rescales its sums.
// w is rounded to f16 (2^-11 relative; products and sums are f32): the
// codes it meets have 4 bits, and the result's type 8 or 11.
//
// The work of all rows is one line of units (64 tokens of one row, key head
// and tile of queries), cut into equal pieces for the blocks, however ragged
// the rows are. A tile whose units fall to several blocks is joined from
// their partial sums, in order, by a second launch.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvcache.cuh"
#include "launch.cuh"

namespace u32scan {

constexpr int kQThreads = 128;
constexpr int kQWarps = kQThreads / 32;
constexpr int kTile = 16;                 // tokens of a warp at a time
constexpr int kUnit = kTile * kQWarps;    // tokens of a unit
constexpr int kMaxDim = 256;
constexpr unsigned int kMaxBlocks = 640;  // bounds the workspace
constexpr uint32_t kTileCost = 2;         // what a tile of queries takes beside its units, in units
constexpr uint64_t kLeastUnits = kTileCost + 2;  // of a block's piece
constexpr int kMaxElements = 2048;        // queries x dimensions of a tile of queries
constexpr int kMaxTileRows = 32;
constexpr float kNoMax = -1e30f;
constexpr float kMaxWeight = 256.0f, kMaxP = 4294967296.0f;

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
    float scale;  // times log2(e)
    bool boxes;   // 16 tokens from a multiple of 16 on lie in one page
    WsHeader *hdr;
    float *partial;      // [2 blocks][elements of a tile]
    float2 *partial_ml;  // [2 blocks][rows of a tile]: reference and sum
    struct Boundary *boundary;
};

// Where a block's piece begins, for the launch that joins.
struct Boundary {
    uint32_t row, head, tile, unit;  // unit: of the tile's, the first in this piece; 0: nothing to join here
    uint64_t units, per;
    uint64_t pad[2];
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

__device__ __forceinline__ RowUnits row_units(const AttendArgs &a, uint64_t s, uint32_t tile_rows) {
    RowUnits r;
    tokens_of(a.v, s, &r.begin, &r.n);
    const int32_t len = a.v.lens[s];
    r.len = len;
    const uint64_t placed = a.v.pages == 0 ? 0 : a.v.width * a.v.page_tokens.d;
    r.limit = (uint32_t)(len <= 0 ? 0 : (uint64_t)len < placed ? (uint64_t)len : placed);
    r.units = r.n == 0 ? 0u : r.limit <= kUnit ? 1u : (r.limit + kUnit - 1) / kUnit;
    r.tiles = (uint32_t)((r.n * a.group.d + tile_rows - 1) / tile_rows);
    return r;
}

// The sizes of one kernel: DP dimensions (dim, up to it), 8 * NT queries. A
// stage holds 16 rows of keys, then of values, of 128 bytes (dimensions past
// 128 in 16 rows more) or 64, 16-byte chunks swizzled as TMA does it.
template <int DP, int NT>
struct Shape {
    static constexpr int kRows = 8 * NT;
    static constexpr int kPitch = DP >= 128 ? 128 : 64;
    static constexpr int kHalves = DP / kPitch;
    static constexpr int kHalfBytes = kTile * kPitch;
    static constexpr int kKeyChunks = DP / 64;                    // of 16 bytes, for each of a lane's two keys
    static constexpr int kValueBytes = DP >= 128 ? 16 : 8;        // for each of a lane's four values and each half
    static constexpr int kBlocks = DP * NT <= 128 ? 4 : 3;        // an SM
    static constexpr int kStageBytes = DP * 2 * kTile;            // of a warp
    static constexpr int kStages = (228 * 1024 / kBlocks - 4096) / (kQWarps * (kStageBytes + 128));
    static constexpr int kRing = kStages * kQWarps * kStageBytes;
    static constexpr int kShared = kRing + kStages * kQWarps * (128 + 8) + 1024;  // scales, barriers, alignment
    static_assert(kQWarps * (kRows * DP + 2 * kRows) * 4 <= kRing, "the warps' sums take the ring's place");
    static_assert(kRows * DP <= kMaxElements && kRows <= kMaxTileRows, "the workspace's slots");
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

// The piece [*from, *to) of block `block`, and the row and unit in it where it begins.
struct Piece {
    uint64_t from, to, per;
    uint64_t row, unit;
};

__device__ Piece piece_of(const AttendArgs &a, uint32_t tile_rows, uint64_t block, uint64_t blocks) {
    __shared__ uint64_t sums[kQWarps], found[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t rows = a.v.rows;
    auto share = [&](uint64_t s) -> uint64_t {
        if (s >= rows) return 0;
        const RowUnits r = row_units(a, s, tile_rows);
        return r.units ? ((uint64_t)r.units + kTileCost) * r.tiles * a.heads : 0;
    };
    auto warp_sum = [&](uint64_t x) {
        for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        return x;
    };
    uint64_t mine = 0;
    for (uint64_t s = threadIdx.x; s < rows; s += kQThreads) mine += share(s);
    mine = warp_sum(mine);
    if (lane == 0) sums[warp] = mine;
    __syncthreads();
    uint64_t total = 0;
    for (int w = 0; w < kQWarps; ++w) total += sums[w];
    Piece p;
    p.per = (total + blocks - 1) / blocks;
    if (p.per < kLeastUnits) p.per = kLeastUnits;
    p.from = block * p.per;
    p.to = p.from + p.per < total ? p.from + p.per : total;
    p.row = p.unit = 0;
    if (p.from >= total) return p;
    uint64_t before = 0;
    for (uint64_t base = 0; base < rows; base += kQThreads) {
        const uint64_t x = share(base + threadIdx.x);
        uint64_t incl = x;
        for (int d = 1; d < 32; d <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += y;
        }
        __syncthreads();  // sums and found were read
        if (lane == 31) sums[warp] = incl;
        if (threadIdx.x == 0) found[0] = ~0ull;
        __syncthreads();
        uint64_t all = 0;
        incl += before;
        for (int w = 0; w < kQWarps; ++w) {
            if (w < warp) incl += sums[w];
            all += sums[w];
        }
        if (p.from < incl && p.from >= incl - x) {
            found[0] = base + threadIdx.x;
            found[1] = p.from - (incl - x);
        }
        before += all;
        __syncthreads();
        if (found[0] != ~0ull) break;
    }
    p.row = found[0];
    p.unit = found[1];
    return p;
}

// Row r of a tile of queries: its token of the row and query head of the key head.
__device__ __forceinline__ bool query_of(const AttendArgs &a, const RowUnits &row, uint32_t tile, uint32_t tile_rows,
                                         uint32_t r, uint32_t *token, uint32_t *j) {
    const uint64_t f = (uint64_t)tile * tile_rows + r;
    if (f >= (uint64_t)row.n * a.group.d) return false;
    // (a tile of n * group rows may pass 2^31; the divisor's bound is that)
    *token = f < (1ull << 31) ? divide((uint32_t)f, a.group) : (uint32_t)(f / a.group.d);
    *j = (uint32_t)(f - (uint64_t)*token * a.group.d);
    return true;
}

template <typename T, int DP, int NT>
__global__ void __launch_bounds__(kQThreads, Shape<DP, NT>::kBlocks)
attend_kernel(const AttendArgs a, const __grid_constant__ CUtensorMap key_map,
              const __grid_constant__ CUtensorMap value_map) {
    using S = Shape<DP, NT>;
    extern __shared__ uint8_t unaligned[];
    const uint32_t ring_at = (smem_u32(unaligned) + 1023u) & ~1023u;
    uint8_t *const ring = unaligned + (ring_at - smem_u32(unaligned));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t g = lane >> 2, t = lane & 3;
    // stage i of this warp: codes at codes_at + i * kNextStage, scales (16 of keys, 16 of values) and barrier behind the ring
    constexpr uint32_t kNextStage = kQWarps * S::kStageBytes, kValuesAt = DP * kTile;
    const uint32_t codes_at = ring_at + warp * S::kStageBytes;
    const uint32_t scales_at = ring_at + S::kRing + warp * S::kStages * 128 + lane * 4;
    const uint32_t bars_at = ring_at + S::kRing + S::kStages * kQWarps * 128 + warp * S::kStages * 8;
    if (a.boxes && lane < S::kStages) mbar_init(bars_at + lane * 8, 1);
    fence_mbar_init();
    const Piece piece = piece_of(a, S::kRows, blockIdx.x, gridDim.x);  // (block barriers within)
    if (piece.from >= piece.to) {
        if (threadIdx.x == 0) a.boundary[blockIdx.x].unit = 0u;
        return;
    }
    uint64_t row_at = piece.row;
    RowUnits row = row_units(a, row_at, S::kRows);
    uint64_t left = piece.to - piece.from;
    const uint64_t width = (uint64_t)row.units + kTileCost;  // of a tile of queries on the line
    uint32_t skip = (uint32_t)(piece.unit % width);          // what of it lies before this piece
    uint32_t tile = (uint32_t)(piece.unit / width % row.tiles);
    uint32_t head = (uint32_t)(piece.unit / width / row.tiles);
    if (threadIdx.x == 0)
        a.boundary[blockIdx.x] = Boundary{(uint32_t)row_at, head, tile, skip > kTileCost ? skip - kTileCost : 0u,
                                          row.units, piece.per, {0, 0}};

    uint32_t stage = 0, parity = 0;  // of the tile that is consumed next
    uint32_t in_flight = 0;
    bool gave_up = false;
    while (true) {
        // units [unit, unit + n_units) of the tile
        const uint64_t here = (uint64_t)row.units + kTileCost - skip;
        const uint32_t taken = (uint32_t)(left < here ? left : here);
        const uint32_t unit = skip > kTileCost ? skip - kTileCost : 0u;
        const uint32_t n_units = skip + taken > kTileCost ? skip + taken - kTileCost - unit : 0u;
        if (n_units > 0) {
            // queries: lane (g, t) holds elements 64 c + 16 t .. + 15 of row g of each eight
            uint32_t q[NT][S::kKeyChunks * 8];
            float factor[NT][2];  // of the queries 2 t, 2 t + 1: what makes a product a score
            int32_t last[NT][2];  // and the last position they see
            int64_t first_last, last_last;
            {
                const int64_t before = row.len - row.n;
                const uint64_t f0 = (uint64_t)tile * S::kRows, f1 = f0 + S::kRows - 1, all = (uint64_t)row.n * a.group.d;
                first_last = before + (int64_t)(f0 / a.group.d);
                last_last = before + (int64_t)((f1 < all ? f1 : all - 1) / a.group.d);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t token = 0, j = 0;
                    const bool real = query_of(a, row, tile, S::kRows, nt * 8 + g, &token, &j);
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

            // the warp's tiles: 16 tokens from (unit + i) * 64 + warp * 16 on
            const uint64_t start = (uint64_t)unit * kUnit + warp * kTile;
            const uint32_t most = start < limit ? (uint32_t)((limit - start + kUnit - 1) / kUnit) : 0u;
            const uint32_t n_tiles = n_units < most ? n_units : most;
            // the page of token `lane mod 16` of tile i
            auto page_at = [&](uint32_t i) -> int32_t {
                const uint64_t at = start + (lane & 15) + (uint64_t)i * kUnit;
                return i < n_tiles && at < limit ? __ldg(table + divide((uint32_t)at, a.v.page_tokens)) : -1;
            };
            auto issue = [&](uint32_t i, int32_t page, uint32_t to_stage) {
                const uint32_t to = codes_at + to_stage * kNextStage;
                const uint32_t at = (uint32_t)start + (lane & 15) + i * kUnit;
                const bool held = page >= 0 && (uint64_t)page < a.v.pages;
                const uint32_t slot = at - divide(at, a.v.page_tokens) * a.v.page_tokens.d;
                in_flight += gave_up ? 0 : 1;
                if (a.boxes && lane == 0 && !gave_up) {
                    const uint32_t bar = bars_at + to_stage * 8;
                    mbar_arrive_expect_tx(bar, S::kStageBytes);
#pragma unroll
                    for (int h = 0; h < S::kHalves; ++h) {
                        copy_box(to + h * S::kHalfBytes, &key_map, bar, S::kPitch * h, (int)head, (int)slot, page);
                        copy_box(to + kValuesAt + h * S::kHalfBytes, &value_map, bar, S::kPitch * h, (int)head, (int)slot, page);
                    }
                }
                if (held) {
                    const uint64_t block = (uint64_t)page * a.scale_stride +
                                           (uint64_t)divide(slot, a.block_tokens) * a.heads + head;
                    copy_async<4>(scales_at + to_stage * 128, (lane < 16 ? a.key_scales : a.value_scales) + block, true);
                } else {
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(scales_at + to_stage * 128), "f"(lane < 16 ? -1.0f : 0.0f)
                                 : "memory");
                }
                if (!a.boxes) {
                    const uint64_t off = held ? (uint64_t)page * a.page_stride + (uint64_t)slot * a.token_stride +
                                                    (uint64_t)head * a.head_stride
                                              : ~0ull;
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

            int32_t page = page_at(0);
            uint32_t ahead = stage;  // the stage that is filled next
#pragma unroll
            for (int i = 0; i < S::kStages - 1; ++i) {
                const int32_t now = page;
                page = page_at(i + 1);
                if ((uint32_t)i < n_tiles) {
                    issue(i, now, ahead);
                    ahead = ahead + 1 == S::kStages ? 0 : ahead + 1;
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
            for (uint32_t i = 0; i < n_tiles; ++i) {
                __syncwarp();  // every lane has read the stage that is filled now
                {
                    const int32_t now = page;
                    page = page_at(i + S::kStages);
                    if (i + S::kStages - 1 < n_tiles) {
                        issue(i + S::kStages - 1, now, ahead);
                        ahead = ahead + 1 == S::kStages ? 0 : ahead + 1;
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                }
                wait_copies<S::kStages - 1>();
                if (a.boxes) {
                    // (having given up, a warp starts no more copies, and waits for those in flight alone)
                    if (in_flight > 0) {
                        --in_flight;
                        if (!__all_sync(0xffffffffu, mbar_wait_bounded(bars_at + stage * 8, parity, kDefaultLimitNs))) {
                            if (lane == 0) report_timeout(a.hdr, blockIdx.x);
                            gave_up = true;
                        }
                    }
                } else {
                    in_flight = 0;
                    __syncwarp();
                }
                const uint8_t *at = ring + warp * S::kStageBytes + stage * kNextStage;
                float own;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(own) : "r"(scales_at + stage * 128) : "memory");
                if (++stage == S::kStages) stage = 0, parity ^= 1;
                const uint32_t base = (uint32_t)start + i * kUnit;

                float s[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[nt][k] = 0.0f;
#pragma unroll
                for (int c = 0; c < S::kKeyChunks; ++c) {
                    const uint8_t *from = at + (DP >= 128 ? c / 2 * S::kHalfBytes : 0) +
                                          S::chunk(S::token(g), DP >= 128 ? t + 4 * (c & 1) : t);
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
                const bool partly = (int64_t)base + kTile - 1 > first_last;  // some query does not see some token
                float p[NT][4], w[NT][4], top_w = 0.0f, top_p = 0.0f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float &x = s[nt][2 * k + j];
                            x = ks[k] < 0.0f ? -INFINITY : x * (ks[k] * factor[nt][j]);
                            if (partly && (int32_t)(base + S::token(g) + 8 * k) > last[nt][j]) x = -INFINITY;
                            p[nt][2 * k + j] = exp2_approx(x - m[nt][j]);
                            w[nt][2 * k + j] = p[nt][2 * k + j] * (vs[k] * c_ref[nt][j]);
                            top_w = fmaxf(top_w, w[nt][2 * k + j]);
                            top_p = fmaxf(top_p, p[nt][2 * k + j]);
                        }
                if (__any_sync(0xffffffffu, top_w > kMaxWeight || top_p > kMaxP)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float by[2];
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
                                heavy = fmaxf(heavy, p[nt][2 * k + j] * vs[k]);
                            }
                            for (int d = 4; d < 32; d <<= 1) heavy = fmaxf(heavy, __shfl_xor_sync(0xffffffffu, heavy, d));
                            const float fit = heavy > 0.0f ? fminf(1.0f / heavy, 0x1p100f) : 0x1p100f;
                            const float c_new = fminf(c_ref[nt][j] * more, fit);
                            by[j] = less > 0.0f ? c_new / c_ref[nt][j] * less : 0.0f;
                            l[nt][j] *= less;
                            m[nt][j] = top;
                            c_ref[nt][j] = c_new;
#pragma unroll
                            for (int k = 0; k < 2; ++k) w[nt][2 * k + j] = p[nt][2 * k + j] * (vs[k] * c_new);
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
                                sees[nt][k] = transposed(pack_half(s[nt][2 * k] == -INFINITY ? 0.0f : 1.0f,
                                                                   s[nt][2 * k + 1] == -INFINITY ? 0.0f : 1.0f));
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
                        const uint32_t r = S::token(2 * t + (k & 1));
                        const uint8_t *from = at + kValuesAt + h * S::kHalfBytes + 8 * (k >> 1) * S::kPitch +
                                              (DP >= 128 ? S::chunk(r, g >> 1 | (g & 1) << 2) : S::chunk(r, g >> 1) + 8 * (g & 1));
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

            // Joins the warps' sums. Element 2 k + j of o[(h * kWords + x) * 2 + i] is dimension 4 x + 2 i + k of the lane's
            // chunk, query 2 t + j.
            wait_copies<0>();
            __syncthreads();
            float *const sums = reinterpret_cast<float *>(ring);
            float2 *const refs = reinterpret_cast<float2 *>(sums + kQWarps * S::kRows * DP);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = l[nt][j];
                    for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                    const uint32_t r = nt * 8 + 2 * t + j;
                    if (g == 0) refs[warp * S::kRows + r] = make_float2(m[nt][j], x);
                    const float out_of = 1.0f / c_ref[nt][j];
#pragma unroll
                    for (int i = 0; i < DP / 16; ++i) {
                        constexpr int kPer = S::kValueBytes / 2;  // of o, for a half
                        const uint32_t chunk = DP >= 128 ? g >> 1 | (g & 1) << 2 : g;
                        const uint32_t d = S::kPitch * (i / kPer) + S::kValueBytes * chunk + 2 * (i % kPer);
                        float2 *to = reinterpret_cast<float2 *>(sums + (warp * S::kRows + r) * DP + d);
                        *to = make_float2(o[i][nt][j] * out_of, o[i][nt][2 + j] * out_of);
                    }
                }
            __syncthreads();
            const bool whole = unit == 0 && n_units == row.units;
            const uint64_t place = 2ull * blockIdx.x + (unit == 0 ? 1 : 0);
            for (int e = threadIdx.x; e < S::kRows * (DP / 2); e += kQThreads) {
                const uint32_t r = e / (DP / 2), d = e % (DP / 2) * 2;
                float top = kNoMax;
#pragma unroll
                for (int w = 0; w < kQWarps; ++w) top = fmaxf(top, refs[w * S::kRows + r].x);
                float x = 0.0f, y = 0.0f, sum = 0.0f;
#pragma unroll
                for (int w = 0; w < kQWarps; ++w) {
                    const float2 ml = refs[w * S::kRows + r];
                    const float by = exp2_approx(ml.x - top);
                    const float2 v = *reinterpret_cast<const float2 *>(sums + (w * S::kRows + r) * DP + d);
                    x += v.x * by;
                    y += v.y * by;
                    sum += ml.y * by;
                }
                if (whole) {
                    uint32_t token, j;
                    if (d < a.dim && query_of(a, row, tile, S::kRows, r, &token, &j)) {
                        T *to = static_cast<T *>(a.out) + (uint64_t)(row.begin + token) * a.out_token_stride +
                                ((uint64_t)head * a.group.d + j) * a.out_head_stride + d;
                        to[0] = QType<T>::put(sum == 0.0f ? 0.0f : x / sum);
                        to[1] = QType<T>::put(sum == 0.0f ? 0.0f : y / sum);
                    }
                } else {
                    *reinterpret_cast<float2 *>(a.partial + place * (S::kRows * DP) + r * DP + d) = make_float2(x, y);
                    if (d == 0) a.partial_ml[place * S::kRows + r] = make_float2(top, sum);
                }
            }
            fence_proxy_async_smem();  // the sums' place becomes the ring again
            __syncthreads();
        }
        left -= taken;
        if (left == 0) break;
        skip = 0;
        if (++tile == row.tiles) {
            tile = 0;
            if (++head == a.heads) {
                head = 0;
                do {
                    if (++row_at >= a.v.rows) return;  // (lens that change meanwhile)
                    row = row_units(a, row_at, S::kRows);
                } while (row.units == 0);
            }
        }
    }
}

// Joins the partial sums of the tile in which block c's piece begins, where that is the first piece to begin within it:
// block c - 1 ended with its first units, the blocks from c on began with the others.
template <typename T, int DP, int NT>
__global__ void __launch_bounds__(kQThreads) join_kernel(const AttendArgs a) {
    using S = Shape<DP, NT>;
    cudaGridDependencySynchronize();  // what the launch before wrote
    const uint64_t block = blockIdx.x + 1;
    const Boundary b = a.boundary[block];
    if (b.unit == 0 || b.unit > b.per) return;
    const uint64_t end = block * b.per - b.unit + b.units;
    const uint64_t stop = (end + b.per - 1) / b.per;  // the first block that begins behind the tile
    const RowUnits row = row_units(a, b.row, S::kRows);
    for (int e = threadIdx.x; e < S::kRows * (DP / 4); e += kQThreads) {
        const uint32_t r = e / (DP / 4), d = e % (DP / 4) * 4;
        uint32_t token, j;
        if (d >= a.dim || !query_of(a, row, b.tile, S::kRows, r, &token, &j)) continue;
        float top = kNoMax, sum = 0.0f, x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (uint64_t k = block - 1; k < stop; ++k) {
            const uint64_t slot = 2 * k + (k == block - 1 ? 1 : 0);
            const float2 ml = a.partial_ml[slot * S::kRows + r];
            const float4 v = *reinterpret_cast<const float4 *>(a.partial + slot * (S::kRows * DP) + r * DP + d);
            const float now = fmaxf(top, ml.x);
            const float old = exp2_approx(top - now), by = exp2_approx(ml.x - now);
            top = now;
            sum = sum * old + ml.y * by;
            x[0] = x[0] * old + v.x * by;
            x[1] = x[1] * old + v.y * by;
            x[2] = x[2] * old + v.z * by;
            x[3] = x[3] * old + v.w * by;
        }
        T *to = static_cast<T *>(a.out) + (uint64_t)(row.begin + token) * a.out_token_stride +
                ((uint64_t)b.head * a.group.d + j) * a.out_head_stride + d;
#pragma unroll
        for (int k = 0; k < 4; ++k) to[k] = QType<T>::put(sum == 0.0f ? 0.0f : x[k] / sum);
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr size_t kPartialBytes = 2ull * kMaxBlocks * kMaxElements * sizeof(float);
constexpr size_t kPartialMlBytes = 2ull * kMaxBlocks * kMaxTileRows * sizeof(float2);
constexpr size_t kBoundaryBytes = kMaxBlocks * sizeof(Boundary);

size_t attend_workspace_bytes() {
    return round_up(round_up(tile_word_reach(), 256) + kPartialBytes + kPartialMlBytes + kBoundaryBytes, 256);
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
    if (cudaFuncSetAttribute(attend_kernel<T, DP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kShared) !=
        cudaSuccess)
        return U32SCAN_ECUDA;
    unsigned int blocks = (unsigned int)sms * S::kBlocks;
    if (blocks > kMaxBlocks) blocks = kMaxBlocks;
    CUtensorMap maps[2] = {};
    if (a.boxes && (!box_map(&maps[0], a.keys, a, DP >= 128) || !box_map(&maps[1], a.values, a, DP >= 128)))
        return U32SCAN_ECUDA;
    attend_kernel<T, DP, NT><<<blocks, kQThreads, S::kShared, s>>>(a, maps[0], maps[1]);
    if (blocks > 1) launch_next(join_kernel<T, DP, NT>, blocks - 1, kQThreads, s, a);
    return cudaGetLastError() == cudaSuccess ? U32SCAN_OK : U32SCAN_ECUDA;
}

// Eight queries at a time, more where a row has them: the codes are read and converted once for all of a tile.
template <typename T>
static int attend_dispatch(const AttendArgs &a, uint64_t rows_of_queries, cudaStream_t s) {
    if (a.dim <= 64) {
        if (rows_of_queries <= 8) return attend_launch<T, 64, 1>(a, s);
        if (rows_of_queries <= 16) return attend_launch<T, 64, 2>(a, s);
        return attend_launch<T, 64, 4>(a, s);
    }
    if (a.dim <= 128) return rows_of_queries <= 8 ? attend_launch<T, 128, 1>(a, s) : attend_launch<T, 128, 2>(a, s);
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
    if (tokens == 0 || rows == 0) return U32SCAN_OK;
    if (queries == nullptr || out == nullptr) return U32SCAN_EINVAL;
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
    a.boxes = cache->page_tokens % kTile == 0 && cache->pages > 0;
    a.hdr = static_cast<WsHeader *>(ws);
    char *w = static_cast<char *>(ws) + round_up(tile_word_reach(), 256);  // past every operation's tile words
    a.partial = reinterpret_cast<float *>(w);
    a.partial_ml = reinterpret_cast<float2 *>(w + kPartialBytes);
    a.boundary = reinterpret_cast<Boundary *>(w + kPartialBytes + kPartialMlBytes);
    // rows of one token have `group` queries a key head; of ragged ones the mean is known here
    const uint64_t mean = starts == nullptr ? 1 : (tokens + rows - 1) / rows;
    const cudaStream_t s = (cudaStream_t)stream;
    if (type == U32SCAN_F16) return attend_dispatch<__half>(a, mean * a.group.d, s);
    return attend_dispatch<__nv_bfloat16>(a, mean * a.group.d, s);
}
