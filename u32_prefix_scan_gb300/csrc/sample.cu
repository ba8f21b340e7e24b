// sample.cu -- the next token of every row of logits, drawn with given u32
// random words under temperature, min-p, top-k and top-p.
//
// Everything after the logits is integer arithmetic, so a row's token does
// not depend on the launch's shape or on the order of any sum, and equals
// the sequential definition's:
//   weight  q = floor(2^31 * 2^-y) as u32, y = (m - l) * (log2 e / T), m the
//           row's largest logit. 2^-y is a recipe of f32 operations rounded
//           one by one (token_weight), the same on every IEEE machine; q = 0
//           from y = 32 on, so a row's sum is within V * 2^-31 of the
//           largest weight of the real one. 31 bits: a u32 with one left
//           over, and sums of 2^22 of them stay below 2^53 (exact in double
//           where top-p multiplies, and exact in u64).
//   order   logit descending, then index ascending; the sort keys are the
//           logits' bits, so no two different logits tie through rounding.
//   filters min-p and top-k zero weights, top-p keeps the shortest prefix in
//           that order whose sum reaches ceil(p * S).
//   draw    r = floor(word * S' / 2^32); the token is the first index whose
//           running sum (in index order) exceeds r. Index order, because an
//           inverse distribution function may run in any order and this one
//           needs no sort.
//
// One cluster of blocks takes a row: each block reads its slice once from
// HBM and keeps it in shared memory (what does not fit is read again, from
// L2), so the passes after the maximum touch no HBM. No row is sorted:
//   top-k   the k-th largest of the maxima of groups of threads is a bound
//           below which no kept token lies; the few logits at or above it
//           (with 2 k groups some 1.4 k) are gathered into one block, which
//           makes the draw.
//   top-p   a histogram of the weights by y (32 bins an octave) gives the bin
//           in which the prefix sum crosses; that bin's logits are gathered
//           (or all above it too, if they are few: then the gathering block
//           makes the draw as well). The histogram also tells each block what
//           it keeps, so that only the block with the draw weighs again.
//   else    (huge k, long ties, infinite logits) radix selection on the
//           logits' bits, 8 a level, on counts or sums of weights.
// A filter ends at an item, (~key, index) as one u64: what stands at or
// before it in order stays, so ties need no count of their own.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.cuh"

namespace u32scan {

typedef unsigned long long u64;

constexpr int kSThreads = 512;
constexpr int kSWarps = kSThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kLocal = 1024;  // logits a block may put forward
constexpr int kList = 2048;   // and all blocks of a row together
constexpr int kRanked = 256;  // up to here items are ranked by counting, past it selected by histograms
constexpr int kBins = 1024;   // histogram of y: 32 bins an octave, 31 octaves
constexpr float kLog2e = 0x1.715476p+0f;
constexpr uint32_t kKeyOfMinusInf = 0x007fffffu;

struct SampleArgs {
    const void *logits;
    u64 rows, vocab, row_stride;
    const float *temperature;
    const int32_t *top_k;
    const float *top_p;
    const float *min_p;
    const uint32_t *random;
    int32_t *tokens;
    float *probs;
    unsigned int per_warp;      // 16-byte vectors of a row a warp takes
    unsigned int staged_iters;  // of its ceil(per_warp / 32) turns, those kept in shared memory
    unsigned int ahead;         // rows between a block's row and the one it asks L2 to fetch, or 0
};

// Exchanges between a cluster's blocks: one slot each, so that none is
// written again while a slow block still reads it.
enum Slot { kSlotMax, kSlotFirst, kSlotSecond, kSlotThird, kSlotSum, kSlotTies, kSlotTieAt, kSlotTies2, kSlotTieAt2, kSlotDraw,
            kSlots };

// Sums of u32 by bin, exact in 64 bits at one native shared-memory atomic an
// addition: the carries out of the low words are counted in the high ones.
template <int N>
struct SumBins {
    uint32_t low[N], high[N];
    __device__ __forceinline__ void add(uint32_t bin, uint32_t v) {
        const uint32_t old = atomicAdd(&low[bin], v);
        if (old + v < v) atomicAdd(&high[bin], 1u);
    }
    __device__ __forceinline__ void clear() {
        for (int b = threadIdx.x; b < N; b += kSThreads) low[b] = high[b] = 0u;
    }
};

struct alignas(16) SampleShared {
    u64 list[kLocal];   // this block's: (~key, index), ascending = in order
    u64 gather[kList];  // the cluster's, in the block of rank 0
    union {
        SumBins<kBins> bins;
        SumBins<256> digits[2];
        struct {
            SumBins<kSThreads> sums;
            uint32_t counts[kSThreads];
        } picks;
    };
    u64 slots[kSlots][kMaxCluster][2];
    u64 warp_a[kSWarps], warp_b[kSWarps], warp_c[kSWarps];
    u64 cast[4];
    uint32_t n_list;
};

// ---------------------------------------------------------------------------
// Logits, keys, weights
// ---------------------------------------------------------------------------

// Unsigned order of the keys = order of the logits (-0 counts as +0).
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// Sixteen bytes of a row as floats, and their maximum (of those that are not
// NaN; -inf or NaN if there is none).
template <typename T>
struct Vec;

template <>
struct Vec<float> {
    static constexpr int N = 4;
    static constexpr uint32_t kFill = 0xff800000u;  // -inf
    static __device__ __forceinline__ void unpack(const uint4 &r, float (&x)[4]) {
        x[0] = __uint_as_float(r.x);
        x[1] = __uint_as_float(r.y);
        x[2] = __uint_as_float(r.z);
        x[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ float max(const uint4 &r) {
        return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)),
                     fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
    }
};

template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static constexpr uint32_t kFill = 0xff80ff80u;
    static __device__ __forceinline__ void unpack(const uint4 &r, float (&x)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ float max(const uint4 &r) {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&r);
        const float2 f = __bfloat1622float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
        return fmaxf(f.x, f.y);
    }
};

template <>
struct Vec<__half> {
    static constexpr int N = 8;
    static constexpr uint32_t kFill = 0xfc00fc00u;
    static __device__ __forceinline__ void unpack(const uint4 &r, float (&x)[8]) {
        const __half2 *h = reinterpret_cast<const __half2 *>(&r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(h[j]);
            x[2 * j] = f.x;
            x[2 * j + 1] = f.y;
        }
    }
    static __device__ __forceinline__ float max(const uint4 &r) {
        const __half2 *h = reinterpret_cast<const __half2 *>(&r);
        const float2 f = __half22float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
        return fmaxf(f.x, f.y);
    }
};

// floor(2^31 * 2^-y) for 0 <= y < 100 (0 from y = 31 on): 2^-n exactly, times
// 2^-f on [-1/2, 1/2] by a degree-5 polynomial with constant term 1 (a minimax
// fit in relative error, 1.9e-7 in f32). Every operation is rounded alone (no
// contraction); the coefficients carry the factor 2^31, which changes no
// rounding, and 2^-n is taken off the exponent's bits.
constexpr float kC0 = 0x1p31f, kC1 = -0x1.62e42ap30f, kC2 = 0x1.ebf9bcp28f, kC3 = -0x1.c6b752p26f,
                kC4 = 0x1.3cea88p24f, kC5 = -0x1.5bba14p21f;
constexpr float kRound = 0x1.8p23f;  // adding and taking it away rounds to an integer, ties to even

// p * 2^-n, n in the low bits of t = n + kRound (whose bits << 23 are n << 23).
__device__ __forceinline__ uint32_t scaled_floor(float p, float t) {
    return __float2uint_rz(__uint_as_float(__float_as_uint(p) - (__float_as_uint(t) << 23)));
}

__device__ __forceinline__ uint32_t exp2_weight(float y) {
    const float t = __fadd_rn(y, kRound);
    const float f = __fsub_rn(y, __fsub_rn(t, kRound));
    float p = __fadd_rn(__fmul_rn(kC5, f), kC4);
    p = __fadd_rn(__fmul_rn(p, f), kC3);
    p = __fadd_rn(__fmul_rn(p, f), kC2);
    p = __fadd_rn(__fmul_rn(p, f), kC1);
    p = __fadd_rn(__fmul_rn(p, f), kC0);
    return scaled_floor(p, t);
}

struct RowRule {
    float m, scale;
    uint32_t qmin;
};

// A logit's weight, any logit, any rule.
__device__ __forceinline__ uint32_t token_weight(float x, const RowRule &rule) {
    if (x == rule.m) return 0x80000000u;
    const float y = __fmul_rn(__fsub_rn(rule.m, x), rule.scale);
    if (!(y < 32.0f) || x == -INFINITY) return 0u;
    const uint32_t q = exp2_weight(y);
    return q >= rule.qmin ? q : 0u;
}

// Two logits' distances y and weights before min-p, two operations an
// instruction (each of the pair rounded alone, as above), for a finite m and
// scale: x = m gives y = 0 by itself, -inf and NaN give the clamp's 40 and
// so weight 0.
__device__ __forceinline__ u64 pack2(float a, float b) {
    u64 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(u64 r, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
// a + b as a * 1 + b: one rounding, an addition's. (CUDA 13.0's assembler
// joins a mul.rn.f32x2 and the add.rn.f32x2 of its product into one rounding:
// one weight in twelve came out different. A product and an fma stay apart.)
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
    u64 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(pack2(1.0f, 1.0f)), "l"(b));
    return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
    u64 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// a - b as b * -1 + a: one rounding, a subtraction's
__device__ __forceinline__ u64 sub2(u64 a, u64 b) {
    u64 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(b), "l"(pack2(-1.0f, -1.0f)), "l"(a));
    return r;
}

__device__ __forceinline__ void weigh2(float x0, float x1, u64 m2, u64 scale2, float (&y)[2], uint32_t (&q)[2]) {
    unpack2(mul2(sub2(m2, pack2(x0, x1)), scale2), y[0], y[1]);
    y[0] = fminf(y[0], 40.0f);
    y[1] = fminf(y[1], 40.0f);
    const u64 y2 = pack2(y[0], y[1]);
    const u64 t2 = add2(y2, pack2(kRound, kRound));
    const u64 f2 = sub2(y2, add2(t2, pack2(-kRound, -kRound)));
    u64 p2 = add2(mul2(pack2(kC5, kC5), f2), pack2(kC4, kC4));
    p2 = add2(mul2(p2, f2), pack2(kC3, kC3));
    p2 = add2(mul2(p2, f2), pack2(kC2, kC2));
    p2 = add2(mul2(p2, f2), pack2(kC1, kC1));
    p2 = add2(mul2(p2, f2), pack2(kC0, kC0));
    float t[2], p[2];
    unpack2(t2, t[0], t[1]);
    unpack2(p2, p[0], p[1]);
    q[0] = scaled_floor(p[0], t[0]);
    q[1] = scaled_floor(p[1], t[1]);
}

// The histogram's bin of a distance: the nearest of the bins' centres, so
// bin b holds y in [b - 1/2, b + 1/2] / 32.
__device__ __forceinline__ uint32_t bin_of(float y) {
    return __float_as_uint(__fmaf_rn(y, 32.0f, 8388608.0f)) & (kBins - 1);
}

// ---------------------------------------------------------------------------
// Block and cluster
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ uint32_t at_rank(const void *p, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, u64 a, u64 b) {
    asm volatile("st.shared::cluster.v2.u64 [%0], {%1, %2};" ::"r"(addr), "l"(a), "l"(b) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ u64 ld_cluster_u64(uint32_t addr) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

// Every block's (a, b), given by its threads below the cluster's size, then
// in sh.slots[slot] of every block. A cluster barrier: what blocks wrote to
// their shared memory before it can be read by the others after it.
__device__ __forceinline__ void exchange(SampleShared &sh, Slot slot, u64 a, u64 b) {
    if (threadIdx.x < cluster_size()) st_cluster(at_rank(sh.slots[slot][cluster_rank()], threadIdx.x), a, b);
    cluster_arrive();
    cluster_wait();
}

__device__ __forceinline__ u64 warp_total(u64 v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// The sum over the block, in every thread.
__device__ __forceinline__ u64 block_total(u64 v, u64 *s_warp) {
    v = warp_total(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
    __syncthreads();
    u64 t = 0;
#pragma unroll
    for (int w = 0; w < kSWarps; ++w) t += s_warp[w];
    return t;
}

// The sum over the threads before this one.
__device__ __forceinline__ u64 block_before(u64 v, u64 *s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const u64 o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    u64 base = 0;
#pragma unroll
    for (int w = 0; w < kSWarps; ++w) base += w < warp ? s_warp[w] : 0ull;
    return base + inc - v;
}

__device__ __forceinline__ u64 warp_min(u64 v) {
    const uint32_t high = __reduce_min_sync(0xffffffffu, (uint32_t)(v >> 32));
    const uint32_t low = __reduce_min_sync(0xffffffffu, (uint32_t)(v >> 32) == high ? (uint32_t)v : 0xffffffffu);
    return (u64)high << 32 | low;
}

constexpr int kOwn = kList / kSThreads;  // gathered items a thread holds

// Over the block's items with a weight (those at distinct places): the place
// at which the running sum of weights, in ascending order of place, reaches
// `target` (1 <= target <= the sum of all), and the sum before it. A histogram
// of the places still in question, 512 bins between the least and the
// greatest, then the same within the bin that holds the crossing, until that
// is one item.
__device__ __noinline__ u64 block_select(SampleShared &sh, const u64 (&places)[kOwn], const uint32_t (&weights)[kOwn],
                                         u64 target, u64 *before_it) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 place[kOwn], base = 0;
    uint32_t weight[kOwn];
#pragma unroll
    for (int c = 0; c < kOwn; ++c) {
        place[c] = places[c];
        weight[c] = weights[c];
    }
    while (true) {
        u64 lo = ~0ull, hi = ~0ull;  // hi: complemented, so that both are minima
#pragma unroll
        for (int c = 0; c < kOwn; ++c)
            if (weight[c]) {
                lo = min(lo, place[c]);
                hi = min(hi, ~place[c]);
            }
        lo = warp_min(lo);
        hi = warp_min(hi);
        sh.picks.sums.clear();
        sh.picks.counts[threadIdx.x] = 0;
        if (lane == 0) {
            sh.warp_a[warp] = lo;
            sh.warp_b[warp] = hi;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kSWarps; ++w) {
            lo = min(lo, sh.warp_a[w]);
            hi = min(hi, sh.warp_b[w]);
        }
        const int shift = 55 - __clzll((~hi - lo) | 511ull);
#pragma unroll
        for (int c = 0; c < kOwn; ++c)
            if (weight[c]) {
                const uint32_t bin = (uint32_t)((place[c] - lo) >> shift);
                sh.picks.sums.add(bin, weight[c]);
                atomicAdd(&sh.picks.counts[bin], 1u);
            }
        __syncthreads();
        const u64 mine = (u64)sh.picks.sums.high[threadIdx.x] << 32 | sh.picks.sums.low[threadIdx.x];
        const u64 before = base + block_before(mine, sh.warp_c);
        if (before < target && target <= before + mine) {
            sh.cast[0] = threadIdx.x;
            sh.cast[1] = before;
            sh.cast[2] = sh.picks.counts[threadIdx.x];
        }
        __syncthreads();
        const u64 bin = sh.cast[0], left = sh.cast[2];
        base = sh.cast[1];
        u64 found = ~0ull;
#pragma unroll
        for (int c = 0; c < kOwn; ++c) {
            if ((place[c] - lo) >> shift != bin) weight[c] = 0;
            if (weight[c]) found = place[c];
        }
        if (left == 1) {
            if (found != ~0ull) sh.cast[3] = found;
            __syncthreads();
            *before_it = base;
            return sh.cast[3];
        }
        __syncthreads();  // cast and the bins are written again
    }
}

// ---------------------------------------------------------------------------
// A block's slice of a row
// ---------------------------------------------------------------------------
template <typename T>
struct Slice {
    using V = Vec<T>;
    const char *base;           // the row's address rounded down to 16 bytes
    unsigned int pad, n;        // elements between base and the row, and in the row
    unsigned int v0, nv;        // this warp's first vector; the row's vectors
    unsigned int per_warp, staged_iters;
    uint4 *stage;               // this lane's vectors: turn i at stage[32 * i]

    // Vector v; past the row's ends filled with -inf.
    __device__ __forceinline__ uint4 load(unsigned int v) const {
        const unsigned int p = v * V::N;
        if (p >= pad && p + V::N <= pad + n) return __ldg(reinterpret_cast<const uint4 *>(base) + v);
        uint32_t w[4] = {V::kFill, V::kFill, V::kFill, V::kFill};
        T *e = reinterpret_cast<T *>(w);
#pragma unroll
        for (int j = 0; j < V::N; ++j)
            if (p + j >= pad && p + j < pad + n) e[j] = reinterpret_cast<const T *>(base)[p + j];
        return make_uint4(w[0], w[1], w[2], w[3]);
    }

    // First reading: keeps the staged vectors, returns this thread's maximum.
    __device__ __forceinline__ float first_pass(int lane) const {
        constexpr int U = 4;
        float m = -INFINITY;
        for (unsigned int j = lane, it = 0; j < per_warp && v0 + j < nv; j += 32 * U, it += U) {
            uint4 r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const unsigned int ju = j + 32 * u;
                if (ju < per_warp && v0 + ju < nv) r[u] = load(v0 + ju);
                else r[u] = make_uint4(V::kFill, V::kFill, V::kFill, V::kFill);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                m = fmaxf(m, V::max(r[u]));
                if (it + u < staged_iters) stage[32 * (it + u)] = r[u];
            }
        }
        return m;
    }

    // f(vector, its number) for this lane's vectors, in ascending order.
    template <typename F>
    __device__ __forceinline__ void each(int lane, F f) const {
        for (unsigned int j = lane, it = 0; j < per_warp && v0 + j < nv; j += 32, ++it)
            f(it < staged_iters ? stage[32 * it] : load(v0 + j), v0 + j);
    }

    __device__ __forceinline__ uint32_t index(unsigned int v, int e) const { return v * V::N + e - pad; }

    // The share of the warp `by` warps on in this block.
    __device__ __forceinline__ Slice of_warp(int by) const {
        Slice s = *this;
        s.v0 += by * (int)per_warp;
        s.stage += by * 32 * (int)staged_iters;
        return s;
    }
};

// A logit's place in the filters' order, ascending.
__device__ __forceinline__ u64 item_of(uint32_t key, uint32_t index) { return (u64)~key << 32 | index; }
__device__ __forceinline__ uint32_t item_weight(u64 item, const RowRule &rule) {
    return token_weight(key_logit(~(uint32_t)(item >> 32)), rule);
}
constexpr u64 kKeepAll = ~0ull;

__device__ __forceinline__ void write_token(const SampleArgs &a, u64 row, uint32_t index, u64 q, u64 total) {
    a.tokens[row] = (int32_t)index;
    if (a.probs) a.probs[row] = (float)((double)q / (double)total);
}

__device__ __forceinline__ u64 draw_of(uint32_t word, u64 total) { return __umul64hi((u64)word << 32, total); }

__device__ __forceinline__ u64 top_p_target(float p, u64 total) {
    return (u64)ceil(__dmul_rn((double)p, (double)total));
}

// The sum of what the blocks put into a slot's first word.
__device__ __forceinline__ u64 slot_total(const SampleShared &sh, Slot slot) {
    u64 t = 0;
    for (uint32_t c = 0; c < cluster_size(); ++c) t += sh.slots[slot][c][0];
    return t;
}

// What this warp keeps of the items up to `last`; FINITE: m and scale are.
template <bool FINITE, typename T>
__device__ __forceinline__ u64 kept_mass(const Slice<T> &sl, const RowRule &rule, u64 last) {
    const float thr = last == kKeepAll ? -INFINITY : key_logit(~(uint32_t)(last >> 32));
    const u64 m2 = pack2(rule.m, rule.m), scale2 = pack2(rule.scale, rule.scale);
    u64 mass = 0;
    sl.each(threadIdx.x & 31, [&](const uint4 &r, unsigned int v) {
        if (!(Vec<T>::max(r) >= thr)) return;
        float x[Vec<T>::N];
        Vec<T>::unpack(r, x);
#pragma unroll
        for (int e = 0; e < Vec<T>::N; e += 2) {
            uint32_t q[2];
            if (FINITE) {
                float y[2];
                weigh2(x[e], x[e + 1], m2, scale2, y, q);
            } else {
                q[0] = token_weight(x[e], rule);
                q[1] = token_weight(x[e + 1], rule);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool keep = x[e + i] > thr || (x[e + i] == thr && sl.index(v, e + i) <= (uint32_t)last);
                mass += keep && q[i] >= rule.qmin ? q[i] : 0u;
            }
        }
    });
    return warp_total(mass);
}

// The draw among the items up to `last`, in index order, from what each block
// keeps (the first words of `slot`) and, where it is known, this warp (else m
// and scale are finite). The
// block that holds the draw finds the warp's share that does, and walks it a
// turn of 32 vectors a warp.
template <bool WARPS_KNOWN, typename T>
__device__ __noinline__ void draw(SampleShared &sh, const Slice<T> &own, const RowRule &rule, u64 last, u64 total,
                                  Slot slot, u64 warp_mass, const SampleArgs &a, u64 row) {
    constexpr int N = Vec<T>::N;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const u64 r = draw_of(a.random[row], total);
    u64 before = 0;
    for (uint32_t c = 0; c < cluster_rank(); ++c) before += sh.slots[slot][c][0];
    if (r < before || r - before >= sh.slots[slot][cluster_rank()][0]) return;
    if (!WARPS_KNOWN) warp_mass = kept_mass<true>(own, rule, last);
    __syncthreads();
    if (lane == 0) sh.warp_a[warp] = warp_mass;
    __syncthreads();
    int w = 0;
    while (r - before >= sh.warp_a[w]) before += sh.warp_a[w++];
    const Slice<T> sl = own.of_warp(w - warp);
    for (unsigned int j0 = 0, it0 = 0; j0 < sl.per_warp; j0 += 32 * kSWarps, it0 += kSWarps) {
        const unsigned int it = it0 + warp, j = 32 * it + lane;
        float x[N];
        uint32_t q[N];
        u64 sum = 0;
        const bool in = j < sl.per_warp && sl.v0 + j < sl.nv;
        if (in) Vec<T>::unpack(it < sl.staged_iters ? sl.stage[32 * it] : sl.load(sl.v0 + j), x);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            q[e] = 0;
            if (in && x[e] > -INFINITY && item_of(key_of(x[e]), sl.index(sl.v0 + j, e)) <= last)
                q[e] = token_weight(x[e], rule);
            sum += q[e];
        }
        u64 inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const u64 o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        __syncthreads();
        if (lane == 31) sh.warp_b[warp] = inc;
        __syncthreads();
        u64 turn = before, at = before;
#pragma unroll
        for (int o = 0; o < kSWarps; ++o) {
            if (o == warp) at = turn;
            turn += sh.warp_b[o];
        }
        at += inc - sum;
        if (at <= r && r - at < sum) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                if (at <= r && r - at < q[e]) write_token(a, row, sl.index(sl.v0 + j, e), q[e], total);
                at += q[e];
            }
        }
        if (r < turn) return;
        before = turn;
    }
}

// A key that at least k of the n maxima reach: the lower edge of the bin that
// holds the k-th largest, of 512 between the least and row_key, the greatest;
// then of 512 in that bin, while it spans more than 1/64 of an octave (a
// maximum of -inf widens the first).
__device__ __forceinline__ uint32_t kth_bound(SampleShared &sh, const uint32_t *maxima, uint32_t n, uint32_t k,
                                              uint32_t row_key) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t *counts = sh.picks.counts;
    uint32_t least = row_key;
    for (uint32_t i = threadIdx.x; i < n; i += kSThreads) least = min(least, maxima[i]);
    least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 0) sh.warp_a[warp] = least;
    counts[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSWarps; ++w) least = min(least, (uint32_t)sh.warp_a[w]);
    int shift = 23 - __clz((row_key - least) | 511u);
    uint32_t nearest = 0;  // distance from row_key at which the bins start
    while (true) {
        for (uint32_t i = threadIdx.x; i < n; i += kSThreads) {
            const uint32_t d = row_key - maxima[i];
            if (d >= nearest && (d - nearest) >> shift < kSThreads) atomicAdd(&counts[(d - nearest) >> shift], 1u);
        }
        __syncthreads();
        const uint32_t mine = counts[threadIdx.x];
        const uint32_t before = (uint32_t)block_before(mine, sh.warp_b);
        if (before < k && k <= before + mine) {
            sh.cast[0] = nearest + (threadIdx.x << shift);
            sh.cast[1] = before;
        }
        counts[threadIdx.x] = 0;
        __syncthreads();
        nearest = (uint32_t)sh.cast[0];
        if (shift <= 17) break;
        k -= (uint32_t)sh.cast[1];
        shift -= 9;
        __syncthreads();  // cast is written again
    }
    const u64 far = (u64)nearest + (1ull << shift) - 1;  // the bin's farthest distance
    return far < row_key ? row_key - (uint32_t)far : 0u;
}

// Puts an item into this block's list.
__device__ __forceinline__ void put(SampleShared &sh, u64 item) {
    const uint32_t at = atomicAdd(&sh.n_list, 1u);
    if (at < kLocal) sh.list[at] = item;
}

// The length of all blocks' lists, after an exchange of their lengths as
// `slot`'s first word; over kList when one of them or all do not fit.
__device__ __forceinline__ uint32_t gathered(const SampleShared &sh, Slot slot) {
    uint32_t n = 0;
    for (uint32_t c = 0; c < cluster_size(); ++c) {
        const uint32_t one = (uint32_t)sh.slots[slot][c][0];
        n += one <= kLocal ? one : kList + 1;
    }
    return n;
}

// All blocks' n items, one list after another, in rank 0's gather (called
// there, when they fit): every thread finds its items' blocks by itself, so
// that all of them are on their way at once.
__device__ __forceinline__ void pull(SampleShared &sh, Slot slot, uint32_t n) {
    for (uint32_t i = threadIdx.x; i < n; i += kSThreads) {
        uint32_t c = 0, at = i;
        while (at >= (uint32_t)sh.slots[slot][c][0]) at -= (uint32_t)sh.slots[slot][c++][0];
        sh.gather[i] = ld_cluster_u64(at_rank(sh.list + at, c));
    }
    __syncthreads();
}

// The token among the n gathered items, which hold all that the filters keep:
// the first k of them in order, and of those the top-p prefix (0 < p < 1),
// measured against `total` if that is not 0, else against their own sum.
__device__ __noinline__ void finish_list(SampleShared &sh, uint32_t n, uint32_t k, float p, u64 total,
                                         const RowRule &rule, const SampleArgs &a, u64 row) {
    const bool cut_p = p > 0.0f && p < 1.0f;
    const uint32_t word = a.random[row];
    if (n <= kRanked) {
        // `team` threads an item count what stands before it
        uint32_t team = 2;
        while (team < 16 && 2 * team * n <= kSThreads) team *= 2;
        const uint32_t i = threadIdx.x / team, part = threadIdx.x % team;
        u64 *weight = sh.list;  // pulled: free
        const u64 item = i < n ? sh.gather[i] : ~0ull;
        const u64 q = i < n ? item_weight(item, rule) : 0u;
        if (part == 0) weight[i] = q;
        __syncthreads();
        uint32_t rank = 0;
        u64 before = 0;
#pragma unroll 4
        for (uint32_t j = part; j < n; j += team) {
            const bool first = sh.gather[j] < item;
            rank += first;
            before += first ? weight[j] : 0ull;
        }
        for (uint32_t d = 1; d < team; d *= 2) {
            rank += __shfl_xor_sync(0xffffffffu, rank, d);
            before += __shfl_xor_sync(0xffffffffu, before, d);
        }
        u64 kept = i < n && rank < k ? q : 0ull;
        if (total == 0) total = block_total(part == 0 ? kept : 0ull, sh.warp_a);
        if (cut_p) {
            if (before >= top_p_target(p, total)) kept = 0;
            total = block_total(part == 0 ? kept : 0ull, sh.warp_b);
        }
        __syncthreads();
        if (part == 0) weight[i] = kept;
        __syncthreads();
        u64 at = 0;
#pragma unroll 4
        for (uint32_t j = part; j < n; j += team) at += (uint32_t)sh.gather[j] < (uint32_t)item ? weight[j] : 0ull;
        for (uint32_t d = 1; d < team; d *= 2) at += __shfl_xor_sync(0xffffffffu, at, d);
        const u64 r = draw_of(word, total);
        if (part == 0 && at <= r && r < at + kept) write_token(a, row, (uint32_t)item, kept, total);
        return;
    }
    u64 item[kOwn], before;
    uint32_t q[kOwn], one[kOwn];
#pragma unroll
    for (int c = 0; c < kOwn; ++c) {
        const uint32_t i = threadIdx.x + c * kSThreads;
        one[c] = i < n;
        item[c] = i < n ? sh.gather[i] : ~0ull;
        q[c] = i < n ? item_weight(item[c], rule) : 0u;
    }
    if (k < n) {
        const u64 last = block_select(sh, item, one, k, &before);
#pragma unroll
        for (int c = 0; c < kOwn; ++c)
            if (item[c] > last) q[c] = 0;
    }
    if (total == 0) {
        u64 sum = 0;
#pragma unroll
        for (int c = 0; c < kOwn; ++c) sum += q[c];
        total = block_total(sum, sh.warp_a);
    }
    if (cut_p) {
        const u64 last = block_select(sh, item, q, top_p_target(p, total), &before);
#pragma unroll
        for (int c = 0; c < kOwn; ++c)
            if (item[c] > last) q[c] = 0;
        total = before + item_weight(last, rule);
    }
#pragma unroll
    for (int c = 0; c < kOwn; ++c) item[c] &= 0xffffffffull;  // the index: the draw's order
    const u64 index = block_select(sh, item, q, draw_of(word, total) + 1, &before);
#pragma unroll
    for (int c = 0; c < kOwn; ++c)
        if (q[c] && item[c] == index) write_token(a, row, (uint32_t)index, q[c], total);
}

// The key at which the running total over the items up to `last`, keys in
// descending order, of counts or of weights (MASS), first reaches `target`
// (1 <= target <= the whole total), and what is missing above it (>= 1).
// `level` numbers the levels of a row's selections (their two buffers swap:
// a slow block may still read the last level's).
template <bool MASS, typename T>
__device__ __noinline__ void radix_select(SampleShared &sh, const Slice<T> &sl, const RowRule &rule, u64 last,
                                          u64 target, int &level, uint32_t *tau, u64 *missing) {
    uint32_t prefix = 0, mask = 0;
    for (int shift = 24; shift >= 0; shift -= 8, ++level) {
        SumBins<256> &hist = sh.digits[level & 1];
        hist.clear();
        __syncthreads();
        sl.each(threadIdx.x & 31, [&](const uint4 &r, unsigned int v) {
            float x[Vec<T>::N];
            Vec<T>::unpack(r, x);
#pragma unroll 1
            for (int e = 0; e < Vec<T>::N; ++e) {
                if (x[e] != x[e]) x[e] = -INFINITY;
                const uint32_t k = key_of(x[e]);
                if ((k & mask) != prefix || item_of(k, sl.index(v, e)) > last) continue;
                const uint32_t w = MASS ? token_weight(x[e], rule) : 1u;
                if (w) hist.add((k >> shift) & 255u, w);
            }
        });
        cluster_arrive();
        cluster_wait();
        // the digits in descending order: thread t has digit 255 - t
        u64 mine = 0;
        if (threadIdx.x < 256)
            for (uint32_t c = 0; c < cluster_size(); ++c)
                mine += (u64)ld_cluster(at_rank(&hist.low[255 - threadIdx.x], c)) +
                        ((u64)ld_cluster(at_rank(&hist.high[255 - threadIdx.x], c)) << 32);
        const u64 before = block_before(mine, sh.warp_a);
        if (before < target && target <= before + mine) {
            sh.cast[0] = 255u - threadIdx.x;
            sh.cast[1] = target - before;
        }
        __syncthreads();
        prefix |= (uint32_t)sh.cast[0] << shift;
        mask |= 255u << shift;
        target = sh.cast[1];
        __syncthreads();
    }
    *tau = prefix;
    *missing = target;
}

// The `nth` logit (from 1, by index) with key tau, as an item; -inf entries
// past the row's ends do not count.
template <typename T>
__device__ __noinline__ u64 nth_tie(SampleShared &sh, const Slice<T> &sl, uint32_t tau, u64 nth, Slot ties_slot,
                                    Slot at_slot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto tied = [&](const uint4 &r, unsigned int v) {  // by element
        float x[Vec<T>::N];
        Vec<T>::unpack(r, x);
        unsigned int t = 0;
#pragma unroll
        for (int e = 0; e < Vec<T>::N; ++e) {
            if (x[e] != x[e]) x[e] = -INFINITY;
            if (key_of(x[e]) == tau && sl.index(v, e) < sl.n) t |= 1u << e;
        }
        return t;
    };
    u64 mine = 0;
    sl.each(lane, [&](const uint4 &r, unsigned int v) { mine += __popc(tied(r, v)); });
    mine = warp_total(mine);
    __syncthreads();
    if (lane == 0) sh.warp_a[warp] = mine;
    if (threadIdx.x == 0) sh.cast[0] = ~0ull;
    __syncthreads();
    u64 before = 0, block_ties = 0;
    for (int w = 0; w < kSWarps; ++w) {
        before += w < warp ? sh.warp_a[w] : 0ull;
        block_ties += sh.warp_a[w];
    }
    exchange(sh, ties_slot, block_ties, 0);
    for (uint32_t c = 0; c < cluster_rank(); ++c) before += sh.slots[ties_slot][c][0];
    if (before < nth && nth <= before + mine)  // this warp's
        for (unsigned int j0 = 0, it = 0; j0 < sl.per_warp; j0 += 32, ++it) {
            const unsigned int j = j0 + lane;
            unsigned int t = 0;
            if (j < sl.per_warp && sl.v0 + j < sl.nv)
                t = tied(it < sl.staged_iters ? sl.stage[32 * it] : sl.load(sl.v0 + j), sl.v0 + j);
            u64 inc = __popc(t);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const u64 o = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += o;
            }
            const u64 at = before + inc - __popc(t);
            if (at < nth && nth <= before + inc) {
                for (u64 skip = nth - at - 1; skip > 0; --skip) t &= t - 1;
                sh.cast[0] = item_of(tau, sl.index(sl.v0 + j, __ffs(t) - 1));
            }
            before += __shfl_sync(0xffffffffu, inc, 31);
        }
    __syncthreads();
    exchange(sh, at_slot, sh.cast[0], 0);
    u64 item = ~0ull;
    for (uint32_t c = 0; c < cluster_size(); ++c) item = min(item, sh.slots[at_slot][c][0]);
    return item;
}

// The filters by selection on the logits' bits, then the draw: right for
// every row, and the way of those the other paths do not take.
template <typename T>
__device__ __noinline__ void sample_by_selection(SampleShared &sh, const Slice<T> &sl, const RowRule &rule, uint32_t k,
                                                 float p, const SampleArgs &a, u64 row) {
    u64 last = kKeepAll, missing;
    uint32_t tau;
    int level = 0;
    if (k > 0) {
        radix_select<false>(sh, sl, rule, kKeepAll, k, level, &tau, &missing);
        if (tau > kKeyOfMinusInf) last = nth_tie(sh, sl, tau, missing, kSlotTies, kSlotTieAt);
    }
    u64 mass = kept_mass<false>(sl, rule, last);
    exchange(sh, kSlotSum, block_total((threadIdx.x & 31) == 0 ? mass : 0ull, sh.warp_c), 0);
    u64 total = slot_total(sh, kSlotSum);
    if (p > 0.0f && p < 1.0f) {
        const u64 want = top_p_target(p, total);
        radix_select<true>(sh, sl, rule, last, want, level, &tau, &missing);
        const u64 q = token_weight(key_logit(tau), rule), ties = (missing + q - 1) / q;
        last = nth_tie(sh, sl, tau, ties, kSlotTies2, kSlotTieAt2);
        total = want - missing + ties * q;
        mass = kept_mass<false>(sl, rule, last);
        exchange(sh, kSlotDraw, block_total((threadIdx.x & 31) == 0 ? mass : 0ull, sh.warp_c), 0);
        draw<true>(sh, sl, rule, last, total, kSlotDraw, mass, a, row);
        return;
    }
    draw<true>(sh, sl, rule, last, total, kSlotSum, mass, a, row);
}

template <typename T>
__global__ void __launch_bounds__(kSThreads, 2) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) unsigned char s_mem[];
    SampleShared &sh = *reinterpret_cast<SampleShared *>(s_mem);
    using V = Vec<T>;
    const uint32_t rank = cluster_rank(), blocks = cluster_size();
    const u64 row = blockIdx.x / blocks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    cluster_arrive();  // paired with the wait before the first exchange: every block has started
    if (threadIdx.x == 0) sh.n_list = 0;

    Slice<T> sl;
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(static_cast<const T *>(a.logits) + row * a.row_stride);
        sl.base = reinterpret_cast<const char *>(at & ~(uintptr_t)15);
        sl.pad = (unsigned int)(at & 15) / sizeof(T);
        sl.n = (unsigned int)a.vocab;
        sl.nv = (sl.pad + sl.n + V::N - 1) / V::N;
        sl.per_warp = a.per_warp;
        sl.staged_iters = a.staged_iters;
        sl.v0 = (rank * kSWarps + warp) * a.per_warp;
        sl.stage = reinterpret_cast<uint4 *>(s_mem + sizeof(SampleShared)) + warp * 32 * a.staged_iters + lane;
    }
    const float t = a.temperature ? a.temperature[row] : 1.0f;
    const int k_arg = a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.0f;
    const float mp = a.min_p ? a.min_p[row] : 0.0f;
    const uint32_t k = k_arg > 0 && (uint32_t)k_arg < sl.n ? (uint32_t)k_arg : 0u;
    const bool cut_p = p > 0.0f && p < 1.0f;

    // The blocks that run after these find their rows in L2: HBM stays busy while these compute
    // (256 rows of 262144 f32: @@ us without, @@ with).
    if (a.ahead && threadIdx.x == 0 && row + a.ahead < a.rows) {
        const uintptr_t from = reinterpret_cast<uintptr_t>(static_cast<const T *>(a.logits) +
                                                           (row + a.ahead) * a.row_stride);
        const uintptr_t first = (from + 15) & ~(uintptr_t)15, end = (from + a.vocab * sizeof(T)) & ~(uintptr_t)15;
        const uintptr_t at = first + (uintptr_t)rank * kSWarps * a.per_warp * 16;
        if (at < end) {
            const uintptr_t bytes = min(end - at, (uintptr_t)kSWarps * a.per_warp * 16);
            bulk_prefetch_l2(reinterpret_cast<const void *>(at), (unsigned int)bytes);
        }
    }

    // the row's largest logit, and for top-k the maxima its bound comes from
    const float thread_max = sl.first_pass(lane);
    const uint32_t thread_key = key_of(thread_max == thread_max ? thread_max : -INFINITY);
    const uint32_t warp_key = __reduce_max_sync(0xffffffffu, thread_key);
    if (lane == 0) sh.warp_a[warp] = warp_key;
    // top-k: maxima of groups of threads, at least 2 k groups in the row
    uint32_t group = 32;
    while (group > 1 && kSThreads / group * blocks < 2 * k) group /= 2;
    const uint32_t groups = kSThreads / group;
    const bool bounded = k > 0 && (sl.n <= kLocal || 2 * k <= groups * blocks);
    const bool by_groups = bounded && sl.n > kLocal;
    uint32_t group_key = warp_key;
    if (by_groups && group < 32) {
        group_key = thread_key;
        for (uint32_t d = 1; d < group; d *= 2) group_key = max(group_key, __shfl_xor_sync(0xffffffffu, group_key, d));
    }
    __syncthreads();
    uint32_t block_key = 0;
#pragma unroll
    for (int w = 0; w < kSWarps; ++w) block_key = max(block_key, (uint32_t)sh.warp_a[w]);
    cluster_wait();
    uint32_t *maxima = reinterpret_cast<uint32_t *>(sh.gather);  // of all the row's groups
    if (by_groups && threadIdx.x % group == 0)
        for (uint32_t c = 0; c < blocks; ++c)
            st_cluster(at_rank(maxima + rank * groups + threadIdx.x / group, c), group_key);
    exchange(sh, kSlotMax, block_key, 0);
    uint32_t row_key = 0;
    for (uint32_t c = 0; c < blocks; ++c) row_key = max(row_key, (uint32_t)sh.slots[kSlotMax][c][0]);
    if (row_key <= kKeyOfMinusInf) {  // the mask leaves nothing
        if (rank == 0 && threadIdx.x == 0) {
            a.tokens[row] = -1;
            if (a.probs) a.probs[row] = 0.0f;
        }
        return;
    }
    RowRule rule;
    rule.m = key_logit(row_key);
    rule.scale = __fdiv_rn(kLog2e, t);
    rule.qmin = mp > 0.0f ? (uint32_t)ceil((double)fminf(mp, 1.0f) * 2147483648.0) : 0u;

    if (!(t > 0.0f)) {  // the first of the largest
        uint32_t first = 0xffffffffu;
        if (block_key == row_key)
            sl.each(lane, [&](const uint4 &r, unsigned int v) {
                if (first != 0xffffffffu || !(V::max(r) >= rule.m)) return;
                float x[V::N];
                V::unpack(r, x);
#pragma unroll
                for (int e = V::N - 1; e >= 0; --e)
                    if (x[e] == rule.m) first = sl.index(v, e);
            });
        first = __reduce_min_sync(0xffffffffu, first);
        if (lane == 0) sh.warp_b[warp] = first;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kSWarps; ++w) first = min(first, (uint32_t)sh.warp_b[w]);
        exchange(sh, kSlotFirst, first, 0);
        if (rank == 0 && threadIdx.x == 0) {
            for (uint32_t c = 0; c < blocks; ++c) first = min(first, (uint32_t)sh.slots[kSlotFirst][c][0]);
            a.tokens[row] = (int32_t)first;
            if (a.probs) a.probs[row] = 1.0f;
        }
        return;
    }
    const bool finite = rule.m < INFINITY && rule.scale < INFINITY;
    if (finite && bounded) {
        const uint32_t bound = by_groups ? kth_bound(sh, maxima, groups * blocks, k, row_key) : 0u;
        const float thr = bound > kKeyOfMinusInf ? key_logit(bound) : -INFINITY;
        sl.each(lane, [&](const uint4 &r, unsigned int v) {
            if (!(V::max(r) >= thr)) return;
            float x[V::N];
            V::unpack(r, x);
#pragma unroll
            for (int e = 0; e < V::N; ++e)
                if (x[e] >= thr && x[e] > -INFINITY) put(sh, item_of(key_of(x[e]), sl.index(v, e)));
        });
        __syncthreads();
        exchange(sh, kSlotFirst, sh.n_list, 0);
        const uint32_t n = gathered(sh, kSlotFirst);
        if (n <= kList) {
            if (rank == 0) pull(sh, kSlotFirst, n);
            cluster_arrive();
            if (rank == 0) finish_list(sh, n, k, p, 0ull, rule, a, row);
            cluster_wait();
            return;
        }
    } else if (finite && k == 0) {
        // All weights; for top-p also their histogram by distance, as far as it can matter: past
        // cut_y the row holds less than (1 - p) of the largest weight. Logits below `zero` weigh
        // nothing (y > 31).
        const u64 m2 = pack2(rule.m, rule.m), scale2 = pack2(rule.scale, rule.scale);
        const float zero = __fsub_rd(rule.m, __fdiv_ru(31.5f, rule.scale));
        u64 mass = 0;
        if (!cut_p) {
            sl.each(lane, [&](const uint4 &r, unsigned int) {
                if (!(V::max(r) >= zero)) return;
                float x[V::N];
                V::unpack(r, x);
#pragma unroll
                for (int e = 0; e < V::N; e += 2) {
                    float y[2];
                    uint32_t q[2];
                    weigh2(x[e], x[e + 1], m2, scale2, y, q);
                    mass += q[0] >= rule.qmin ? q[0] : 0u;
                    mass += q[1] >= rule.qmin ? q[1] : 0u;
                }
            });
            mass = warp_total(mass);
            exchange(sh, kSlotFirst, block_total(lane == 0 ? mass : 0ull, sh.warp_c), 0);
            draw<true>(sh, sl, rule, kKeepAll, slot_total(sh, kSlotFirst), kSlotFirst, mass, a, row);
            return;
        }
        const float cut_y = fminf(31.0f, log2f((float)sl.n / (1.0f - p)) + 0.1f);
        const uint32_t floor_q = max(max(rule.qmin, exp2_weight(cut_y)), 1u);  // the histogram's least weight
        sh.bins.clear();
        __syncthreads();
        sl.each(lane, [&](const uint4 &r, unsigned int) {
            if (!(V::max(r) >= zero)) return;
            float x[V::N];
            V::unpack(r, x);
#pragma unroll
            for (int e = 0; e < V::N; e += 2) {
                float y[2];
                uint32_t q[2];
                weigh2(x[e], x[e + 1], m2, scale2, y, q);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mass += q[i] >= rule.qmin ? q[i] : 0u;
                    if (q[i] >= floor_q) sh.bins.add(bin_of(y[i]), q[i]);
                }
            }
        });
        exchange(sh, kSlotFirst, block_total(mass, sh.warp_c), 0);
        const u64 total = slot_total(sh, kSlotFirst), want = top_p_target(p, total);
        // the bin in which the running sum reaches `want`, two bins a thread
        u64 low[kMaxCluster], high[kMaxCluster];
#pragma unroll
        for (uint32_t c = 0; c < kMaxCluster; ++c) {
            low[c] = c < blocks ? ld_cluster_u64(at_rank(&sh.bins.low[2 * threadIdx.x], c)) : 0ull;
            high[c] = c < blocks ? ld_cluster_u64(at_rank(&sh.bins.high[2 * threadIdx.x], c)) : 0ull;
        }
        u64 bin_mass[2] = {0, 0};
#pragma unroll
        for (uint32_t c = 0; c < kMaxCluster; ++c) {
            bin_mass[0] += (low[c] & 0xffffffffull) | high[c] << 32;
            bin_mass[1] += low[c] >> 32 | (high[c] >> 32) << 32;
        }
        // at most so many logits with a weight lie in a bin: none weighs less than its far end,
        // less more than the recipe's error
        u64 at_most[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t far = exp2_weight(((float)(2 * threadIdx.x + i) + 0.5f) * (1.0f / 32.0f));
            const uint32_t slack = (far >> 16) + 2;
            const uint32_t least = max(far > slack ? far - slack : 0u, floor_q);
            at_most[i] = (u64)(__fdividef((float)bin_mass[i], (float)least) * 1.001f) + (bin_mass[i] ? 1u : 0u);
        }
        const u64 own[2] = {(u64)sh.bins.high[2 * threadIdx.x] << 32 | sh.bins.low[2 * threadIdx.x],
                            (u64)sh.bins.high[2 * threadIdx.x + 1] << 32 | sh.bins.low[2 * threadIdx.x + 1]};
        const u64 before = block_before(bin_mass[0] + bin_mass[1], sh.warp_a);
        const u64 count_before = block_before(at_most[0] + at_most[1], sh.warp_b);
        if (before < want && want <= before + bin_mass[0] + bin_mass[1]) {
            const bool second = want > before + bin_mass[0];
            sh.cast[0] = 2 * threadIdx.x + second;
            sh.cast[1] = before + (second ? bin_mass[0] : 0ull);
            sh.cast[2] = count_before + at_most[0] + (second ? at_most[1] : 0ull);
        }
        __syncthreads();
        const uint32_t bin = (uint32_t)sh.cast[0];
        const u64 above = sh.cast[1];
        const bool all = sh.cast[2] <= kList;
        const u64 block_above = block_total((2 * threadIdx.x < bin ? own[0] : 0ull) +
                                                (2 * threadIdx.x + 1 < bin ? own[1] : 0ull), sh.warp_c);
        // every logit in a bin up to this one is at or above thr, every one in a bin from it on at
        // or below cap
        const float thr = __fsub_rd(rule.m, __fdiv_ru(((float)bin + 1.0f) * (1.0f / 32.0f), rule.scale));
        const float cap = all || bin == 0 ? INFINITY
                                          : __fsub_ru(rule.m, __fdiv_rd(((float)bin - 1.0f) * (1.0f / 32.0f), rule.scale));
        sl.each(lane, [&](const uint4 &r, unsigned int v) {
            if (!(V::max(r) >= thr)) return;
            float x[V::N];
            V::unpack(r, x);
            unsigned int near = 0;
#pragma unroll
            for (int e = 0; e < V::N; ++e)
                if (x[e] >= thr && x[e] <= cap) near |= 1u << e;
#pragma unroll 1
            for (; near; near &= near - 1) {
                const int e = __ffs(near) - 1;
                float xe = x[0];
#pragma unroll
                for (int i = 1; i < V::N; ++i) xe = e == i ? x[i] : xe;
                const float y = __fmul_rn(__fsub_rn(rule.m, xe), rule.scale);
                if (!(y < 32.0f) || exp2_weight(y) < floor_q) continue;
                const uint32_t b = bin_of(y);
                if (all ? b <= bin : b == bin) put(sh, item_of(key_of(xe), sl.index(v, e)));
            }
        });
        __syncthreads();
        exchange(sh, kSlotSecond, sh.n_list, 0);
        const uint32_t n = gathered(sh, kSlotSecond);
        if (n <= kList) {
            if (rank == 0) pull(sh, kSlotSecond, n);
            if (all) {
                cluster_arrive();
                if (rank == 0) finish_list(sh, n, 0xffffffffu, p, total, rule, a, row);
                cluster_wait();
                return;
            }
            u64 last = 0, left = 0;
            if (rank == 0) {  // the crossing among the gathered
                u64 item[kOwn];
                uint32_t q[kOwn];
#pragma unroll
                for (int c = 0; c < kOwn; ++c) {
                    const uint32_t i = threadIdx.x + c * kSThreads;
                    item[c] = i < n ? sh.gather[i] : ~0ull;
                    q[c] = i < n ? item_weight(item[c], rule) : 0u;
                }
                last = block_select(sh, item, q, want - above, &left);
                left += above + item_weight(last, rule);
            }
            exchange(sh, kSlotThird, last, left);
            last = sh.slots[kSlotThird][0][0];
            left = sh.slots[kSlotThird][0][1];
            // this block's part: its bins before the crossing one, and its items up to the crossing
            u64 part = 0;
            for (uint32_t i = threadIdx.x; i < sh.n_list; i += kSThreads)
                if (sh.list[i] <= last) part += item_weight(sh.list[i], rule);
            exchange(sh, kSlotDraw, block_total(part, sh.warp_c) + block_above, 0);
            draw<false>(sh, sl, rule, last, left, kSlotDraw, 0ull, a, row);
            return;
        }
    }
    sample_by_selection(sh, sl, rule, k, p, a, row);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Turns of 32 vectors a warp keeps in shared memory: two blocks an SM.
constexpr unsigned int kStageBytes = kSWarps * 32 * 16;
constexpr unsigned int kMaxStaged = 9;
static_assert(sizeof(SampleShared) % 16 == 0 && offsetof(SampleShared, slots) % 16 == 0, "16-byte accesses");
static_assert(2 * (sizeof(SampleShared) + kMaxStaged * kStageBytes + 1024) <= 228 * 1024, "two blocks an SM");

template <typename T>
static int sample_launch(SampleArgs a, cudaStream_t stream) {
    // The smallest cluster whose slices fit shared memory, then larger while
    // blocks are fewer than the GPU holds and a thread keeps a vector.
    const unsigned int nv = (unsigned int)((a.vocab + 2 * Vec<T>::N - 2) / Vec<T>::N);
    unsigned int blocks = 1;
    while (blocks < kMaxCluster &&
           (nv > blocks * kMaxStaged * kSThreads || (a.rows * blocks < 256 && nv > blocks * kSThreads)))
        blocks *= 2;
    const unsigned int per_block = (nv + blocks - 1) / blocks;
    a.per_warp = ((per_block + kSWarps - 1) / kSWarps + 7) / 8 * 8;
    const unsigned int iters = (a.per_warp + 31) / 32;
    a.staged_iters = iters < kMaxStaged ? iters : kMaxStaged;
    const size_t smem = sizeof(SampleShared) + (size_t)a.staged_iters * kStageBytes;
    if (cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(sizeof(SampleShared) + kMaxStaged * kStageBytes)) != cudaSuccess)
        return U32SCAN_ECUDA;
    const unsigned int resident = 2 * 152 / blocks;  // rows at a time
    a.ahead = a.rows > resident ? resident : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned int)a.rows * blocks);
    cfg.blockDim = dim3(kSThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<T>, (const SampleArgs)a) == cudaSuccess ? U32SCAN_OK : U32SCAN_ECUDA;
}

}  // namespace u32scan

using namespace u32scan;
extern "C" int sample_tokens(const void *logits, int type, size_t rows, size_t vocab, size_t row_stride,
                             const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                             const uint32_t *random, int32_t *tokens, float *probs, u32scan_stream_t stream) {
    if (type != U32SCAN_F32 && type != U32SCAN_F16 && type != U32SCAN_BF16) return U32SCAN_EINVAL;
    if (rows >= (1ull << 28) || vocab > U32SCAN_MAX_VOCAB || row_stride >= (1ull << 32)) return U32SCAN_EINVAL;
    if (rows == 0) return U32SCAN_OK;
    const uintptr_t elem = type == U32SCAN_F32 ? 3 : 1;
    if ((vocab > 0 && logits == nullptr) || random == nullptr || tokens == nullptr) return U32SCAN_EINVAL;
    if (reinterpret_cast<uintptr_t>(logits) & elem) return U32SCAN_EINVAL;
    for (const void *p : {(const void *)temperature, (const void *)top_k, (const void *)top_p, (const void *)min_p,
                          (const void *)random, (const void *)tokens, (const void *)probs})
        if (reinterpret_cast<uintptr_t>(p) & 3) return U32SCAN_EINVAL;
    const SampleArgs a{logits, rows, vocab, row_stride, temperature, top_k, top_p, min_p, random, tokens, probs, 0, 0, 0};
    const cudaStream_t s = (cudaStream_t)stream;
    if (type == U32SCAN_F32) return sample_launch<float>(a, s);
    if (type == U32SCAN_F16) return sample_launch<__half>(a, s);
    return sample_launch<__nv_bfloat16>(a, s);
}
