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
// L2), so the passes after the maximum touch no HBM, and skips what lies below
// a bound 32 vectors at a time. No row is sorted:
//   top-k   the k-th largest of the maxima of groups of threads is a bound
//           below which no kept token lies; the few logits at or above it
//           (with 2 k groups some 1.4 k) are gathered into one block, which
//           makes the draw. Where a row has fewer than 2 k groups: as top-p,
//           with counts for weights.
//   top-p   a histogram of the weights by y (32 bins an octave) gives the bin
//           in which the prefix sum crosses; that bin's logits are gathered
//           (or all above it too, if they are few: then the gathering block
//           makes the draw as well). The histogram also tells each half of a
//           block what it keeps, so that only the half with the draw weighs
//           again. A bin with more logits than are gathered (long ties, flat
//           rows) is searched by radix selection on its logits' bits.
// A filter ends at an item, (~key, index) as one u64: what stands at or
// before it in order stays, so ties need no count of their own.
//
// What every row runs is in line, from the first reading to the draw: a call
// spills the slice and the rule that stay in registers otherwise (256 x 131072
// f32 under top-p 137 us with calls, 119 without; 64 x 131072 bf16 38.6, 35.4).
// Only what few rows need (long ties, rows' ends) and the selections are calls.
//
// Measured on one GB300, launches back to back: a row of 32000 bf16 under
// top-k and top-p 8 us; 7 x 50257 f32 greedy 4, without filters 7, under top-k
// 50 9, under top-p 12 (peaked) to 16 (flat); 64 x 131072 bf16 without
// filters 16, under top-p 35; 256 x 262144 f32, a fifth of the rows greedy, most
// others under top-k, top-p or both, 112 (268 MB: 2.4 TB/s, where reading alone
// takes 40; DRAM 30 % busy). What bounds it is waiting more than issue, and
// neither is HBM's rate. A logit's weight is 15 f32 operations that round one by
// one, and some 30 instructions with its place in the histogram (3.6 logits a
// clock and SM); with the later passes top-p takes 66 instructions a bf16 logit,
// which the SMs would issue in 14 of the 35 us. The rest are barriers and short steps
// between them, a cluster's 500 clocks or more each. Of the 256 rows' 112 us issue
// is 30: three quarters of an f32 slice are not staged and come from L2 in every
// pass, one load a lane ahead, and rows of unequal work leave SMs idle at the end.
// (Instructions are issued in 50 and 39 % of the cycles in which an SM is at work.)
// Two blocks of 16 warps an SM, 64 registers a thread: while one waits at a barrier
// the other weighs.
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
constexpr int kHits = kLocal;  // vectors with such logits (warp, its vector: 16 bits each)
constexpr int kList = 2048;   // and all blocks of a row together
constexpr int kRanked = 256;  // up to here items are ranked by counting, past it selected by histograms
constexpr int kTurns = 64;    // turns (of 32 vectors) a warp remembers the maximum of
constexpr int kFew = 64;      // up to here a selection's last items are (eight threads each)
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
    unsigned int per_warp;      // vectors of a row a warp takes
    unsigned int staged_iters;  // of its ceil(per_warp / 32) turns, those kept in shared memory
};

// Exchanges between a cluster's blocks: one slot each, so that none is
// written again while a slow block still reads it.
enum Slot {
    kSlotBound,     // lengths of the lists above the bound
    kSlotFirst,     // greedy: the least index; no list: weights
    kSlotCountList, // top-k by histogram: lengths of lists, ties, the tie
    kSlotCountTies,
    kSlotCountTie,
    kSlotSumList,   // top-p: lengths of lists and weights above, ties, the tie
    kSlotSumTies,
    kSlotSumTie,
    kSlots
};

// Sums of u32 by bin, exact in 64 bits at one native shared-memory atomic an
// addition: the carries out of the low words are counted in the high ones.
template <int N>
struct SumBins {
    uint32_t low[N], high[N];
    __device__ __forceinline__ void add(uint32_t bin, uint32_t v) {
        const uint32_t old = atomicAdd(&low[bin], v);
        if (old + v < v) atomicAdd(&high[bin], 1u);
    }
    // add() of those that are at least floor, all on their way before the
    // first carry is looked at.
    template <int M>
    __device__ __forceinline__ void add_from(uint32_t floor, const uint32_t (&bin)[M], const uint32_t (&v)[M]) {
        uint32_t old[M];
#pragma unroll
        for (int i = 0; i < M; ++i) {
            old[i] = 0;
            if (v[i] >= floor) old[i] = atomicAdd(&low[bin[i]], v[i]);
        }
        bool carry = false;
#pragma unroll
        for (int i = 0; i < M; ++i) carry |= old[i] > ~v[i];
        if (carry) {
#pragma unroll
            for (int i = 0; i < M; ++i)
                if (old[i] > ~v[i]) atomicAdd(&high[bin[i]], 1u);
        }
    }
    __device__ __forceinline__ void clear() {
        for (int b = threadIdx.x; b < N; b += kSThreads) low[b] = high[b] = 0u;
    }
};

struct alignas(16) SampleShared {
    u64 items[kLocal + kList];  // (~key, index), ascending = in order: this block's list, then all blocks'
    union {
        SumBins<kBins> bins[2];  // of the block's two halves
        SumBins<256> digits[2];
        struct {
            union {
                SumBins<kSThreads> sums;
                struct {
                    u64 place[kFew];
                    uint32_t weight[kFew], from[kFew];
                } few;
            };
            uint32_t counts[kSThreads];
            uint32_t weights[kList];
        } picks;
        uint32_t hits[kHits];
    };
    u64 slots[kSlots][kMaxCluster][2];
    uint32_t turn_key[kSWarps][kTurns];  // the key of a turn's largest logit
    uint32_t warp_keys[kMaxCluster][kSWarps];  // the keys of all warps' largest logits
    u64 warp[3][kSWarps];
    u64 cast[6];
    uint32_t n_list, n_hits;
};

// The block's, at the start of its dynamic shared memory; named here and not
// handed on by reference, so that every access is known to be to shared memory.
__device__ __forceinline__ SampleShared &block_shared() {
    extern __shared__ __align__(16) unsigned char s_mem[];
    return *reinterpret_cast<SampleShared *>(s_mem);
}

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

// Eight logits of a row, as they are read (Raw) and as floats; their maximum
// (of those that are not NaN; -inf or NaN if there is none); whether any lies in
// [from(lo), upto(hi)], the bounds rounded inwards to the logits' type. Staged,
// a turn's vectors lie 16 bytes of each lane after 16 bytes of each. (With four
// f32 a vector the loops' own instructions weigh twice as much: 256 x 131072
// under top-p 149 us and 138, 256 x 262144 of mixed settings 135 and 130.)
struct Vec16 {  // what f16 and bf16 share
    static constexpr int N = 8;
    typedef uint4 Raw;
    static __device__ __forceinline__ Raw load(const char *p) { return __ldg(reinterpret_cast<const uint4 *>(p)); }
    static __device__ __forceinline__ void put(uint4 *stage, const Raw &r) { *stage = r; }
    static __device__ __forceinline__ Raw get(const uint4 *stage) { return *stage; }
};

template <typename T>
struct Vec;

template <>
struct Vec<float> {
    static constexpr int N = 8;
    static constexpr uint32_t kFill = 0xff800000u;  // -inf
    struct Raw {
        uint4 a, b;
    };
    static __device__ __forceinline__ Raw load(const char *p) {
        Raw r;
        asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=r"(r.a.x), "=r"(r.a.y), "=r"(r.a.z), "=r"(r.a.w), "=r"(r.b.x), "=r"(r.b.y), "=r"(r.b.z), "=r"(r.b.w)
            : "l"(p));
        return r;
    }
    static __device__ __forceinline__ void put(uint4 *stage, const Raw &r) {
        stage[0] = r.a;
        stage[32] = r.b;
    }
    static __device__ __forceinline__ Raw get(const uint4 *stage) { return {stage[0], stage[32]}; }
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[8]) {
        const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(w[e]);
    }
    typedef float Bound;
    static __device__ __forceinline__ Bound from(float lo) { return lo; }
    static __device__ __forceinline__ Bound upto(float hi) { return hi; }
    static __device__ __forceinline__ bool any_in(const Raw &r, Bound lo, Bound hi) {
        float x[8];
        unpack(r, x);
        bool any = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) any |= x[e] >= lo && x[e] <= hi;
        return any;
    }
    static __device__ __forceinline__ float max(const Raw &r) {
        float x[8];
        unpack(r, x);
        return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    }
};

template <>
struct Vec<__nv_bfloat16> : Vec16 {
    static constexpr uint32_t kFill = 0xff80ff80u;
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
    typedef __nv_bfloat162 Bound;
    static __device__ __forceinline__ Bound from(float lo) { return __bfloat162bfloat162(__float2bfloat16_ru(lo)); }
    static __device__ __forceinline__ Bound upto(float hi) { return __bfloat162bfloat162(__float2bfloat16_rd(hi)); }
    static __device__ __forceinline__ bool any_in(const Raw &r, Bound lo, Bound hi) {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&r);
        unsigned int any = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) any |= __hge2_mask(h[j], lo) & __hle2_mask(h[j], hi);
        return any != 0;
    }
    static __device__ __forceinline__ float max(const Raw &r) {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&r);
        const float2 f = __bfloat1622float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
        return fmaxf(f.x, f.y);
    }
};

template <>
struct Vec<__half> : Vec16 {
    static constexpr uint32_t kFill = 0xfc00fc00u;
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[8]) {
        const __half2 *h = reinterpret_cast<const __half2 *>(&r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(h[j]);
            x[2 * j] = f.x;
            x[2 * j + 1] = f.y;
        }
    }
    typedef __half2 Bound;
    static __device__ __forceinline__ Bound from(float lo) { return __half2half2(__float2half_ru(lo)); }
    static __device__ __forceinline__ Bound upto(float hi) { return __half2half2(__float2half_rd(hi)); }
    static __device__ __forceinline__ bool any_in(const Raw &r, Bound lo, Bound hi) {
        const __half2 *h = reinterpret_cast<const __half2 *>(&r);
        unsigned int any = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) any |= __hge2_mask(h[j], lo) & __hle2_mask(h[j], hi);
        return any != 0;
    }
    static __device__ __forceinline__ float max(const Raw &r) {
        const __half2 *h = reinterpret_cast<const __half2 *>(&r);
        const float2 f = __half22float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
        return fmaxf(f.x, f.y);
    }
};

// floor(2^31 * 2^-y) for 0 <= y < 100 (1 at y = 31, 0 past it): 2^-n exactly, times
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

// Where a row's result goes, and the word it is drawn with.
struct RowEnd {
    int32_t *token;
    float *prob;
    uint32_t word;
    unsigned int per_warp;
};

// A logit's weight, any logit, any rule.
__device__ __noinline__ uint32_t token_weight(float x, RowRule rule) {
    if (x == rule.m) return 0x80000000u;
    const float y = __fmul_rn(__fsub_rn(rule.m, x), rule.scale);
    if (!(y < 32.0f) || x == -INFINITY) return 0u;
    const uint32_t q = exp2_weight(y);
    return q >= rule.qmin ? q : 0u;
}

// Two f32 operations an instruction, each of the pair rounded alone.
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

// Weighs a vector's logits for a row of finite m and scale, as token_weight
// does but before min-p: distances y and weights q. x = m gives y = 0 by
// itself; -inf and NaN give the clamp's 40, past the weights' range. 6 logits a
// clock and SM from shared memory (clamping 16-bit logits two at a time before
// they are widened, or rounding the other way round, measured 5.6).
template <typename T>
struct Weigher {
    u64 m2, scale2;

    __device__ __forceinline__ explicit Weigher(const RowRule &rule)
        : m2(pack2(rule.m, rule.m)), scale2(pack2(rule.scale, rule.scale)) {}

    __device__ __forceinline__ void operator()(const typename Vec<T>::Raw &r, float (&x)[Vec<T>::N],
                                               float (&y)[Vec<T>::N], uint32_t (&q)[Vec<T>::N]) const {
        constexpr int N = Vec<T>::N;
        Vec<T>::unpack(r, x);
        u64 y2[N / 2];
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            y2[e / 2] = mul2(sub2(m2, pack2(x[e], x[e + 1])), scale2);
            unpack2(y2[e / 2], y[e], y[e + 1]);
            y[e] = fminf(y[e], 40.0f);
            y[e + 1] = fminf(y[e + 1], 40.0f);
            y2[e / 2] = pack2(y[e], y[e + 1]);
        }
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const u64 t2 = add2(y2[e / 2], pack2(kRound, kRound));
            const u64 f2 = sub2(y2[e / 2], add2(t2, pack2(-kRound, -kRound)));
            u64 p2 = add2(mul2(pack2(kC5, kC5), f2), pack2(kC4, kC4));
            p2 = add2(mul2(p2, f2), pack2(kC3, kC3));
            p2 = add2(mul2(p2, f2), pack2(kC2, kC2));
            p2 = add2(mul2(p2, f2), pack2(kC1, kC1));
            p2 = add2(mul2(p2, f2), pack2(kC0, kC0));
            float t[2], p[2];
            unpack2(t2, t[0], t[1]);
            unpack2(p2, p[0], p[1]);
            q[e] = scaled_floor(p[0], t[0]);
            q[e + 1] = scaled_floor(p[1], t[1]);
        }
    }
};

// The histogram's bin of a distance: the nearest of the bins' centres, so
// bin b holds y in [b - 1/2, b + 1/2] / 32.
// (y below 31.9.)
__device__ __forceinline__ uint32_t bin_of(float y) {
    return __float_as_uint(__fmaf_rn(y, 32.0f, 8388608.0f)) - 0x4b000000u;
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
__device__ __forceinline__ void ld_cluster_u64x2(uint32_t addr, u64 &a, u64 &b) {
    asm volatile("ld.shared::cluster.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}
__device__ __forceinline__ u64 ld_cluster_u64(uint32_t addr) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

// Every block's (a, b), given by its threads below the cluster's size, then
// in sh.slots[slot] of every block. A cluster barrier: what blocks wrote to
// their shared memory before it can be read by the others after it.
__device__ __forceinline__ void exchange(Slot slot, u64 a, u64 b) {
    SampleShared &sh = block_shared();
    if (threadIdx.x < cluster_size()) st_cluster(at_rank(sh.slots[slot][cluster_rank()], threadIdx.x), a, b);
    cluster_arrive();
    cluster_wait();
}

// The sum over the warp of values below 2^54 (a row's sums are below 2^53).
__device__ __forceinline__ u64 warp_total(u64 v) {
    const uint32_t low = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x7ffffffu);
    const uint32_t high = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 27));
    return ((u64)high << 27) + low;
}

__device__ __forceinline__ u64 warp_min(u64 v) {
    const uint32_t high = __reduce_min_sync(0xffffffffu, (uint32_t)(v >> 32));
    const uint32_t low = __reduce_min_sync(0xffffffffu, (uint32_t)(v >> 32) == high ? (uint32_t)v : 0xffffffffu);
    return (u64)high << 32 | low;
}

__device__ __forceinline__ u64 warp_inclusive(u64 v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const u64 o = __shfl_up_sync(0xffffffffu, v, d);
        v += lane >= d ? o : 0ull;
    }
    return v;
}

// Warp w's value of sh.warp[which], for lanes w below the number of warps,
// after every warp has given one.
__device__ __forceinline__ u64 of_warps(u64 v, int which, u64 none) {
    SampleShared &sh = block_shared();
    const int lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) sh.warp[which][threadIdx.x >> 5] = v;
    __syncthreads();
    return lane < kSWarps ? sh.warp[which][lane] : none;
}

// The sum over the block, in every thread.
__device__ __forceinline__ u64 block_total(u64 v) { return warp_total(of_warps(warp_total(v), 0, 0ull)); }

// The same of several values at once.
template <int K>
__device__ __forceinline__ void block_totals(u64 (&v)[K]) {
    SampleShared &sh = block_shared();
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = warp_total(v[i]);
    __syncthreads();
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < K; ++i) sh.warp[i][threadIdx.x >> 5] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = warp_total(lane < kSWarps ? sh.warp[i][lane] : 0ull);
}

// The sum over the threads before this one.
__device__ __forceinline__ u64 block_before(u64 v) {
    const u64 inc = warp_inclusive(v);
    const u64 warps = of_warps(__shfl_sync(0xffffffffu, inc, 31), 1, 0ull);
    return warp_total((threadIdx.x & 31) < (threadIdx.x >> 5) ? warps : 0ull) + inc - v;
}

// The least over the block, in every thread.
__device__ __forceinline__ u64 block_min(u64 v) { return warp_min(of_warps(warp_min(v), 2, ~0ull)); }

// The least lo and the greatest hi over the block, in every thread.
__device__ __forceinline__ void block_range(u64 &lo, u64 &hi) {
    SampleShared &sh = block_shared();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    lo = warp_min(lo);
    hi = warp_min(~hi);
    __syncthreads();
    if (lane == 0) {
        sh.warp[0][warp] = lo;
        sh.warp[1][warp] = hi;
    }
    __syncthreads();
    lo = warp_min(lane < kSWarps ? sh.warp[0][lane] : ~0ull);
    hi = ~warp_min(lane < kSWarps ? sh.warp[1][lane] : ~0ull);
}

// ---------------------------------------------------------------------------
// A block's slice of a row
// ---------------------------------------------------------------------------
// Vector v of base, the elements outside [first, end) as -inf.
template <typename T>
__device__ __noinline__ typename Vec<T>::Raw load_edge(const T *base, unsigned int v, unsigned int first,
                                                       unsigned int end) {
    typedef typename Vec<T>::Raw Raw;
    constexpr int bits = 8 * sizeof(T), per_word = 32 / bits, words = sizeof(Raw) / 4;
    union {
        Raw r;
        uint32_t w[words];
    };
#pragma unroll
    for (int j = 0; j < words; ++j) {
        w[j] = Vec<T>::kFill;
#pragma unroll
        for (int i = 0; i < per_word; ++i) {
            const unsigned int at = v * Vec<T>::N + j * per_word + i;
            if (at >= first && at < end) {
                const uint32_t one = sizeof(T) == 4 ? reinterpret_cast<const uint32_t *>(base)[at]
                                                    : reinterpret_cast<const uint16_t *>(base)[at];
                w[j] = sizeof(T) == 4 ? one : (w[j] & ~(0xffffu << bits * i)) | one << bits * i;
            }
        }
    }
    return r;
}

template <typename T>
struct Slice {
    using V = Vec<T>;
    typedef typename V::Raw Raw;
    static constexpr int kLane = sizeof(Raw) / 16;  // 16-byte words of a vector
    const char *base;           // the row's address rounded down to a vector
    unsigned int pad, n;        // elements between base and the row, and in the row
    unsigned int v0, count;     // this warp's first vector and how many it has
    unsigned int staged_iters;
    uint4 *stage;               // this lane's vectors: turn i at stage + 32 * kLane * i

    // Vector v; past the row's ends filled with -inf.
    __device__ __forceinline__ Raw load(unsigned int v) const {
        const unsigned int first = pad ? 1u : 0u, end = (pad + n) / V::N;  // those between are whole
        if (v - first < end - first) return V::load(base + (size_t)v * sizeof(Raw));
        return load_edge<T>(reinterpret_cast<const T *>(base), v, pad, pad + n);
    }

    // First reading: keeps the staged vectors and the turns' maxima, returns the
    // warp's (as a key) and, if asked, this thread's.
    __device__ __forceinline__ uint32_t first_pass(uint32_t *thread_key) const {
        constexpr int U = 4 / kLane;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        uint32_t *turn_key = block_shared().turn_key[warp];
        const char *whole = base + (size_t)(v0 + lane) * sizeof(Raw);
        const unsigned int whole_end = (pad + n) / V::N;  // vectors from here on, and 0 with a pad, are cut
        float m = -INFINITY;
        uint32_t most = 0;
#pragma unroll 1
        for (unsigned int it = 0; 32 * it < count; it += U) {
            Raw r[U];
            const unsigned int end = 32 * (it + U);
            if (end <= count && v0 + end <= whole_end && (pad == 0 || v0 + it > 0)) {
#pragma unroll
                for (int u = 0; u < U; ++u) r[u] = V::load(whole + 32 * (it + u) * sizeof(Raw));
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const unsigned int j = 32 * (it + u) + lane;
                    r[u] = fill();
                    if (has(j)) r[u] = load(v0 + j);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float top = V::max(r[u]);
                m = fmaxf(m, top);
                const uint32_t key = __reduce_max_sync(0xffffffffu, key_of(top == top ? top : -INFINITY));
                most = max(most, key);
                if (it + u < kTurns && lane == 0) turn_key[it + u] = key;
                if (it + u < staged_iters) V::put(stage + 32 * kLane * (it + u), r[u]);
            }
        }
        __syncwarp();
        *thread_key = key_of(m);
        return max(most, kKeyOfMinusInf);
    }

    __device__ __forceinline__ bool has(unsigned int j) const { return j < count; }
    static __device__ __forceinline__ Raw fill() {
        const uint4 four = make_uint4(V::kFill, V::kFill, V::kFill, V::kFill);
        if constexpr (kLane == 2) return {four, four};
        else return four;
    }
    __device__ __forceinline__ Raw turn(unsigned int it, unsigned int j) const {
        return it < staged_iters ? V::get(stage + 32 * kLane * it) : load(v0 + j);
    }

    // f(vector, its number) for this lane's vectors, in ascending order, in
    // the turns that may hold a logit at or above thr; the next one that is
    // not in shared memory is on its way meanwhile.
    template <typename F>
    __device__ __forceinline__ void each(float thr, F f) const {
        const unsigned int lane = threadIdx.x & 31;
        const uint32_t *turn_key = block_shared().turn_key[threadIdx.x >> 5];
        static_assert(kTurns == 64, "two words of turns");
        const uint32_t key = key_of(thr);
        const unsigned int turns = (count + 31) / 32;
        // the remembered turns to take; those past them are all taken
        unsigned int low = __ballot_sync(0xffffffffu, lane < turns && turn_key[lane] >= key);
        unsigned int high = __ballot_sync(0xffffffffu, 32 + lane < turns && turn_key[32 + lane] >= key);
        unsigned int past = kTurns - 1;
        auto take = [&]() -> unsigned int {
            if (low) {
                const unsigned int it = __ffs(low) - 1;
                low &= low - 1;
                return it;
            }
            if (high) {
                const unsigned int it = __ffs(high) + 31;
                high &= high - 1;
                return it;
            }
            return ++past;
        };
        unsigned int it = take();
        Raw ahead = {};
        if (it >= staged_iters && has(32 * it + lane)) ahead = load(v0 + 32 * it + lane);
#pragma unroll 1
        while (has(32 * it + lane)) {
            const unsigned int v = v0 + 32 * it + lane;
            Raw r = ahead;
            if (it < staged_iters) r = V::get(stage + 32 * kLane * it);
            it = take();
            if (it >= staged_iters && has(32 * it + lane)) ahead = load(v0 + 32 * it + lane);
            f(r, v);
        }
    }

    __device__ __forceinline__ uint32_t index(unsigned int v, int e) const { return v * V::N + e - pad; }

    // The share of the warp `by` warps on in this block.
    __device__ __forceinline__ Slice of_warp(int by, unsigned int per_warp, unsigned int nv) const {
        Slice s = *this;
        s.v0 += by * (int)per_warp;
        s.count = s.v0 < nv ? min(per_warp, nv - s.v0) : 0u;
        s.stage += by * 32 * kLane * (int)staged_iters;
        return s;
    }
};

// A logit's place in the filters' order, ascending.
__device__ __forceinline__ u64 item_of(uint32_t key, uint32_t index) { return (u64)~key << 32 | index; }
__device__ __forceinline__ uint32_t item_weight(u64 item, RowRule rule) {
    return token_weight(key_logit(~(uint32_t)(item >> 32)), rule);
}
constexpr u64 kKeepAll = ~0ull;
constexpr u64 kNoItem = ~0ull;  // an item without weight, past all others

// The gathered items' weights (of one each with COUNT), 0 past `limit`, for
// block_select.
template <bool COUNT>
__device__ __forceinline__ void weigh_items(uint32_t n, u64 limit, RowRule rule) {
    SampleShared &sh = block_shared();
#pragma unroll 1
    for (uint32_t i = threadIdx.x; i < n; i += kSThreads) {
        const u64 item = sh.items[kLocal + i];
        sh.picks.weights[i] = item > limit || item == kNoItem ? 0u : COUNT ? 1u : item_weight(item, rule);
    }
}

// Over the n gathered items with a weight (weigh_items, by the same threads):
// the first, in order (or by index), at which the running sum of weights
// reaches `target` (1 <= target <= the sum of all), and the sum before it. A
// histogram of the places still in question, 512 bins between the least and
// the greatest, gives the bin that holds the crossing; its items, where they
// are at most kFew, find it by counting what stands before them, else
// they are the next histogram's.
__device__ __noinline__ u64 block_select(uint32_t n, bool by_index, u64 target, u64 *before_it, u64 low = 0,
                                         u64 high = ~0ull) {
    SampleShared &sh = block_shared();
    const u64 place_bits = by_index ? 0xffffffffull : ~0ull;
    u64 base = 0;
    bool narrow = high != ~0ull;
    while (true) {
        sh.picks.sums.low[threadIdx.x] = sh.picks.sums.high[threadIdx.x] = sh.picks.counts[threadIdx.x] = 0;
        u64 lo = low, hi = high;
        if (narrow) {
            __syncthreads();
        } else {
            lo = ~0ull;
            hi = 0;
#pragma unroll 1
            for (uint32_t i = threadIdx.x; i < n; i += kSThreads) {
                const u64 place = sh.items[kLocal + i] & place_bits;
                if (sh.picks.weights[i] && place >= low && place <= high) {
                    lo = min(lo, place);
                    hi = max(hi, place);
                }
            }
            block_range(lo, hi);
        }
        narrow = false;
        const int shift = 55 - __clzll((hi - lo) | 511ull);
#pragma unroll 1
        for (uint32_t i = threadIdx.x; i < n; i += kSThreads) {
            const u64 place = sh.items[kLocal + i] & place_bits;
            const uint32_t w = sh.picks.weights[i];
            if (w && place >= low && place <= high) {
                const uint32_t bin = (uint32_t)((place - lo) >> shift);
                sh.picks.sums.add(bin, w);
                atomicAdd(&sh.picks.counts[bin], 1u);
            }
        }
        __syncthreads();
        const u64 mine = (u64)sh.picks.sums.high[threadIdx.x] << 32 | sh.picks.sums.low[threadIdx.x];
        const u64 before = base + block_before(mine);
        if (before < target && target <= before + mine) {
            sh.cast[0] = threadIdx.x;
            sh.cast[1] = before;
            sh.cast[2] = sh.picks.counts[threadIdx.x];
        }
        __syncthreads();
        base = sh.cast[1];
        low = lo + (sh.cast[0] << shift);
        high = min(high, low + ((1ull << shift) - 1));  // the last bin may reach past the places in question
        const uint32_t few = (uint32_t)sh.cast[2];
        __syncthreads();  // cast and the bins are written again
        if (few > kFew) continue;
        if (threadIdx.x == 0) sh.picks.counts[0] = 0;
        __syncthreads();
#pragma unroll 1
        for (uint32_t i = threadIdx.x; i < n; i += kSThreads) {
            const u64 place = sh.items[kLocal + i] & place_bits;
            if (sh.picks.weights[i] && place >= low && place <= high) {
                const uint32_t at = atomicAdd(&sh.picks.counts[0], 1u);
                sh.picks.few.place[at] = place;
                sh.picks.few.weight[at] = sh.picks.weights[i];
                sh.picks.few.from[at] = i;
            }
        }
        __syncthreads();
        constexpr uint32_t team = kSThreads / kFew;
        const uint32_t i = threadIdx.x / team, part = threadIdx.x % team;
        const u64 place = i < few ? sh.picks.few.place[i] : 0ull;
        u64 sum = 0;
        for (uint32_t j = part; j < few; j += team)
            sum += sh.picks.few.place[j] < place ? sh.picks.few.weight[j] : 0u;
#pragma unroll
        for (uint32_t d = 1; d < team; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        sum += base;
        if (part == 0 && i < few && sum < target && target <= sum + sh.picks.few.weight[i]) {
            sh.cast[0] = sh.items[kLocal + sh.picks.few.from[i]];
            sh.cast[1] = sum;
        }
        __syncthreads();
        *before_it = sh.cast[1];
        return sh.cast[0];
    }
}

// (float)((double)q / (double)total), 1 <= q <= total <= 2^53, q <= 2^31, in
// integers: the double division takes 0.45 us at every row's end. From a quotient
// a few units off, the one rounded down (in `units` of the last place) and what
// is left of it; a remainder that a double would round to half a unit is a tie.
__device__ __forceinline__ float quotient(u64 q, u64 total) {
    const uint32_t near = __float_as_uint(__fdividef(__ull2float_rn(q), __ull2float_rn(total)));
    int exponent = (int)(near >> 23) - 127;
    u64 units = (near & 0x7fffffu) | 0x800000u;
    const int shift = 23 - exponent;
    long long left = (long long)((shift < 64 ? q << shift : 0ull) - units * total);  // modulo 2^64: it is small
#pragma unroll 1
    for (; left < 0; left += total) --units;
#pragma unroll 1
    for (; left >= (long long)total; left -= total) ++units;
    if (units < 1u << 23) {  // the quotient lies below a power of two, the one near it does not
        left *= 2;
        units *= 2;
        --exponent;
        if (left >= (long long)total) {
            left -= total;
            ++units;
        }
    } else if (units >= 1u << 24) {
        left += units & 1 ? total : 0ull;
        total *= 2;
        units /= 2;
        ++exponent;
    }
    const u64 twice = 2 * (u64)left, apart = twice > total ? twice - total : total - twice;
    const bool up = apart <= total >> 29 ? units & 1 : twice > total;
    return __uint_as_float(((uint32_t)(exponent + 127) << 23) + (uint32_t)(units - (1u << 23)) + up);
}

__device__ __forceinline__ void write_token(RowEnd end, uint32_t index, u64 q, u64 total) {
    *end.token = (int32_t)index;
    if (end.prob) *end.prob = quotient(q, total);
}

__device__ __forceinline__ u64 draw_of(uint32_t word, u64 total) { return __umul64hi((u64)word << 32, total); }

__device__ __forceinline__ u64 top_p_target(float p, u64 total) {
    // The product's 77 bits in integers (doubles are few on this chip, and slow when every warp
    // wants one: 780 clocks a block), to 53 bits as a double's are, ties to even, then up.
    const uint32_t bits = __float_as_uint(p), exponent = max(bits >> 23, 1u);  // p = digits * 2^(exponent - 150)
    const uint32_t digits = (bits & 0x7fffffu) | (bits >> 23 ? 0x800000u : 0u);
    u64 low = total * digits, high = __umul64hi(total, digits);
    int below = 150 - (int)exponent;  // binary places
    const int length = high ? 128 - __clzll(high) : 64 - __clzll(low);
    if (length > 53) {
        const int drop = length - 53;  // at most 24
        const u64 rest = low & ((1ull << drop) - 1), tie = 1ull << (drop - 1);
        low = low >> drop | high << (64 - drop);
        low += rest > tie || (rest == tie && (low & 1));
        below -= drop;
    }
    if (below > 53) return 1;
    return (low >> below) + ((low & ((1ull << below) - 1)) != 0);
}

// The sum of what the first `blocks` blocks put into a slot.
__device__ __forceinline__ u64 slot_total(Slot slot, uint32_t blocks, int word = 0) {
    SampleShared &sh = block_shared();
    const uint32_t lane = threadIdx.x & 31;
    return warp_total(lane < blocks ? sh.slots[slot][lane][word] : 0ull);
}

// The weights of a vector's logits up to `last`, 0 for the others, for a
// finite m and scale.
template <typename T>
__device__ __forceinline__ u64 kept_weights(const Slice<T> &sl, const typename Vec<T>::Raw &r, unsigned int v,
                                            const Weigher<T> &weigh, uint32_t qmin, u64 last,
                                            uint32_t (&q)[Vec<T>::N]) {
    float x[Vec<T>::N], y[Vec<T>::N];
    weigh(r, x, y, q);
#pragma unroll
    for (int e = 0; e < Vec<T>::N; ++e) q[e] = q[e] >= qmin ? q[e] : 0u;
    if (last != kKeepAll) {
        const float thr = key_logit(~(uint32_t)(last >> 32));
#pragma unroll
        for (int e = 0; e < Vec<T>::N; ++e)
            if (x[e] < thr || (x[e] == thr && sl.index(v, e) > (uint32_t)last)) q[e] = 0;
    }
    u64 sum = 0;
#pragma unroll
    for (int e = 0; e < Vec<T>::N; ++e) sum += q[e];
    return sum;
}

// The draw among the items up to `last`, in index order, by the block that
// holds it: `before` is what the blocks before this one keep, `mass` in lane i
// what its i-th group of `group` warps does. It weighs the group with the draw
// again, a turn of 32 vectors a warp, and walks the turn with the draw.
template <typename T>
__device__ __forceinline__ void draw(Slice<T> own, RowRule rule, u64 last, u64 total, u64 before, u64 mass,
                                  unsigned int group, RowEnd end) {
    SampleShared &sh = block_shared();
    constexpr int N = Vec<T>::N;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const u64 r = draw_of(end.word, total), upto = before + warp_inclusive(mass);
    if (r < before || r >= __shfl_sync(0xffffffffu, upto, 31)) return;
    const unsigned int at_group = __ffs(__ballot_sync(0xffffffffu, r < upto)) - 1;
    before = __shfl_sync(0xffffffffu, upto - mass, at_group);
    const int warp0 = (int)(at_group * group);
    const unsigned int per_warp = end.per_warp, nv = (own.pad + own.n + N - 1) / N;
    const unsigned int per = (per_warp + 31) / 32, turns = group * per;
    const Weigher<T> weigh(rule);
    u64 *of_turn = sh.items;
    u64 at = 0;
    bool walk = false;  // first all turns, then the one
    unsigned int t = warp;
#pragma unroll 1
    while (true) {
        uint32_t q[N];
#pragma unroll
        for (int e = 0; e < N; ++e) q[e] = 0;
        u64 sum = 0;
        const Slice<T> sl = own.of_warp(warp0 + (int)(t / per) - warp, per_warp, nv);
        const unsigned int it = t % per, j = 32 * it + lane;
        if (t < turns && sl.has(j)) sum = kept_weights(sl, sl.turn(it, j), sl.v0 + j, weigh, rule.qmin, last, q);
        if (walk) {
            at += warp_inclusive(sum) - sum;
            if (at <= r && r - at < sum) {
                int chosen = 0;
                uint32_t weight = 0;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    if (at <= r && r - at < q[e]) {
                        chosen = e;
                        weight = q[e];
                    }
                    at += q[e];
                }
                write_token(end, sl.index(sl.v0 + j, chosen), weight, total);
            }
            return;
        }
        sum = warp_total(sum);
        if (lane == 0 && t < turns) of_turn[t] = sum;
        t += kSWarps;
        if (t < turns) continue;
        __syncthreads();
        const unsigned int each = (turns + kSThreads - 1) / kSThreads, first = threadIdx.x * each;
        sum = 0;
        for (t = first; t < first + each && t < turns; ++t) sum += of_turn[t];
        at = before + block_before(sum);
        if (at <= r && r - at < sum) {
            t = first;
            while (r - at >= of_turn[t]) at += of_turn[t++];
            sh.cast[0] = t;
            sh.cast[1] = at;
        }
        __syncthreads();
        if (warp != 0) return;
        t = (unsigned int)sh.cast[0];
        at = sh.cast[1];
        walk = true;
    }
}

// A key that at least k of the n maxima reach. Of up to 512 (a multiple of 16)
// the k-th largest, by counting; of more the lower edge of the bin that holds
// it, of 512 between the least and row_key, the greatest, then of 512 in that
// bin, while it spans more than 1/64 of an octave (a maximum of -inf widens
// the first).
__device__ __forceinline__ uint32_t kth_bound(const uint32_t *maxima, uint32_t n, uint32_t k,
                                              uint32_t row_key) {
    SampleShared &sh = block_shared();
    if (n <= kSThreads) {
        uint32_t team = 1;  // threads that count for one maximum
        while (team < 16 && 2 * team * n <= kSThreads) team *= 2;
        const uint32_t i = threadIdx.x / team, part = threadIdx.x % team;
        const uint32_t mine = i < n ? maxima[i] : 0u;
        const uint4 *four = reinterpret_cast<const uint4 *>(maxima);
        uint32_t above = 0;
        if (i < n)
#pragma unroll 2
            for (uint32_t j = 4 * part; j < n; j += 4 * team) {
                const uint4 o = four[j / 4];
                above += (o.x > mine || (o.x == mine && j < i)) + (o.y > mine || (o.y == mine && j + 1 < i)) +
                         (o.z > mine || (o.z == mine && j + 2 < i)) + (o.w > mine || (o.w == mine && j + 3 < i));
            }
        for (uint32_t d = 1; d < team; d *= 2) above += __shfl_xor_sync(0xffffffffu, above, d);
        if (part == 0 && i < n && above == k - 1) sh.cast[0] = mine;
        __syncthreads();
        return (uint32_t)sh.cast[0];
    }
    uint32_t *counts = sh.picks.counts;
    uint32_t least = row_key;
    for (uint32_t i = threadIdx.x; i < n; i += kSThreads) least = min(least, maxima[i]);
    counts[threadIdx.x] = 0;
    least = (uint32_t)block_min(least);
    int shift = 23 - __clz((row_key - least) | 511u);
    uint32_t nearest = 0;  // distance from row_key at which the bins start
    while (true) {
        for (uint32_t i = threadIdx.x; i < n; i += kSThreads) {
            const uint32_t d = row_key - maxima[i];
            if (d >= nearest && (d - nearest) >> shift < kSThreads) atomicAdd(&counts[(d - nearest) >> shift], 1u);
        }
        __syncthreads();
        const uint32_t mine = counts[threadIdx.x];
        const uint32_t before = (uint32_t)block_before(mine);
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
__device__ __forceinline__ void put(u64 item) {
    SampleShared &sh = block_shared();
    const uint32_t at = atomicAdd(&sh.n_list, 1u);
    if (at < kLocal) sh.items[at] = item;
}

// f(x[e], e) for the elements that `test` names: few, so one copy of f.
template <int N, typename Test, typename F>
__device__ __forceinline__ void each_of(const float (&x)[N], Test test, F f) {
    unsigned int mask = 0;
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (test(x[e])) mask |= 1u << e;
#pragma unroll 1
    for (; mask; mask &= mask - 1) {
        const int e = __ffs(mask) - 1;
        float xe = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) xe = e == i ? x[i] : xe;
        f(xe, e);
    }
}

// Gathers the logits in [thr, cap] (-inf not among them) into this block's
// list. In a long slice first the vectors that hold one (few, and a few
// instructions each, where taking such a vector apart would stop its whole
// warp), then, a thread a vector, the logits: 64 x 131072 bf16 under top-p
// 38.7 us, 40.2 with all at once. In a short slice, up to 64 vectors a warp,
// all at once: a row of 32000 bf16 under top-k 8.6 us, 9.0 in two steps.
template <typename T>
__device__ __forceinline__ void collect(Slice<T> sl, unsigned int per_warp, float thr, float cap) {
    SampleShared &sh = block_shared();
    using V = Vec<T>;
    const int warp = threadIdx.x >> 5;
    thr = fmaxf(thr, -3.402823466e38f);  // the least finite logit
    auto take = [&](const auto &r, unsigned int v) {
        float x[V::N];
        V::unpack(r, x);
        each_of<V::N>(x, [&](float xe) { return xe >= thr && xe <= cap; },
                      [&](float xe, int e) { put(item_of(key_of(xe), sl.index(v, e))); });
    };
    const typename V::Bound lo = V::from(thr), hi = V::upto(cap);
    if (per_warp <= 64) {
        sl.each(thr, [&](const auto &r, unsigned int v) {
            if (V::any_in(r, lo, hi)) take(r, v);
        });
        __syncthreads();
        return;
    }
    __syncthreads();
    if (threadIdx.x == 0) sh.n_hits = 0;
    __syncthreads();
    sl.each(thr, [&](const auto &r, unsigned int v) {
        if (!V::any_in(r, lo, hi)) return;
        const uint32_t at = atomicAdd(&sh.n_hits, 1u);
        if (at < kHits) sh.hits[at] = (uint32_t)warp << 16 | (v - sl.v0);
    });
    __syncthreads();
#pragma unroll 1
    for (uint32_t i = threadIdx.x; i < min(sh.n_hits, (uint32_t)kHits); i += kSThreads) {
        const int by = (int)(sh.hits[i] >> 16) - warp;
        const unsigned int j = sh.hits[i] & 0xffffu, it = j / 32;
        const unsigned int v = sl.v0 + by * (int)per_warp + j;
        const uint4 *stage = sl.stage + by * 32 * sl.kLane * (int)sl.staged_iters;
        stage += (int)(j % 32) - (int)(threadIdx.x % 32);
        take(it < sl.staged_iters ? V::get(stage + 32 * sl.kLane * it) : sl.load(v), v);
    }
    __syncthreads();
    if (threadIdx.x == 0 && sh.n_hits > kHits) sh.n_list = kLocal + 1;  // too many
    __syncthreads();
}

// The length of all blocks' lists, after an exchange of their lengths as
// `slot`'s first word; over kList when one of them or all do not fit.
__device__ __forceinline__ uint32_t gathered(Slot slot) {
    SampleShared &sh = block_shared();
    const uint32_t lane = threadIdx.x & 31, one = lane < cluster_size() ? (uint32_t)sh.slots[slot][lane][0] : 0u;
    return __reduce_add_sync(0xffffffffu, one <= kLocal ? one : kList + 1);
}

// All blocks' n items, one list after another, in this block (when they fit):
// every thread finds its items' blocks by itself, so that all of them are on
// their way at once.
__device__ __forceinline__ void pull(Slot slot, uint32_t n) {
    SampleShared &sh = block_shared();
    for (uint32_t i = threadIdx.x; i < n; i += kSThreads) {
        uint32_t c = 0, at = i;
        while (at >= (uint32_t)sh.slots[slot][c][0]) at -= (uint32_t)sh.slots[slot][c++][0];
        sh.items[kLocal + i] = ld_cluster_u64(at_rank(sh.items + at, c));
    }
    __syncthreads();
}

// The token among the n gathered items, which hold all that the filters keep:
// the first k of them in order, and of those the top-p prefix (0 < p < 1),
// measured against `total` if that is not 0, else against their own sum.
__device__ __noinline__ void finish_list(uint32_t n, uint32_t k, float p, u64 total,
                                         RowRule rule, RowEnd end) {
    SampleShared &sh = block_shared();
    const bool cut_p = p > 0.0f && p < 1.0f;
    const uint32_t word = end.word;
    if (n <= kRanked) {
        // `team` threads an item count what stands before it
        uint32_t team = 2;
        while (team < 16 && 2 * team * n <= kSThreads) team *= 2;
        const uint32_t i = threadIdx.x / team, part = threadIdx.x % team;
        u64 *weight = sh.items;  // pulled: free
        const u64 item = i < n ? sh.items[kLocal + i] : ~0ull;
        const u64 q = i < n ? item_weight(item, rule) : 0u;
        if (part == 0) weight[i] = q;
        __syncthreads();
        uint32_t rank = 0;
        u64 before = 0;
        if (i < n)
#pragma unroll 2
            for (uint32_t j = part; j < n; j += team) {
                const bool first = sh.items[kLocal + j] < item;
                rank += first;
                before += first ? weight[j] : 0ull;
            }
        for (uint32_t d = 1; d < team; d *= 2) {
            rank += __shfl_xor_sync(0xffffffffu, rank, d);
            before += __shfl_xor_sync(0xffffffffu, before, d);
        }
        u64 kept = i < n && rank < k ? q : 0ull;
        if (total == 0) total = block_total(part == 0 ? kept : 0ull);
        if (cut_p) {
            if (before >= top_p_target(p, total)) kept = 0;
            total = block_total(part == 0 ? kept : 0ull);
        }
        __syncthreads();
        if (part == 0) weight[i] = kept;
        __syncthreads();
        u64 at = 0;
        if (i < n)
#pragma unroll 2
            for (uint32_t j = part; j < n; j += team)
                at += (uint32_t)sh.items[kLocal + j] < (uint32_t)item ? weight[j] : 0ull;
        for (uint32_t d = 1; d < team; d *= 2) at += __shfl_xor_sync(0xffffffffu, at, d);
        const u64 r = draw_of(word, total);
        if (part == 0 && at <= r && r < at + kept) write_token(end, (uint32_t)item, kept, total);
        return;
    }
    u64 last = kKeepAll, before;
    if (k < n) {
        weigh_items<true>(n, last, rule);
        last = block_select(n, false, k, &before);
    }
    weigh_items<false>(n, last, rule);
    if (total == 0) {
        u64 sum = 0;
#pragma unroll 1
        for (uint32_t i = threadIdx.x; i < n; i += kSThreads) sum += sh.picks.weights[i];
        total = block_total(sum);
    }
    if (cut_p) {
        last = block_select(n, false, top_p_target(p, total), &before);
        total = before + item_weight(last, rule);
        weigh_items<false>(n, last, rule);
    }
    const u64 chosen = block_select(n, true, draw_of(word, total) + 1, &before);
    if (threadIdx.x == 0) write_token(end, (uint32_t)chosen, item_weight(chosen, rule), total);
}

// The `nth` logit (from 1, by index) with key tau, as an item; -inf entries
// past the row's ends do not count.
template <typename T>
__device__ __noinline__ u64 nth_tie(Slice<T> sl, uint32_t tau, u64 nth, Slot ties_slot,
                                    Slot at_slot) {
    SampleShared &sh = block_shared();
    const int lane = threadIdx.x & 31;
    auto tied = [&](const auto &r, unsigned int v) {  // by element
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
    sl.each(key_logit(tau), [&](const auto &r, unsigned int v) { mine += __popc(tied(r, v)); });
    mine = warp_total(mine);
    u64 before = block_before(lane == 0 ? mine : 0ull);  // of lane 0: the warps' before
    before = __shfl_sync(0xffffffffu, before, 0);
    // past block_before's barriers every thread has read what the caller left in cast, and the
    // exchange's barrier comes before the tie is written
    if (threadIdx.x == 0) sh.cast[0] = ~0ull;
    exchange(ties_slot, block_total(lane == 0 ? mine : 0ull), 0);
    before += slot_total(ties_slot, cluster_rank());
    if (before < nth && nth <= before + mine)  // this warp's
        for (unsigned int j0 = 0, it = 0; j0 < sl.count; j0 += 32, ++it) {
            const unsigned int j = j0 + lane;
            unsigned int t = 0;
            if (sl.has(j)) t = tied(sl.turn(it, j), sl.v0 + j);
            const u64 inc = warp_inclusive(__popc(t));
            const u64 at = before + inc - __popc(t);
            if (at < nth && nth <= before + inc) {
                for (u64 skip = nth - at - 1; skip > 0; --skip) t &= t - 1;
                sh.cast[0] = item_of(tau, sl.index(sl.v0 + j, __ffs(t) - 1));
            }
            before += __shfl_sync(0xffffffffu, inc, 31);
        }
    __syncthreads();
    exchange(at_slot, sh.cast[0], 0);
    return warp_min(lane < (int)cluster_size() ? sh.slots[at_slot][lane][0] : ~0ull);
}

// The histogram bin in which a filter ends, and what lies in it.
struct Crossing {
    uint32_t bin;
    uint32_t floor_q;  // the least weight in the histogram (counts: all that weigh, y <= 31)
    float thr, cap;    // every logit of the bin is in [thr, cap], few others are
    u64 limit;         // items past it do not count
    bool upto;         // the bins before it too
};

// Is the logit x (in [thr, cap]) with this index one of the crossing's?
template <bool COUNT>
__device__ __forceinline__ bool in_crossing(const Crossing &c, RowRule rule, float x, u64 item) {
    const float y = __fmul_rn(__fsub_rn(rule.m, x), rule.scale);
    if (!(y <= 31.0f)) return false;  // it weighs nothing
    const uint32_t b = bin_of(y);
    return (c.upto ? b <= c.bin : b == c.bin) && (COUNT || (exp2_weight(y) >= c.floor_q && item <= c.limit));
}

// The item at which the running sum of the bin's weights (counts) reaches
// target, over the whole cluster: its key by radix selection, 8 bits a level,
// then the tie. *left: the sum up to it.
template <bool COUNT, typename T>
__device__ __noinline__ u64 select_in_bin(Slice<T> sl, RowRule rule, const Crossing &c, u64 target, u64 *left) {
    SampleShared &sh = block_shared();
    uint32_t prefix = 0, mask = 0;
    u64 missing = target;
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
        SumBins<256> &hist = sh.digits[shift / 8 & 1];  // two in turn: a slow block may still read the last one
        __syncthreads();
        hist.clear();
        __syncthreads();
        sl.each(c.thr, [&](const auto &r, unsigned int v) {
            if (!(Vec<T>::max(r) >= c.thr)) return;
            float x[Vec<T>::N];
            Vec<T>::unpack(r, x);
            each_of<Vec<T>::N>(x, [&](float xe) { return xe >= c.thr && xe <= c.cap; },
                               [&](float xe, int e) {
                                   const uint32_t k = key_of(xe);
                                   if ((k & mask) != prefix) return;
                                   if (!in_crossing<COUNT>(c, rule, xe, item_of(k, sl.index(v, e)))) return;
                                   hist.add((k >> shift) & 255u, COUNT ? 1u : token_weight(xe, rule));
                               });
        });
        cluster_arrive();
        cluster_wait();
        // the digits in descending order: thread t has digit 255 - t
        u64 mine = 0;
        if (threadIdx.x < 256)
            for (uint32_t b = 0; b < cluster_size(); ++b)
                mine += (u64)ld_cluster(at_rank(&hist.low[255 - threadIdx.x], b)) +
                        ((u64)ld_cluster(at_rank(&hist.high[255 - threadIdx.x], b)) << 32);
        const u64 before = block_before(mine);
        if (before < missing && missing <= before + mine) {
            sh.cast[0] = 255u - threadIdx.x;
            sh.cast[1] = missing - before;
        }
        __syncthreads();
        prefix |= (uint32_t)sh.cast[0] << shift;
        mask |= 255u << shift;
        missing = sh.cast[1];
    }
    const u64 q = COUNT ? 1ull : token_weight(key_logit(prefix), rule), ties = (missing + q - 1) / q;
    *left = target - missing + ties * q;
    return nth_tie(sl, prefix, ties, COUNT ? kSlotCountTies : kSlotSumTies, COUNT ? kSlotCountTie : kSlotSumTie);
}

// The draw among all items up to `last`, weighed first.
template <typename T>
__device__ __noinline__ void weigh_and_draw(Slice<T> sl, RowRule rule, u64 last, RowEnd end) {
    using V = Vec<T>;
    const Weigher<T> weigh(rule);
    u64 mass = 0;
    sl.each(__fsub_rd(rule.m, 31.5f * __frcp_rn(rule.scale)), [&](const auto &r, unsigned int v) {
        uint32_t q[V::N];
        mass += kept_weights(sl, r, v, weigh, rule.qmin, last, q);
    });
    mass = of_warps(warp_total(mass), 0, 0ull);
    exchange(kSlotFirst, warp_total(mass), 0);
    draw(sl, rule, last, slot_total(kSlotFirst, cluster_size()), slot_total(kSlotFirst, cluster_rank()), mass, 1, end);
}

// A filter over a row of finite m and scale: top-k (COUNT) or top-p over the
// items up to `limit`, by a histogram of counts or weights. Returns true when
// the row's token is written (top-p: always), else *last is the item at
// which the filter ends.
template <bool COUNT, typename T>
__device__ __forceinline__ bool filter(Slice<T> sl, RowRule rule, uint32_t k, float p, u64 limit,
                                    RowEnd end, u64 *last, bool clean) {
    SampleShared &sh = block_shared();
    using V = Vec<T>;
    const uint32_t rank = cluster_rank(), blocks = cluster_size();
    const int warp = threadIdx.x >> 5;
    const Slot list_slot = COUNT ? kSlotCountList : kSlotSumList;
    // top-p: the histogram goes as far as it can matter (past cut_y the row holds less than (1 - p)
    // of the largest weight); with min-p it takes all that is kept, and its sum is the row's
    const float cut_y = fminf(31.0f, log2f((float)sl.n / (1.0f - p)) + 0.1f);
    const bool min_p = rule.qmin > 0;
    Crossing c;
    c.limit = limit;
    c.floor_q = COUNT ? 1u : min_p ? rule.qmin : max(exp2_weight(cut_y), 1u);
    if (!clean) {
        __syncthreads();
        sh.bins[0].clear();
        sh.bins[1].clear();
        if (threadIdx.x == 0) sh.n_list = 0;
        __syncthreads();
    }
    SumBins<kBins> &bins = sh.bins[warp / (kSWarps / 2)];
    const Weigher<T> weigh(rule);
    const float octave = __frcp_rn(rule.scale);  // the bounds below leave room for its rounding
    const float zero = __fsub_rd(rule.m, 31.5f * octave);  // logits below it weigh nothing (y > 31)
    const bool limited = limit != kKeepAll;
    const float limit_x = limited ? key_logit(~(uint32_t)(limit >> 32)) : -INFINITY;
    u64 mass = 0;
    sl.each(zero, [&](const auto &r, unsigned int v) {
        float x[V::N], y[V::N];
        if constexpr (COUNT) {
            V::unpack(r, x);
#pragma unroll
            for (int e = 0; e < V::N; e += 2) {
                unpack2(mul2(sub2(weigh.m2, pack2(x[e], x[e + 1])), weigh.scale2), y[e], y[e + 1]);
                if (y[e] <= 31.0f) atomicAdd(&bins.low[bin_of(y[e])], 1u);
                if (y[e + 1] <= 31.0f) atomicAdd(&bins.low[bin_of(y[e + 1])], 1u);
            }
        } else {
            uint32_t q[V::N];
            weigh(r, x, y, q);
            if (limited)
#pragma unroll
                for (int e = 0; e < V::N; ++e) {
                    const bool past = x[e] == limit_x && sl.index(v, e) > (uint32_t)limit;
                    if (x[e] < limit_x || past) q[e] = 0;
                }
#pragma unroll
            for (int e = 0; e < V::N; e += 2) mass += (u64)q[e] + q[e + 1];
#pragma unroll
            for (int e = 0; e < V::N; e += 4) {
                const uint32_t b[4] = {bin_of(y[e]), bin_of(y[e + 1]), bin_of(y[e + 2]), bin_of(y[e + 3])};
                const uint32_t w[4] = {q[e], q[e + 1], q[e + 2], q[e + 3]};
                bins.add_from(c.floor_q, b, w);
            }
        }
    });
    __syncthreads();
    // two bins a thread, of both halves and (for the cluster) their sum, and that of every 16 bins
    u64 own[2][2], *sums = sh.items + kLocal, *coarse = sums + kBins, *of_block = coarse + kBins / 16;
    u64 sixteen = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int b = 2 * threadIdx.x + i;
        own[0][i] = (u64)sh.bins[0].high[b] << 32 | sh.bins[0].low[b];
        own[1][i] = (u64)sh.bins[1].high[b] << 32 | sh.bins[1].low[b];
        sums[b] = own[0][i] + own[1][i];
        sixteen += sums[b];
    }
#pragma unroll
    for (int d = 1; d < 8; d *= 2) sixteen += __shfl_xor_sync(0xffffffffu, sixteen, d);
    if (threadIdx.x % 8 == 0) coarse[threadIdx.x / 8] = sixteen;
    mass = block_total(COUNT || min_p ? own[0][0] + own[0][1] + own[1][0] + own[1][1] : mass);
    if (threadIdx.x == 0) *of_block = mass;
    cluster_arrive();
    cluster_wait();
    // The bin in which the running sum reaches what is wanted: of the cluster's sums by 16 bins,
    // then by bin, by one warp (4 KB from the other blocks; all bins to all threads are 64 KB).
    if (warp == 0) {
        const uint32_t lane = threadIdx.x;
        u64 pair[2] = {0, 0}, one = 0;
        if (lane < blocks) one = ld_cluster_u64(at_rank(of_block, lane));
        u64 part[kMaxCluster][2];
#pragma unroll
        for (uint32_t b = 0; b < kMaxCluster; ++b) {
            part[b][0] = part[b][1] = 0;
            if (b < blocks) ld_cluster_u64x2(at_rank(coarse + 2 * lane, b), part[b][0], part[b][1]);
        }
#pragma unroll
        for (uint32_t b = 0; b < kMaxCluster; ++b) {
            pair[0] += part[b][0];
            pair[1] += part[b][1];
        }
        const u64 total = warp_total(one), want = COUNT ? k : top_p_target(p, total);
        u64 inc = warp_inclusive(pair[0] + pair[1]), before = inc - pair[0] - pair[1];
        unsigned int at = __ffs(__ballot_sync(0xffffffffu, want <= inc)) - 1;  // (none: bin 1023)
        at = min(at, 31u);
        const bool upper = want > before + pair[0];
        if (upper) before += pair[0];
        before = __shfl_sync(0xffffffffu, before, at);
        const uint32_t first = 16 * (2 * at + __shfl_sync(0xffffffffu, (unsigned int)upper, at));
        u64 v = 0;
#pragma unroll
        for (uint32_t b = 0; b < kMaxCluster; b += 2)
            if (b + lane / 16 < blocks) v += ld_cluster_u64(at_rank(sums + first + lane % 16, b + lane / 16));
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        inc = before + warp_inclusive(lane < 16 ? v : 0ull);
        at = __ffs(__ballot_sync(0xffffffffu, want <= inc)) - 1;
        if (lane == min(at, 15u)) {
            sh.cast[0] = first + lane;
            sh.cast[1] = inc - v;
            sh.cast[2] = inc;
            sh.cast[3] = total;
            sh.cast[4] = want;
        }
    }
    __syncthreads();
    const u64 total = sh.cast[3], want = sh.cast[4];
    if (COUNT && total <= want) {  // all that have a weight are kept
        cluster_arrive();  // the sums are written again
        cluster_wait();
        *last = limit;
        return false;
    }
    c.bin = (uint32_t)sh.cast[0];
    const u64 above = sh.cast[1];
    // Are there few enough to gather all up to this bin? None there weighs less than the bin's far
    // end, less more than the recipe's error.
    const uint32_t far = exp2_weight(((float)c.bin + 0.5f) * (1.0f / 32.0f)), slack = (far >> 16) + 2;
    c.upto = sh.cast[2] <= (COUNT ? (u64)kList : (u64)max(far > slack ? far - slack : 0u, c.floor_q) * kList);
    u64 half[2] = {0, 0};  // weights of the bins before it
    if (!COUNT) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            half[h] = (2 * threadIdx.x < c.bin ? own[h][0] : 0ull) + (2 * threadIdx.x + 1 < c.bin ? own[h][1] : 0ull);
        block_totals(half);
    }
    // Every logit in a bin up to this one is at or above thr, every one in a bin from it on at or
    // below cap; the few others between them are taken out of the list afterwards.
    c.thr = __fsub_rd(rule.m, __fmul_ru(((float)c.bin + 0.51f) * (1.0f / 32.0f), octave));
    c.cap = c.upto || c.bin == 0 ? INFINITY
                                 : __fsub_ru(rule.m, __fmul_rd(((float)c.bin - 0.51f) * (1.0f / 32.0f), octave));
    collect(sl, end.per_warp, c.thr, c.cap);
#pragma unroll 1
    for (uint32_t i = threadIdx.x; i < min(sh.n_list, (uint32_t)kLocal); i += kSThreads)
        if (!in_crossing<COUNT>(c, rule, key_logit(~(uint32_t)(sh.items[i] >> 32)), sh.items[i])) sh.items[i] = kNoItem;
    exchange(list_slot, sh.n_list, half[0] + half[1]);
    const uint32_t n = gathered(list_slot);
    u64 left;
    if (n > kList) {
        c.upto = false;
        *last = select_in_bin<COUNT>(sl, rule, c, want - above, &left);
        if (COUNT) return false;
        weigh_and_draw(sl, rule, *last, end);
        return true;
    }
    if (!c.upto || rank == 0) pull(list_slot, n);
    cluster_arrive();  // no block leaves, or writes over its list, while others read it
    if (c.upto) {
        if (rank == 0) finish_list(n, COUNT ? k : 0xffffffffu, p, COUNT ? 0ull : total, rule, end);
        cluster_wait();
        return true;
    }
    // every block finds the crossing among the gathered, and what is kept of them where
    weigh_items<COUNT>(n, kKeepAll, rule);
    *last = block_select(n, false, want - above, &left, item_of(key_of(fminf(c.cap, rule.m)), 0),
                         item_of(key_of(c.thr), 0xffffffffu));
    if (!COUNT) {
        left += above + item_weight(*last, rule);
        const uint32_t from = (uint32_t)slot_total(list_slot, rank), to = from + sh.n_list;
        const uint32_t second = (rank * kSWarps + kSWarps / 2) * end.per_warp * V::N;  // its first element
        u64 kept[3] = {0, 0, 0};  // by the blocks before, and by this one's halves
#pragma unroll 1
        for (uint32_t i = threadIdx.x; i < to; i += kSThreads) {
            const u64 item = sh.items[kLocal + i];
            if (item > *last) continue;
            const u64 q = sh.picks.weights[i];
            if (i < from) kept[0] += q;
            else if ((uint32_t)item + sl.pad < second) kept[1] += q;
            else kept[2] += q;
        }
        block_totals(kept);
        half[0] += kept[1];
        half[1] += kept[2];
        cluster_wait();
        draw(sl, rule, *last, left, kept[0] + slot_total(list_slot, rank, 1),
             threadIdx.x % 32 == 0 ? half[0] : threadIdx.x % 32 == 1 ? half[1] : 0ull, kSWarps / 2, end);
        return true;
    }
    cluster_wait();
    return false;
}

// A row whose largest logit is infinite, or whose scale is: only the largest
// have a weight, 2^31 each.
template <typename T>
__device__ __noinline__ void sample_largest(Slice<T> sl, uint32_t row_key, uint32_t k, float p,
                                            RowEnd end) {
    u64 ties = 0;
    sl.each(key_logit(row_key), [&](const auto &r, unsigned int) {
        float x[Vec<T>::N];
        Vec<T>::unpack(r, x);
#pragma unroll
        for (int e = 0; e < Vec<T>::N; ++e) ties += x[e] == key_logit(row_key);
    });
    exchange(kSlotFirst, block_total(ties), 0);
    ties = slot_total(kSlotFirst, cluster_size());
    if (k > 0 && k < ties) ties = k;
    if (p > 0.0f && p < 1.0f) ties = (top_p_target(p, ties << 31) + (1ull << 31) - 1) >> 31;
    const u64 nth = (draw_of(end.word, ties << 31) >> 31) + 1;
    const u64 item = nth_tie(sl, row_key, nth, kSlotSumTies, kSlotSumTie);
    if (cluster_rank() == 0 && threadIdx.x == 0) write_token(end, (uint32_t)item, 1ull << 31, ties << 31);
}

template <typename T>
__global__ void __launch_bounds__(kSThreads, 2) sample_kernel(const SampleArgs a) {
    SampleShared &sh = block_shared();
    using V = Vec<T>;
    const uint32_t rank = cluster_rank(), blocks = cluster_size();
    const u64 row = blockIdx.x / blocks;
    const RowEnd end{a.tokens + row, a.probs ? a.probs + row : nullptr, a.random[row], a.per_warp};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // paired with the wait before the first exchange: every block has started (nothing written yet)
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    if (threadIdx.x == 0) sh.n_list = 0;

    Slice<T> sl;
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(static_cast<const T *>(a.logits) + row * a.row_stride);
        constexpr uintptr_t within = sizeof(typename V::Raw) - 1;
        sl.base = reinterpret_cast<const char *>(at & ~within);
        sl.pad = (unsigned int)(at & within) / sizeof(T);
        sl.n = (unsigned int)a.vocab;
        const unsigned int nv = (sl.pad + sl.n + V::N - 1) / V::N;
        sl.staged_iters = a.staged_iters;
        sl.v0 = (rank * kSWarps + warp) * a.per_warp;
        sl.count = sl.v0 < nv ? min(a.per_warp, nv - sl.v0) : 0u;
        sl.stage = reinterpret_cast<uint4 *>(&sh + 1) + warp * 32 * sl.kLane * a.staged_iters + lane;
    }
    const float t = a.temperature ? a.temperature[row] : 1.0f;
    const int k_arg = a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.0f;
    const float mp = a.min_p ? a.min_p[row] : 0.0f;
    const uint32_t k = k_arg > 0 && (uint32_t)k_arg < sl.n ? (uint32_t)k_arg : 0u;
    const bool cut_p = p > 0.0f && p < 1.0f;

    // the row's largest logit, and for top-k the maxima its bound comes from
    uint32_t thread_key;
    const uint32_t warp_key = sl.first_pass(&thread_key);
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
    if ((k > 0 || cut_p) && !bounded) {  // a histogram comes first
        sh.bins[0].clear();
        sh.bins[1].clear();
    }
    cluster_wait();
    uint32_t *maxima = reinterpret_cast<uint32_t *>(sh.items + kLocal);  // of all the row's groups
    if (by_groups && threadIdx.x % group == 0)
        for (uint32_t c = 0; c < blocks; ++c)
            st_cluster(at_rank(maxima + rank * groups + threadIdx.x / group, c), group_key);
    if (lane < (int)blocks) st_cluster(at_rank(&sh.warp_keys[rank][warp], lane), warp_key);
    cluster_arrive();
    cluster_wait();
    uint32_t row_key = 0;
#pragma unroll
    for (uint32_t i = 0; i < kMaxCluster; i += 32 / kSWarps)
        if (i + lane / kSWarps < blocks) row_key = max(row_key, sh.warp_keys[i + lane / kSWarps][lane % kSWarps]);
    row_key = __reduce_max_sync(0xffffffffu, row_key);
    if (row_key <= kKeyOfMinusInf) {  // the mask leaves nothing
        if (rank == 0 && threadIdx.x == 0) {
            *end.token = -1;
            if (end.prob) *end.prob = 0.0f;
        }
        return;
    }
    RowRule rule;
    rule.m = key_logit(row_key);
    rule.scale = __fdiv_rn(kLog2e, t);
    rule.qmin = mp > 0.0f ? __float2uint_ru(__fmul_rn(fminf(mp, 1.0f), 0x1p31f)) : 0u;  // (the product is exact)

    if (!(t > 0.0f)) {  // the first of the largest
        uint32_t first = 0xffffffffu;
        if (warp_key == row_key)
            sl.each(rule.m, [&](const auto &r, unsigned int v) {
                if (first != 0xffffffffu || !(V::max(r) >= rule.m)) return;
                float x[V::N];
                V::unpack(r, x);
#pragma unroll
                for (int e = V::N - 1; e >= 0; --e)
                    if (x[e] == rule.m) first = sl.index(v, e);
            });
        exchange(kSlotFirst, block_min(first), 0);
        first = __reduce_min_sync(0xffffffffu, lane < (int)blocks ? (uint32_t)sh.slots[kSlotFirst][lane][0] : first);
        if (rank == 0 && threadIdx.x == 0) {
            *end.token = (int32_t)first;
            if (end.prob) *end.prob = 1.0f;
        }
        return;
    }
    if (!(rule.m < INFINITY) || !(rule.scale < INFINITY)) {
        sample_largest(sl, row_key, k, p, end);
        return;
    }
    if (bounded) {
        const uint32_t bound = by_groups ? kth_bound(maxima, groups * blocks, k, row_key) : 0u;
        collect(sl, end.per_warp, bound > kKeyOfMinusInf ? key_logit(bound) : -INFINITY, INFINITY);
        exchange(kSlotBound, sh.n_list, 0);
        const uint32_t n = gathered(kSlotBound);
        if (n <= kList) {
            if (rank == 0) pull(kSlotBound, n);
            cluster_arrive();
            if (rank == 0) finish_list(n, k, p, 0ull, rule, end);
            cluster_wait();
            return;
        }
    }
    u64 last = kKeepAll;
    if (k > 0 && filter<true>(sl, rule, k, p, kKeepAll, end, &last, !bounded)) return;
    if (cut_p) {
        u64 cut;
        filter<false>(sl, rule, k, p, last, end, &cut, k == 0);
        return;
    }
    weigh_and_draw(sl, rule, last, end);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Blocks a row, where a test fixes them; 0: by the rule in sample_launch.
#ifndef U32SCAN_SAMPLE_BLOCKS
#define U32SCAN_SAMPLE_BLOCKS 0
#endif

// Bytes of a row a block keeps in shared memory: two blocks an SM.
constexpr unsigned int kMaxStage = 64 * 1024;
// Blocks at a time: two on each of a GB300's 152 SMs. (With fewer SMs at hand, as in a
// partition, the rule below takes more rows for one wave than run in it; results are the same.)
constexpr unsigned int kResident = 304;
static_assert(sizeof(SampleShared) % 16 == 0 && offsetof(SampleShared, slots) % 16 == 0 && kLocal % 2 == 0,
              "16-byte accesses");
static_assert(U32SCAN_MAX_VOCAB / 8 / kMaxCluster / kSWarps + 8 < 65536, "a warp's vectors in 16 bits");
static_assert(2 * (sizeof(SampleShared) + kMaxStage + 1024) <= 228 * 1024, "two blocks an SM");

template <typename T>
static int sample_launch(SampleArgs a, cudaStream_t stream) {
    // The largest cluster with which all rows run at a time, a thread still having a vector, and
    // slices of at most 65536 logits. Fewer and larger slices pay the barriers and the
    // serial steps less often, more and smaller ones share a long row's passes: 256 x 262144 f32 mixed
    // takes 132, 112, 125 us with 2, 4, 8 blocks a row, 64 x 131072 bf16 top-p 38, 35, 46, 256 x 32000
    // bf16 top-p 32, 38, 53 with 1, 2, 4, 7 x 50257 f32 top-p 34, 24, 19, 16 with 1, 2, 4, 8.
    constexpr unsigned int vec_bytes = sizeof(typename Vec<T>::Raw);
    const bool aligned = reinterpret_cast<uintptr_t>(a.logits) % vec_bytes == 0 && a.row_stride % Vec<T>::N == 0;
    const unsigned int nv = (unsigned int)((a.vocab + (aligned ? 1 : 2) * (Vec<T>::N - 1)) / Vec<T>::N);
    unsigned int blocks = 1;
    while (blocks < kMaxCluster &&
           (a.vocab > blocks * 65536ull || (2 * a.rows * blocks <= kResident && nv > blocks * kSThreads)))
        blocks *= 2;
#if U32SCAN_SAMPLE_BLOCKS
    blocks = U32SCAN_SAMPLE_BLOCKS;
#endif
    const unsigned int per_block = (nv + blocks - 1) / blocks;
    a.per_warp = ((per_block + kSWarps - 1) / kSWarps + 7) / 8 * 8;
    const unsigned int iters = (a.per_warp + 31) / 32;
    constexpr unsigned int turn_bytes = kSThreads * vec_bytes;
    a.staged_iters = iters < kMaxStage / turn_bytes ? iters : kMaxStage / turn_bytes;
    const size_t smem = sizeof(SampleShared) + (size_t)a.staged_iters * turn_bytes;
    if (cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(sizeof(SampleShared) + kMaxStage)) != cudaSuccess)
        return U32SCAN_ECUDA;
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
    if (rows >= (1ull << 28) || vocab > U32SCAN_MAX_VOCAB) return U32SCAN_EINVAL;
    if (rows > 1 && row_stride >= (1ull << 32)) return U32SCAN_EINVAL;  // one row's is not used
    if (rows == 0) return U32SCAN_OK;
    const uintptr_t elem = type == U32SCAN_F32 ? 3 : 1;
    if ((vocab > 0 && logits == nullptr) || random == nullptr || tokens == nullptr) return U32SCAN_EINVAL;
    if (reinterpret_cast<uintptr_t>(logits) & elem) return U32SCAN_EINVAL;
    for (const void *p : {(const void *)temperature, (const void *)top_k, (const void *)top_p, (const void *)min_p,
                          (const void *)random, (const void *)tokens, (const void *)probs})
        if (reinterpret_cast<uintptr_t>(p) & 3) return U32SCAN_EINVAL;
    const SampleArgs a{logits, rows, vocab, row_stride, temperature, top_k, top_p, min_p, random, tokens, probs, 0, 0};
    const cudaStream_t s = (cudaStream_t)stream;
    if (type == U32SCAN_F32) return sample_launch<float>(a, s);
    if (type == U32SCAN_F16) return sample_launch<__half>(a, s);
    return sample_launch<__nv_bfloat16>(a, s);
}
