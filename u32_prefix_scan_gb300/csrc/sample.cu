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
//   top-k   the bound pass: the ceil(k / blocks)-th largest of each block's
//           512 thread maxima is a bound below which no kept token lies;
//           the few logits at or above it are gathered into one block, which
//           ranks them.
//   top-p   a histogram of the weights by y (32 bins an octave) gives the bin
//           in which the prefix sum crosses; that bin's logits are gathered
//           and sorted (or all above it too, if they are few: then the
//           gathering block makes the draw as well).
//   else    (huge k, long ties, infinite logits) radix selection on the
//           logits' bits, 8 a level, on counts or sums of weights.
// A filter ends at a key `tau` and at how many of the logits equal to it stay
// (those with the lowest indices).
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
constexpr int kRanked = 256;  // of them, ranked by counting rather than by sorting
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
};

// Exchanges between a cluster's blocks: one slot each, so that none is
// written again while a slow block still reads it.
enum Slot { kSlotMax, kSlotFirst, kSlotSecond, kSlotThird, kSlotAbove, kSlotDraw, kSlots };

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
// contraction).
constexpr float kC1 = -0x1.62e42ap-1f, kC2 = 0x1.ebf9bcp-3f, kC3 = -0x1.c6b752p-5f, kC4 = 0x1.3cea88p-7f,
                kC5 = -0x1.5bba14p-10f;
constexpr float kRound = 0x1.8p23f;  // adding and taking it away rounds to an integer, ties to even

__device__ __forceinline__ uint32_t exp2_weight(float y) {
    const float t = __fadd_rn(y, kRound);
    const float f = __fsub_rn(y, __fsub_rn(t, kRound));
    float p = __fadd_rn(__fmul_rn(kC5, f), kC4);
    p = __fadd_rn(__fmul_rn(p, f), kC3);
    p = __fadd_rn(__fmul_rn(p, f), kC2);
    p = __fadd_rn(__fmul_rn(p, f), kC1);
    p = __fadd_rn(__fmul_rn(p, f), 1.0f);
    // times 2^(31 - n), exact; n is in t's low bits, and 0x4b400000 << 23 = 0
    return __float2uint_rz(__fmul_rn(p, __uint_as_float((158u << 23) - (__float_as_uint(t) << 23))));
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
    p2 = add2(mul2(p2, f2), pack2(1.0f, 1.0f));
    float t[2], w[2];
    unpack2(t2, t[0], t[1]);
    unpack2(mul2(p2, pack2(__uint_as_float((158u << 23) - (__float_as_uint(t[0]) << 23)),
                           __uint_as_float((158u << 23) - (__float_as_uint(t[1]) << 23)))),
            w[0], w[1]);
    q[0] = __float2uint_rz(w[0]);
    q[1] = __float2uint_rz(w[1]);
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

// Ascending sort of the first `size` (a power of two) words by the block.
__device__ __forceinline__ void block_sort(u64 *a, unsigned int size) {
    for (unsigned int k = 2; k <= size; k <<= 1)
        for (unsigned int j = k >> 1; j > 0; j >>= 1) {
            for (unsigned int c = threadIdx.x; c < size / 2; c += kSThreads) {
                const unsigned int i = 2 * c - (c & (j - 1)), o = i + j;  // c-th pair at distance j
                const u64 x = a[i], y = a[o];
                if ((x > y) == ((i & k) == 0)) {
                    a[i] = y;
                    a[o] = x;
                }
            }
            __syncthreads();
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
};

// Where a filter ends: keys above tau stay, and the first `ties` (by index)
// of those equal to it.
struct Cut {
    uint32_t tau;
    u64 ties;
};

// The key at which the running total over keys in descending order, of counts
// or of weights (MASS) of the keys from floor_key on, first reaches `target`
// (1 <= target <= the whole total), and what is missing above it (>= 1).
// `level` numbers the levels of a row's selections (their two buffers swap:
// a slow block may still read the last level's).
template <bool MASS, typename T>
__device__ __noinline__ void radix_select(SampleShared &sh, const Slice<T> &sl, const RowRule &rule,
                                          uint32_t floor_key, u64 target, int &level, uint32_t *tau, u64 *missing) {
    const int lane = threadIdx.x & 31;
    uint32_t prefix = 0, mask = 0;
    for (int shift = 24; shift >= 0; shift -= 8, ++level) {
        SumBins<256> &hist = sh.digits[level & 1];
        hist.clear();
        __syncthreads();
        sl.each(lane, [&](const uint4 &r, unsigned int) {
            float x[Vec<T>::N];
            Vec<T>::unpack(r, x);
#pragma unroll
            for (int e = 0; e < Vec<T>::N; ++e) {
                if (x[e] != x[e]) x[e] = -INFINITY;
                const uint32_t k = key_of(x[e]);
                if ((k & mask) != prefix || k < floor_key) continue;
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

__device__ __forceinline__ void write_token(const SampleArgs &a, u64 row, uint32_t index, u64 q, u64 total) {
    a.tokens[row] = (int32_t)index;
    if (a.probs) a.probs[row] = (float)((double)q / (double)total);
}

__device__ __forceinline__ u64 draw_of(uint32_t word, u64 total) { return __umul64hi((u64)word << 32, total); }

__device__ __forceinline__ u64 top_p_target(float p, u64 total) {
    return (u64)ceil(__dmul_rn((double)p, (double)total));
}

// The draw among what `cut` leaves, in index order. mass and ties: what this
// warp's vectors hold above tau and at it.
template <typename T>
__device__ __noinline__ void draw(SampleShared &sh, const Slice<T> &sl, const RowRule &rule, const Cut &cut,
                                  u64 q_tau, u64 total, u64 mass, u64 ties, const SampleArgs &a, u64 row) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const u64 r = draw_of(a.random[row], total);
    __syncthreads();
    if (lane == 0) {
        sh.warp_a[warp] = mass;
        sh.warp_b[warp] = ties;
    }
    __syncthreads();
    u64 block_mass = 0, block_ties = 0;
#pragma unroll
    for (int w = 0; w < kSWarps; ++w) {
        block_mass += sh.warp_a[w];
        block_ties += sh.warp_b[w];
    }
    exchange(sh, kSlotDraw, block_mass, block_ties);
    u64 before = 0, tie_left = cut.ties;
    for (uint32_t c = 0; c < cluster_rank(); ++c) {
        const u64 t = min(tie_left, sh.slots[kSlotDraw][c][1]);
        before += sh.slots[kSlotDraw][c][0] + t * q_tau;
        tie_left -= t;
    }
    for (int w = 0; w < warp; ++w) {
        const u64 t = min(tie_left, sh.warp_b[w]);
        before += sh.warp_a[w] + t * q_tau;
        tie_left -= t;
    }
    if (!(before <= r && r - before < mass + min(tie_left, ties) * q_tau)) return;
    // this warp's: 32 vectors a turn
    for (unsigned int j0 = 0, it = 0; j0 < sl.per_warp && sl.v0 + j0 < sl.nv; j0 += 32, ++it) {
        const unsigned int j = j0 + lane;
        float x[Vec<T>::N];
        const bool in = j < sl.per_warp && sl.v0 + j < sl.nv;
        if (in) Vec<T>::unpack(it < sl.staged_iters ? sl.stage[32 * it] : sl.load(sl.v0 + j), x);
        unsigned int tied = 0;  // by element
        u64 sum = 0;
#pragma unroll
        for (int e = 0; e < Vec<T>::N; ++e) {
            if (!in || x[e] != x[e]) x[e] = -INFINITY;
            const uint32_t k = key_of(x[e]);
            if (k > cut.tau) sum += token_weight(x[e], rule);
            if (k == cut.tau) tied |= 1u << e;
        }
        u64 t_inc = __popc(tied);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const u64 o = __shfl_up_sync(0xffffffffu, t_inc, d);
            if (lane >= d) t_inc += o;
        }
        u64 my_ties = t_inc - __popc(tied);  // before this lane's
        my_ties = my_ties < tie_left ? tie_left - my_ties : 0ull;
        sum += min(my_ties, (u64)__popc(tied)) * q_tau;
        u64 inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const u64 o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        const unsigned int hit = __ballot_sync(0xffffffffu, before + inc > r);
        if (hit) {
            if (lane != __ffs(hit) - 1) return;
            u64 at = before + inc - sum;
#pragma unroll
            for (int e = 0; e < Vec<T>::N; ++e) {
                u64 q = 0;
                if (key_of(x[e]) > cut.tau) q = token_weight(x[e], rule);
                else if ((tied >> e & 1u) && my_ties > 0) {
                    q = q_tau;
                    --my_ties;
                }
                if (at <= r && r < at + q) write_token(a, row, sl.index(sl.v0 + j, e), q, total);
                at += q;
            }
            return;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
        const u64 used = __shfl_sync(0xffffffffu, t_inc, 31);
        tie_left -= min(tie_left, used);
    }
}

// What the vectors of this warp hold above the cut's key, and at it.
template <typename T>
__device__ __forceinline__ void cut_pass(const Slice<T> &sl, const RowRule &rule, const Cut &cut, u64 *mass,
                                         u64 *ties) {
    const float thr = cut.tau ? key_logit(cut.tau) : -INFINITY;
    u64 m = 0;
    unsigned int t = 0;
    sl.each(threadIdx.x & 31, [&](const uint4 &r, unsigned int) {
        if (!(Vec<T>::max(r) >= thr)) return;
        float x[Vec<T>::N];
        Vec<T>::unpack(r, x);
#pragma unroll
        for (int e = 0; e < Vec<T>::N; ++e) {
            if (x[e] > thr) m += token_weight(x[e], rule);
            t += x[e] == thr;
        }
    });
    *mass = warp_total(m);
    *ties = __reduce_add_sync(0xffffffffu, t);
}

// Gathers the logits that keep(x) names into this block's list.
template <typename T, typename Keep>
__device__ __forceinline__ void collect(SampleShared &sh, const Slice<T> &sl, float thr, Keep keep) {
    sl.each(threadIdx.x & 31, [&](const uint4 &r, unsigned int v) {
        if (!(Vec<T>::max(r) >= thr)) return;
        float x[Vec<T>::N];
        Vec<T>::unpack(r, x);
#pragma unroll
        for (int e = 0; e < Vec<T>::N; ++e)
            if (x[e] >= thr && x[e] > -INFINITY && keep(x[e])) {
                const uint32_t at = atomicAdd(&sh.n_list, 1u);
                if (at < kLocal) sh.list[at] = (u64)~key_of(x[e]) << 32 | sl.index(v, e);
            }
    });
    __syncthreads();
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

// All blocks' lists, one after another in rank 0's gather (called there, when
// they fit).
__device__ __forceinline__ void pull(SampleShared &sh, Slot slot) {
    uint32_t at = 0;
    for (uint32_t c = 0; c < cluster_size(); ++c) {
        const uint32_t n = (uint32_t)sh.slots[slot][c][0];
        for (uint32_t i = threadIdx.x; i < n; i += kSThreads) sh.gather[at + i] = ld_cluster_u64(at_rank(sh.list + i, c));
        at += n;
    }
    __syncthreads();
}

__device__ __forceinline__ uint32_t item_weight(u64 item, const RowRule &rule) {
    return token_weight(key_logit(~(uint32_t)(item >> 32)), rule);
}

// The token among the n gathered logits, which hold all that the filters
// keep: the first k of them in order, and of those the top-p prefix (p < 1),
// measured against `total` if that is not 0, else against their own sum.
__device__ __noinline__ void finish_list(SampleShared &sh, uint32_t n, uint32_t k, float p, u64 total,
                                         const RowRule &rule, const SampleArgs &a, u64 row) {
    const bool cut_p = p > 0.0f && p < 1.0f;
    const uint32_t word = a.random[row];
    u64 *weight = sh.list;  // pulled: free
    if (n <= kRanked) {
        // two threads an item count what stands before it
        const uint32_t i = threadIdx.x >> 1, half = threadIdx.x & 1;
        const u64 item = i < n ? sh.gather[i] : ~0ull;
        const u64 q = i < n ? item_weight(item, rule) : 0u;
        if (half == 0) weight[i] = q;
        __syncthreads();
        uint32_t rank = 0;
        u64 before = 0;
        for (uint32_t j = half; j < n; j += 2)
            if (sh.gather[j] < item) {
                ++rank;
                before += weight[j];
            }
        rank += __shfl_xor_sync(0xffffffffu, rank, 1);
        before += __shfl_xor_sync(0xffffffffu, before, 1);
        u64 kept = i < n && rank < k ? q : 0ull;
        if (total == 0) total = block_total(half == 0 ? kept : 0ull, sh.warp_a);
        if (cut_p) {
            if (before >= top_p_target(p, total)) kept = 0;
            total = block_total(half == 0 ? kept : 0ull, sh.warp_a);
        }
        __syncthreads();
        if (half == 0) weight[i] = kept;
        __syncthreads();
        u64 at = 0;
        for (uint32_t j = half; j < n; j += 2)
            if ((uint32_t)sh.gather[j] < (uint32_t)item) at += weight[j];
        at += __shfl_xor_sync(0xffffffffu, at, 1);
        const u64 r = draw_of(word, total);
        if (half == 0 && at <= r && r < at + kept) write_token(a, row, (uint32_t)item, kept, total);
        return;
    }
    unsigned int size = 512;
    while (size < n) size <<= 1;
    for (unsigned int i = n + threadIdx.x; i < size; i += kSThreads) sh.gather[i] = ~0ull;
    __syncthreads();
    block_sort(sh.gather, size);
    constexpr int C = kList / kSThreads;
    const unsigned int per = size / kSThreads;
    u64 q[C], sum = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const unsigned int i = threadIdx.x * per + c;
        q[c] = c < (int)per && i < n && i < k ? item_weight(sh.gather[i], rule) : 0u;
        sum += q[c];
    }
    if (total == 0) total = block_total(sum, sh.warp_a);
    if (cut_p) {
        const u64 want = top_p_target(p, total);
        u64 before = block_before(sum, sh.warp_a);
        sum = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const u64 own = q[c];
            if (before >= want) q[c] = 0;
            before += own;
            sum += q[c];
        }
        total = block_total(sum, sh.warp_a);
    }
    // the same items by index
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const unsigned int i = threadIdx.x * per + c;
        if (c < (int)per) sh.gather[i] = i < n ? sh.gather[i] << 32 | q[c] : ~0ull << 32;
    }
    __syncthreads();
    block_sort(sh.gather, size);
    sum = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        q[c] = c < (int)per ? (uint32_t)sh.gather[threadIdx.x * per + c] : 0u;
        sum += q[c];
    }
    u64 at = block_before(sum, sh.warp_a);
    const u64 r = draw_of(word, total);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (at <= r && r < at + q[c])
            write_token(a, row, (uint32_t)(sh.gather[threadIdx.x * per + c] >> 32), q[c], total);
        at += q[c];
    }
}

// The filters by selection on the logits' bits, then the draw: right for
// every row, and the way of those the other paths do not take.
template <typename T>
__device__ __noinline__ void sample_by_selection(SampleShared &sh, const Slice<T> &sl, const RowRule &rule, uint32_t k,
                                                 float p, const SampleArgs &a, u64 row) {
    Cut cut{0u, 0ull};  // no key is 0: everything stays
    int level = 0;
    if (k > 0) radix_select<false>(sh, sl, rule, 0u, k, level, &cut.tau, &cut.ties);
    u64 q_tau = k > 0 ? token_weight(key_logit(cut.tau), rule) : 0u;
    u64 mass, ties;
    cut_pass(sl, rule, cut, &mass, &ties);
    const u64 above_block = block_total((threadIdx.x & 31) == 0 ? mass : 0ull, sh.warp_c);
    exchange(sh, kSlotAbove, above_block, 0);
    u64 above = 0;
    for (uint32_t c = 0; c < cluster_size(); ++c) above += sh.slots[kSlotAbove][c][0];
    u64 total = above + cut.ties * q_tau;
    if (p > 0.0f && p < 1.0f) {
        const u64 want = top_p_target(p, total);
        if (want > above) {  // ends among the ties
            cut.ties = (want - above + q_tau - 1) / q_tau;
            total = above + cut.ties * q_tau;
        } else {
            u64 missing;
            radix_select<true>(sh, sl, rule, cut.tau + 1u, want, level, &cut.tau, &missing);
            q_tau = token_weight(key_logit(cut.tau), rule);
            cut.ties = (missing + q_tau - 1) / q_tau;
            total = want - missing + cut.ties * q_tau;
            cut_pass(sl, rule, cut, &mass, &ties);
        }
    }
    draw(sh, sl, rule, cut, q_tau, total, mass, ties, a, row);
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

    // the row's largest logit, and for top-k the bound
    const float thread_max = sl.first_pass(lane);
    const uint32_t thread_key = key_of(thread_max == thread_max ? thread_max : -INFINITY);
    const uint32_t warp_key = __reduce_max_sync(0xffffffffu, thread_key);
    if (lane == 0) sh.warp_a[warp] = warp_key;
    const uint32_t share = (k + blocks - 1) / blocks;
    const bool bounded = k > 0 && (sl.n <= kLocal || share <= kSThreads / 2);
    uint32_t bound = 0;
    if (bounded && sl.n > kLocal) {
        // the largest 16-bit prefix that at least `share` thread maxima reach
        for (uint32_t bit = 0x80000000u; bit >= 0x10000u; bit >>= 1)
            if (__syncthreads_count(thread_key >= (bound | bit)) >= (int)share) bound |= bit;
    } else {
        __syncthreads();
    }
    uint32_t block_key = 0;
#pragma unroll
    for (int w = 0; w < kSWarps; ++w) block_key = max(block_key, (uint32_t)sh.warp_a[w]);
    cluster_wait();
    exchange(sh, kSlotMax, block_key, bound);
    uint32_t row_key = 0;
    for (uint32_t c = 0; c < blocks; ++c) {
        row_key = max(row_key, (uint32_t)sh.slots[kSlotMax][c][0]);
        bound = min(bound, (uint32_t)sh.slots[kSlotMax][c][1]);
    }
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
        collect(sh, sl, bound > kKeyOfMinusInf ? key_logit(bound) : -INFINITY, [](float) { return true; });
        exchange(sh, kSlotFirst, sh.n_list, 0);
        const uint32_t n = gathered(sh, kSlotFirst);
        if (n <= kList) {
            if (rank == 0) pull(sh, kSlotFirst);
            cluster_arrive();
            if (rank == 0) finish_list(sh, n, k, p, 0ull, rule, a, row);
            cluster_wait();
            return;
        }
    } else if (finite && k == 0) {
        // all weights; for top-p also the histogram of the distances that can matter: past
        // cut_y the row holds less than (1 - p) of the largest weight
        const float cut_y = cut_p ? fminf(31.0f, log2f((float)sl.n / (1.0f - p)) + 0.1f) : 0.0f;
        if (cut_p) {
            sh.bins.clear();
            __syncthreads();
        }
        const u64 m2 = pack2(rule.m, rule.m), scale2 = pack2(rule.scale, rule.scale);
        u64 mass = 0;
        sl.each(lane, [&](const uint4 &r, unsigned int) {
            float x[V::N];
            V::unpack(r, x);
#pragma unroll
            for (int e = 0; e < V::N; e += 2) {
                float y[2];
                uint32_t q[2];
                weigh2(x[e], x[e + 1], m2, scale2, y, q);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t w = q[i] >= rule.qmin ? q[i] : 0u;
                    mass += w;
                    if (y[i] < cut_y && w) sh.bins.add(bin_of(y[i]), w);
                }
            }
        });
        mass = warp_total(mass);
        if (!cut_p) {
            const u64 block_mass = block_total(lane == 0 ? mass : 0ull, sh.warp_c);
            exchange(sh, kSlotFirst, block_mass, 0);
            u64 total = 0;
            for (uint32_t c = 0; c < blocks; ++c) total += sh.slots[kSlotFirst][c][0];
            draw(sh, sl, rule, Cut{0u, 0ull}, 0ull, total, mass, 0ull, a, row);
            return;
        }
        const u64 block_mass = block_total(lane == 0 ? mass : 0ull, sh.warp_c);
        exchange(sh, kSlotFirst, block_mass, 0);
        u64 total = 0;
        for (uint32_t c = 0; c < blocks; ++c) total += sh.slots[kSlotFirst][c][0];
        const u64 want = top_p_target(p, total);
        // the bin in which the running sum reaches `want`, two bins a thread
        u64 bin_mass[2] = {0, 0};
        for (uint32_t c = 0; c < blocks; ++c) {
            const u64 low = ld_cluster_u64(at_rank(&sh.bins.low[2 * threadIdx.x], c));
            const u64 high = ld_cluster_u64(at_rank(&sh.bins.high[2 * threadIdx.x], c));
            bin_mass[0] += (low & 0xffffffffull) | high << 32;
            bin_mass[1] += low >> 32 | (high >> 32) << 32;
        }
        // at most so many logits with a weight lie in a bin: none weighs less than its far end,
        // less more than the recipe's error
        u64 at_most[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t far = exp2_weight(((float)(2 * threadIdx.x + i) + 0.5f) * (1.0f / 32.0f));
            const uint32_t slack = (far >> 16) + 2;
            const uint32_t least = max(far > slack ? far - slack : 0u, max(rule.qmin, 1u));
            at_most[i] = (u64)((float)bin_mass[i] / (float)least * 1.001f) + (bin_mass[i] ? 1u : 0u);
        }
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
        // every logit in a bin up to this one is at or above
        const float thr = __fsub_rd(rule.m, __fdiv_ru(((float)bin + 1.0f) * (1.0f / 32.0f), rule.scale));
        collect(sh, sl, thr, [&](float x) {
            const float y = __fmul_rn(__fsub_rn(rule.m, x), rule.scale);
            if (!(y < cut_y) || token_weight(x, rule) == 0u) return false;
            const uint32_t b = bin_of(y);
            return all ? b <= bin : b == bin;
        });
        exchange(sh, kSlotSecond, sh.n_list, 0);
        const uint32_t n = gathered(sh, kSlotSecond);
        if (n <= kList) {
            if (rank == 0) pull(sh, kSlotSecond);
            if (all) {
                cluster_arrive();
                if (rank == 0) finish_list(sh, n, 0xffffffffu, p, total, rule, a, row);
                cluster_wait();
                return;
            }
            u64 tau = 0, ties = 0;
            if (rank == 0) {  // the crossing among the gathered
                unsigned int size = 512;
                while (size < n) size <<= 1;
                for (unsigned int i = n + threadIdx.x; i < size; i += kSThreads) sh.gather[i] = ~0ull;
                __syncthreads();
                block_sort(sh.gather, size);
                const unsigned int per = size / kSThreads;
                u64 sum = 0;
                for (unsigned int c = 0; c < per; ++c) {
                    const unsigned int i = threadIdx.x * per + c;
                    if (i < n) sum += item_weight(sh.gather[i], rule);
                }
                u64 at = above + block_before(sum, sh.warp_a);
                for (unsigned int c = 0; c < per; ++c) {
                    const unsigned int i = threadIdx.x * per + c;
                    if (i >= n) break;
                    const u64 q = item_weight(sh.gather[i], rule);
                    if (at < want && want <= at + q) {
                        const uint32_t high = (uint32_t)(sh.gather[i] >> 32);
                        unsigned int first = i;
                        while (first > 0 && (uint32_t)(sh.gather[first - 1] >> 32) == high) --first;
                        sh.cast[0] = (u64)~high << 32 | (i - first + 1);
                        sh.cast[1] = at + q;
                    }
                    at += q;
                }
                __syncthreads();
                tau = sh.cast[0];
                ties = sh.cast[1];
            }
            exchange(sh, kSlotThird, tau, ties);
            const u64 packed = sh.slots[kSlotThird][0][0], left = sh.slots[kSlotThird][0][1];
            const Cut cut{(uint32_t)(packed >> 32), packed & 0xffffffffull};
            const u64 q_tau = token_weight(key_logit(cut.tau), rule);
            u64 kept, tied;
            cut_pass(sl, rule, cut, &kept, &tied);
            draw(sh, sl, rule, cut, q_tau, left, kept, tied, a, row);
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
    const SampleArgs a{logits, rows, vocab, row_stride, temperature, top_k, top_p, min_p, random, tokens, probs, 0, 0};
    const cudaStream_t s = (cudaStream_t)stream;
    if (type == U32SCAN_F32) return sample_launch<float>(a, s);
    if (type == U32SCAN_F16) return sample_launch<__half>(a, s);
    return sample_launch<__nv_bfloat16>(a, s);
}
