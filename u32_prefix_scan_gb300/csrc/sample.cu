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
// No sort is made: a filter's end is a key `tau` and how many of the logits
// equal to it stay (the lowest indices), found by a radix selection, 8 bits
// a level from the top, on counts (top-k) or sums of weights (top-p).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.cuh"

namespace u32scan {

constexpr int kSThreads = 1024;
constexpr int kSWarps = kSThreads / 32;
constexpr float kLog2e = 0x1.715476p+0f;

typedef unsigned long long u64;

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
};

// A logit as f32; NaN is masked out like -inf.
__device__ __forceinline__ float logit_of(float x) { return x == x ? x : -INFINITY; }
__device__ __forceinline__ float logit_of(__half x) { return logit_of(__half2float(x)); }
__device__ __forceinline__ float logit_of(__nv_bfloat16 x) { return logit_of(__bfloat162float(x)); }

// Unsigned order of the keys = order of the logits (-0 counts as +0).
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// floor(2^31 * 2^-y) for 0 <= y < 32: 2^-n exactly, times 2^-f on [-1/2, 1/2]
// by a degree-5 polynomial with constant term 1 (a minimax fit in relative
// error, 1.9e-7 in f32). Every operation is rounded alone (no contraction).
__device__ __forceinline__ uint32_t exp2_weight(float y) {
    const float n = __fsub_rn(__fadd_rn(y, 0x1.8p23f), 0x1.8p23f);  // nearest integer, ties to even
    const float f = __fsub_rn(y, n);
    float p = __fadd_rn(__fmul_rn(-0x1.5bba14p-10f, f), 0x1.3cea88p-7f);
    p = __fadd_rn(__fmul_rn(p, f), -0x1.c6b752p-5f);
    p = __fadd_rn(__fmul_rn(p, f), 0x1.ebf9bcp-3f);
    p = __fadd_rn(__fmul_rn(p, f), -0x1.62e42ap-1f);
    p = __fadd_rn(__fmul_rn(p, f), 1.0f);
    // times 2^(31 - n), n in [0, 32]: exact
    return __float2uint_rz(__fmul_rn(p, __uint_as_float((uint32_t)(158 - (int)n) << 23)));
}

struct RowRule {
    float m, scale;
    uint32_t qmin;
};

__device__ __forceinline__ uint32_t token_weight(float x, const RowRule &rule) {
    if (x == rule.m) return 0x80000000u;
    const float y = __fmul_rn(__fsub_rn(rule.m, x), rule.scale);
    if (!(y < 32.0f) || x == -INFINITY) return 0u;
    const uint32_t q = exp2_weight(y);
    return q >= rule.qmin ? q : 0u;
}

template <typename V>
__device__ __forceinline__ V block_sum(V v, V *s_red) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
    __syncthreads();
    V t = 0;
    for (int w = 0; w < kSWarps; ++w) t += s_red[w];
    return t;
}

// Where a filter ends: keys above tau stay, and the first `ties` (by index)
// of those equal to it.
struct Cut {
    uint32_t tau;
    u64 ties;
};

// The key at which the running total, taken over keys in descending order,
// first reaches `target` (1 <= target <= the whole total): of counts, or of
// weights. Returns the key and what is still missing above it (1 <= missing).
template <bool MASS, typename T>
__device__ __forceinline__ void radix_select(const T *x, u64 n, const RowRule &rule, uint32_t floor_key, u64 target,
                                             u64 *s_hist, uint32_t *s_pick, u64 *s_left, uint32_t *tau, u64 *missing) {
    uint32_t prefix = 0, mask = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        __syncthreads();
        for (int b = threadIdx.x; b < 256; b += kSThreads) s_hist[b] = 0;
        __syncthreads();
        for (u64 i = threadIdx.x; i < n; i += kSThreads) {
            const float v = logit_of(x[i]);
            const uint32_t k = key_of(v);
            if ((k & mask) != prefix || k < floor_key) continue;
            const u64 w = MASS ? (u64)token_weight(v, rule) : 1ull;
            if (w) atomicAdd(&s_hist[(k >> shift) & 255u], w);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            u64 left = target;
            int b = 255;
            for (; b > 0 && s_hist[b] < left; --b) left -= s_hist[b];
            *s_pick = (uint32_t)b;
            *s_left = left;
        }
        __syncthreads();
        prefix |= *s_pick << shift;
        mask |= 255u << shift;
        target = *s_left;
    }
    *tau = prefix;
    *missing = target;
}

template <typename T>
__global__ void __launch_bounds__(kSThreads) sample_row_kernel(SampleArgs a) {
    __shared__ u64 s_hist[256];
    __shared__ u64 s_red[kSWarps];
    __shared__ u64 s_seg_mass[kSWarps], s_seg_ties[kSWarps];
    __shared__ float s_max[kSWarps];
    __shared__ uint32_t s_pick;
    __shared__ u64 s_left;
    const u64 row = blockIdx.x, n = a.vocab;
    const T *x = static_cast<const T *>(a.logits) + row * a.row_stride;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    float m = -INFINITY;
    for (u64 i = threadIdx.x; i < n; i += kSThreads) m = fmaxf(m, logit_of(x[i]));
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
    for (int w = 0; w < kSWarps; ++w) m = fmaxf(m, s_max[w]);
    if (m == -INFINITY) {  // the mask leaves nothing
        if (threadIdx.x == 0) {
            a.tokens[row] = -1;
            if (a.probs) a.probs[row] = 0.0f;
        }
        return;
    }
    const float t = a.temperature ? a.temperature[row] : 1.0f;
    const bool greedy = !(t > 0.0f);
    const int k = a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.0f;
    const float mp = a.min_p ? a.min_p[row] : 0.0f;
    RowRule rule;
    rule.m = m;
    rule.scale = __fdiv_rn(kLog2e, t);
    rule.qmin = mp > 0.0f ? (uint32_t)ceil((double)fminf(mp, 1.0f) * 2147483648.0) : 0u;

    Cut cut{0u, 0ull};  // no key is 0: everything stays
    u64 r = 0, total = 0;
    if (greedy) {  // the first of the largest
        cut.tau = key_of(m);
        cut.ties = 1;
    } else {
        if (k > 0 && (u64)k < n) {
            u64 missing;
            radix_select<false>(x, n, rule, 0u, (u64)k, s_hist, &s_pick, &s_left, &cut.tau, &missing);
            cut.ties = missing;
        }
        // the weight that the filters so far leave
        const uint32_t q_tau = cut.tau ? token_weight(key_logit(cut.tau), rule) : 0u;
        u64 above = 0;
        for (u64 i = threadIdx.x; i < n; i += kSThreads) {
            const float v = logit_of(x[i]);
            if (key_of(v) > cut.tau) above += token_weight(v, rule);
        }
        above = block_sum(above, s_red);
        total = above + cut.ties * q_tau;
        if (p > 0.0f && p < 1.0f) {
            const u64 want = (u64)ceil(__dmul_rn((double)p, (double)total));
            if (want > above) {  // ends among the ties
                cut.ties = (want - above + q_tau - 1) / q_tau;
                total = above + cut.ties * q_tau;
            } else {
                u64 missing;
                radix_select<true>(x, n, rule, cut.tau + 1u, want, s_hist, &s_pick, &s_left, &cut.tau, &missing);
                const uint32_t q = token_weight(key_logit(cut.tau), rule);
                cut.ties = (missing + q - 1) / q;
                total = want - missing + cut.ties * q;
            }
        }
        r = __umul64hi((u64)a.random[row] << 32, total);
    }
    // the draw: each warp's share of the index range, then one warp's walk
    const uint32_t q_tau = greedy ? 1u : cut.tau ? token_weight(key_logit(cut.tau), rule) : 0u;
    const u64 per = (n + kSWarps - 1) / kSWarps;
    const u64 lo = min((u64)warp * per, n), hi = min(lo + per, n);
    u64 mass = 0, ties = 0;
    for (u64 i = lo + lane; i < hi; i += 32) {
        const float v = logit_of(x[i]);
        const uint32_t key = key_of(v);
        if (key > cut.tau) mass += token_weight(v, rule);
        if (key == cut.tau) ++ties;
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        mass += __shfl_xor_sync(0xffffffffu, mass, d);
        ties += __shfl_xor_sync(0xffffffffu, ties, d);
    }
    __syncthreads();
    if (lane == 0) {
        s_seg_mass[warp] = mass;
        s_seg_ties[warp] = ties;
    }
    __syncthreads();
    u64 before = 0, tie_left = cut.ties;
    for (int w = 0; w < warp; ++w) {
        const u64 tk = min(tie_left, s_seg_ties[w]);
        before += s_seg_mass[w] + tk * q_tau;
        tie_left -= tk;
    }
    const u64 own = mass + min(tie_left, ties) * q_tau;
    if (!(before <= r && r < before + own)) return;
    for (u64 i0 = lo; i0 < hi; i0 += 32) {
        const u64 i = i0 + lane;
        const float v = i < hi ? logit_of(x[i]) : -INFINITY;
        const uint32_t key = key_of(v);
        const bool tie = i < hi && key == cut.tau;
        const unsigned int tm = __ballot_sync(0xffffffffu, tie);
        const bool tie_in = tie && (u64)__popc(tm & lanemask_lt(lane)) < tie_left;
        const u64 q = i < hi && key > cut.tau ? token_weight(v, rule) : tie_in ? q_tau : 0ull;
        u64 inc = q;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const u64 o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        const unsigned int hit = __ballot_sync(0xffffffffu, before + inc > r);
        if (hit) {
            if (lane == __ffs(hit) - 1) {
                a.tokens[row] = (int32_t)i;
                if (a.probs) a.probs[row] = greedy ? 1.0f : (float)((double)q / (double)total);
            }
            return;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
        const u64 used = (u64)__popc(tm);
        tie_left -= min(tie_left, used);
    }
}

template <typename T>
static int sample_launch(const SampleArgs &a, cudaStream_t stream) {
    sample_row_kernel<T><<<(unsigned int)a.rows, kSThreads, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? U32SCAN_OK : U32SCAN_ECUDA;
}

}  // namespace u32scan

using namespace u32scan;

extern "C" int sample_tokens(const void *logits, int type, size_t rows, size_t vocab, size_t row_stride,
                             const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                             const uint32_t *random, int32_t *tokens, float *probs, u32scan_stream_t stream) {
    if (type != U32SCAN_F32 && type != U32SCAN_F16 && type != U32SCAN_BF16) return U32SCAN_EINVAL;
    if (rows >= (1ull << 31) || vocab > U32SCAN_MAX_VOCAB || row_stride >= (1ull << 32)) return U32SCAN_EINVAL;
    if (rows == 0) return U32SCAN_OK;
    const uintptr_t elem = type == U32SCAN_F32 ? 3 : 1;
    if ((vocab > 0 && logits == nullptr) || random == nullptr || tokens == nullptr) return U32SCAN_EINVAL;
    if (reinterpret_cast<uintptr_t>(logits) & elem) return U32SCAN_EINVAL;
    for (const void *p : {(const void *)temperature, (const void *)top_k, (const void *)top_p, (const void *)min_p,
                          (const void *)random, (const void *)tokens, (const void *)probs})
        if (reinterpret_cast<uintptr_t>(p) & 3) return U32SCAN_EINVAL;
    const SampleArgs a{logits, rows, vocab, row_stride, temperature, top_k, top_p, min_p, random, tokens, probs};
    const cudaStream_t s = (cudaStream_t)stream;
    if (type == U32SCAN_F32) return sample_launch<float>(a, s);
    if (type == U32SCAN_F16) return sample_launch<__half>(a, s);
    return sample_launch<__nv_bfloat16>(a, s);
}
