// adjust.cu -- a request's rules applied to its logits: penalties for tokens
// of the history, biases of listed tokens, a mask of allowed ones.
//
// A block takes one slice of a row: every thread starts the loads of its
// logits (one or four vectors of 16 bytes), the block counts the history's
// tokens that fall into its slice (and marks those of the list) in shared memory
// meanwhile, and each thread then changes and stores what it holds. The whole
// history passes every slice of its row, from L2, 16 bytes a thread. Every f32
// operation rounds alone, so the result is the definition's bit for bit.
//
// Measured on one GB300, launches back to back: 256 x 262144 f32 with 2048
// tokens of history, 300 biases and a mask (547 MB) 119 us, 4.6 TB/s, bound by
// instructions (70 % of the issue slots: some 190 for a warp's vectors, half of
// which hold a touched logit); with no lists and no mask 82 us, 6.5 TB/s, the
// memory's rate. 48 x 131072 bf16 with 32768 of history (30 MB, in L2) 25 us: each
// slice's block goes over the whole history. One row of 32000 bf16 2.8 us: the
// launch and two dependent loads.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.cuh"
#include "launch.cuh"

namespace u32scan {

typedef unsigned long long u64;

constexpr int kAThreads = 512;
constexpr uint32_t kSeen = 0x80000000u;   // a prompt's token
constexpr uint32_t kNamed = 0x40000000u;  // a token of the list; the bits below count the history past the prompt
constexpr uint32_t kCount = kNamed - 1u;
constexpr uint32_t kNames = 512;          // list entries of one slice that are kept in shared memory

struct AdjustArgs {
    const void *logits;
    void *out;
    u64 rows, vocab, row_stride, out_stride;
    u32scan_logit_rules r;
    unsigned int slices;
};

template <typename T>
struct Logit;
template <>
struct Logit<float> {
    static __device__ float get(float x) { return x; }
    static __device__ float put(float x) { return x; }
};
template <>
struct Logit<__half> {
    static __device__ float get(__half x) { return __half2float(x); }
    static __device__ __half put(float x) { return __float2half_rn(x); }
};
template <>
struct Logit<__nv_bfloat16> {
    static __device__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

// A penalty that is not finite counts as none.
__device__ __forceinline__ float finite_or(const float *p, u64 row, float none) {
    const float x = p ? p[row] : none;
    return x - x == 0.0f ? x : none;
}

// VEC elements at a time, at addresses that are multiples of their size.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vector {
    T x[VEC];
};

// Element e of a vector that stays in registers.
template <typename T, int VEC>
__device__ __forceinline__ T element(const Vector<T, VEC> &v, uint32_t e) {
    T x = v.x[0];
#pragma unroll
    for (int i = 1; i < VEC; ++i)
        if (e == (uint32_t)i) x = v.x[i];
    return x;
}

template <int N>
__device__ __forceinline__ void read(uint32_t (&to)[N], const uint32_t *from) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(from + i);
            to[i] = x.x, to[i + 1] = x.y, to[i + 2] = x.z, to[i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) to[i] = from[i];
    }
}

// PER vectors of VEC logits a thread. A row's logits and results may start anywhere within a vector, both at the same
// place: token i is element i + shift of vectors that are aligned. (Tokens and places of the history stay below 2^30.)
template <typename T, int VEC, int PER>
__global__ void __launch_bounds__(kAThreads, sizeof(T) == 4 ? 3 : 2) adjust_kernel(const AdjustArgs a) {
    constexpr uint32_t kSlice = kAThreads * PER * VEC;
    extern __shared__ __align__(16) uint32_t count[];  // kSlice
    __shared__ uint32_t n_names, name_at[kNames], name_i[kNames];
    const u64 row = blockIdx.x / a.slices;
    const T *in = static_cast<const T *>(a.logits) + row * a.row_stride;
    T *out = static_cast<T *>(a.out) + row * a.out_stride;
    const int32_t vocab = (int32_t)a.vocab;
    const int32_t shift = VEC > 1 ? (int32_t)(reinterpret_cast<uintptr_t>(in) / sizeof(T) % VEC) : 0;
    const int32_t first = (int32_t)((blockIdx.x % a.slices) * kSlice) - shift;  // the token of the slice's first element
    if (first >= vocab) return;

    // All that does not wait for another load is started at once: the row's settings, the first of the history (as
    // much as there may be) and of the list, the logits.
    const uint32_t biases = (uint32_t)a.r.biases;
    const bool lists = a.r.history != nullptr || biases > 0;
    int32_t held = (int32_t)a.r.history_width, prompt = 0;
    if (a.r.history_lens) held = min(held, max(a.r.history_lens[row], 0));
    if (a.r.prompt_lens) prompt = max(a.r.prompt_lens[row], 0);
    const float rep = finite_or(a.r.repetition, row, 0.0f), freq = finite_or(a.r.frequency, row, 0.0f);
    const float pres = finite_or(a.r.presence, row, 0.0f);
    // the history one at a time up to the first multiple of 16 bytes, then four
    const int32_t *h = a.r.history ? a.r.history + row * a.r.history_stride : nullptr;
    const int32_t wide = h ? (int32_t)a.r.history_width : 0;
    const int32_t lead = min(wide, (int32_t)(-(reinterpret_cast<uintptr_t>(h) / 4) & 3)), fours = (wide - lead) / 4;
    const int4 *h4 = reinterpret_cast<const int4 *>(h + lead);
    const int32_t mine = (int32_t)threadIdx.x;
    const int4 soon = mine < fours ? __ldg(h4 + mine) : int4{-1, -1, -1, -1};
    const int32_t *names = a.r.bias_tokens + row * biases;
    const int32_t soon_name = threadIdx.x < biases ? __ldg(names + threadIdx.x) : -1;

    const uint32_t *allowed = a.r.allowed ? a.r.allowed + row * a.r.allowed_stride : nullptr;
    Vector<T, VEC> l[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int32_t t = first + (k * kAThreads + mine) * VEC;
        if (t >= 0 && t + VEC <= vocab) {
            l[k] = *reinterpret_cast<const Vector<T, VEC> *>(in + t);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (t + e >= 0 && t + e < vocab) l[k].x[e] = in[t + e];
        }
    }

    if (lists) {
        for (uint32_t i = threadIdx.x; i < kSlice / 4; i += kAThreads) reinterpret_cast<uint4 *>(count)[i] = uint4{0, 0, 0, 0};
        if (threadIdx.x == 0) n_names = 0u;
        __syncthreads();
        // the row's tokens [low, low + size) fall into this slice
        const uint32_t low = (uint32_t)max(first, 0), size = (uint32_t)min(vocab - (int32_t)low, (int32_t)(first + kSlice - low));
        uint32_t *const at_low = count + (low - first);
        auto note = [&](int32_t i, int32_t token) {
            const uint32_t at = (uint32_t)token - low;
            if (at >= size || i >= held) return;
            if (i < prompt) atomicOr(at_low + at, kSeen);
            else atomicAdd(at_low + at, 1u);
        };
        auto note4 = [&](int32_t i, const int4 &x) {
            const int32_t at = lead + 4 * i;
            note(at, x.x), note(at + 1, x.y), note(at + 2, x.z), note(at + 3, x.w);
        };
        if (mine < lead) note(mine, h[mine]);
        if (mine < fours) note4(mine, soon);
        const int32_t held_fours = min(fours, (held - lead + 3) / 4);
#pragma unroll 4
        for (int32_t i = mine + kAThreads; i < held_fours; i += kAThreads) note4(i, __ldg(h4 + i));
        const int32_t tail = lead + 4 * fours + mine;
        if (tail < wide) note(tail, h[tail]);
        auto name = [&](uint32_t i, int32_t token) {
            const uint32_t at = (uint32_t)token - low;
            if (at >= size) return;
            atomicOr(at_low + at, kNamed);
            const uint32_t n = atomicAdd(&n_names, 1u);
            if (n < kNames) name_at[n] = at + (low - first), name_i[n] = i;
        };
        if (threadIdx.x < biases) name(threadIdx.x, soon_name);
        for (uint32_t i = threadIdx.x + kAThreads; i < biases; i += kAThreads) name(i, names[i]);
        __syncthreads();
    }
    // The last entry of the list that names element `at` of the slice: among the slice's own, which are few, or in the
    // whole list, from its end.
    auto bias_of = [&](uint32_t at) {
        uint32_t i = 0;
        if (n_names <= kNames) {
            for (uint32_t n = 0; n < n_names; ++n)
                if (name_at[n] == at) i = max(i, name_i[n]);
        } else {
            i = biases - 1u;
            while (names[i] != (int32_t)at + first) --i;
        }
        return a.r.bias[row * biases + i];
    };

#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const uint32_t at = (uint32_t)(k * kAThreads + mine) * VEC;
        const int32_t t = first + (int32_t)at;
        if (t >= vocab) break;
        if (lists) {
            // (one turn for each touched element: few lanes have more than one, and written out for every
            // element of a vector the division and the search would be passed VEC times)
            uint32_t c[VEC], any = 0;
            read<VEC>(c, count + at);
#pragma unroll
            for (int e = 0; e < VEC; ++e) any |= c[e] ? 1u << e : 0u;
            if (any) {
                for (uint32_t todo = any; todo; todo &= todo - 1) {
                    const uint32_t e = __ffs(todo) - 1, what = count[at + e];
                    float x = Logit<T>::get(element(l[k], e));
                    if ((what & ~kNamed) && rep > 0.0f) x = x > 0.0f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
                    if (what & kCount) x = __fsub_rn(__fsub_rn(x, __fmul_rn(freq, __uint2float_rn(what & kCount))), pres);
                    if (what & kNamed) x = __fadd_rn(x, bias_of(at + e));
                    *reinterpret_cast<T *>(&count[at + e]) = Logit<T>::put(x);
                }
                read<VEC>(c, count + at);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (any >> e & 1u) l[k].x[e] = *reinterpret_cast<const T *>(&c[e]);
            }
        }
        if (allowed) {
            // (loaded beside the logits, the words cost registers and more time than they hide: 158 us instead of 120)
            const int32_t t0 = max(t, 0);
            const uint32_t lo = allowed[t0 >> 5], hi = shift == 0 ? lo : allowed[(min(t + VEC, vocab) - 1) >> 5];
            uint32_t bits = __funnelshift_r(lo, hi, (uint32_t)t0 & 31);  // bit 0: token t0
            bits <<= (uint32_t)(t0 - t);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (!(bits >> e & 1u)) l[k].x[e] = Logit<T>::put(-INFINITY);
        }
        if (t >= 0 && t + VEC <= vocab) {
            *reinterpret_cast<Vector<T, VEC> *>(out + t) = l[k];
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (t + e >= 0 && t + e < vocab) out[t + e] = l[k].x[e];
        }
    }
}

template <typename T, int VEC, int PER>
static int adjust_launch(AdjustArgs a, cudaStream_t stream) {
    constexpr u64 kSlice = (u64)kAThreads * PER * VEC;
    // a row that does not begin at a vector's first element reaches one further
    const bool begins = reinterpret_cast<uintptr_t>(a.logits) % (VEC * sizeof(T)) == 0 && a.row_stride % VEC == 0;
    const u64 slices = (a.vocab + (begins ? 0 : VEC - 1) + kSlice - 1) / kSlice;
    if (slices * a.rows >= (1ull << 31)) return U32SCAN_EINVAL;
    a.slices = (unsigned int)slices;
    const size_t shared = a.r.biases > 0 || a.r.history ? 4 * kSlice : 0;
    if (cudaFuncSetAttribute(adjust_kernel<T, VEC, PER>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(4 * kSlice)) !=
        cudaSuccess)
        return U32SCAN_ECUDA;
    adjust_kernel<T, VEC, PER><<<(unsigned int)(slices * a.rows), kAThreads, shared, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? U32SCAN_OK : U32SCAN_ECUDA;
}

template <typename T>
static int adjust_dispatch(const AdjustArgs &a, cudaStream_t stream) {
    constexpr int kVec = 16 / sizeof(T);
    const uintptr_t from = reinterpret_cast<uintptr_t>(a.logits), to = reinterpret_cast<uintptr_t>(a.out);
    // logits and results start at the same place within 16 bytes, in every row
    const bool alike = (from - to) % 16 == 0 && (a.row_stride - a.out_stride) % kVec == 0;
    if (!alike) return adjust_launch<T, 1, 4>(a, stream);
    // four vectors a thread where that leaves a wave of blocks
    if (a.rows * (a.vocab / (kAThreads * kVec * 4)) < 304) return adjust_launch<T, kVec, 1>(a, stream);
    return adjust_launch<T, kVec, 4>(a, stream);
}

}  // namespace u32scan

using namespace u32scan;

extern "C" int adjust_logits(const void *logits, int type, size_t rows, size_t vocab, size_t row_stride, void *out,
                             size_t out_stride, const u32scan_logit_rules *rules, u32scan_stream_t stream) {
    if (type != U32SCAN_F32 && type != U32SCAN_F16 && type != U32SCAN_BF16) return U32SCAN_EINVAL;
    if (rows >= (1ull << 28) || vocab > U32SCAN_MAX_VOCAB || rules == nullptr) return U32SCAN_EINVAL;
    const u32scan_logit_rules &r = *rules;
    if (rows > 1 && (row_stride >= (1ull << 32) || out_stride >= (1ull << 32) || out_stride < vocab))
        return U32SCAN_EINVAL;
    if (r.history_width >= kNamed || r.biases >= (1ull << 31)) return U32SCAN_EINVAL;
    if (rows > 1 && (r.history_stride >= (1ull << 32) || r.allowed_stride >= (1ull << 32))) return U32SCAN_EINVAL;
    for (const void *p : {(const void *)r.history, (const void *)r.history_lens, (const void *)r.prompt_lens,
                          (const void *)r.repetition, (const void *)r.presence, (const void *)r.frequency,
                          (const void *)r.bias_tokens, (const void *)r.bias, (const void *)r.allowed})
        if (reinterpret_cast<uintptr_t>(p) & 3) return U32SCAN_EINVAL;
    const uintptr_t elem = type == U32SCAN_F32 ? 4 : 2;
    const uintptr_t from = reinterpret_cast<uintptr_t>(logits), to = reinterpret_cast<uintptr_t>(out);
    if ((from | to) & (elem - 1)) return U32SCAN_EINVAL;
    if (rows == 0 || vocab == 0) return U32SCAN_OK;
    if (logits == nullptr || out == nullptr) return U32SCAN_EINVAL;
    if (r.history_width > 0 && r.history == nullptr) return U32SCAN_EINVAL;
    if (r.biases > 0 && (r.bias_tokens == nullptr || r.bias == nullptr)) return U32SCAN_EINVAL;
    const bool in_place = from == to && (rows == 1 || row_stride == out_stride);
    if (!in_place && share_memory(Strided{logits, vocab * elem, {rows, 1, 1}, {row_stride * elem, 0, 0}},
                                  Strided{out, vocab * elem, {rows, 1, 1}, {out_stride * elem, 0, 0}}))
        return U32SCAN_EINVAL;
    AdjustArgs a{logits, out, rows, vocab, rows > 1 ? row_stride : 0, rows > 1 ? out_stride : 0, r, 0};
    if (a.r.history_width == 0) a.r.history = nullptr;
    const cudaStream_t s = (cudaStream_t)stream;
    if (type == U32SCAN_F32) return adjust_dispatch<float>(a, s);
    if (type == U32SCAN_F16) return adjust_dispatch<__half>(a, s);
    return adjust_dispatch<__nv_bfloat16>(a, s);
}
