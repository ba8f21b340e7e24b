// adjust.cu -- a request's rules applied to its logits: penalties for tokens
// of the history, biases of listed tokens, a mask of allowed ones.
//
// A block takes one slice of a row. It counts the history's tokens that fall
// into its slice (and marks those of the list) in shared memory, then passes
// over the slice once. Every f32 operation rounds alone, so the result is the
// definition's bit for bit.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.cuh"

namespace u32scan {

typedef unsigned long long u64;

constexpr int kAThreads = 256;
constexpr unsigned int kASlice = 4096;  // logits of a block
constexpr uint32_t kSeen = 0x80000000u; // a prompt's token; the bits below count the others

struct AdjustArgs {
    const void *logits;
    void *out;
    u64 rows, vocab, row_stride, out_stride;
    u32scan_logit_rules r;
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

template <typename T>
__global__ void __launch_bounds__(kAThreads) adjust_kernel(const AdjustArgs a, const unsigned int slices) {
    __shared__ uint32_t count[kASlice], named[kASlice];
    const u64 row = blockIdx.x / slices;
    const uint32_t first = blockIdx.x % slices * kASlice;
    const uint32_t n = (uint32_t)(a.vocab - first < kASlice ? a.vocab - first : kASlice);
    for (uint32_t i = threadIdx.x; i < n; i += kAThreads) count[i] = named[i] = 0u;
    __syncthreads();
    if (a.r.history) {
        int64_t held = (int64_t)a.r.history_width, prompt = 0;
        if (a.r.history_lens) held = min(held, (int64_t)max(a.r.history_lens[row], 0));
        if (a.r.prompt_lens) prompt = min(held, (int64_t)max(a.r.prompt_lens[row], 0));
        const int32_t *h = a.r.history + row * a.r.history_stride;
        for (int64_t i = threadIdx.x; i < held; i += kAThreads) {
            const uint32_t at = (uint32_t)h[i] - first;
            if (at < n) {
                if (i < prompt) atomicOr(&count[at], kSeen);
                else atomicAdd(&count[at], 1u);
            }
        }
    }
    for (u64 i = threadIdx.x; i < a.r.biases; i += kAThreads) {
        const uint32_t at = (uint32_t)a.r.bias_tokens[row * a.r.biases + i] - first;
        if (at < n) atomicMax(&named[at], (uint32_t)i + 1u);
    }
    __syncthreads();
    const float rep = finite_or(a.r.repetition, row, 0.0f), freq = finite_or(a.r.frequency, row, 0.0f);
    const float pres = finite_or(a.r.presence, row, 0.0f);
    const T *in = static_cast<const T *>(a.logits) + row * a.row_stride + first;
    T *out = static_cast<T *>(a.out) + row * a.out_stride + first;
    for (uint32_t i = threadIdx.x; i < n; i += kAThreads) {
        T l = in[i];
        const uint32_t c = count[i], b = named[i];
        if (c | b) {
            float x = Logit<T>::get(l);
            if (c && rep > 0.0f) x = x > 0.0f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
            if (c & ~kSeen)
                x = __fsub_rn(__fsub_rn(x, __fmul_rn(freq, __uint2float_rn(c & ~kSeen))), pres);
            if (b) x = __fadd_rn(x, a.r.bias[row * a.r.biases + b - 1u]);
            l = Logit<T>::put(x);
        }
        if (a.r.allowed) {
            const uint32_t t = first + i;
            if (!(a.r.allowed[row * a.r.allowed_stride + t / 32] >> (t % 32) & 1u)) l = Logit<T>::put(-INFINITY);
        }
        out[i] = l;
    }
}

template <typename T>
static int adjust_launch(const AdjustArgs &a, cudaStream_t stream) {
    const u64 slices = (a.vocab + kASlice - 1) / kASlice;
    if (slices * a.rows >= (1ull << 31)) return U32SCAN_EINVAL;
    adjust_kernel<T><<<(unsigned int)(slices * a.rows), kAThreads, 0, stream>>>(a, (unsigned int)slices);
    return cudaGetLastError() == cudaSuccess ? U32SCAN_OK : U32SCAN_ECUDA;
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
    if (r.history_width >= (1ull << 31) || r.biases >= (1ull << 31)) return U32SCAN_EINVAL;
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
    const u64 in_span = ((rows - 1) * row_stride + vocab) * elem, out_span = ((rows - 1) * out_stride + vocab) * elem;
    const bool in_place = from == to && (rows == 1 || row_stride == out_stride);
    if (!in_place && from < to + out_span && to < from + in_span) return U32SCAN_EINVAL;
    AdjustArgs a{logits, out, rows, vocab, rows > 1 ? row_stride : 0, rows > 1 ? out_stride : 0, r};
    if (a.r.history_width == 0) a.r.history = nullptr;
    const cudaStream_t s = (cudaStream_t)stream;
    if (type == U32SCAN_F32) return adjust_launch<float>(a, s);
    if (type == U32SCAN_F16) return adjust_launch<__half>(a, s);
    return adjust_launch<__nv_bfloat16>(a, s);
}
