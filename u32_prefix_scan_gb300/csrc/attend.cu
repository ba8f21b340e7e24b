// attend.cu -- attention over a paged cache of 8-bit keys and values.
//
// A block takes one query head of one token: 128 scores at a time, the
// running maximum and sum of the softmax, then the values weighted by them.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "kvcache.cuh"

namespace u32scan {

constexpr int kQThreads = 128;
constexpr int kMaxDim = 256;

struct AttendArgs {
    RowsView v;
    const uint8_t *keys, *values;
    const float *key_scales, *value_scales;
    uint64_t page_stride, token_stride, head_stride, scale_stride;
    Divisor block_tokens;
    uint32_t heads, group, dim;
    const void *queries;
    void *out;
    uint64_t q_token_stride, q_head_stride, out_token_stride, out_head_stride;
    float scale;
};

__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(__half *y, float x) { *y = __float2half_rn(x); }
__device__ __forceinline__ void from_float(__nv_bfloat16 *y, float x) { *y = __float2bfloat16_rn(x); }

__device__ __forceinline__ float code_value(uint8_t code) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
}

template <typename T>
__global__ void __launch_bounds__(kQThreads) attend_kernel(const AttendArgs a) {
    __shared__ float q[kMaxDim], weight[kQThreads], fold[kQThreads / 32];
    __shared__ const uint8_t *value_at[kQThreads];
    const uint64_t token = blockIdx.x / (a.heads * a.group);
    const uint32_t qh = blockIdx.x % (a.heads * a.group), head = qh / a.group;
    int64_t begin, n;
    const int64_t row = row_of(a.v, token, &begin, &n);
    if (row < 0) return;
    const T *x = static_cast<const T *>(a.queries) + token * a.q_token_stride + qh * a.q_head_stride;
    for (uint32_t d = threadIdx.x; d < a.dim; d += kQThreads) q[d] = to_float(x[d]);
    __syncthreads();
    const int64_t seen = (int64_t)a.v.lens[row] - n + ((int64_t)token - begin) + 1;
    float m = -INFINITY, l = 0.0f, o[kMaxDim / kQThreads] = {};
    for (int64_t j0 = 0; j0 < seen; j0 += kQThreads) {
        const int64_t j = j0 + threadIdx.x;
        float s = -INFINITY, sv = 0.0f;
        value_at[threadIdx.x] = nullptr;
        if (j < seen) {
            const uint32_t nth = divide((uint32_t)j, a.v.page_tokens);
            const int32_t page = nth < a.v.width ? a.v.table[(uint64_t)row * a.v.table_stride + nth] : -1;
            if (page >= 0 && (uint64_t)page < a.v.pages) {
                const uint32_t slot = (uint32_t)j - nth * a.v.page_tokens.d;
                const uint64_t at = (uint64_t)page * a.page_stride + (uint64_t)slot * a.token_stride +
                                    (uint64_t)head * a.head_stride;
                const uint64_t block = (uint64_t)page * a.scale_stride +
                                       (uint64_t)divide(slot, a.block_tokens) * a.heads + head;
                float dot = 0.0f;
                for (uint32_t d = 0; d < a.dim; ++d) dot += q[d] * code_value(a.keys[at + d]);
                s = dot * a.key_scales[block] * a.scale;
                sv = a.value_scales[block];
                value_at[threadIdx.x] = a.values + at;
            }
        }
        float top = s;
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        if ((threadIdx.x & 31) == 0) fold[threadIdx.x >> 5] = top;
        __syncthreads();
        for (int w = 0; w < kQThreads / 32; ++w) top = fmaxf(top, fold[w]);
        top = fmaxf(top, m);
        const float p = s == -INFINITY ? 0.0f : expf(s - top);
        const float old = m == top ? 1.0f : expf(m - top);
        m = top;
        l = l * old + p;  // each thread's own tokens
        weight[threadIdx.x] = p * sv;
        __syncthreads();
        for (int k = 0; k < kMaxDim / kQThreads; ++k) {
            const uint32_t d = threadIdx.x + k * kQThreads;
            if (d >= a.dim) break;
            o[k] *= old;
            for (int t = 0; t < kQThreads; ++t)
                if (value_at[t]) o[k] += weight[t] * code_value(value_at[t][d]);
        }
        __syncthreads();
    }
    for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if ((threadIdx.x & 31) == 0) fold[threadIdx.x >> 5] = l;
    __syncthreads();
    l = 0.0f;
    for (int w = 0; w < kQThreads / 32; ++w) l += fold[w];
    T *y = static_cast<T *>(a.out) + token * a.out_token_stride + qh * a.out_head_stride;
    for (int k = 0; k < kMaxDim / kQThreads; ++k) {
        const uint32_t d = threadIdx.x + k * kQThreads;
        if (d < a.dim) from_float(&y[d], l == 0.0f ? 0.0f : o[k] / l);
    }
}

size_t attend_workspace_bytes() { return kHeaderBytes; }

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
    if (tokens * q_heads >= (1ull << 31)) return U32SCAN_EINVAL;
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
    a.group = (uint32_t)(q_heads / cache->heads);
    a.dim = (uint32_t)cache->dim;
    a.queries = queries;
    a.out = out;
    a.q_token_stride = query_token_stride;
    a.q_head_stride = query_head_stride;
    a.out_token_stride = out_token_stride;
    a.out_head_stride = out_head_stride;
    a.scale = scale;
    const cudaStream_t s = (cudaStream_t)stream;
    const unsigned int grid = (unsigned int)(tokens * q_heads);
    if (type == U32SCAN_F16) attend_kernel<__half><<<grid, kQThreads, 0, s>>>(a);
    else attend_kernel<__nv_bfloat16><<<grid, kQThreads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? U32SCAN_OK : U32SCAN_ECUDA;
}
