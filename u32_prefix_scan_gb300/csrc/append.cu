// append.cu -- new keys and values written into the pages of a paged cache,
// keys (and queries) rotated by their position on the way.
//
// A warp takes one head of one token at a time; for the 8-bit cache, the new
// tokens of one block of a page.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "kvcache.cuh"

namespace u32scan {

constexpr int kNThreads = 256;
constexpr int kNWarps = kNThreads / 32;

struct Heads {
    const void *data;
    uint64_t heads, token_stride, head_stride;
};

struct AppendArgs {
    RowsView v;
    const int32_t *status;
    Heads keys, values, queries, out;
    const float *cos, *sin;
    uint64_t positions;
    uint32_t pairs, dim;
    int interleaved;
    void *cache_keys, *cache_values;
    uint64_t page_stride, token_stride, head_stride;
    float *key_scales, *value_scales;
    uint64_t scale_stride;
    Divisor block_tokens;
};

template <typename T>
struct Num;
template <>
struct Num<float> {
    static __device__ __forceinline__ float get(float x) { return x; }
    static __device__ __forceinline__ float put(float x) { return x; }
};
template <>
struct Num<__half> {
    static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <>
struct Num<__nv_bfloat16> {
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

__device__ __forceinline__ float code_value(uint8_t code) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
}
__device__ __forceinline__ uint8_t value_code(float x) { return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3); }

// Where a token lies.
struct Place {
    bool held;     // its page is the pool's
    int64_t row, position, first;  // first: the row's first new position
    uint64_t page;
    uint32_t slot;
};

__device__ Place place_of(const AppendArgs &a, uint64_t token) {
    Place p;
    int64_t begin, n;
    p.row = row_of(a.v, token, &begin, &n);
    p.held = false;
    if (p.row < 0) return p;
    p.first = (int64_t)a.v.lens[p.row] - n;
    p.position = p.first + ((int64_t)token - begin);
    if (p.position < 0 || (a.status && a.status[p.row] < 0)) return p;
    const uint32_t nth = divide((uint32_t)p.position, a.v.page_tokens);
    if (nth >= a.v.width) return p;
    const int32_t page = a.v.table[(uint64_t)p.row * a.v.table_stride + nth];
    if (page < 0 || (uint64_t)page >= a.v.pages) return p;
    if (a.cos && (uint64_t)p.position >= a.positions) return p;
    p.held = true;
    p.page = (uint64_t)page;
    p.slot = (uint32_t)p.position - nth * a.v.page_tokens.d;
    return p;
}

// Element d of a head, rotated.
template <typename T>
__device__ __forceinline__ float rotated(const AppendArgs &a, const T *x, uint32_t d, int64_t position, bool turn) {
    const float own = Num<T>::get(x[d]);
    if (!turn || d >= 2 * a.pairs) return own;
    const bool second = a.interleaved ? (d & 1u) : d >= a.pairs;
    const uint32_t pair = a.interleaved ? d / 2 : second ? d - a.pairs : d;
    const uint32_t at = a.interleaved ? d ^ 1u : second ? d - a.pairs : d + a.pairs;
    const float other = Num<T>::get(x[at]);
    const float c = a.cos[(uint64_t)position * a.pairs + pair], s = a.sin[(uint64_t)position * a.pairs + pair];
    return second ? __fadd_rn(__fmul_rn(own, c), __fmul_rn(other, s)) : __fsub_rn(__fmul_rn(own, c), __fmul_rn(other, s));
}

template <typename T>
__device__ __forceinline__ const T *head_of(const Heads &h, uint64_t token, uint64_t head) {
    return static_cast<const T *>(h.data) + token * h.token_stride + head * h.head_stride;
}

// One block of one head: the scale that its new values need beside the old ones, then the codes.
template <typename T>
__device__ void append_block(const AppendArgs &a, const Place &p, uint64_t token, uint64_t head, bool key, int lane) {
    const Heads &src = key ? a.keys : a.values;
    uint8_t *codes = static_cast<uint8_t *>(key ? a.cache_keys : a.cache_values) + p.page * a.page_stride +
                     head * a.head_stride;
    const uint32_t nth = divide(p.slot, a.block_tokens), size = a.block_tokens.d;
    const uint32_t before = p.slot - nth * size;  // older tokens of the block
    float *scale_at = (key ? a.key_scales : a.value_scales) + p.page * a.scale_stride +
                      (uint64_t)nth * a.keys.heads + head;
    const int64_t len = a.v.lens[p.row];
    uint32_t n = size - before;
    if ((int64_t)n > len - p.position) n = (uint32_t)(len - p.position);
    if (a.cos && (int64_t)n > (int64_t)a.positions - p.position) n = (uint32_t)((int64_t)a.positions - p.position);
    const bool turn = key && a.cos;
    float m = 0.0f;
    for (uint32_t i = 0; i < n; ++i) {
        const T *x = head_of<T>(src, token + i, head);
        for (uint32_t d = lane; d < a.dim; d += 32) {
            const float y = fabsf(rotated(a, x, d, p.position + i, turn));
            if (y < INFINITY) m = fmaxf(m, y);
        }
    }
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    // least e with m <= 1.75 * 2^(8 + e)
    int e = (int)(__float_as_uint(m) >> 23) - 127 - 8 + ((__float_as_uint(m) & 0x7fffffu) > 0x600000u ? 1 : 0);
    if (e < -100) e = -100;
    float scale = __uint_as_float((uint32_t)(e + 127) << 23);
    if (before) {
        float old = *scale_at;
        if (!(old > 0.0f && old < INFINITY)) old = 0.0f;
        if (old >= scale) {
            scale = old;
        } else {
            const float ratio = __fdiv_rn(old, scale);
            for (uint32_t t = 0; t < before; ++t)
                for (uint32_t d = lane; d < a.dim; d += 32) {
                    uint8_t *c = codes + (uint64_t)(p.slot - before + t) * a.token_stride + d;
                    *c = value_code(__fmul_rn(code_value(*c), ratio));
                }
        }
    }
    const float inv = __fdiv_rn(1.0f, scale);
    for (uint32_t i = 0; i < n; ++i) {
        const T *x = head_of<T>(src, token + i, head);
        for (uint32_t d = lane; d < a.dim; d += 32)
            codes[(uint64_t)(p.slot + i) * a.token_stride + d] =
                value_code(__fmul_rn(rotated(a, x, d, p.position + i, turn), inv));
    }
    __syncwarp();
    if (lane == 0) *scale_at = scale;
}

template <typename T, bool CODED>
__global__ void __launch_bounds__(kNThreads) append_kernel(const AppendArgs a) {
    const uint64_t token = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Place p = place_of(a, token);
    if (p.row < 0) return;
    const bool turn = a.cos != nullptr, reached = !turn || (p.position >= 0 && (uint64_t)p.position < a.positions);
    for (uint64_t h = warp; h < a.queries.heads; h += kNWarps) {
        const T *x = head_of<T>(a.queries, token, h);
        T *y = const_cast<T *>(head_of<T>(a.out, token, h));
        float r[32];
        int k = 0;
        for (uint32_t d = lane; d < a.dim; d += 32) r[k++] = reached ? rotated(a, x, d, p.position, turn) : NAN;
        __syncwarp();  // in place: every element read before any is written
        k = 0;
        for (uint32_t d = lane; d < a.dim; d += 32) y[d] = Num<T>::put(r[k++]);
    }
    if (!p.held) return;
    if (CODED) {
        const uint32_t within = p.slot - divide(p.slot, a.block_tokens) * a.block_tokens.d;
        if (within != 0 && p.position != p.first) return;  // the block's first new token writes it
        for (uint64_t h = warp; h < 2 * a.keys.heads; h += kNWarps)
            append_block<T>(a, p, token, h >> 1, !(h & 1), lane);
    } else {
        for (uint64_t h = warp; h < 2 * a.keys.heads; h += kNWarps) {
            const bool key = !(h & 1);
            const T *x = head_of<T>(key ? a.keys : a.values, token, h >> 1);
            T *y = static_cast<T *>(key ? a.cache_keys : a.cache_values) + p.page * a.page_stride +
                   (uint64_t)p.slot * a.token_stride + (h >> 1) * a.head_stride;
            for (uint32_t d = lane; d < a.dim; d += 32) y[d] = Num<T>::put(rotated(a, x, d, p.position, key && turn));
        }
    }
}

template <typename T>
static void append_launch(const AppendArgs &a, bool coded, cudaStream_t s) {
    const unsigned int grid = (unsigned int)a.v.tokens;
    if (coded) append_kernel<T, true><<<grid, kNThreads, 0, s>>>(a);
    else append_kernel<T, false><<<grid, kNThreads, 0, s>>>(a);
}

}  // namespace u32scan

using namespace u32scan;

extern "C" int pages_append(const u32scan_kv_cache *cache, const int32_t *table, size_t table_stride, size_t rows,
                            size_t width, const int32_t *lens, const int32_t *starts, const int32_t *status,
                            const u32scan_new_tokens *new_tokens, u32scan_stream_t stream) {
    if (!cache_ok(cache) || new_tokens == nullptr) return U32SCAN_EINVAL;
    const u32scan_new_tokens &t = *new_tokens;
    if (!rows_ok(table, table_stride, rows, width, lens, starts, t.tokens) || misaligned(status, 4))
        return U32SCAN_EINVAL;
    if (t.type < U32SCAN_F32 || t.type > U32SCAN_BF16 || (cache->type != U32SCAN_E4M3 && cache->type != t.type))
        return U32SCAN_EINVAL;
    const size_t elem = element_bytes(t.type);
    if (misaligned(t.keys, elem) || misaligned(t.values, elem) || misaligned(t.queries, elem) ||
        misaligned(t.queries_out, elem) || misaligned(t.cos, 4) || misaligned(t.sin, 4))
        return U32SCAN_EINVAL;
    if (!strides_ok(t.key_token_stride, t.key_head_stride) || !strides_ok(t.value_token_stride, t.value_head_stride) ||
        !strides_ok(t.query_token_stride, t.query_head_stride) || !strides_ok(t.out_token_stride, t.out_head_stride))
        return U32SCAN_EINVAL;
    if ((t.cos == nullptr) != (t.sin == nullptr) || t.positions >= (1ull << 31) || t.pairs > cache->dim / 2)
        return U32SCAN_EINVAL;
    if (t.queries != nullptr && t.q_heads >= (1ull << 16)) return U32SCAN_EINVAL;
    if (t.tokens == 0 || rows == 0) return U32SCAN_OK;
    if (t.keys == nullptr || t.values == nullptr) return U32SCAN_EINVAL;
    if (t.queries != nullptr && t.q_heads > 0 && t.queries_out == nullptr) return U32SCAN_EINVAL;
    const bool turn = t.cos != nullptr && t.pairs > 0;
    AppendArgs a{};
    a.v = RowsView{table, lens, starts, table_stride, rows, width, t.tokens, cache->pages,
                   divisor((uint32_t)cache->page_tokens)};
    a.status = status;
    a.keys = Heads{t.keys, cache->heads, t.key_token_stride, t.key_head_stride};
    a.values = Heads{t.values, cache->heads, t.value_token_stride, t.value_head_stride};
    a.queries = Heads{t.queries, t.queries ? t.q_heads : 0, t.query_token_stride, t.query_head_stride};
    a.out = Heads{t.queries_out, a.queries.heads, t.out_token_stride, t.out_head_stride};
    a.cos = turn ? t.cos : nullptr;
    a.sin = t.sin;
    a.positions = t.positions;
    a.pairs = (uint32_t)t.pairs;
    a.dim = (uint32_t)cache->dim;
    a.interleaved = t.interleaved;
    a.cache_keys = cache->keys;
    a.cache_values = cache->values;
    a.page_stride = cache->page_stride;
    a.token_stride = cache->token_stride;
    a.head_stride = cache->head_stride;
    const bool coded = cache->type == U32SCAN_E4M3;
    if (coded) {
        a.key_scales = cache->key_scales;
        a.value_scales = cache->value_scales;
        a.scale_stride = cache->scale_stride;
        a.block_tokens = divisor((uint32_t)(cache->page_tokens / cache->blocks));
    }
    const cudaStream_t s = (cudaStream_t)stream;
    if (t.type == U32SCAN_F32) append_launch<float>(a, coded, s);
    else if (t.type == U32SCAN_F16) append_launch<__half>(a, coded, s);
    else append_launch<__nv_bfloat16>(a, coded, s);
    return cudaGetLastError() == cudaSuccess ? U32SCAN_OK : U32SCAN_ECUDA;
}
