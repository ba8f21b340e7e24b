// append.cu -- new keys and values written into the pages of a paged cache,
// keys (and queries) rotated by their position on the way.
//
// A block takes one token. Heads are handled in units of two vectors: the two
// halves of eight (f32: four) pairs, or two adjacent vectors; a thread keeps to one
// unit of a head and goes over the heads, its angles in registers. For the
// 8-bit cache a warp takes one head of one block of a page: the largest
// magnitude of its new tokens first, the codes in a second pass (the tokens
// come from L1 then). The tokens of a block share its heads between them.
// Heads of other sizes, strides or addresses go element by element.
//
// Measured on one GB300, launches back to back: 8192 tokens of 64 + 16 heads of
// 128 (bf16 into bf16, 340 MB) 57 us, 5.9 TB/s, bound by the memory; 16384 tokens
// of 16 + 32 heads of 64 into 8 bits (170 MB) 80 us, bound by latency and
// instructions: the chain from a token's row over its page to the scale, and two
// passes over the values; 64 rows' next tokens into 8 bits 5 us, one row's into
// bf16 2.8, a launch and that chain. The 5 us are of scales that hold: where a
// new token raises its block's, a warp tells the older codes anew a byte a lane
// at a time, and the launch lasts as long as the slowest: with 2, 20, 100 % of
// the (64 x 16, blocks of 16 tokens of 128) scales growing 15, 22, 27 us, in blocks of
// 64 tokens of 256 96, 172, 190 us (5.8 with none).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "kvcache.cuh"
#include "launch.cuh"

namespace u32scan {

constexpr int kNThreads = 256;  // at most

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

// A rotated pair.
__device__ __forceinline__ void turn_pair(float &x, float &y, float c, float s) {
    const float a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
    x = a;
}

template <typename T, int N>
struct alignas(sizeof(T) * N) Vector {
    T x[N];
};

// Unit u of a head, two vectors of N elements: where they begin, and the first pair if it is turned.
struct Unit {
    uint32_t at[2], pair;
    bool turned;
};

template <int N>
__device__ __forceinline__ Unit unit_of(const AppendArgs &a, uint32_t u, bool turn) {
    Unit x;
    x.turned = turn && u * N < a.pairs;
    x.pair = x.turned ? u * N : 0;
    x.at[0] = x.turned && !a.interleaved ? u * N : 2 * u * N;
    x.at[1] = x.turned && !a.interleaved ? a.pairs + u * N : x.at[0] + N;
    return x;
}

template <int N>
__device__ __forceinline__ void angles_of(const AppendArgs &a, const Unit &u, int64_t position, float (&c)[N], float (&s)[N]) {
    if (!u.turned) return;
    const uint64_t from = (uint64_t)position * a.pairs + u.pair;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 x = __ldg(reinterpret_cast<const float4 *>(a.cos + from + i));
        const float4 y = __ldg(reinterpret_cast<const float4 *>(a.sin + from + i));
        c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
        s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
    }
}

// The unit's values, turned.
template <typename T, int N>
__device__ __forceinline__ void turned_unit(const AppendArgs &a, const Unit &u, const Vector<T, N> &x, const Vector<T, N> &y,
                                            const float (&c)[N], const float (&s)[N], float (&v)[2][N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[0][i] = Num<T>::get(x.x[i]), v[1][i] = Num<T>::get(y.x[i]);
    if (!u.turned) return;
    if (!a.interleaved) {
#pragma unroll
        for (int i = 0; i < N; ++i) turn_pair(v[0][i], v[1][i], c[i], s[i]);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < N; i += 2) turn_pair(v[h][i], v[h][i + 1], c[(h * N + i) / 2], s[(h * N + i) / 2]);
    }
}

// Where a block of a page stands, and the part of it that is new.
struct Part {
    float *scale;
    uint8_t *codes;     // of the first new slot
    uint32_t n, before; // new tokens, older ones in front of them
    int64_t position;   // of the first new one
    uint64_t token;
    bool key;
};

// The largest magnitudes' scale: the least power of two that holds them, or the old one if it does; the older codes are
// told in it (by the warp, element by element: they are few and seldom).
__device__ float part_scale(const AppendArgs &a, const Part &p, float m, int lane) {
    // least e with m <= 1.75 * 2^(8 + e)
    int e = (int)(__float_as_uint(m) >> 23) - 127 - 8 + ((__float_as_uint(m) & 0x7fffffu) > 0x600000u ? 1 : 0);
    if (e < -100) e = -100;
    float scale = __uint_as_float((uint32_t)(e + 127) << 23);
    if (p.before) {
        float old = *p.scale;
        if (!(old > 0.0f && old < INFINITY)) old = 0.0f;
        if (old >= scale) return old;
        const float ratio = __fdiv_rn(old, scale);
        for (uint32_t t = 1; t <= p.before; ++t)
            for (uint32_t d = lane; d < a.dim; d += 32) {
                uint8_t *c = p.codes - (uint64_t)t * a.token_stride + d;
                *c = value_code(__fmul_rn(code_value(*c), ratio));
            }
    }
    return scale;
}

template <typename T>
__device__ __forceinline__ T *cache_at(const AppendArgs &a, bool key, uint64_t page, uint64_t slot, uint64_t head) {
    return static_cast<T *>(key ? a.cache_keys : a.cache_values) + page * a.page_stride + slot * a.token_stride +
           head * a.head_stride;
}

// The part's codes and scale. N: vectors of N elements, or 0: one element at a time.
template <typename T, int N>
__device__ void append_part(const AppendArgs &a, const Part &p, uint64_t head, int lane) {
    const Heads &src = p.key ? a.keys : a.values;
    const bool turn = p.key && a.cos;
    float m = 0.0f, inv = 0.0f;
    for (int pass = 0; pass < 2; ++pass) {
        if constexpr (N > 0) {
            const uint32_t units = a.dim / (2 * N), abreast = 32 / units;  // of a token; tokens beside each other
            const uint32_t mine = lane / units;
            const Unit u = unit_of<N>(a, lane % units, turn);
            if (mine < abreast) {
#pragma unroll 1
                for (uint32_t i = mine; i < p.n; i += abreast) {
                    const T *x = head_of<T>(src, p.token + i, head);
                    float c[N], s[N], v[2][N];
                    angles_of<N>(a, u, p.position + i, c, s);
                    turned_unit<T, N>(a, u, *reinterpret_cast<const Vector<T, N> *>(x + u.at[0]),
                                      *reinterpret_cast<const Vector<T, N> *>(x + u.at[1]), c, s, v);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (pass == 0) {
#pragma unroll
                            for (int k = 0; k < N; ++k)
                                if (fabsf(v[h][k]) < INFINITY) m = fmaxf(m, fabsf(v[h][k]));
                        } else {
                            uint32_t w = 0;
#pragma unroll
                            for (int k = 0; k < N; k += 2)
                                w |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[h][k], inv), __fmul_rn(v[h][k + 1], inv)),
                                                                        __NV_SATFINITE, __NV_E4M3)
                                     << 8 * k;
                            *reinterpret_cast<uint32_t *>(p.codes + (uint64_t)i * a.token_stride + u.at[h]) = w;
                        }
                    }
                }
            }
        } else {
            for (uint32_t i = 0; i < p.n; ++i) {
                const T *x = head_of<T>(src, p.token + i, head);
                for (uint32_t d = lane; d < a.dim; d += 32) {
                    const float y = rotated(a, x, d, p.position + i, turn);
                    if (pass == 0) {
                        if (fabsf(y) < INFINITY) m = fmaxf(m, fabsf(y));
                    } else {
                        p.codes[(uint64_t)i * a.token_stride + d] = value_code(__fmul_rn(y, inv));
                    }
                }
            }
        }
        if (pass == 0) {
            m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
            const float scale = part_scale(a, p, m, lane);
            inv = __fdiv_rn(1.0f, scale);
            __syncwarp();  // every lane has read the old scale
            if (lane == 0) *p.scale = scale;
        }
    }
}

// WIDE: vectors of 16 bytes (for codes: of four values), else elements. (At 48 registers a thread, five blocks of 256 an SM,
// with 24 to 48 bytes a thread spilled: 8192 tokens of 64 + 16 heads of 128 bf16 57 us, 16384 into 8 bits 80, 64 rows' next 5.2,
// one row's 2.7; at 64, four, 60, 80, 5.0, 2.7; at 40, six, 87, 79, 5.6, 3.2.)
template <typename T, bool CODED, bool WIDE>
__global__ void __launch_bounds__(kNThreads, 5) append_kernel(const AppendArgs a) {
    const uint64_t token = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Place p = place_of(a, token);
    if (p.row < 0) return;
    const bool turn = a.cos != nullptr, reached = !turn || (p.position >= 0 && (uint64_t)p.position < a.positions);
    if (CODED && p.held) {
        // the block's new tokens, of which this is number `rank`; they take its heads in turn
        const uint32_t size = a.block_tokens.d, nth = divide(p.slot, a.block_tokens), within = p.slot - nth * size;
        const int64_t back = p.position - p.first;  // new tokens of the row before this one
        const uint32_t rank = back < (int64_t)within ? (uint32_t)back : within, before = within - rank;
        const int64_t position = p.position - rank;
        int64_t n = (int64_t)a.v.lens[p.row] - position;
        if (n > (int64_t)(size - before)) n = size - before;
        if (turn && n > (int64_t)a.positions - position) n = (int64_t)a.positions - position;
        for (uint64_t task = rank + (uint64_t)n * warp; task < 2 * a.keys.heads; task += (uint64_t)n * (blockDim.x / 32)) {
            const uint64_t head = task >> 1;
            const bool key = !(task & 1);
            const Part part{(key ? a.key_scales : a.value_scales) + p.page * a.scale_stride + (uint64_t)nth * a.keys.heads + head,
                            cache_at<uint8_t>(a, key, p.page, p.slot - rank, head), (uint32_t)n, before, position, token - rank,
                            key};
            append_part<T, WIDE ? 4 : 0>(a, part, head, lane);
        }
    }
    if constexpr (WIDE) {
        constexpr int N = 16 / sizeof(T);
        const uint32_t units = a.dim / (2 * N), abreast = blockDim.x / units, mine = threadIdx.x / units;
        if (mine >= abreast) return;
        const Unit u = unit_of<N>(a, threadIdx.x % units, turn), plain = unit_of<N>(a, threadIdx.x % units, false);
        float c[N], s[N];
        if (reached) angles_of<N>(a, u, p.position, c, s);
        const uint64_t heads = a.queries.heads + (!CODED && p.held ? 2 * a.keys.heads : 0);
#pragma unroll 4
        for (uint64_t h = mine; h < heads; h += abreast) {
            const bool query = h < a.queries.heads, key = h < a.queries.heads + a.keys.heads;
            const uint64_t head = query ? h : key ? h - a.queries.heads : h - a.queries.heads - a.keys.heads;
            const Unit &x = key ? u : plain;
            const T *from = head_of<T>(query ? a.queries : key ? a.keys : a.values, token, head);
            T *to = query ? const_cast<T *>(head_of<T>(a.out, token, head)) : cache_at<T>(a, key, p.page, p.slot, head);
            Vector<T, N> v[2] = {*reinterpret_cast<const Vector<T, N> *>(from + x.at[0]),
                                 *reinterpret_cast<const Vector<T, N> *>(from + x.at[1])};
            if (x.turned || !reached) {
                float y[2][N];
                turned_unit<T, N>(a, x, v[0], v[1], c, s, y);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    v[0].x[i] = Num<T>::put(reached ? y[0][i] : NAN);
                    v[1].x[i] = Num<T>::put(reached ? y[1][i] : NAN);
                }
            }
            *reinterpret_cast<Vector<T, N> *>(to + x.at[0]) = v[0];
            *reinterpret_cast<Vector<T, N> *>(to + x.at[1]) = v[1];
        }
    } else {
        for (uint64_t h = warp; h < a.queries.heads; h += blockDim.x / 32) {
            const T *x = head_of<T>(a.queries, token, h);
            T *y = const_cast<T *>(head_of<T>(a.out, token, h));
            float r[32];
            int k = 0;
            for (uint32_t d = lane; d < a.dim; d += 32) r[k++] = reached ? rotated(a, x, d, p.position, turn) : NAN;
            __syncwarp();  // in place: every element read before any is written
            k = 0;
            for (uint32_t d = lane; d < a.dim; d += 32) y[d] = Num<T>::put(r[k++]);
        }
        for (uint64_t h = warp; !CODED && p.held && h < 2 * a.keys.heads; h += blockDim.x / 32) {
            const bool key = !(h & 1);
            const T *x = head_of<T>(key ? a.keys : a.values, token, h >> 1);
            T *y = cache_at<T>(a, key, p.page, p.slot, h >> 1);
            for (uint32_t d = lane; d < a.dim; d += 32) y[d] = Num<T>::put(rotated(a, x, d, p.position, key && turn));
        }
    }
}

// Whether the rotated queries would lie over what other blocks still read. (Queries themselves, place by place, may.)
static bool queries_over_inputs(const AppendArgs &a, size_t elem) {
    auto view = [&](const Heads &h) {
        return Strided{h.data, a.dim * elem, {a.v.tokens, h.heads, 1}, {h.token_stride * elem, h.head_stride * elem, 0}};
    };
    const Heads &q = a.queries, &o = a.out;
    const bool in_place = q.data == o.data && (a.v.tokens == 1 || q.token_stride == o.token_stride) &&
                          (q.heads == 1 || q.head_stride == o.head_stride);
    return q.heads > 0 && ((!in_place && share_memory(view(o), view(q))) || share_memory(view(o), view(a.keys)) ||
                           share_memory(view(o), view(a.values)));
}

// Whether every address that a vector kernel forms is a multiple of its vector's size (16 bytes; codes: 4).
static bool wide(const AppendArgs &a, size_t elem, bool coded) {
    const uint64_t n = 16 / elem;
    if (a.dim % (2 * n) != 0 || a.dim > 256 || (a.cos && (a.pairs % n != 0 || misaligned(a.cos, 16) || misaligned(a.sin, 16))))
        return false;
    for (const Heads *h : {&a.keys, &a.values, &a.queries, &a.out})
        if (h->heads > 0 && (misaligned(h->data, 16) || (h->token_stride | h->head_stride) % n != 0)) return false;
    const uint64_t m = coded ? 4 : n;
    return !misaligned(a.cache_keys, coded ? 4 : 16) && !misaligned(a.cache_values, coded ? 4 : 16) &&
           (a.page_stride | a.token_stride | a.head_stride) % m == 0;
}

template <typename T>
static void append_launch(const AppendArgs &a, bool coded, cudaStream_t s) {
    const unsigned int grid = (unsigned int)a.v.tokens;
    if (!wide(a, sizeof(T), coded)) {
        if (coded) append_kernel<T, true, false><<<grid, kNThreads, 0, s>>>(a);
        else append_kernel<T, false, false><<<grid, kNThreads, 0, s>>>(a);
        return;
    }
    // Of many tokens (more blocks of 64 threads than run at a time) a thread takes several units, whose loads overlap; of few
    // as many threads as a token has units, or warps as it has heads of its block. 64, 128, 256 threads: 8192 tokens of 64 +
    // 16 heads of 128 bf16 57, 57, 64 us, 16384 tokens of 16 + 32 heads of 64 into 8 bits 80, 81, 112; 64 tokens of 32 + 16 heads into
    // 8 bits 10.9, 6.8, 5.2, one of them into bf16 4.2, 3.0, 2.7.
    const uint64_t units = a.queries.heads * (a.dim * sizeof(T) / 32) + (coded ? 0 : 2 * a.keys.heads * (a.dim * sizeof(T) / 32));
    const uint64_t work = coded && units < 64 * a.keys.heads ? 64 * a.keys.heads : units;
    const int threads = a.v.tokens >= 2432 || work <= 64 ? 64 : work <= 128 ? 128 : kNThreads;
    if (coded) append_kernel<T, true, true><<<grid, threads, 0, s>>>(a);
    else append_kernel<T, false, true><<<grid, threads, 0, s>>>(a);
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
    if (queries_over_inputs(a, elem)) return U32SCAN_EINVAL;
    const cudaStream_t s = (cudaStream_t)stream;
    if (t.type == U32SCAN_F32) append_launch<float>(a, coded, s);
    else if (t.type == U32SCAN_F16) append_launch<__half>(a, coded, s);
    else append_launch<__nv_bfloat16>(a, coded, s);
    return cudaGetLastError() == cudaSuccess ? U32SCAN_OK : U32SCAN_ECUDA;
}
