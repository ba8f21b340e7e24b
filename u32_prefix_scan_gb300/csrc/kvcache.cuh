// kvcache.cuh -- one layer's keys and values in a paged cache, as the kernels
// that write (append.cu) and read (attend.cu) them see it: the arguments'
// checks on the host, a token's place on the device.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "internal.cuh"

namespace u32scan {

// Division by a number fixed for a launch, for numerators below 2^31: floor(x
// * m / 2^s) with s = 31 + ceil(log2 d) and m = ceil(2^s / d) is floor(x / d),
// as m d - 2^s < d <= 2^(s - 31) makes the error x (m d - 2^s) / (d 2^s)
// less than 1 / d.
struct Divisor {
    uint32_t d, shift;
    uint64_t m;
};

static inline Divisor divisor(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    return Divisor{d, 31 + l, ((1ull << (31 + l)) + d - 1) / d};
}

__device__ __forceinline__ uint32_t divide(uint32_t x, const Divisor &d) {
    return (uint32_t)((uint64_t)x * d.m >> d.shift);  // m <= 2^32, x < 2^31: the product fits
}

// The rows' tables and the tokens that belong to them.
struct RowsView {
    const int32_t *table, *lens, *starts;
    uint64_t table_stride, rows, width, tokens, pages;
    Divisor page_tokens;
};

// Row s's tokens [begin, begin + n) of the call.
__device__ __forceinline__ void tokens_of(const RowsView &v, uint64_t s, int64_t *begin, int64_t *n) {
    if (v.starts == nullptr) {
        *begin = (int64_t)s;
        *n = 1;
        return;
    }
    const int64_t most = (int64_t)v.tokens;
    const int64_t a = v.starts[s], b = v.starts[s + 1];
    const int64_t lo = a < 0 ? 0 : a > most ? most : a, hi = b < 0 ? 0 : b > most ? most : b;
    *begin = lo;
    *n = hi > lo ? hi - lo : 0;
}

// The row of a token of the call, or -1 behind the last row's tokens: the
// last row that begins at or before it. A whole warp looks, 32 rows at a time
// (one after the other, in halves, the loads are what a small append waits for).
__device__ __forceinline__ int64_t row_of(const RowsView &v, uint64_t token, int64_t *begin, int64_t *n) {
    uint64_t lo = token;
    if (v.starts) {
        uint64_t left = v.rows;  // the row is one of lo .. lo + left - 1, or none
        lo = 0;
        do {
            const uint64_t step = (left + 31) / 32, at = (threadIdx.x & 31) * step;
            const bool before = at < left && (int64_t)v.starts[lo + at] <= (int64_t)token;
            const int found = __popc(__ballot_sync(0xffffffffu, before));
            if (found == 0) return -1;
            const uint64_t skip = (found - 1) * step;
            lo += skip;
            left = left - skip < step ? left - skip : step;
        } while (left > 1);
    }
    tokens_of(v, lo, begin, n);
    return (int64_t)token < *begin + *n ? (int64_t)lo : -1;
}

static inline bool misaligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

static inline size_t element_bytes(int type) { return type == U32SCAN_F32 ? 4 : type == U32SCAN_E4M3 ? 1 : 2; }

static inline bool cache_ok(const u32scan_kv_cache *c) {
    if (c == nullptr || c->type < U32SCAN_F32 || c->type > U32SCAN_E4M3) return false;
    if (c->pages >= (1ull << 31) || c->page_tokens == 0 || c->page_tokens >= (1ull << 31)) return false;
    if (c->heads == 0 || c->heads >= (1ull << 16) || c->dim == 0 || c->dim > 1024) return false;
    if (c->page_stride >= (1ull << 40) || c->token_stride >= (1ull << 40) || c->head_stride >= (1ull << 40)) return false;
    if ((c->pages > 1 && c->page_stride == 0) || (c->page_tokens > 1 && c->token_stride == 0) ||
        (c->heads > 1 && c->head_stride == 0))
        return false;
    if (c->pages > 0 && (c->keys == nullptr || c->values == nullptr)) return false;
    if (misaligned(c->keys, element_bytes(c->type)) || misaligned(c->values, element_bytes(c->type))) return false;
    if (c->type == U32SCAN_E4M3) {
        if (c->blocks == 0 || c->page_tokens % c->blocks != 0 || c->scale_stride >= (1ull << 40)) return false;
        if (c->pages > 0 && (c->key_scales == nullptr || c->value_scales == nullptr)) return false;
        if (misaligned(c->key_scales, 4) || misaligned(c->value_scales, 4)) return false;
    }
    return true;
}

static inline bool rows_ok(const int32_t *table, size_t stride, size_t rows, size_t width, const int32_t *lens,
                           const int32_t *starts, size_t tokens) {
    if (rows >= (1ull << 31) || width >= (1ull << 31) || tokens >= (1ull << 31)) return false;
    if (stride < width || stride >= (1ull << 31)) return false;
    if (rows > 0 && (lens == nullptr || (width > 0 && table == nullptr))) return false;
    if (starts == nullptr && rows != tokens) return false;
    return !misaligned(table, 4) && !misaligned(lens, 4) && !misaligned(starts, 4);
}

static inline bool strides_ok(size_t token, size_t head) { return token < (1ull << 40) && head < (1ull << 40); }

}  // namespace u32scan
