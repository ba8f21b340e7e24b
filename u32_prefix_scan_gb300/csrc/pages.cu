// pages.cu -- the pages of a paged cache: copied, forked between rows,
// released and packed.
//
// A cache is a pool of `pages` pages (in every plane: one layer's keys or
// values), a table of page numbers a row, the rows' lengths in tokens and
// refs, how many table entries hold each page (0 = free). Each operation is
// a prefix sum over flags of refs (which pages are free, or live) joined to
// one over the rows:
//   fork     need[s] = pages row s lacks; ends = inclusive sum of need in row
//            order; the free page of rank f (ascending) goes to the row with
//            ends[s-1] <= f < ends[s], as its (f - ends[s-1])-th fresh page.
//   free     refs -= 1 over the released rows' entries.
//   compact  L = live pages; the k-th live page at or above L goes to the
//            k-th free page below L (sources and destinations are disjoint,
//            so all pages move at once).
// All of it is integer, so results do not depend on the order of atomics.
//
// Three launches, each reading what the one before wrote: plan (count the free
// or live pages of every 4096 refs; the last block scans the counts and the
// rows' needs), place (list the pages by rank) and act (table entries, refs,
// bytes). A cache of up to 4096 pages is planned and placed by one block in
// one launch. refs is read twice, the second time from L2 (4 MB at a million
// pages): a single pass that carries the rank from tile to tile would have
// every tile wait for the one before, and the rows' needs, which decide how
// far the list goes, are known only after the scan.
//
// Measured on one GB300, launches back to back: copying 509 pages of 64 x 32
// KiB 312 us (2.1 GB read and written, 6.8 TB/s, the rate of a plain copy),
// packing 65537 half-live pages of 2 x 16 KiB 165 us (1.06 GB, 6.4 TB/s): bound
// by HBM. Forking 512 of 2048 rows in 262147 pages 16 us, releasing half of
// 8192 rows of up to 500 pages 10 us, the same on 16 rows and 1024 pages 8 and 4 us
// and packing those 7 us: bound by latency, the launches that wait for one
// another and in each a chain of loads (row, entry, count).
#include <cstdint>
#include <mutex>
#include <cuda_runtime.h>

#include "internal.cuh"

namespace u32scan {

typedef unsigned long long u64;

constexpr int kPThreads = 256;      // free, copies and act
constexpr int kPWarps = kPThreads / 32;
constexpr int kPlanThreads = 1024;  // plan and place
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPerThread = 4;       // refs of a thread of plan and place
constexpr int kRefTile = kPlanThreads * kPerThread;
constexpr int kEntryChunk = 512;    // table entries handled by one warp
constexpr size_t kCopyUnit = 16384; // bytes of a page copied by one block at a time

struct Pool {
    const u64 *planes;
    u64 n_planes, pages, page_bytes, page_stride;
};

// What the launches of one call hand on to each other (in the workspace,
// past every other operation's tile words).
struct PagesCtrl {
    u64 free_pages;    // fork: F
    u64 taken;         // fork: fresh pages of the rows that are served
    u64 jobs;          // fork: children whose parent's last page is partly filled
    u64 live;          // compact: L
    u64 moved;         // compact: pages that move
    u64 pad[27];
};
static_assert(sizeof(PagesCtrl) == 256, "one line group");

struct PagesWs {
    WsHeader *hdr;
    PagesCtrl *ctrl;
    u64 *tile_base;   // [tiles] counts, then exclusive bases
    u64 *ends;        // fork: [rows]
    int32_t *old_len; // fork: [rows] length before the call (of the parent, for a child)
    int32_t *jobs;    // fork: [rows]
    int32_t *fresh;   // fork: [pages] the free pages by rank
    uint32_t *freed;  // free: [blocks]
    int32_t *holes, *movers, *rank;  // compact: [pages] each
};

static u64 ref_tiles(u64 pages) { return (pages + kRefTile - 1) / kRefTile; }

// n = pages + rows: 8 bytes a tile, and at most 16 bytes a row and 4 a page
// (fork) or 12 a page (compact).
size_t pages_workspace_bytes(u64 n) {
    return round_up(tile_word_reach(), 256) + sizeof(PagesCtrl) + round_up(8 * (n / kRefTile + 2), 256) +
           round_up(16 * n, 256) + 4 * 256;
}

static PagesWs carve(void *ws, u64 pages, u64 rows) {
    char *p = static_cast<char *>(ws) + round_up(tile_word_reach(), 256);
    PagesWs w;
    w.hdr = static_cast<WsHeader *>(ws);
    w.ctrl = reinterpret_cast<PagesCtrl *>(p);
    p += sizeof(PagesCtrl);
    w.tile_base = reinterpret_cast<u64 *>(p);
    p += round_up(8 * ref_tiles(pages) + 8, 256);
    w.ends = reinterpret_cast<u64 *>(p);
    w.old_len = reinterpret_cast<int32_t *>(p + round_up(8 * rows, 256));
    w.jobs = reinterpret_cast<int32_t *>(p + round_up(8 * rows, 256) + round_up(4 * rows, 256));
    w.fresh = reinterpret_cast<int32_t *>(p + round_up(8 * rows, 256) + 2 * round_up(4 * rows, 256));
    w.freed = reinterpret_cast<uint32_t *>(p);
    w.holes = reinterpret_cast<int32_t *>(p);
    w.movers = reinterpret_cast<int32_t *>(p + round_up(4 * pages, 256));
    w.rank = reinterpret_cast<int32_t *>(p + 2 * round_up(4 * pages, 256));
    return w;
}

// ---------------------------------------------------------------------------
// Block-wide pieces
// ---------------------------------------------------------------------------
__device__ __forceinline__ u64 warp_inclusive_u64(u64 x, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    return x;
}

// Exclusive sum over the block's threads; *total is the block's (all threads
// call it; s_warp holds one value a warp, at most 32).
__device__ __forceinline__ u64 block_exclusive(u64 x, u64 *s_warp, u64 *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const u64 inc = warp_inclusive_u64(x, lane);
    __syncthreads();
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    const u64 sums = warp_inclusive_u64(lane < warps ? s_warp[lane] : 0ull, lane);
    *total = __shfl_sync(0xffffffffu, sums, 31);
    const u64 base = __shfl_sync(0xffffffffu, sums, warp ? warp - 1 : 0);
    return (warp ? base : 0ull) + inc - x;
}

// True in every thread of the block that finishes last (each block's earlier
// writes are then visible to it). The counter is left at zero.
__device__ __forceinline__ bool last_block(WsHeader *hdr) {
    __shared__ uint32_t s_last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        const bool last = atom_add_acq_rel(&hdr->done, 1u) == gridDim.x - 1u;
        if (last) st_relaxed_u32(&hdr->done, 0u);
        s_last = last ? 1u : 0u;
    }
    __syncthreads();
    return s_last != 0u;
}

// f(i, base) for i < n by one block, where base is the sum of the values v(k),
// k < i; returns the sum of all. A thread takes neighbouring i, so that one
// block-wide scan serves many (4 a thread at a time).
template <typename V, typename F>
__device__ __forceinline__ u64 scan_by_block(u64 n, u64 *s_warp, V v, F f) {
    constexpr int C = 4;
    u64 carry = 0;
    for (u64 i0 = 0; i0 < n; i0 += (u64)C * blockDim.x) {
        const u64 left = n - i0, per = left < (u64)C * blockDim.x ? (left + blockDim.x - 1) / blockDim.x : C;
        const u64 first = i0 + threadIdx.x * per;
        u64 x[C], sum = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = c < (int)per && first + c < n ? v(first + c) : 0ull;
#pragma unroll
        for (int c = 0; c < C; ++c) sum += x[c];
        u64 total, base = carry + block_exclusive(sum, s_warp, &total);
        carry += total;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (c < (int)per && first + c < n) f(first + c, base, x[c]);
            base += x[c];
        }
    }
    return carry;
}

// Which of this thread's kPerThread refs of a tile are free (zero), a bit each.
__device__ __forceinline__ unsigned int free_mask(const int32_t *refs, u64 tile, u64 pages) {
    const u64 first = tile * kRefTile + (u64)threadIdx.x * kPerThread;
    unsigned int m = 0;
    if (first + kPerThread <= pages && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) {
        int4 r[kPerThread / 4];
#pragma unroll
        for (int j = 0; j < kPerThread / 4; ++j) r[j] = reinterpret_cast<const int4 *>(refs + first)[j];
#pragma unroll
        for (int j = 0; j < kPerThread / 4; ++j)
            m |= ((r[j].x == 0) | (r[j].y == 0) << 1 | (r[j].z == 0) << 2 | (r[j].w == 0) << 3) << (4 * j);
    } else {
#pragma unroll
        for (int j = 0; j < kPerThread; ++j)
            if (first + j < pages && refs[first + j] == 0) m |= 1u << j;
    }
    return m;
}

// The bits of free_mask's refs that exist.
__device__ __forceinline__ unsigned int page_mask(u64 tile, u64 pages) {
    const u64 first = tile * kRefTile + (u64)threadIdx.x * kPerThread;
    if (first >= pages) return 0u;
    return pages - first >= kPerThread ? (1u << kPerThread) - 1u : (1u << (unsigned int)(pages - first)) - 1u;
}

// ---------------------------------------------------------------------------
// Copying bytes
// ---------------------------------------------------------------------------
__device__ __forceinline__ void copy_bytes(char *dst, const char *src, size_t n) {
    const uintptr_t d = reinterpret_cast<uintptr_t>(dst), s = reinterpret_cast<uintptr_t>(src);
    if (((d | s | n) & 15) == 0) {
        const uint4 *sv = reinterpret_cast<const uint4 *>(src);
        uint4 *dv = reinterpret_cast<uint4 *>(dst);
        const size_t nv = n / 16;
        size_t i = threadIdx.x;
        for (; i + 3 * kPThreads < nv; i += 4 * kPThreads) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __ldcs(sv + i + j * kPThreads);
#pragma unroll
            for (int j = 0; j < 4; ++j) __stcs(dv + i + j * kPThreads, v[j]);
        }
        for (; i < nv; i += kPThreads) __stcs(dv + i, __ldcs(sv + i));
    } else if (((d | s | n) & 3) == 0) {
        const uint32_t *sv = reinterpret_cast<const uint32_t *>(src);
        uint32_t *dv = reinterpret_cast<uint32_t *>(dst);
        for (size_t i = threadIdx.x; i < n / 4; i += kPThreads) dv[i] = sv[i];
    } else {
        for (size_t i = threadIdx.x; i < n; i += kPThreads) dst[i] = src[i];
    }
}

// Copies of `count` pairs of pages in every plane, unit by unit over the
// grid. pair(k, &src, &dst) gives pair k, or false to skip it.
template <typename Pair>
__device__ __forceinline__ void copy_pages(const Pool &pool, u64 count, u64 block, u64 blocks, Pair pair) {
    const u64 per_page = (pool.page_bytes + kCopyUnit - 1) / kCopyUnit;
    const u64 per_pair = per_page * pool.n_planes;
    for (u64 u = block; u < count * per_pair; u += blocks) {
        const u64 k = u / per_pair, rest = u - k * per_pair;
        const u64 plane = rest / per_page, part = rest - plane * per_page;
        u64 src, dst;
        if (!pair(k, &src, &dst) || src >= pool.pages || dst >= pool.pages || src == dst) continue;
        char *base = reinterpret_cast<char *>(pool.planes[plane]);
        const size_t at = part * kCopyUnit;
        const size_t n = pool.page_bytes - at < kCopyUnit ? pool.page_bytes - at : kCopyUnit;
        copy_bytes(base + dst * pool.page_stride + at, base + src * pool.page_stride + at, n);
    }
}

// A page number as an index; anything below zero becomes too large for a pool.
__device__ __forceinline__ u64 page_of(int32_t p) { return p < 0 ? ~0ull : (u64)p; }

__global__ void __launch_bounds__(kPThreads)
pages_copy_kernel(Pool pool, const int32_t *src, const int32_t *dst, u64 n, const int32_t *count) {
    u64 m = n;
    if (count) {
        const int32_t c = *count;
        m = c < 0 ? 0ull : (u64)c < n ? (u64)c : n;
    }
    copy_pages(pool, m, blockIdx.x, gridDim.x, [&](u64 k, u64 *s, u64 *d) {
        *s = page_of(src[k]);
        *d = page_of(dst[k]);
        return true;
    });
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
struct ForkArgs {
    int32_t *table;
    u64 stride, rows, width;
    int32_t *lens;
    int32_t *refs;
    u64 pages;
    uint32_t page_tokens;
    const int32_t *parent, *grow;
    int32_t *status, *free_pages;
};

constexpr int32_t kBadRow = -1;  // old_len of a row whose arguments are refused

// Both below 2^31, so that 32 bits are enough.
__device__ __forceinline__ uint32_t pages_for(uint32_t tokens, uint32_t page_tokens) {
    return (tokens + page_tokens - 1) / page_tokens;
}

// Pages row s holds before its fresh ones: a child's shared full pages, or
// the row's own.
__device__ __forceinline__ uint32_t held_pages(bool child, uint32_t old_len, uint32_t page_tokens) {
    return child ? old_len / page_tokens : pages_for(old_len, page_tokens);
}

__device__ __forceinline__ bool is_child(const ForkArgs &a, u64 s) { return a.parent && a.parent[s] >= 0; }

__device__ __forceinline__ u64 row_need(const ForkArgs &a, u64 s, int32_t *old_len) {
    *old_len = kBadRow;
    const bool child = is_child(a, s);
    const int32_t own = a.lens[s];
    int32_t old = own;
    if (child) {
        const u64 p = (u64)a.parent[s];
        if (p >= a.rows || own != 0 || a.parent[p] >= 0) return 0;
        old = a.lens[p];
    }
    const int32_t g = a.grow ? a.grow[s] : 0;
    if (old < 0 || g < 0) return 0;
    const uint32_t total = (uint32_t)old + (uint32_t)g;
    if (total > 0x7fffffffu || pages_for(total, a.page_tokens) > a.width) return 0;
    *old_len = old;
    return pages_for(total, a.page_tokens) - held_pages(child, (uint32_t)old, a.page_tokens);
}

// What the rows ask for, by one block: ends, the jobs, and the number of pages
// the served rows take (returned).
__device__ __forceinline__ u64 plan_rows(const ForkArgs &a, const PagesWs &w, u64 free_pages, u64 *s_warp) {
    __shared__ u64 s_taken;
    u64 taken = 0, jobs = 0;
    if (threadIdx.x == 0) s_taken = 0;
    auto need_of = [&](u64 s, int32_t *old) {
        const u64 need = row_need(a, s, old);
        w.old_len[s] = *old;
        return need;
    };
    auto place_row = [&](u64 s, u64 base, u64 need) {
        w.ends[s] = base + need;
        if (need && base + need <= free_pages) taken = base + need;
    };
    // a child whose parent's last page is partly filled
    auto is_job = [&](u64 s, int32_t old) {
        return old > 0 && is_child(a, s) && (uint32_t)old % a.page_tokens != 0;
    };
    if (a.rows <= 65535) {
        // one scan of both: needs (their sum is below 65535 * 2^31) and, from bit 48 on, jobs
        constexpr u64 kNeeds = (1ull << 48) - 1;
        const u64 sums = scan_by_block(
            a.rows, s_warp,
            [&](u64 s) -> u64 {
                int32_t old;
                const u64 need = need_of(s, &old);
                return need | (is_job(s, old) ? 1ull << 48 : 0ull);
            },
            [&](u64 s, u64 base, u64 x) {
                place_row(s, base & kNeeds, x & kNeeds);
                if (x >> 48) w.jobs[base >> 48] = (int32_t)s;
            });
        jobs = sums >> 48;
    } else {
        scan_by_block(
            a.rows, s_warp,
            [&](u64 s) -> u64 {
                int32_t old;
                return need_of(s, &old);
            },
            place_row);
        jobs = scan_by_block(  // a thread reads what it wrote
            a.rows, s_warp, [&](u64 s) -> u64 { return is_job(s, w.old_len[s]); },
            [&](u64 s, u64 base, u64 job) {
                if (job) w.jobs[base] = (int32_t)s;
            });
    }
    if (taken) atomicMax(&s_taken, taken);
    __syncthreads();
    if (threadIdx.x == 0) {
        w.ctrl->free_pages = free_pages;
        w.ctrl->taken = s_taken;
        w.ctrl->jobs = jobs;
        if (a.free_pages) *a.free_pages = (int32_t)(free_pages - s_taken);
    }
    return s_taken;
}

// The tile's free pages of rank below `taken` become fresh ones.
__device__ __forceinline__ void place_fresh(const ForkArgs &a, const PagesWs &w, u64 tile, unsigned int mask, u64 rank,
                                            u64 taken) {
    const u64 first = tile * kRefTile + (u64)threadIdx.x * kPerThread;
    for (; mask && rank < taken; mask &= mask - 1, ++rank) {
        const u64 page = first + (__ffs(mask) - 1);
        w.fresh[rank] = (int32_t)page;
        a.refs[page] = 1;
    }
}

// ONE: a single block, which also places (a cache of one tile).
template <bool ONE>
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(ForkArgs a, PagesWs w, u64 tiles) {
    __shared__ u64 s_warp[kPlanWarps];
    cudaTriggerProgrammaticLaunchCompletion();  // the next launch may come to its wait
    u64 total;
    const unsigned int mask = blockIdx.x < tiles ? free_mask(a.refs, blockIdx.x, a.pages) : 0u;
    const u64 rank = block_exclusive(__popc(mask), s_warp, &total);
    if (ONE) {
        const u64 taken = plan_rows(a, w, total, s_warp);
        place_fresh(a, w, 0, mask, rank, taken);
        return;
    }
    if (threadIdx.x == 0) w.tile_base[blockIdx.x] = total;
    if (!last_block(w.hdr)) return;
    const u64 free_pages = scan_by_block(
        tiles, s_warp, [&](u64 t) { return ld_relaxed(w.tile_base + t); },
        [&](u64 t, u64 base, u64) { w.tile_base[t] = base; });
    plan_rows(a, w, free_pages, s_warp);
}

__global__ void __launch_bounds__(kPlanThreads) fork_place_kernel(ForkArgs a, PagesWs w) {
    __shared__ u64 s_warp[kPlanWarps];
    cudaTriggerProgrammaticLaunchCompletion();  // the next launch may come to its wait
    cudaGridDependencySynchronize();  // what the launch before wrote
    const u64 base = w.tile_base[blockIdx.x], taken = w.ctrl->taken;
    if (base >= taken) return;
    const unsigned int mask = free_mask(a.refs, blockIdx.x, a.pages);
    u64 total;
    const u64 rank = base + block_exclusive(__popc(mask), s_warp, &total);
    place_fresh(a, w, blockIdx.x, mask, rank, taken);
}

// Row s gets all it asks for.
__device__ __forceinline__ bool row_served(const PagesWs &w, u64 s, u64 begin, u64 free_pages) {
    return w.old_len[s] != kBadRow && (w.ends[s] == begin || w.ends[s] <= free_pages);
}

__device__ __forceinline__ u64 row_begin(const PagesWs &w, u64 s) { return s ? w.ends[s - 1] : 0ull; }

// Table entries, lengths and states (the first row_blocks blocks, a warp to
// kEntryChunk entries of a row), and the bytes of the partly filled pages.
__global__ void __launch_bounds__(kPThreads)
fork_act_kernel(ForkArgs a, PagesWs w, Pool pool, unsigned int row_blocks, u64 chunks) {
    cudaGridDependencySynchronize();  // what the launch before wrote
    const u64 free_pages = w.ctrl->free_pages;
    if (blockIdx.x >= row_blocks) {
        copy_pages(pool, w.ctrl->jobs, blockIdx.x - row_blocks, gridDim.x - row_blocks,
                   [&](u64 k, u64 *src, u64 *dst) {
                       const u64 s = (u64)w.jobs[k], begin = row_begin(w, s);
                       if (!row_served(w, s, begin, free_pages)) return false;
                       *src = page_of(a.table[(u64)a.parent[s] * a.stride + (uint32_t)w.old_len[s] / a.page_tokens]);
                       *dst = page_of(w.fresh[begin]);
                       return true;
                   });
        return;
    }
    const u64 item = (u64)blockIdx.x * kPWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const u64 s = item / chunks, chunk = item - s * chunks;
    if (s >= a.rows) return;
    const u64 begin = row_begin(w, s), need = w.ends[s] - begin;
    const bool served = row_served(w, s, begin, free_pages), child = is_child(a, s);
    const int32_t old = w.old_len[s];
    if (chunk == 0 && lane == 0) {
        a.status[s] = served ? (int32_t)need : old == kBadRow ? -1 : -2;
        if (served) a.lens[s] = old + (a.grow ? a.grow[s] : 0);
    }
    if (!served) return;
    const u64 held = held_pages(child, (uint32_t)old, a.page_tokens), total = held + need;
    const int32_t *from = a.table + (child ? (u64)a.parent[s] : s) * a.stride;
    int32_t *to = a.table + s * a.stride;
    const u64 first = chunk * kEntryChunk, end = chunk + 1 == chunks ? total : min(total, first + kEntryChunk);
    for (u64 j = (child ? first : max(first, held)) + lane; j < end; j += 32) {
        const int32_t e = j < held ? from[j] : w.fresh[begin + (j - held)];
        to[j] = e;
        if (j < held && page_of(e) < a.pages) atomicAdd(a.refs + e, 1);
    }
}

// ---------------------------------------------------------------------------
// free
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPThreads)
free_kernel(int32_t *table, u64 stride, u64 rows, u64 width, int32_t *lens, int32_t *refs, u64 pages,
            uint32_t page_tokens, const int32_t *release, int32_t *freed, PagesWs w) {
    constexpr int U = 4;
    __shared__ u64 s_warp[kPWarps];
    const int lane = threadIdx.x & 31;
    u64 gone = 0;
    for (u64 s = (u64)blockIdx.x * kPWarps + (threadIdx.x >> 5); s < rows; s += (u64)gridDim.x * kPWarps) {
        const int32_t gone_row = release[s], len = lens[s];  // on their way together
        if (gone_row == 0) continue;
        const u64 n = len > 0 ? min((u64)pages_for((uint32_t)len, page_tokens), width) : 0ull;
        int32_t *row = table + s * stride;
        for (u64 j = lane; j < n; j += 32 * U) {  // U entries and their counts on the way together
            int32_t e[U], was[U];
#pragma unroll
            for (int u = 0; u < U; ++u) e[u] = j + 32 * u < n ? row[j + 32 * u] : -1;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                was[u] = page_of(e[u]) < pages ? atomicSub(refs + e[u], 1) : 0;
                if (j + 32 * u < n) row[j + 32 * u] = -1;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) gone += was[u] == 1;
        }
        __syncwarp();
        if (lane == 0) lens[s] = 0;
    }
    u64 total;
    block_exclusive(gone, s_warp, &total);
    if (threadIdx.x == 0) w.freed[blockIdx.x] = (uint32_t)total;
    if (!last_block(w.hdr)) return;
    u64 mine = 0;
    for (u64 b = threadIdx.x; b < gridDim.x; b += kPThreads) mine += ld_relaxed_u32(w.freed + b);
    block_exclusive(mine, s_warp, &total);
    if (threadIdx.x == 0 && freed) *freed = (int32_t)total;
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
struct CompactArgs {
    int32_t *table;
    u64 stride, rows, width;
    const int32_t *lens;
    int32_t *refs;
    u64 pages;
    uint32_t page_tokens;
    int32_t *live, *remap;
};

// The tile's free pages below `live` are holes, its live ones from there on
// movers; `rank` counts the live pages before this thread's, `stay` those
// below `live`.
__device__ __forceinline__ void place_moves(const CompactArgs &a, const PagesWs &w, u64 tile, unsigned int live_mask,
                                            u64 rank, u64 live, u64 stay) {
    const u64 first = tile * kRefTile + (u64)threadIdx.x * kPerThread;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
        const u64 i = first + j;
        if (i >= a.pages) break;
        const bool is_live = live_mask >> j & 1u;
        if (i < live && !is_live) w.holes[i - rank] = (int32_t)i;
        if (i >= live && is_live) {
            w.movers[rank - stay] = (int32_t)i;
            w.rank[i] = (int32_t)(rank - stay);
        }
        if (a.remap && !(i >= live && is_live)) a.remap[i] = is_live ? (int32_t)i : -1;
        rank += is_live;
    }
}

// How many of the live pages lie below page `live`, given the tile that holds
// it (`rank`: those before this thread's refs).
__device__ __forceinline__ void count_below(u64 tile, unsigned int live_mask, u64 rank, u64 live, u64 *below) {
    const u64 first = tile * kRefTile + (u64)threadIdx.x * kPerThread;
    if (first <= live && live < first + kPerThread)
        *below = rank + __popc(live_mask & ((1u << (unsigned int)(live - first)) - 1u));
}

template <bool ONE>
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(CompactArgs a, PagesWs w) {
    __shared__ u64 s_warp[kPlanWarps];
    cudaTriggerProgrammaticLaunchCompletion();  // the next launch may come to its wait
    __shared__ u64 s_below;
    unsigned int mask = ~free_mask(a.refs, blockIdx.x, a.pages) & page_mask(blockIdx.x, a.pages);
    u64 total, tile = blockIdx.x;
    u64 rank = block_exclusive(__popc(mask), s_warp, &total);
    u64 live = total;
    if (!ONE) {
        if (threadIdx.x == 0) w.tile_base[blockIdx.x] = total;
        if (!last_block(w.hdr)) return;
        live = scan_by_block(
            gridDim.x, s_warp, [&](u64 t) { return ld_relaxed(w.tile_base + t); },
            [&](u64 t, u64 base, u64) { w.tile_base[t] = base; });
        __syncthreads();
        tile = live / kRefTile;
        if (live < a.pages) {
            mask = ~free_mask(a.refs, tile, a.pages) & page_mask(tile, a.pages);
            rank = w.tile_base[tile] + block_exclusive(__popc(mask), s_warp, &total);
        }
    }
    if (threadIdx.x == 0) s_below = live;
    __syncthreads();
    if (live < a.pages) count_below(tile, mask, rank, live, &s_below);
    __syncthreads();
    if (threadIdx.x == 0) {
        w.ctrl->live = live;
        w.ctrl->moved = live - s_below;
        if (a.live) *a.live = (int32_t)live;
    }
    if (ONE) place_moves(a, w, 0, mask, rank, live, s_below);
}

__global__ void __launch_bounds__(kPlanThreads) compact_place_kernel(CompactArgs a, PagesWs w) {
    __shared__ u64 s_warp[kPlanWarps];
    cudaTriggerProgrammaticLaunchCompletion();  // the next launch may come to its wait
    cudaGridDependencySynchronize();  // what the launch before wrote
    const u64 live = w.ctrl->live, stay = live - w.ctrl->moved;
    const unsigned int mask = ~free_mask(a.refs, blockIdx.x, a.pages) & page_mask(blockIdx.x, a.pages);
    u64 total;
    const u64 rank = w.tile_base[blockIdx.x] + block_exclusive(__popc(mask), s_warp, &total);
    place_moves(a, w, blockIdx.x, mask, rank, live, stay);
}

__global__ void __launch_bounds__(kPThreads)
compact_act_kernel(CompactArgs a, PagesWs w, Pool pool, unsigned int row_blocks, unsigned int ref_blocks) {
    cudaGridDependencySynchronize();  // what the launch before wrote
    const u64 live = w.ctrl->live, moved = w.ctrl->moved;
    const int lane = threadIdx.x & 31;
    if (blockIdx.x < row_blocks) {  // table entries
        for (u64 s = (u64)blockIdx.x * kPWarps + (threadIdx.x >> 5); s < a.rows; s += (u64)row_blocks * kPWarps) {
            const int32_t len = a.lens[s];
            const u64 n = len > 0 ? min((u64)pages_for((uint32_t)len, a.page_tokens), a.width) : 0ull;
            int32_t *row = a.table + s * a.stride;
            for (u64 j = lane; j < n; j += 32) {
                const u64 e = page_of(row[j]);
                if (e < live || e >= a.pages) continue;
                const u64 k = page_of(w.rank[e]);  // unset for a free page: checked against movers
                if (k < moved && w.movers[k] == (int32_t)e) row[j] = w.holes[k];
            }
        }
        return;
    }
    if (blockIdx.x < row_blocks + ref_blocks) {
        const u64 step = (u64)ref_blocks * kPThreads;
        for (u64 k = (u64)(blockIdx.x - row_blocks) * kPThreads + threadIdx.x; k < moved; k += step) {
            const int32_t from = w.movers[k], to = w.holes[k];
            a.refs[to] = a.refs[from];
            a.refs[from] = 0;
            if (a.remap) a.remap[from] = to;
        }
        return;
    }
    copy_pages(pool, moved, blockIdx.x - row_blocks - ref_blocks, gridDim.x - row_blocks - ref_blocks,
               [&](u64 k, u64 *src, u64 *dst) {
                   *src = (u64)w.movers[k];
                   *dst = (u64)w.holes[k];
                   return true;
               });
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static std::mutex g_pages_mu;
static int g_pages_sms[64];

static int sm_count(int *sms) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return U32SCAN_ECUDA;
    std::lock_guard<std::mutex> lock(g_pages_mu);
    if (g_pages_sms[dev] == 0 &&
        cudaDeviceGetAttribute(&g_pages_sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return U32SCAN_ECUDA;
    *sms = g_pages_sms[dev];
    return U32SCAN_OK;
}

static int launched() { return cudaGetLastError() == cudaSuccess ? U32SCAN_OK : U32SCAN_ECUDA; }

// A launch that may be set up while the one before it in the stream (of the
// same call) still runs, and waits for its end before it reads anything
// (forking 16 rows 8.2 and 7.7 us, of 2048 rows 16.8 and 16.0).
template <typename... P, typename... A>
static void launch_next(void (*kernel)(P...), unsigned int grid, int threads, cudaStream_t s, A... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned int)threads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kernel, P(args)...);  // launched() sees its error
}

static bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) != 0; }

// A pool's arguments are sound; an absent pool is one without planes.
static bool pool_ok(const u32scan_page_pool *pool, size_t pages, Pool *out) {
    *out = Pool{nullptr, 0, pages, 0, 0};
    if (pool == nullptr || pool->n_planes == 0 || pool->page_bytes == 0) return pool == nullptr || pool->pages == pages;
    if (pool->pages != pages || pool->planes == nullptr || (reinterpret_cast<uintptr_t>(pool->planes) & 7))
        return false;
    if (pool->n_planes >= (1u << 20) || pool->page_bytes >= (1ull << 40) || pool->page_stride < pool->page_bytes ||
        pool->page_stride >= (1ull << 40))
        return false;
    *out = Pool{reinterpret_cast<const u64 *>(pool->planes), pool->n_planes, pages, pool->page_bytes,
                pool->page_stride};
    return true;
}

static bool table_ok(const int32_t *table, size_t stride, size_t rows, size_t width, const int32_t *lens,
                     const int32_t *refs, size_t pages, size_t page_tokens) {
    if (rows >= (1ull << 31) || width >= (1ull << 31) || pages >= (1ull << 31)) return false;
    if (page_tokens == 0 || page_tokens >= (1ull << 31) || stride < width || stride >= (1ull << 31)) return false;
    if (rows > 0 && (lens == nullptr || (width > 0 && table == nullptr))) return false;
    if (pages > 0 && refs == nullptr) return false;
    return !misaligned(table) && !misaligned(lens) && !misaligned(refs);
}

static bool ws_ok(const void *ws, size_t ws_bytes, size_t pages, size_t rows) {
    return ws != nullptr && !(reinterpret_cast<uintptr_t>(ws) & 255) &&
           ws_bytes >= pages_workspace_bytes((u64)pages + rows);
}

// Blocks for `units` copy units: one a unit up to 128 an SM (8 at a time; the
// rest are handed out as those finish, which keeps the SMs level: 509 pages of
// 64 x 32 KiB take 342, 312, 311 us with 8, 64, 128 an SM, and 314 would at the
// rate of a plain copy of 2 GB; a packing whose number of pages only the device knows
// 179, 167, 165, and 177 with 512).
static unsigned int copy_grid(u64 units, int sms) {
    const u64 full = (u64)sms * 128;
    return (unsigned int)(units < full ? (units ? units : 1) : full);
}

static u64 units_per_pair(const Pool &p) { return p.n_planes * ((p.page_bytes + kCopyUnit - 1) / kCopyUnit); }

}  // namespace u32scan

using namespace u32scan;

extern "C" int pages_copy(const u32scan_page_pool *pool, const int32_t *src, const int32_t *dst, size_t n,
                          const int32_t *count, u32scan_stream_t stream) {
    Pool p;
    if (pool == nullptr || pool->pages >= (1ull << 31) || !pool_ok(pool, pool->pages, &p)) return U32SCAN_EINVAL;
    if (n >= (1ull << 31) || (n > 0 && (src == nullptr || dst == nullptr))) return U32SCAN_EINVAL;
    if (misaligned(src) || misaligned(dst) || misaligned(count)) return U32SCAN_EINVAL;
    if (n == 0 || p.n_planes == 0 || p.pages == 0) return U32SCAN_OK;
    int sms = 0;
    const int rc = sm_count(&sms);
    if (rc != U32SCAN_OK) return rc;
    pages_copy_kernel<<<copy_grid(n * units_per_pair(p), sms), kPThreads, 0, (cudaStream_t)stream>>>(p, src, dst, n,
                                                                                                   count);
    return launched();
}

extern "C" int pages_fork(int32_t *table, size_t table_stride, size_t rows, size_t width, int32_t *lens, int32_t *refs,
                          size_t pages, size_t page_tokens, const int32_t *parent, const int32_t *grow,
                          const u32scan_page_pool *pool, int32_t *status, int32_t *free_pages, void *ws,
                          size_t ws_bytes, u32scan_stream_t stream) {
    Pool p;
    if (!table_ok(table, table_stride, rows, width, lens, refs, pages, page_tokens) || !pool_ok(pool, pages, &p))
        return U32SCAN_EINVAL;
    if ((rows > 0 && status == nullptr) || misaligned(parent) || misaligned(grow) || misaligned(status) ||
        misaligned(free_pages))
        return U32SCAN_EINVAL;
    if (rows == 0 && free_pages == nullptr) return U32SCAN_OK;
    if (!ws_ok(ws, ws_bytes, pages, rows)) return U32SCAN_EWORKSPACE;
    int sms = 0;
    int rc = sm_count(&sms);
    if (rc != U32SCAN_OK) return rc;
    const cudaStream_t s = (cudaStream_t)stream;
    const ForkArgs a{table, table_stride, rows,   width, lens,   refs,
                     pages, (uint32_t)page_tokens, parent, grow, status, free_pages};
    const PagesWs w = carve(ws, pages, rows);
    const u64 tiles = ref_tiles(pages), chunks = parent && width ? (width + kEntryChunk - 1) / kEntryChunk : 1;
    const u64 row_blocks = (rows * chunks + kPWarps - 1) / kPWarps;
    const unsigned int data_blocks = parent && p.n_planes ? copy_grid(rows * units_per_pair(p), sms) : 0u;
    if (row_blocks + data_blocks >= (1ull << 31)) return U32SCAN_EINVAL;
    // One block plans a cache of one tile, and places too: the rows are planned by one block either
    // way, and a launch less is 3.6 us (4096 pages, with 16, 4096, 16384, 65535 rows that grow 5.4,
    // 10.4, 25.8, 86.7 us, and 9.0, 14.0, 29.4, 90.4 us in three launches).
    if (tiles <= 1) {
        fork_plan_kernel<true><<<1, kPlanThreads, 0, s>>>(a, w, tiles);
    } else {
        fork_plan_kernel<false><<<(unsigned int)tiles, kPlanThreads, 0, s>>>(a, w, tiles);
        launch_next(fork_place_kernel, (unsigned int)tiles, kPlanThreads, s, a, w);
    }
    if (row_blocks)
        launch_next(fork_act_kernel, (unsigned int)row_blocks + data_blocks, kPThreads, s, a, w, p,
                    (unsigned int)row_blocks, chunks);
    return launched();
}

extern "C" int pages_free(int32_t *table, size_t table_stride, size_t rows, size_t width, int32_t *lens, int32_t *refs,
                          size_t pages, size_t page_tokens, const int32_t *release, int32_t *freed, void *ws,
                          size_t ws_bytes, u32scan_stream_t stream) {
    if (!table_ok(table, table_stride, rows, width, lens, refs, pages, page_tokens)) return U32SCAN_EINVAL;
    if ((rows > 0 && release == nullptr) || misaligned(release) || misaligned(freed)) return U32SCAN_EINVAL;
    if (rows == 0 && freed == nullptr) return U32SCAN_OK;
    if (!ws_ok(ws, ws_bytes, pages, rows)) return U32SCAN_EWORKSPACE;
    int sms = 0;
    const int rc = sm_count(&sms);
    if (rc != U32SCAN_OK) return rc;
    const u64 want = (rows + kPWarps - 1) / kPWarps, full = (u64)sms * 8;
    const unsigned int grid = (unsigned int)(want < full ? (want ? want : 1) : full);
    free_kernel<<<grid, kPThreads, 0, (cudaStream_t)stream>>>(table, table_stride, rows, width, lens, refs, pages,
                                                              (uint32_t)page_tokens, release, freed,
                                                              carve(ws, pages, rows));
    return launched();
}

extern "C" int pages_compact(const u32scan_page_pool *pool, int32_t *table, size_t table_stride, size_t rows,
                             size_t width, const int32_t *lens, int32_t *refs, size_t pages, size_t page_tokens,
                             int32_t *live, int32_t *remap, void *ws, size_t ws_bytes, u32scan_stream_t stream) {
    Pool p;
    if (!table_ok(table, table_stride, rows, width, lens, refs, pages, page_tokens) || !pool_ok(pool, pages, &p))
        return U32SCAN_EINVAL;
    if (misaligned(live) || misaligned(remap)) return U32SCAN_EINVAL;
    const cudaStream_t s = (cudaStream_t)stream;
    if (pages == 0) {
        if (live && cudaMemsetAsync(live, 0, 4, s) != cudaSuccess) return U32SCAN_ECUDA;
        return U32SCAN_OK;
    }
    if (!ws_ok(ws, ws_bytes, pages, rows)) return U32SCAN_EWORKSPACE;
    int sms = 0;
    const int rc = sm_count(&sms);
    if (rc != U32SCAN_OK) return rc;
    const CompactArgs a{table, table_stride, rows, width, lens, refs, pages, (uint32_t)page_tokens, live, remap};
    const PagesWs w = carve(ws, pages, rows);
    const unsigned int tiles = (unsigned int)ref_tiles(pages);
    if (tiles == 1) {
        compact_plan_kernel<true><<<1, kPlanThreads, 0, s>>>(a, w);
    } else {
        compact_plan_kernel<false><<<tiles, kPlanThreads, 0, s>>>(a, w);
        launch_next(compact_place_kernel, tiles, kPlanThreads, s, a, w);
    }
    const u64 want = (rows + kPWarps - 1) / kPWarps, ref_want = (pages / 2 + kPThreads - 1) / kPThreads;
    const unsigned int row_blocks = (unsigned int)(want < (u64)sms ? want : (u64)sms);
    const unsigned int ref_blocks = (unsigned int)(ref_want < (u64)sms ? (ref_want ? ref_want : 1) : (u64)sms);
    const unsigned int data_blocks = p.n_planes ? copy_grid(pages / 2 * units_per_pair(p), sms) : 0u;
    launch_next(compact_act_kernel, row_blocks + ref_blocks + data_blocks, kPThreads, s, a, w, p, row_blocks,
                ref_blocks);
    return launched();
}
