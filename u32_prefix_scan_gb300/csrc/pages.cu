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
// Reduce, then scan: the count kernel reads refs once in tiles and its last
// block scans the tiles' counts and the rows' needs, so the second kernel
// knows every base without waiting on other blocks. refs is read twice, the
// second time from L2 (4 MB at a million pages).
#include <cstdint>
#include <mutex>
#include <cuda_runtime.h>

#include "internal.cuh"

namespace u32scan {

typedef unsigned long long u64;

constexpr int kPThreads = 256;
constexpr int kPWarps = kPThreads / 32;
constexpr int kRefTile = 4096;      // refs counted by one block
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
    u64 jobs;          // fork: rows whose partly filled page is copied
    u64 live;          // compact: L
    u64 moved;         // compact: pages that move
    u64 pad[28];
};
static_assert(sizeof(PagesCtrl) == 256, "one line group");

struct PagesWs {
    WsHeader *hdr;
    PagesCtrl *ctrl;
    u64 *tile_base;   // [tiles] counts, then exclusive bases
    u64 *ends;        // fork: [rows]
    int32_t *old_len; // fork: [rows] length before the call (of the parent, for a child)
    int32_t *jobs;    // fork: [rows]
    uint32_t *freed;  // free: [blocks]
    int32_t *holes, *movers, *rank;  // compact: [pages] each
};

static u64 ref_tiles(u64 pages) { return (pages + kRefTile - 1) / kRefTile; }

// n = pages + rows: 8 bytes a tile and at most 16 bytes a row or 12 a page.
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
// call it; s_warp holds kPWarps values).
__device__ __forceinline__ u64 block_exclusive(u64 x, u64 *s_warp, u64 *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const u64 inc = warp_inclusive_u64(x, lane);
    __syncthreads();
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    u64 base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPWarps; ++w) {
        if (w < warp) base += s_warp[w];
        all += s_warp[w];
    }
    *total = all;
    return base + inc - x;
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

// a[i] <- a[0] + .. + a[i] (INCLUSIVE) or a[i-1], by one block; returns the
// total. The values are read past L1: other blocks wrote them.
template <bool INCLUSIVE>
__device__ __forceinline__ u64 scan_by_block(u64 *a, u64 n, u64 *s_warp) {
    u64 carry = 0;
    for (u64 i0 = 0; i0 < n; i0 += kPThreads) {
        const u64 i = i0 + threadIdx.x;
        const u64 x = i < n ? ld_relaxed(a + i) : 0ull;
        u64 total;
        const u64 ex = block_exclusive(x, s_warp, &total);
        if (i < n) a[i] = carry + ex + (INCLUSIVE ? x : 0ull);
        carry += total;
    }
    return carry;
}

// Number of refs in [begin, end) that are zero (ZERO) or not, by one block.
template <bool ZERO>
__device__ __forceinline__ u64 count_refs(const int32_t *refs, u64 begin, u64 end, u64 *s_warp) {
    u64 c = 0;
    for (u64 i = begin + threadIdx.x; i < end; i += kPThreads) c += (refs[i] == 0) == ZERO;
    u64 total;
    block_exclusive(c, s_warp, &total);
    return total;
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
    u64 page_tokens;
    const int32_t *parent, *grow;
    int32_t *status, *free_pages;
};

constexpr int32_t kBadRow = -1;  // old_len of a row whose arguments are refused

__device__ __forceinline__ u64 pages_for(u64 tokens, u64 page_tokens) {
    return (tokens + page_tokens - 1) / page_tokens;
}

// Pages row s holds before its fresh ones: a child's shared full pages, or
// the row's own.
__device__ __forceinline__ u64 held_pages(bool child, u64 old_len, u64 page_tokens) {
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
    const u64 total = (u64)old + (u64)g;
    if (total > 0x7fffffffull || pages_for(total, a.page_tokens) > a.width) return 0;
    *old_len = old;
    return pages_for(total, a.page_tokens) - held_pages(child, (u64)old, a.page_tokens);
}

__global__ void __launch_bounds__(kPThreads) fork_count_kernel(ForkArgs a, PagesWs w, u64 tiles) {
    __shared__ u64 s_warp[kPWarps];
    if (blockIdx.x < tiles) {
        const u64 begin = (u64)blockIdx.x * kRefTile;
        const u64 c = count_refs<true>(a.refs, begin, min(begin + kRefTile, a.pages), s_warp);
        if (threadIdx.x == 0) w.tile_base[blockIdx.x] = c;
    } else {
        const u64 s = (blockIdx.x - tiles) * kPThreads + threadIdx.x;
        if (s < a.rows) {
            int32_t old;
            w.ends[s] = row_need(a, s, &old);
            w.old_len[s] = old;
        }
    }
    if (!last_block(w.hdr)) return;
    const u64 free_pages = scan_by_block<false>(w.tile_base, tiles, s_warp);
    scan_by_block<true>(w.ends, a.rows, s_warp);
    // the children whose parent's last page is partly filled, in row order
    u64 jobs = 0;
    for (u64 s0 = 0; s0 < a.rows; s0 += kPThreads) {
        const u64 s = s0 + threadIdx.x;
        bool job = false;
        if (s < a.rows && is_child(a, s)) {
            const int32_t old = (int32_t)ld_relaxed_u32(reinterpret_cast<const unsigned int *>(w.old_len + s));
            job = old > 0 && (u64)old % a.page_tokens != 0;
        }
        u64 total;
        const u64 at = jobs + block_exclusive(job ? 1ull : 0ull, s_warp, &total);
        if (job) w.jobs[at] = (int32_t)s;
        jobs += total;
    }
    if (threadIdx.x == 0) {
        w.ctrl->free_pages = free_pages;
        w.ctrl->jobs = jobs;
    }
}

// Row s gets all it asks for.
__device__ __forceinline__ bool row_served(const PagesWs &w, u64 s, u64 free_pages) {
    if (w.old_len[s] == kBadRow) return false;
    const u64 end = w.ends[s], begin = s ? w.ends[s - 1] : 0ull;
    return end == begin || end <= free_pages;
}

// The number of ends at or below x.
__device__ __forceinline__ u64 ends_upto(const u64 *ends, u64 rows, u64 x) {
    u64 lo = 0, hi = rows;
    while (lo < hi) {
        const u64 mid = (lo + hi) / 2;
        if (ends[mid] <= x) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPThreads) fork_assign_kernel(ForkArgs a, PagesWs w, u64 tiles, u64 chunks) {
    __shared__ u64 s_warp[kPWarps];
    const u64 free_pages = w.ctrl->free_pages;
    const u64 asked = a.rows ? w.ends[a.rows - 1] : 0ull;
    if (blockIdx.x < tiles) {  // hand out this tile's free pages
        u64 rank = w.tile_base[blockIdx.x];
        const u64 begin = (u64)blockIdx.x * kRefTile, end = min(begin + kRefTile, a.pages);
        for (u64 i0 = begin; i0 < end && rank < asked; i0 += kPThreads) {
            const u64 i = i0 + threadIdx.x;
            const bool is_free = i < end && a.refs[i] == 0;
            u64 total;
            const u64 f = rank + block_exclusive(is_free ? 1ull : 0ull, s_warp, &total);
            rank += total;
            if (!is_free || f >= asked) continue;
            const u64 s = ends_upto(w.ends, a.rows, f);  // the row with ends[s-1] <= f < ends[s]
            if (w.ends[s] > free_pages) continue;        // it cannot have all its pages: it takes none
            const u64 first = s ? w.ends[s - 1] : 0ull;
            const u64 slot = held_pages(is_child(a, s), (u64)w.old_len[s], a.page_tokens) + (f - first);
            a.table[s * a.stride + slot] = (int32_t)i;
            a.refs[i] = 1;
        }
        return;
    }
    const u64 item = (blockIdx.x - tiles) * kPWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const u64 s = item / chunks, chunk = item - s * chunks;
    if (item == 0 && lane == 0 && a.free_pages) {  // what the served rows leave
        const u64 fit = ends_upto(w.ends, a.rows, free_pages);
        *a.free_pages = (int32_t)(free_pages - (fit ? w.ends[fit - 1] : 0ull));
    }
    if (s >= a.rows) return;
    const bool served = row_served(w, s, free_pages);
    const bool child = is_child(a, s);
    if (chunk == 0 && lane == 0) {
        const u64 need = w.ends[s] - (s ? w.ends[s - 1] : 0ull);
        a.status[s] = served ? (int32_t)need : w.old_len[s] == kBadRow ? -1 : -2;
        if (served) a.lens[s] = w.old_len[s] + (a.grow ? a.grow[s] : 0);
    }
    if (!served || !child) return;
    const u64 shared = (u64)w.old_len[s] / a.page_tokens;
    const int32_t *from = a.table + (u64)a.parent[s] * a.stride;
    int32_t *to = a.table + s * a.stride;
    for (u64 j = chunk * kEntryChunk + lane; j < min(shared, (chunk + 1) * kEntryChunk); j += 32) {
        const int32_t e = from[j];
        to[j] = e;
        if (page_of(e) < a.pages) atomicAdd(a.refs + e, 1);
    }
}

__global__ void __launch_bounds__(kPThreads) fork_copy_kernel(ForkArgs a, PagesWs w, Pool pool) {
    const u64 free_pages = w.ctrl->free_pages;
    copy_pages(pool, w.ctrl->jobs, blockIdx.x, gridDim.x, [&](u64 k, u64 *src, u64 *dst) {
        const u64 s = (u64)w.jobs[k];
        if (!row_served(w, s, free_pages)) return false;
        const u64 slot = (u64)w.old_len[s] / a.page_tokens;
        *src = page_of(a.table[(u64)a.parent[s] * a.stride + slot]);
        *dst = page_of(a.table[s * a.stride + slot]);
        return true;
    });
}

// ---------------------------------------------------------------------------
// free
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPThreads)
free_kernel(int32_t *table, u64 stride, u64 rows, u64 width, int32_t *lens, int32_t *refs, u64 pages, u64 page_tokens,
            const int32_t *release, int32_t *freed, PagesWs w) {
    __shared__ u64 s_warp[kPWarps];
    const int lane = threadIdx.x & 31;
    u64 gone = 0;
    for (u64 s = (u64)blockIdx.x * kPWarps + (threadIdx.x >> 5); s < rows; s += (u64)gridDim.x * kPWarps) {
        if (release[s] == 0) continue;
        const int32_t len = lens[s];
        const u64 n = len > 0 ? min(pages_for((u64)len, page_tokens), width) : 0ull;
        int32_t *row = table + s * stride;
        for (u64 j = lane; j < n; j += 32) {
            const int32_t e = row[j];
            row[j] = -1;
            if (page_of(e) < pages && atomicSub(refs + e, 1) == 1) ++gone;
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
    u64 pages, page_tokens;
    int32_t *live, *remap;
};

__global__ void __launch_bounds__(kPThreads) compact_count_kernel(CompactArgs a, PagesWs w) {
    __shared__ u64 s_warp[kPWarps];
    const u64 begin = (u64)blockIdx.x * kRefTile;
    const u64 c = count_refs<false>(a.refs, begin, min(begin + kRefTile, a.pages), s_warp);
    if (threadIdx.x == 0) w.tile_base[blockIdx.x] = c;
    if (!last_block(w.hdr)) return;
    const u64 live = scan_by_block<false>(w.tile_base, gridDim.x, s_warp);
    __syncthreads();
    u64 below = live;  // live pages below `live`: those that stay
    if (live < a.pages) {
        const u64 tile = live / kRefTile;
        below = w.tile_base[tile] + count_refs<false>(a.refs, tile * kRefTile, live, s_warp);
    }
    if (threadIdx.x == 0) {
        w.ctrl->live = live;
        w.ctrl->moved = live - below;
        if (a.live) *a.live = (int32_t)live;
    }
}

__global__ void __launch_bounds__(kPThreads) compact_pair_kernel(CompactArgs a, PagesWs w) {
    __shared__ u64 s_warp[kPWarps];
    const u64 live = w.ctrl->live, stay = live - w.ctrl->moved;
    u64 rank = w.tile_base[blockIdx.x];
    const u64 begin = (u64)blockIdx.x * kRefTile, end = min(begin + kRefTile, a.pages);
    for (u64 i0 = begin; i0 < end; i0 += kPThreads) {
        const u64 i = i0 + threadIdx.x;
        const bool is_live = i < end && a.refs[i] != 0;
        u64 total;
        const u64 r = rank + block_exclusive(is_live ? 1ull : 0ull, s_warp, &total);
        rank += total;
        if (i >= end) continue;
        if (i < live && !is_live) w.holes[i - r] = (int32_t)i;
        if (i >= live && is_live) {
            w.movers[r - stay] = (int32_t)i;
            w.rank[i] = (int32_t)(r - stay);
        }
        if (a.remap && !(i >= live && is_live)) a.remap[i] = is_live ? (int32_t)i : -1;
    }
}

__global__ void __launch_bounds__(kPThreads)
compact_move_kernel(CompactArgs a, PagesWs w, Pool pool, unsigned int row_blocks, unsigned int ref_blocks) {
    const u64 live = w.ctrl->live, moved = w.ctrl->moved;
    const int lane = threadIdx.x & 31;
    if (blockIdx.x < row_blocks) {  // table entries
        for (u64 s = (u64)blockIdx.x * kPWarps + (threadIdx.x >> 5); s < a.rows; s += (u64)row_blocks * kPWarps) {
            const int32_t len = a.lens[s];
            const u64 n = len > 0 ? min(pages_for((u64)len, a.page_tokens), a.width) : 0ull;
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

static bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) != 0; }

// A pool's arguments are sound; an absent pool is one without planes.
static bool pool_ok(const u32scan_page_pool *pool, size_t pages, Pool *out) {
    *out = Pool{nullptr, 0, pages, 0, 0};
    if (pool == nullptr || pool->n_planes == 0 || pool->page_bytes == 0) return pool == nullptr || pool->pages == pages;
    if (pool->pages != pages || pool->planes == nullptr || (reinterpret_cast<uintptr_t>(pool->planes) & 7)) return false;
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
    if ((rows > 0 && (lens == nullptr || (width > 0 && table == nullptr))) || (pages > 0 && refs == nullptr)) return false;
    return !misaligned(table) && !misaligned(lens) && !misaligned(refs);
}

static bool ws_ok(const void *ws, size_t ws_bytes, size_t pages, size_t rows) {
    return ws != nullptr && !(reinterpret_cast<uintptr_t>(ws) & 255) &&
           ws_bytes >= pages_workspace_bytes((u64)pages + rows);
}

// Blocks for `units` copy units: enough to fill the GPU, no more than units.
static unsigned int copy_grid(u64 units, int sms) {
    const u64 full = (u64)sms * 8;
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
    const ForkArgs a{table, table_stride, rows, width, lens, refs, pages, page_tokens, parent, grow, status, free_pages};
    const PagesWs w = carve(ws, pages, rows);
    const u64 tiles = ref_tiles(pages), row_blocks = (rows + kPThreads - 1) / kPThreads;
    const u64 chunks = parent ? (width + kEntryChunk - 1) / kEntryChunk + (width == 0) : 1;
    const u64 warps = (rows ? rows : 1) * chunks, assign_blocks = (warps + kPWarps - 1) / kPWarps;
    if (tiles + assign_blocks >= (1ull << 31)) return U32SCAN_EINVAL;
    fork_count_kernel<<<(unsigned int)(tiles + row_blocks + (tiles + row_blocks == 0)), kPThreads, 0, s>>>(a, w, tiles);
    fork_assign_kernel<<<(unsigned int)(tiles + assign_blocks), kPThreads, 0, s>>>(a, w, tiles, chunks);
    if (parent && p.n_planes)
        fork_copy_kernel<<<copy_grid(rows * units_per_pair(p), sms), kPThreads, 0, s>>>(a, w, p);
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
                                                              page_tokens, release, freed, carve(ws, pages, rows));
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
    const CompactArgs a{table, table_stride, rows, width, lens, refs, pages, page_tokens, live, remap};
    const PagesWs w = carve(ws, pages, rows);
    const unsigned int tiles = (unsigned int)ref_tiles(pages);
    compact_count_kernel<<<tiles, kPThreads, 0, s>>>(a, w);
    compact_pair_kernel<<<tiles, kPThreads, 0, s>>>(a, w);
    const u64 want = (rows + kPWarps - 1) / kPWarps, ref_want = (pages / 2 + kPThreads - 1) / kPThreads;
    const unsigned int row_blocks = (unsigned int)(want < (u64)sms ? want : (u64)sms);
    const unsigned int ref_blocks = (unsigned int)(ref_want < (u64)sms ? (ref_want ? ref_want : 1) : (u64)sms);
    const unsigned int data_blocks = p.n_planes ? copy_grid(pages / 2 * units_per_pair(p), sms) : 0u;
    compact_move_kernel<<<row_blocks + ref_blocks + data_blocks, kPThreads, 0, s>>>(a, w, p, row_blocks, ref_blocks);
    return launched();
}
