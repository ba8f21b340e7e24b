// launch.cuh -- what the host side of several kernels shares: the device's SMs,
// a launch that overlaps the one before it, whether two arrays share memory.
#pragma once

#include <algorithm>
#include <cstdint>
#include <mutex>
#include <cuda_runtime.h>

#include "u32scan.h"

namespace u32scan {

static std::mutex g_sms_mu;
static int g_sms[64];

static int sm_count(int *sms) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return U32SCAN_ECUDA;
    std::lock_guard<std::mutex> lock(g_sms_mu);
    if (g_sms[dev] == 0 &&
        cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return U32SCAN_ECUDA;
    *sms = g_sms[dev];
    return U32SCAN_OK;
}

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

// Runs of bytes at every sum of multiples of up to three strides (a count of 0: none, of 1: no stride).
struct Strided {
    const void *at;
    uint64_t run, count[3], stride[3];  // bytes
};

// Whether two of them share a byte. With c the distance from a's first run to
// b's, that is whether some sum c + k_0 s_0 + k_1 s_1 + .. lies in (-b.run,
// a.run), k_i from 0 to b's counts or from minus a's to 0 (of a stride that both have,
// the two ranges' sum). Axis by axis, the widest first, only those multiples are tried
// that the narrower ones can bring back into reach: few where the strides are
// nested, as those of views of one tensor are.
static inline bool share_memory(const Strided &a, const Strided &b) {
    typedef __int128 wide;
    struct Axis {
        wide stride, lo, hi;
    } axis[6];
    int n = 0;
    for (const Strided *x : {&a, &b}) {
        if (x->run == 0) return false;
        for (int i = 0; i < 3; ++i) {
            if (x->count[i] == 0) return false;
            if (x->count[i] == 1 || x->stride[i] == 0) continue;
            int at = 0;
            while (at < n && axis[at].stride != (wide)x->stride[i]) ++at;
            if (at == n) axis[n++] = Axis{(wide)x->stride[i], 0, 0};
            (x == &a ? axis[at].lo : axis[at].hi) += (x == &a ? -1 : 1) * (wide)(x->count[i] - 1);
        }
    }
    std::sort(axis, axis + n, [](const Axis &x, const Axis &y) { return x.stride > y.stride; });
    wide lo[7], hi[7];  // what the axes from i on add
    lo[n] = hi[n] = 0;
    for (int i = n - 1; i >= 0; --i) lo[i] = lo[i + 1] + axis[i].lo * axis[i].stride, hi[i] = hi[i + 1] + axis[i].hi * axis[i].stride;
    struct Search {
        const Axis *axis;
        const wide *lo, *hi;
        wide above, below;  // the sums sought lie between these two
        int n;
        bool from(int i, wide c) const {
            if (c + lo[i] >= below || c + hi[i] <= above) return false;
            if (i == n) return true;
            const wide s = axis[i].stride, least = above - c - hi[i + 1], most = below - c - lo[i + 1];  // k s between them
            const wide k0 = (least >= 0 ? least / s : -((-least + s - 1) / s)) + 1;
            const wide k1 = (most > 0 ? (most + s - 1) / s : -(-most / s)) - 1;
            for (wide k = std::max(k0, axis[i].lo); k <= std::min(k1, axis[i].hi); ++k)
                if (from(i + 1, c + k * s)) return true;
            return false;
        }
    } const search{axis, lo, hi, -(wide)b.run, (wide)a.run, n};
    return search.from(0, (wide)reinterpret_cast<uintptr_t>(b.at) - (wide)reinterpret_cast<uintptr_t>(a.at));
}

}  // namespace u32scan
