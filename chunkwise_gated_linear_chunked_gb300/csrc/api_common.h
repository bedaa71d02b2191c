// Host-side helpers shared by the translation units that implement libgla's C ABI: workspace alignment,
// pointer and overlap checks, the SM count and the per-thread measurement hook.
#pragma once

#include <cstddef>
#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>

namespace gla {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline int sm_count()
{
    static std::mutex mu;
    static int cache[128] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128)
        return 148;
    std::lock_guard<std::mutex> lock(mu);
    if (!cache[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            n = 148;
        cache[dev] = n;
    }
    return cache[dev];
}

// Per-thread measurement hook state (gla_profile_events).
struct Profile {
    cudaEvent_t *events = nullptr;
    int n_events = 0;
    int *ids = nullptr;
    int launches = 0;
};
inline thread_local Profile g_prof;

enum KernelId {
    K_PLAN = 1, K_STATE_FFMA = 2, K_SCAN = 3, K_OUT_FFMA = 4, K_FUSED_TC = 7,
    K_BWD_SUMS = 8, K_BWD_SCAN = 9, K_BWD_GRADS = 10, K_BWD_DG = 11, K_TTT = 12, K_WY = 13,
    K_WY_TC = 14, K_BWD_SUMS_TC = 15, K_BWD_GRADS_TC = 16, K_TTT_TC = 17,
    K_SCAN_FWD = 18, K_SCAN_BWD = 19, K_SCAN_STEP = 20, K_GLA_STEP = 21, K_NORM_FWD = 22, K_NORM_QUANT = 23,
    K_NORM_BWD = 24, K_NORM_DW = 25, K_SCAN_FWD_ROWS = 26, K_SCAN_BWD_ROWS = 27,
    K_DELTA_COLS = 28, K_DELTA_COLS_BACK = 29, K_DELTA_ROWS = 30, K_DELTA_ROWS_BACK = 31, K_DELTA_JOIN = 32, K_DELTA_GATES = 33,
    K_DELTA_STEP = 34, K_DELTA_PREP = 35, K_DELTA_CHAIN = 36, K_DELTA_CHAIN_BACK = 37, K_DELTA_GRADS = 38, K_GN_TOKENS = 39,
    K_GN_SUMS = 40, K_GN_APPLY = 41, K_GN_TOKENS_BACK = 42, K_GN_GRAD_SUMS = 43, K_GN_GRAD = 44, K_GN_DW = 45
};

// Launch one kernel through `fn`, bracketed by the profiling events when they are armed.
template <typename Fn>
cudaError_t profiled(int id, cudaStream_t s, Fn fn)
{
    Profile &p = g_prof;
    const int i = p.launches++;
    const bool rec = p.events && 2 * i + 1 < p.n_events;
    if (rec && cudaEventRecord(p.events[2 * i], s) != cudaSuccess)
        return cudaErrorUnknown;
    cudaError_t e = fn();
    if (e != cudaSuccess)
        return e;
    if (rec) {
        if (p.ids)
            p.ids[i] = id;
        return cudaEventRecord(p.events[2 * i + 1], s);
    }
    return cudaSuccess;
}

inline bool misaligned(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u); }

struct Range {
    uintptr_t lo, hi;
};
inline Range range_of(const void *p, size_t bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + bytes};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

}  // namespace gla
