// Vector-state gated linear recurrence: forward and backward.
#include "gla_internal.h"
#include "layer_internal.h"

namespace gla {
namespace {

// Rows [begin, end) of sequence n; false (and a status) where the offsets are bad.
__device__ __forceinline__ bool sequence_rows(const ScanArgs &a, int n, long long &begin, long long &end)
{
    if (!a.cu) {
        begin = (long long)n * a.T;
        end = begin + a.T;
        return true;
    }
    begin = a.cu[n];
    end = a.cu[n + 1];
    const bool ok = begin >= 0 && end >= begin && end <= a.T && (n > 0 || begin == 0) && (n < a.N - 1 || end == a.T);
    if (!ok && threadIdx.x == 0)
        report(a.status, GLA_ERR_INVALID_ARG);
    return ok;
}

// One thread per channel, rows in order.
template <typename Tx, typename Tg, typename To>
__global__ void __launch_bounds__(128) scan_fwd_serial(ScanArgs a, int tiles)
{
    const int n = blockIdx.x / tiles, d = (blockIdx.x % tiles) * 128 + threadIdx.x;
    long long begin, end;
    if (!sequence_rows(a, n, begin, end) || d >= a.D)
        return;
    const Tx *x = static_cast<const Tx *>(a.x) + d;
    const Tg *g = static_cast<const Tg *>(a.g) + d;
    To *o = static_cast<To *>(a.h) + d;
    float h = a.h0 ? a.h0[(size_t)n * a.D + d] : 0.f;
#pragma unroll 8
    for (long long r = begin; r < end; ++r) {
        h = fmaf(expf(widen(g[r * a.ldg])), h, widen(x[r * a.ldx]));
        o[r * a.D] = narrow<To>(h);
    }
    if (a.ht)
        a.ht[(size_t)n * a.D + d] = h;
}

template <typename Tx, typename Tg, typename To>
__global__ void __launch_bounds__(128) scan_bwd_serial(ScanArgs a, int tiles)
{
    const int n = blockIdx.x / tiles, d = (blockIdx.x % tiles) * 128 + threadIdx.x;
    long long begin, end;
    if (!sequence_rows(a, n, begin, end) || d >= a.D)
        return;
    const Tg *g = static_cast<const Tg *>(a.g) + d;
    const To *h = static_cast<const To *>(a.h_in) + d, *dh = static_cast<const To *>(a.dh) + d;
    Tx *dx = static_cast<Tx *>(a.dx) + d;
    Tg *dg = static_cast<Tg *>(a.dg) + d;
    float mu = a.dht ? a.dht[(size_t)n * a.D + d] : 0.f;
#pragma unroll 8
    for (long long r = end - 1; r >= begin; --r) {
        const float lam = widen(dh[r * a.D]) + mu;
        const float prev = r > begin ? widen(h[(r - 1) * a.D]) : a.h0 ? a.h0[(size_t)n * a.D + d] : 0.f;
        mu = expf(widen(g[r * a.ldg])) * lam;
        dx[r * a.lddx] = narrow<Tx>(lam);
        dg[r * a.lddg] = narrow<Tg>(mu * prev);
    }
    if (a.dh0)
        a.dh0[(size_t)n * a.D + d] = mu;
}

}  // namespace

cudaError_t launch_scan_fwd(const ScanArgs &a, int dtype, cudaStream_t s)
{
    const int tiles = (a.D + 127) / 128;
    return by_types(dtype, [&](auto x, auto g, auto o) {
        scan_fwd_serial<std::remove_pointer_t<decltype(x)>, std::remove_pointer_t<decltype(g)>,
                        std::remove_pointer_t<decltype(o)>><<<a.N * tiles, 128, 0, s>>>(a, tiles);
        return cudaGetLastError();
    });
}

cudaError_t launch_scan_bwd(const ScanArgs &a, int dtype, cudaStream_t s)
{
    const int tiles = (a.D + 127) / 128;
    return by_types(dtype, [&](auto x, auto g, auto o) {
        scan_bwd_serial<std::remove_pointer_t<decltype(x)>, std::remove_pointer_t<decltype(g)>,
                        std::remove_pointer_t<decltype(o)>><<<a.N * tiles, 128, 0, s>>>(a, tiles);
        return cudaGetLastError();
    });
}

}  // namespace gla
