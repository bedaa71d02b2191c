// One-token state updates: the vector-state recurrence and the GLA recurrence.
#include "gla_internal.h"
#include "layer_internal.h"

namespace gla {
namespace {

// The state of sequence b, or -1 for an idle one (and for a slot outside the pool, which is reported).
__device__ __forceinline__ int state_of(const StepArgs &a, int b)
{
    if (!a.slots)
        return b;
    const int s = a.slots[b];
    if (s >= 0 && s < a.S)
        return s;
    if (s != -1 && threadIdx.x == 0)
        report(a.status, GLA_ERR_INVALID_ARG);
    return -1;
}

template <typename Tx, typename Tg, typename To>
__global__ void __launch_bounds__(128) scan_step_kernel(StepArgs a, int tiles)
{
    const int b = blockIdx.x / tiles, d = (blockIdx.x % tiles) * 128 + threadIdx.x;
    const int s = state_of(a, b);
    if (d >= a.D)
        return;
    float h = 0.f;
    if (s >= 0) {
        const size_t at = (size_t)s * a.D + d;
        h = fmaf(decay(widen(static_cast<const Tg *>(a.g)[b * a.ldg + d])), a.h0[at],
                 widen(static_cast<const Tx *>(a.x)[b * a.ldx + d]));
        a.ht[at] = h;
    }
    static_cast<To *>(a.h)[(size_t)b * a.D + d] = narrow<To>(h);
}

// One CTA per (sequence, head), one thread per value column.
template <typename Tx, typename Tg, typename To>
__global__ void __launch_bounds__(256) gla_step_kernel(StepArgs a)
{
    const int b = blockIdx.x / a.H, j = threadIdx.x;
    const int slot = state_of(a, b);
    const size_t bh = blockIdx.x;
    float o = 0.f;
    if (slot >= 0) {
        const size_t at = ((size_t)slot * a.H + blockIdx.x % a.H) * a.K * a.V + j;
        const float v = widen(static_cast<const Tx *>(a.v)[bh * a.V + j]);
        for (int i = 0; i < a.K; ++i) {
            const size_t e = bh * a.K + i;
            const float s = fmaf(decay(widen(static_cast<const Tg *>(a.g)[e])), a.h0[at + (size_t)i * a.V],
                                 widen(static_cast<const Tx *>(a.k)[e]) * v);
            a.ht[at + (size_t)i * a.V] = s;
            o = fmaf(widen(static_cast<const Tx *>(a.x)[e]), s, o);
        }
    }
    static_cast<To *>(a.h)[bh * a.V + j] = narrow<To>(a.scale * o);
}

}  // namespace

cudaError_t launch_scan_step(const StepArgs &a, int dtype, cudaStream_t s)
{
    const int tiles = (a.D + 127) / 128;
    return by_types(dtype, [&](auto x, auto g, auto o) {
        scan_step_kernel<std::remove_pointer_t<decltype(x)>, std::remove_pointer_t<decltype(g)>,
                         std::remove_pointer_t<decltype(o)>><<<a.B * tiles, 128, 0, s>>>(a, tiles);
        return cudaGetLastError();
    });
}

cudaError_t launch_gla_step(const StepArgs &a, int dtype, cudaStream_t s)
{
    return by_types(dtype, [&](auto x, auto g, auto o) {
        gla_step_kernel<std::remove_pointer_t<decltype(x)>, std::remove_pointer_t<decltype(g)>,
                        std::remove_pointer_t<decltype(o)>><<<a.B * a.H, a.V, 0, s>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace gla
