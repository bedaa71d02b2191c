// One-token state updates: the vector-state recurrence and the GLA recurrence.  Both are bound by the states' bytes
// (read once, written once) for many sequences and by launch and memory latency for few.
#include <type_traits>

#include "gla_internal.h"
#include "layer_internal.h"
#include "tc_ptx.cuh"

namespace gla {
namespace {

constexpr int kThreads = 128;
constexpr int kCols = 32;   // value columns of a GLA tile: 128 bytes of a state row

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

template <typename T>
struct alignas(4 * sizeof(T)) Four {
    T v[4];
    __device__ __forceinline__ float4 wide() const { return make_float4(widen(v[0]), widen(v[1]), widen(v[2]), widen(v[3])); }
    static __device__ __forceinline__ Four of(float4 f)
    {
        return {narrow<T>(f.x), narrow<T>(f.y), narrow<T>(f.z), narrow<T>(f.w)};
    }
};

// Four channels a thread: adjacent ones (FOUR: rows start and end on whole fours), or a CTA's width apart.
template <typename Tx, typename Tg, typename To, bool FOUR>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(StepArgs a, int tiles)
{
    tc::grid_dep_wait();
    const int b = blockIdx.x / tiles, d = (blockIdx.x - b * tiles) * 4 * kThreads + threadIdx.x * (FOUR ? 4 : 1);
    const int s = state_of(a, b);
    const Tx *x = static_cast<const Tx *>(a.x) + b * a.ldx + d;
    const Tg *g = static_cast<const Tg *>(a.g) + b * a.ldg + d;
    To *o = static_cast<To *>(a.h) + (size_t)b * a.D + d;
    const size_t at = (size_t)(s < 0 ? 0 : s) * a.D + d;
    if constexpr (FOUR) {
        if (d >= a.D)
            return;
        float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s >= 0) {
            const float4 xs = reinterpret_cast<const Four<Tx> *>(x)->wide(), gs = reinterpret_cast<const Four<Tg> *>(g)->wide();
            h = *reinterpret_cast<const float4 *>(a.h0 + at);
            h = make_float4(fmaf(decay(gs.x), h.x, xs.x), fmaf(decay(gs.y), h.y, xs.y), fmaf(decay(gs.z), h.z, xs.z),
                            fmaf(decay(gs.w), h.w, xs.w));
            *reinterpret_cast<float4 *>(a.ht + at) = h;
        }
        *reinterpret_cast<Four<To> *>(o) = Four<To>::of(h);
    } else {
        float h[4] = {}, xs[4], gs[4];
        bool on[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            on[i] = d + i * kThreads < a.D;
            if (s >= 0 && on[i]) {
                h[i] = a.h0[at + i * kThreads];
                xs[i] = widen(x[i * kThreads]);
                gs[i] = widen(g[i * kThreads]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (s >= 0 && on[i]) {
                h[i] = fmaf(decay(gs[i]), h[i], xs[i]);
                a.ht[at + i * kThreads] = h[i];
            }
            if (on[i])
                o[i * kThreads] = narrow<To>(h[i]);
        }
    }
}

// S' = diag(a) S + k^T v and o = scale q S' touch every state element once, so a CTA takes K rows by 32 columns: small
// enough that 8 heads of one sequence already make 32 CTAs, and all of a thread's K / 16 loads of 16 bytes are under
// way at once (16 KB a CTA).  128 sequences of 16 heads, 128 x 256: 81 us, 6.7 TB/s; one of 8 heads: 1.65 us.  Eight
// lanes hold a row's columns, so a warp covers four rows; the sum over rows that o takes is finished over the lanes and
// then over the four warps.
template <typename Tx, typename Tg, typename To, int K>
__global__ void __launch_bounds__(kThreads) gla_step_kernel(StepArgs a, int tiles)
{
    constexpr int kRows = kThreads / 8, kTurns = K / kRows;   // rows of a turn
    __shared__ float4 akq[K];                                 // decay, key and query of each row
    __shared__ float4 part[kThreads / 32][8];
    tc::grid_dep_wait();
    const int bh = blockIdx.x / tiles, b = bh / a.H, head = bh - b * a.H;
    const int lane8 = threadIdx.x % 8, row0 = threadIdx.x / 8, c = (blockIdx.x - bh * tiles) * kCols + 4 * lane8;
    const int slot = state_of(a, b);
    To *o = static_cast<To *>(a.h) + (size_t)bh * a.V + c;
    if (slot < 0) {
        if (threadIdx.x < 8)
            *reinterpret_cast<Four<To> *>(o) = Four<To>::of(make_float4(0.f, 0.f, 0.f, 0.f));
        return;
    }
    const size_t at = (((size_t)slot * a.H + head) * K + row0) * a.V + c;
    float4 s[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i)
        s[i] = *reinterpret_cast<const float4 *>(a.h0 + at + (size_t)i * kRows * a.V);
    if (threadIdx.x < K) {
        const size_t e = (size_t)bh * K + threadIdx.x;
        akq[threadIdx.x] = make_float4(decay(widen(static_cast<const Tg *>(a.g)[e])), widen(static_cast<const Tx *>(a.k)[e]),
                                       widen(static_cast<const Tx *>(a.x)[e]), 0.f);
    }
    const float4 v = reinterpret_cast<const Four<Tx> *>(static_cast<const Tx *>(a.v) + (size_t)bh * a.V + c)->wide();
    __syncthreads();
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const float4 r = akq[row0 + i * kRows];
        s[i] = make_float4(fmaf(r.x, s[i].x, r.y * v.x), fmaf(r.x, s[i].y, r.y * v.y), fmaf(r.x, s[i].z, r.y * v.z),
                           fmaf(r.x, s[i].w, r.y * v.w));
        *reinterpret_cast<float4 *>(a.ht + at + (size_t)i * kRows * a.V) = s[i];
        sum = make_float4(fmaf(r.z, s[i].x, sum.x), fmaf(r.z, s[i].y, sum.y), fmaf(r.z, s[i].z, sum.z),
                          fmaf(r.z, s[i].w, sum.w));
    }
#pragma unroll
    for (int m = 8; m < 32; m *= 2) {
        sum.x += __shfl_xor_sync(~0u, sum.x, m);
        sum.y += __shfl_xor_sync(~0u, sum.y, m);
        sum.z += __shfl_xor_sync(~0u, sum.z, m);
        sum.w += __shfl_xor_sync(~0u, sum.w, m);
    }
    if (threadIdx.x % 32 < 8)
        part[threadIdx.x / 32][lane8] = sum;
    __syncthreads();
    if (threadIdx.x >= 8)
        return;
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) {
        const float4 p = part[i][lane8];
        sum = make_float4(sum.x + p.x, sum.y + p.y, sum.z + p.z, sum.w + p.w);
    }
    *reinterpret_cast<Four<To> *>(o) = Four<To>::of(make_float4(a.scale * sum.x, a.scale * sum.y, a.scale * sum.z, a.scale * sum.w));
}

}  // namespace

cudaError_t launch_scan_step(const StepArgs &a, int dtype, cudaStream_t s)
{
    const bool four = a.D % 4 == 0 && a.ldx % 4 == 0 && a.ldg % 4 == 0;
    const int tiles = (a.D + 4 * kThreads - 1) / (4 * kThreads);
    return by_types(dtype, [&](auto x, auto g, auto o) {
        typedef std::remove_pointer_t<decltype(x)> Tx;
        typedef std::remove_pointer_t<decltype(g)> Tg;
        typedef std::remove_pointer_t<decltype(o)> To;
        if (four)
            return launch_early(scan_step_kernel<Tx, Tg, To, true>, a.B * tiles, kThreads, s, a, tiles);
        else
            return launch_early(scan_step_kernel<Tx, Tg, To, false>, a.B * tiles, kThreads, s, a, tiles);
    });
}

cudaError_t launch_gla_step(const StepArgs &a, int dtype, cudaStream_t s)
{
    const int tiles = a.V / kCols;
    return by_types(dtype, [&](auto x, auto g, auto o) {
        typedef std::remove_pointer_t<decltype(x)> Tx;
        typedef std::remove_pointer_t<decltype(g)> Tg;
        typedef std::remove_pointer_t<decltype(o)> To;
        if (a.K == 128)
            return launch_early(gla_step_kernel<Tx, Tg, To, 128>, a.B * a.H * tiles, kThreads, s, a, tiles);
        else
            return launch_early(gla_step_kernel<Tx, Tg, To, 64>, a.B * a.H * tiles, kThreads, s, a, tiles);
    });
}

}  // namespace gla
