// One token of the gated delta rule for each of B sequences, states in a pool:
//
//     S~ = exp(g) S,   n = beta (v - k S~),   S' = S~ + k^T n,   o = scale q S' = scale (q S~ + (q.k) n)
//
// so that one pass over the state gives both sums, k S and q S, and the state is read and written once from registers.
// Bound by the states' bytes for many sequences, by launch and memory latency for few.
#include <type_traits>

#include "delta_internal.h"
#include "tc_ptx.cuh"

namespace gla {
namespace {

constexpr int kThreads = 128;
constexpr int kCols = 32;   // value columns of a CTA: 128 bytes of a state row

// A CTA takes K rows (up to P) by 32 columns, as gla_step does: eight lanes hold a row's columns (four adjacent ones
// where FOUR, else eight apart), a warp four rows, all of a thread's P / 16 loads under way at once.  128 sequences of 32
// heads, 128 x 128: 82 us, 6.5 TB/s, with six CTAs an SM (five, at 95 registers: 90; eight: 91).
template <typename Tx, typename To, int P, bool FOUR>
__global__ void __launch_bounds__(kThreads, P <= 128 ? 6 : 4) delta_step_kernel(DeltaStepArgs a, int tiles)
{
    constexpr int kRows = kThreads / 8, kTurns = P / kRows;
    __shared__ float2 kq[P];
    __shared__ float2 part[kThreads / 32][kCols];
    __shared__ float qk[kThreads / 32];
    tc::grid_dep_wait();
    const int bh = blockIdx.x / tiles, b = bh / a.HV, hv = bh - b * a.HV, tid = threadIdx.x, lane = tid % 8, row0 = tid / 8;
    const int c0 = (blockIdx.x - bh * tiles) * kCols + (FOUR ? 4 * lane : lane), step = FOUR ? 1 : 8;
    int slot = a.slots ? a.slots[b] : b;
    if (slot < 0 || slot >= a.S) {
        if (slot != -1 && tid == 0)
            report(a.status, GLA_ERR_INVALID_ARG);
        slot = -1;
    }
    To *o = static_cast<To *>(a.o) + (size_t)bh * a.V;
    if (slot < 0) {   // idle
        if (tid < 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c0 + e * step < a.V)
                    o[c0 + e * step] = narrow<To>(0.f);
        return;
    }
    const size_t at = (((size_t)slot * a.HV + hv) * a.K + row0) * a.V + c0;
    float s[kTurns][4];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const float *p = a.h0 + at + (size_t)i * kRows * a.V;
        const bool on = row0 + i * kRows < a.K;
        if constexpr (FOUR) {
            const float4 f = on && c0 < a.V ? *reinterpret_cast<const float4 *>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
            s[i][0] = f.x, s[i][1] = f.y, s[i][2] = f.z, s[i][3] = f.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[i][e] = on && c0 + e * step < a.V ? p[e * step] : 0.f;
        }
    }
    const size_t key = ((size_t)b * a.H + hv / (a.HV / a.H)) * a.K;
    const float decay_ = expf(a.g[bh]), beta = a.beta[bh];
    float dotted = 0.f;
#pragma unroll
    for (int d = tid; d < P; d += kThreads) {
        const float2 f = d < a.K ? make_float2(widen(static_cast<const Tx *>(a.k)[key + d]), widen(static_cast<const Tx *>(a.q)[key + d]))
                                 : make_float2(0.f, 0.f);
        kq[d] = f;
        dotted = fmaf(f.x, f.y, dotted);
    }
#pragma unroll
    for (int m = 16; m; m /= 2)
        dotted += __shfl_xor_sync(~0u, dotted, m);
    if (tid % 32 == 0)
        qk[tid / 32] = dotted;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = c0 + e * step < a.V ? widen(static_cast<const Tx *>(a.v)[(size_t)bh * a.V + c0 + e * step]) : 0.f;
    __syncthreads();
    float2 sum[4] = {};
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const float2 f = kq[row0 + i * kRows];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[i][e] *= decay_;
            sum[e] = make_float2(fmaf(f.x, s[i][e], sum[e].x), fmaf(f.y, s[i][e], sum[e].y));
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int m = 8; m < 32; m *= 2) {
            sum[e].x += __shfl_xor_sync(~0u, sum[e].x, m);
            sum[e].y += __shfl_xor_sync(~0u, sum[e].y, m);
        }
        if (tid % 32 < 8)
            part[tid / 32][4 * lane + e] = sum[e];
    }
    __syncthreads();
    const float all = (qk[0] + qk[1]) + (qk[2] + qk[3]);
    float n[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float2 t = part[0][4 * lane + e];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) {
            const float2 p = part[i][4 * lane + e];
            t = make_float2(t.x + p.x, t.y + p.y);
        }
        n[e] = beta * (v[e] - t.x);
        if (tid < 8 && c0 + e * step < a.V)
            o[c0 + e * step] = narrow<To>(a.scale * fmaf(all, n[e], t.y));
    }
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        float *p = a.ht + at + (size_t)i * kRows * a.V;
        if (row0 + i * kRows >= a.K)
            continue;
        const float k = kq[row0 + i * kRows].x;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s[i][e] = fmaf(k, n[e], s[i][e]);
        if constexpr (FOUR) {
            if (c0 < a.V)
                *reinterpret_cast<float4 *>(p) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c0 + e * step < a.V)
                    p[e * step] = s[i][e];
        }
    }
}

}  // namespace

cudaError_t launch_delta_step(const DeltaStepArgs &a, int dtype, cudaStream_t s)
{
    const int tiles = (a.V + kCols - 1) / kCols;
    const unsigned grid = (unsigned)((size_t)a.B * a.HV * tiles);
    return delta_types(dtype, [&](auto x, auto o) {
        typedef std::remove_pointer_t<decltype(x)> Tx;
        typedef std::remove_pointer_t<decltype(o)> To;
        auto go = [&](auto p) {
            constexpr int P = decltype(p)::value;
            return a.V % 4 == 0 ? launch_early(delta_step_kernel<Tx, To, P, true>, grid, kThreads, s, a, tiles)
                                : launch_early(delta_step_kernel<Tx, To, P, false>, grid, kThreads, s, a, tiles);
        };
        return a.K <= 64 ? go(std::integral_constant<int, 64>()) : a.K <= 128 ? go(std::integral_constant<int, 128>())
                                                                              : go(std::integral_constant<int, 256>());
    });
}

}  // namespace gla
