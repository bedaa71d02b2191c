// Residual addition and root-mean-square norm: forward (fp32 / 16-bit or e4m3 output) and backward.
#include <algorithm>

#include "api_common.h"
#include "layer_internal.h"

namespace gla {
namespace {

constexpr int kThreads = 256;

// Maximum that keeps a NaN of either side.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <typename F>
__device__ __forceinline__ float block_reduce(float v, float *sh, F f)
{
    for (int m = 16; m; m >>= 1)
        v = f(v, __shfl_xor_sync(~0u, v, m));
    __syncthreads();
    if (threadIdx.x % 32 == 0)
        sh[threadIdx.x / 32] = v;
    __syncthreads();
    v = sh[0];
    for (int i = 1; i < kThreads / 32; ++i)
        v = f(v, sh[i]);
    return v;
}

__device__ __forceinline__ float sum_of(float v, float *sh)
{
    return block_reduce(v, sh, [](float a, float b) { return a + b; });
}

// One CTA per row.
template <typename Tx, typename Tr>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(NormArgs a)
{
    __shared__ float sh[kThreads / 32];
    const Tx *x = static_cast<const Tx *>(a.x);
    const Tr *res = static_cast<const Tr *>(a.res);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t at = row * a.D;
        auto total = [&](int d) { return widen(x[at + d]) + (res ? widen(res[at + d]) : 0.f); };
        float sq = 0.f;
        for (int d = threadIdx.x; d < a.D; d += kThreads)
            sq = fmaf(total(d), total(d), sq);
        const float rstd = rsqrtf(sum_of(sq, sh) / a.D + a.eps);
        if (a.rstd && threadIdx.x == 0)
            a.rstd[row] = rstd;
        auto normed = [&](int d) { return total(d) * rstd * (a.w ? a.w[d] : 1.f); };
        const int group = a.group ? a.group : a.D, groups = (a.D + group - 1) / group;
        for (int c = 0; c < (a.scales ? groups : 1); ++c) {
            const int lo = a.scales ? c * group : 0, hi = a.scales ? min(a.D, lo + group) : a.D;
            float inv = 1.f;
            if (a.scales) {
                float m = 0.f;
                for (int d = lo + threadIdx.x; d < hi; d += kThreads)
                    m = max_nan(m, fabsf(normed(d)));
                m = block_reduce(m, sh, max_nan);
                const float scale = max_nan(m / 448.f, 1e-30f);
                inv = 1.f / scale;
                if (threadIdx.x == 0)
                    a.scales[row * groups + c] = scale;
            }
            for (int d = lo + threadIdx.x; d < hi; d += kThreads) {
                const float y = normed(d);
                if (a.scales)
                    static_cast<__nv_fp8_storage_t *>(a.y)[at + d] =
                        __nv_cvt_float_to_fp8(y * inv, __NV_SATFINITE, __NV_E4M3);
                else
                    static_cast<Tx *>(a.y)[at + d] = narrow<Tx>(y);
                if (a.s)   // last: s may be res itself
                    static_cast<Tr *>(a.s)[at + d] = narrow<Tr>(total(d));
            }
        }
    }
}

template <typename Tx, typename Tr>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(NormArgs a)
{
    __shared__ float sh[kThreads / 32];
    const Tr *s = static_cast<const Tr *>(a.s_in), *ds = static_cast<const Tr *>(a.ds);
    const Tx *dy = static_cast<const Tx *>(a.dy);
    float *part = a.part + (size_t)blockIdx.x * a.D;
    for (int d = threadIdx.x; d < a.D; d += kThreads)
        part[d] = 0.f;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t at = row * a.D;
        const float r = a.rstd_in[row];
        float c = 0.f;
        for (int d = threadIdx.x; d < a.D; d += kThreads)
            c = fmaf((a.w ? a.w[d] : 1.f) * widen(dy[at + d]), widen(s[at + d]) * r, c);
        c = sum_of(c, sh) / a.D;
        for (int d = threadIdx.x; d < a.D; d += kThreads) {
            const float n = widen(s[at + d]) * r, g = widen(dy[at + d]);
            const float grad = r * ((a.w ? a.w[d] : 1.f) * g - n * c) + (ds ? widen(ds[at + d]) : 0.f);
            part[d] = fmaf(g, n, part[d]);
            if (a.dx)
                static_cast<Tx *>(a.dx)[at + d] = narrow<Tx>(grad);
            if (a.dres)
                static_cast<Tr *>(a.dres)[at + d] = narrow<Tr>(grad);
        }
    }
}

__global__ void __launch_bounds__(kThreads) norm_dw_kernel(NormArgs a)
{
    const int d = blockIdx.x * kThreads + threadIdx.x;
    if (d >= a.D)
        return;
    float sum = 0.f;
    for (int i = 0; i < (a.rows ? a.ctas : 0); ++i)
        sum += a.part[(size_t)i * a.D + d];
    a.dw[d] = sum;
}

template <typename F>
cudaError_t by_norm_types(int dtype, bool res_f32, F f)
{
    typedef __nv_bfloat16 bf;
    if (dtype == GLA_F32)
        return f((float *)0, (float *)0);
    if (dtype == GLA_BF16)
        return res_f32 ? f((bf *)0, (float *)0) : f((bf *)0, (bf *)0);
    return res_f32 ? f((__half *)0, (float *)0) : f((__half *)0, (__half *)0);
}

}  // namespace

int norm_bwd_ctas(int64_t rows, int) { return (int)std::min<int64_t>(rows, 2 * sm_count()); }

cudaError_t launch_norm_fwd(const NormArgs &a, int dtype, bool res_f32, cudaStream_t s)
{
    return by_norm_types(dtype, res_f32, [&](auto x, auto r) {
        norm_fwd_kernel<std::remove_pointer_t<decltype(x)>, std::remove_pointer_t<decltype(r)>>
            <<<(unsigned)std::min<int64_t>(a.rows, 1 << 20), kThreads, 0, s>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t launch_norm_bwd(const NormArgs &a, int dtype, bool res_f32, cudaStream_t s)
{
    return by_norm_types(dtype, res_f32, [&](auto x, auto r) {
        norm_bwd_kernel<std::remove_pointer_t<decltype(x)>, std::remove_pointer_t<decltype(r)>>
            <<<a.ctas, kThreads, 0, s>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t launch_norm_dw(const NormArgs &a, cudaStream_t s)
{
    norm_dw_kernel<<<(a.D + kThreads - 1) / kThreads, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace gla
