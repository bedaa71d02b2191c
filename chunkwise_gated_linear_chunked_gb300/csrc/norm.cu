// Residual addition and root-mean-square norm: forward (fp32 / 16-bit or e4m3 output) and backward.
//
// Up to 8192 columns a row lives in registers, 16 values a thread: it is read once, reduced, and written.  A warp holds
// 512 adjacent columns (so a group of 128 columns never leaves a warp), up to 16 warps a row; rows of at most 256
// columns share a warp.  A CTA keeps its share of the weights in registers, walks rows a grid apart, and asks for its
// next row before it reduces the present one.  Wider rows are read again from cache instead, by one CTA a row.
#include <algorithm>

#include "api_common.h"
#include "layer_internal.h"

namespace gla {
namespace {

constexpr int kThreads = 256;        // threads of a CTA (more where a row needs them)
constexpr int kHeld = 16;            // values of a row in a thread
constexpr int kMaxHeld = 8192;       // columns of a row that 16 warps hold
constexpr float kE4m3Max = 448.f, kScaleMin = 1e-30f;

// Maximum that keeps a NaN of either side.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Threads of a row and rows of a CTA.
struct Split {
    int lanes, rows, threads;
};
inline Split split_of(int D)
{
    Split s;
    if (D <= 256) {
        s.lanes = 1;
        while (s.lanes * kHeld < D)
            s.lanes *= 2;
    } else {
        s.lanes = (D + 32 * kHeld - 1) / (32 * kHeld) * 32;
    }
    s.rows = s.lanes < kThreads ? kThreads / s.lanes : 1;
    s.threads = s.rows * s.lanes;
    return s;
}

// VEC adjacent values of a row as they lie in memory.
template <typename T, int VEC>
struct Vec {
    T v[VEC];
    __device__ __forceinline__ void load(const T *p)
    {
        if constexpr (VEC * sizeof(T) == 32) {
            reinterpret_cast<uint4 *>(v)[0] = reinterpret_cast<const uint4 *>(p)[0];
            reinterpret_cast<uint4 *>(v)[1] = reinterpret_cast<const uint4 *>(p)[1];
        } else if constexpr (VEC * sizeof(T) == 16) {
            *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(p);
        } else {
            static_assert(VEC == 1, "whole 16-byte units or single values");
            v[0] = *p;
        }
    }
    __device__ __forceinline__ void store(T *p) const
    {
        if constexpr (VEC * sizeof(T) == 32) {
            reinterpret_cast<uint4 *>(p)[0] = reinterpret_cast<const uint4 *>(v)[0];
            reinterpret_cast<uint4 *>(p)[1] = reinterpret_cast<const uint4 *>(v)[1];
        } else if constexpr (VEC * sizeof(T) == 16) {
            *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(v);
        } else {
            *p = v[0];
        }
    }
};

// A thread's part of a row: kHeld / VEC vectors.
template <typename T, int VEC>
struct Part {
    static constexpr int N = kHeld / VEC;
    alignas(16) Vec<T, VEC> vec[N];
    __device__ __forceinline__ void load(const T *row, const int (&col)[N], int D)
    {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (col[j] < D)
                vec[j].load(row + col[j]);
            else
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    vec[j].v[i] = T(0.f);
    }
    __device__ __forceinline__ float at(int i) const { return widen(vec[i / VEC].v[i % VEC]); }
    __device__ __forceinline__ void set(int i, float f) { vec[i / VEC].v[i % VEC] = narrow<T>(f); }
    __device__ __forceinline__ void store(T *row, const int (&col)[N], int D) const
    {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (col[j] < D)
                vec[j].store(row + col[j]);
    }
};

// The first column of each of a thread's vectors: lane l of a row.
template <int VEC>
__device__ __forceinline__ void columns(int (&col)[kHeld / VEC], int l, int lanes)
{
    constexpr int N = kHeld / VEC;
#pragma unroll
    for (int j = 0; j < N; ++j)
        col[j] = (lanes < 32 ? j * lanes + l : (l / 32 * N + j) * 32 + l % 32) * VEC;
}

template <int VEC>
__device__ __forceinline__ void load_weights(float (&w)[kHeld], const float *p, const int (&col)[kHeld / VEC], int D)
{
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int c = col[i / VEC];
        w[i] = c >= D ? 0.f : p ? p[c + i % VEC] : 1.f;
    }
}

// Sum (and maximum) over the lanes of a row.  `part` has a slot per warp; a CTA's rows come here together, and two
// calls in a row use different `part`s.
template <bool MAX>
__device__ __forceinline__ void reduce_row(float &sum, float &most, int lanes, float2 *part)
{
    for (int m = min(lanes, 32) / 2; m; m >>= 1) {
        sum += __shfl_xor_sync(~0u, sum, m);
        if (MAX)
            most = max_nan(most, __shfl_xor_sync(~0u, most, m));
    }
    if (lanes <= 32)
        return;
    const int warp = threadIdx.x / 32, count = lanes / 32, first = warp / count * count;
    if (threadIdx.x % 32 == 0)
        part[warp] = make_float2(sum, most);
    __syncthreads();
    float2 t = part[first];
    sum = t.x;
    most = t.y;
    for (int i = 1; i < count; ++i) {
        t = part[first + i];
        sum += t.x;
        if (MAX)
            most = max_nan(most, t.y);
    }
}

// Groups of 128 columns.  Where a row has whole warps, kGroupLanes lanes' kGroupVecs vectors make one up, and a thread's
// vectors lie in kHeld / VEC / kGroupVecs of them; where rows share a warp, a row has at most two.
template <int VEC>
constexpr int kGroupLanes = VEC >= 4 ? 128 / VEC : 32;
template <int VEC>
constexpr int kGroupVecs = VEC >= 4 ? 1 : 4 / VEC;
constexpr int kGroups = 4;   // most of a thread

template <int VEC>
__device__ __forceinline__ void group_maxima(float (&m)[kGroups], const float (&v)[kHeld], const int (&col)[kHeld / VEC],
                                             int lanes)
{
#pragma unroll
    for (int k = 0; k < kGroups; ++k)
        m[k] = 0.f;
    if (lanes < 32) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            if (col[i / VEC] < 128)
                m[0] = max_nan(m[0], fabsf(v[i]));
            else
                m[1] = max_nan(m[1], fabsf(v[i]));
        }
        for (int d = lanes / 2; d; d >>= 1) {
            m[0] = max_nan(m[0], __shfl_xor_sync(~0u, m[0], d));
            m[1] = max_nan(m[1], __shfl_xor_sync(~0u, m[1], d));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        m[i / VEC / kGroupVecs<VEC>] = max_nan(m[i / VEC / kGroupVecs<VEC>], fabsf(v[i]));
#pragma unroll
    for (int k = 0; k < kHeld / VEC / kGroupVecs<VEC>; ++k)
#pragma unroll
        for (int d = kGroupLanes<VEC> / 2; d; d >>= 1)
            m[k] = max_nan(m[k], __shfl_xor_sync(~0u, m[k], d));
}

// The row's group that a thread's k-th maximum belongs to (past the last for those it does not have).
template <int VEC>
__device__ __forceinline__ int group_of(int k, int l, int lanes)
{
    constexpr int kOwn = kHeld / VEC / kGroupVecs<VEC>;   // of a thread
    if (lanes < 32)
        return k < 2 ? k : 1 << 30;
    // a warp's 512 columns are four groups: k-th of a thread is a block of 32 / kGroupLanes adjacent ones
    return k < kOwn ? l / 32 * 4 + k * (32 / kGroupLanes<VEC>) + l % 32 / kGroupLanes<VEC> : 1 << 30;
}

// VEC adjacent values v * rstd * inv in e4m3.
template <int VEC>
__device__ __forceinline__ void put_e4m3(uint8_t *q, const float *v, float rstd, float inv)
{
    if constexpr (VEC == 1) {
        *q = __nv_cvt_float_to_fp8(v[0] * rstd * inv, __NV_SATFINITE, __NV_E4M3);
    } else {
        alignas(8) __nv_fp8x2_storage_t b[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
            b[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * rstd * inv, v[2 * i + 1] * rstd * inv),
                                            __NV_SATFINITE, __NV_E4M3);
        if constexpr (VEC == 8)
            *reinterpret_cast<uint2 *>(q) = *reinterpret_cast<const uint2 *>(b);
        else
            *reinterpret_cast<uint32_t *>(q) = *reinterpret_cast<const uint32_t *>(b);
    }
}

template <typename Tx, typename Tr, int VEC, bool QUANT>
__global__ void __launch_bounds__(512) norm_fwd_rows(NormArgs a, Split sp)
{
    constexpr int N = kHeld / VEC;
    __shared__ float2 part[2][16];
    const int l = threadIdx.x % sp.lanes, D = a.D;
    int col[N];
    columns<VEC>(col, l, sp.lanes);
    const int64_t stride = (int64_t)gridDim.x * sp.rows;
    int64_t row = (int64_t)blockIdx.x * sp.rows + threadIdx.x / sp.lanes;
    Part<Tx, VEC> x;
    Part<Tr, VEC> res;
    auto fetch = [&](int64_t r) {
        if (r < a.rows) {
            x.load(static_cast<const Tx *>(a.x) + r * D, col, D);
            if (a.res)
                res.load(static_cast<const Tr *>(a.res) + r * D, col, D);
        }
    };
    fetch(row);
    float w[kHeld];
    load_weights<VEC>(w, a.w, col, D);
    // every thread of the CTA takes the same number of turns (they meet in the reduction)
    for (int64_t first = (int64_t)blockIdx.x * sp.rows, turn = 0; first < a.rows; first += stride, row += stride, ++turn) {
        const bool on = row < a.rows;
        float v[kHeld], sum = 0.f, most = 0.f, most_of[kGroups];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            v[i] = x.at(i);
            if (a.res)
                v[i] += res.at(i);
            sum = fmaf(v[i], v[i], sum);
        }
        if (on && a.s) {
            Part<Tr, VEC> s;
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                s.set(i, v[i]);
            s.store(static_cast<Tr *>(a.s) + row * D, col, D);
        }
        fetch(row + stride);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            v[i] *= w[i];
            if (QUANT)
                most = max_nan(most, fabsf(v[i]));
        }
        if (QUANT && a.group)
            group_maxima<VEC>(most_of, v, col, sp.lanes);
        reduce_row<QUANT>(sum, most, sp.lanes, part[turn & 1]);
        const float rstd = rsqrtf(sum / D + a.eps);
        if (!on)
            continue;
        if (a.rstd && l == 0)
            a.rstd[row] = rstd;
        if constexpr (!QUANT) {
            Part<Tx, VEC> y;
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                y.set(i, v[i] * rstd);
            y.store(static_cast<Tx *>(a.y) + row * D, col, D);
        } else {
            const int groups = a.group ? (D + 127) / 128 : 1;
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                most_of[k] = max_nan((a.group ? most_of[k] : most) * rstd / kE4m3Max, kScaleMin);
                const int g = a.group ? group_of<VEC>(k, l, sp.lanes) : 0;
                const bool lead = a.group ? (sp.lanes < 32 ? l == 0 : l % kGroupLanes<VEC> == 0) : l == 0 && k == 0;
                if (lead && g < groups)
                    a.scales[row * groups + g] = most_of[k];
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                // a vector lies in one group: by its columns where a row shares a warp, else by its number
                const float scale = !a.group ? most_of[0]
                                    : sp.lanes < 32 ? (col[j] < 128 ? most_of[0] : most_of[1])
                                                    : most_of[j / kGroupVecs<VEC>];
                if (col[j] < D)
                    put_e4m3<VEC>(static_cast<uint8_t *>(a.y) + row * D + col[j], v + j * VEC, rstd, 1.f / scale);
            }
        }
    }
}

template <typename Tx, typename Tr, int VEC>
__global__ void __launch_bounds__(512) norm_bwd_rows(NormArgs a, Split sp)
{
    constexpr int N = kHeld / VEC;
    constexpr bool kEarly = VEC == 8 && sizeof(Tr) == 2;   // registers for the next row beside the present one
    __shared__ float2 part[2][16];
    __shared__ float acc[2048];   // a CTA of several rows has at most so many columns
    const int l = threadIdx.x % sp.lanes, D = a.D;
    int col[N];
    columns<VEC>(col, l, sp.lanes);
    const int64_t stride = (int64_t)gridDim.x * sp.rows;
    int64_t row = (int64_t)blockIdx.x * sp.rows + threadIdx.x / sp.lanes;
    Part<Tr, VEC> s, ds;
    Part<Tx, VEC> dy;
    float rstd = 0.f;
    auto fetch = [&](int64_t r) {
        if (r < a.rows) {
            s.load(static_cast<const Tr *>(a.s_in) + r * D, col, D);
            dy.load(static_cast<const Tx *>(a.dy) + r * D, col, D);
            if (a.ds)
                ds.load(static_cast<const Tr *>(a.ds) + r * D, col, D);
            rstd = a.rstd_in[r];
        }
    };
    if (kEarly)
        fetch(row);
    float w[kHeld], dw[kHeld];
    load_weights<VEC>(w, a.w, col, D);
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        dw[i] = 0.f;
    for (int64_t first = (int64_t)blockIdx.x * sp.rows, turn = 0; first < a.rows; first += stride, row += stride, ++turn) {
        const bool on = row < a.rows;
        if (!kEarly)
            fetch(row);
        const float r = rstd;
        float n[kHeld], g[kHeld], up[kHeld], c = 0.f, none = 0.f;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            n[i] = s.at(i) * r;
            g[i] = dy.at(i);
            up[i] = a.ds ? ds.at(i) : 0.f;
            if (on)
                dw[i] = fmaf(g[i], n[i], dw[i]);
            g[i] *= w[i];
            c = fmaf(g[i], n[i], c);
        }
        if (kEarly)
            fetch(row + stride);
        reduce_row<false>(c, none, sp.lanes, part[turn & 1]);
        if (!on)
            continue;
        c /= D;
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            up[i] = fmaf(r, g[i] - n[i] * c, up[i]);
        if (a.dx) {
            Part<Tx, VEC> out;
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                out.set(i, up[i]);
            out.store(static_cast<Tx *>(a.dx) + row * D, col, D);
        }
        if (a.dres) {
            Part<Tr, VEC> out;
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                out.set(i, up[i]);
            out.store(static_cast<Tr *>(a.dres) + row * D, col, D);
        }
    }
    if (!a.dw)
        return;
    // the CTA's sum of dw: over the rows of a warp, then over the warps in order
    for (int m = sp.lanes; m < 32; m *= 2)
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            dw[i] += __shfl_xor_sync(~0u, dw[i], m);
    float *out = a.part + (size_t)blockIdx.x * D;
    const int wide = max(sp.lanes, 32), turns = sp.threads / wide, mine = threadIdx.x / wide;
    const bool lead = threadIdx.x % wide < sp.lanes;
    for (int t = 0; t < turns; ++t) {
        if (t == mine && lead)
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int d = col[i / VEC] + i % VEC;
                if (col[i / VEC] >= D)
                    continue;
                const float sum = t > 0 ? acc[d] + dw[i] : dw[i];
                if (t == turns - 1)
                    out[d] = sum;
                else
                    acc[d] = sum;
            }
        if (turns > 1)
            __syncthreads();
    }
}

// --- rows wider than kMaxHeld: one CTA a row, read again from cache -----------------------------------------------

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

__device__ __forceinline__ float block_sum(float v, float *sh)
{
    return block_reduce(v, sh, [](float a, float b) { return a + b; });
}

template <typename Tx, typename Tr>
__global__ void __launch_bounds__(kThreads) norm_fwd_wide(NormArgs a)
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
        const float rstd = rsqrtf(block_sum(sq, sh) / a.D + a.eps);
        if (a.rstd && threadIdx.x == 0)
            a.rstd[row] = rstd;
        auto normed = [&](int d) { return total(d) * (a.w ? a.w[d] : 1.f) * rstd; };
        const int group = a.group ? a.group : a.D, groups = (a.D + group - 1) / group;
        for (int c = 0; c < (a.scales ? groups : 1); ++c) {
            const int lo = a.scales ? c * group : 0, hi = a.scales ? min(a.D, lo + group) : a.D;
            float inv = 1.f;
            if (a.scales) {
                float m = 0.f;
                for (int d = lo + threadIdx.x; d < hi; d += kThreads)
                    m = max_nan(m, fabsf(normed(d)));
                const float scale = max_nan(block_reduce(m, sh, max_nan) / kE4m3Max, kScaleMin);
                inv = 1.f / scale;
                if (threadIdx.x == 0)
                    a.scales[row * groups + c] = scale;
            }
            for (int d = lo + threadIdx.x; d < hi; d += kThreads) {
                const float y = normed(d), s = total(d);
                if (a.scales)
                    static_cast<__nv_fp8_storage_t *>(a.y)[at + d] =
                        __nv_cvt_float_to_fp8(y * inv, __NV_SATFINITE, __NV_E4M3);
                else
                    static_cast<Tx *>(a.y)[at + d] = narrow<Tx>(y);
                if (a.s)   // last: s may be res itself
                    static_cast<Tr *>(a.s)[at + d] = narrow<Tr>(s);
            }
        }
    }
}

template <typename Tx, typename Tr>
__global__ void __launch_bounds__(kThreads) norm_bwd_wide(NormArgs a)
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
        c = block_sum(c, sh) / a.D;
        for (int d = threadIdx.x; d < a.D; d += kThreads) {
            const float n = widen(s[at + d]) * r, g = widen(dy[at + d]);
            const float grad = fmaf(r, (a.w ? a.w[d] : 1.f) * g - n * c, ds ? widen(ds[at + d]) : 0.f);
            part[d] = fmaf(g, n, part[d]);
            if (a.dx)
                static_cast<Tx *>(a.dx)[at + d] = narrow<Tx>(grad);
            if (a.dres)
                static_cast<Tr *>(a.dres)[at + d] = narrow<Tr>(grad);
        }
    }
}

// dw from the CTAs' partial sums: 32 columns a CTA, 32 threads a column, in a fixed order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(NormArgs a)
{
    __shared__ float sh[32][33];
    const int c = threadIdx.x % 32, k = threadIdx.x / 32, d = blockIdx.x * 32 + c;
    float sum = 0.f;
    if (d < a.D)
        for (int i = k; i < a.ctas; i += 32)
            sum += a.part[(size_t)i * a.D + d];
    sh[k][c] = sum;
    __syncthreads();
    sum = sh[c][k];
    for (int m = 16; m; m >>= 1)
        sum += __shfl_xor_sync(~0u, sum, m);
    if (c == 0 && blockIdx.x * 32 + k < a.D)
        a.dw[blockIdx.x * 32 + k] = sum;
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

// Persistent CTAs: as many as an SM holds of them, or one for each of its rows where there are fewer.
template <typename K>
int grid_of(K kernel, int64_t rows, const Split &sp)
{
    int per_sm = 1;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, sp.threads, 0) != cudaSuccess || per_sm < 1)
        per_sm = 1;
    return (int)std::min<int64_t>((rows + sp.rows - 1) / sp.rows, (int64_t)per_sm * sm_count());
}

template <typename Tx, typename Tr, int VEC, bool QUANT>
cudaError_t fwd_rows(const NormArgs &a, cudaStream_t s)
{
    const Split sp = split_of(a.D);
    auto kernel = norm_fwd_rows<Tx, Tr, VEC, QUANT>;
    kernel<<<grid_of(kernel, a.rows, sp), sp.threads, 0, s>>>(a, sp);
    return cudaGetLastError();
}

}  // namespace

int norm_bwd_ctas(int64_t rows, int D)
{
    const Split sp = split_of(D);
    return (int)std::min<int64_t>(D > kMaxHeld ? rows : (rows + sp.rows - 1) / sp.rows, 2 * sm_count());
}

cudaError_t launch_norm_fwd(const NormArgs &a, int dtype, bool res_f32, cudaStream_t s)
{
    return by_norm_types(dtype, res_f32, [&](auto x, auto r) {
        typedef std::remove_pointer_t<decltype(x)> Tx;
        typedef std::remove_pointer_t<decltype(r)> Tr;
        if (a.D > kMaxHeld) {
            norm_fwd_wide<Tx, Tr><<<(unsigned)std::min<int64_t>(a.rows, 16 * sm_count()), kThreads, 0, s>>>(a);
            return cudaGetLastError();
        }
        constexpr int VEC = 16 / sizeof(Tx);
        if (a.D % VEC == 0)   // rows start on 16-byte units
            return a.scales ? fwd_rows<Tx, Tr, VEC, true>(a, s) : fwd_rows<Tx, Tr, VEC, false>(a, s);
        return a.scales ? fwd_rows<Tx, Tr, 1, true>(a, s) : fwd_rows<Tx, Tr, 1, false>(a, s);
    });
}

cudaError_t launch_norm_bwd(const NormArgs &a, int dtype, bool res_f32, cudaStream_t s)
{
    return by_norm_types(dtype, res_f32, [&](auto x, auto r) {
        typedef std::remove_pointer_t<decltype(x)> Tx;
        typedef std::remove_pointer_t<decltype(r)> Tr;
        constexpr int VEC = 16 / sizeof(Tx);
        const Split sp = split_of(a.D);
        if (a.D > kMaxHeld)
            norm_bwd_wide<Tx, Tr><<<a.ctas, kThreads, 0, s>>>(a);
        else if (a.D % VEC == 0)
            norm_bwd_rows<Tx, Tr, VEC><<<a.ctas, sp.threads, 0, s>>>(a, sp);
        else
            norm_bwd_rows<Tx, Tr, 1><<<a.ctas, sp.threads, 0, s>>>(a, sp);
        return cudaGetLastError();
    });
}

cudaError_t launch_norm_dw(const NormArgs &a, cudaStream_t s)
{
    norm_dw_kernel<<<(a.D + 31) / 32, 1024, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace gla
