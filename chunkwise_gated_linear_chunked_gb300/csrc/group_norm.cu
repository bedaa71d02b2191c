// Group norm with an activation, channels last.  For sample n and group j of W = C / G channels, over all its positions:
//
//     mean, var over S x W values,   rstd = 1 / sqrt(var + eps),   xh = (x - mean) rstd,   z = xh w + b,   y = act(z)
//     dz = dy act'(z),   a = w dz,   dx = rstd (a - mean(a) - xh mean(a xh)),   dw = sum dz xh,   db = sum dz
//
// Bound by HBM (two instructions an element a byte or so).  Two ways:
//
// One position a sample (tokens) and at most 4096 channels a group: a group is a run of memory that up to 256 lanes hold
// in registers, so that it is read once; variances are sums of squares about the mean.  A lane keeps its channels from
// sample to sample, with their weights and its share of dw and db in registers.
//
// Otherwise (maps): samples are cut into slices of positions.  A CTA walks a slice with a vector of channels a thread and
// sums per channel, about the thread's first value (a value of the group itself, so the sum of squares loses at most the
// thread's count of units to the cancellation), joins the threads' means and squares by group, and a second kernel joins
// the slices and writes y (dx); it reads x again, from L2 where the tensor fits.  Every join has a fixed order, so results
// do not depend on timing.
#include <algorithm>
#include <numeric>
#include <type_traits>

#include "api_common.h"
#include "group_norm.h"
#include "layer_internal.h"
#include "tc_ptx.cuh"

namespace gla {
namespace {

constexpr int kThreads = 256;

template <typename T, int VEC>
struct alignas(VEC * sizeof(T)) Vec {
    T v[VEC];
};

// sigmoid(z); its error is that of ex2 and rcp, about 3 units in the last place.
__device__ __forceinline__ float sigmoid(float z)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp2_fast(-z * kLog2e)));
    return r;
}

template <bool SILU>
__device__ __forceinline__ float activated(float z)
{
    if constexpr (SILU)
        return z * sigmoid(z);
    return z;
}

// The gradient before the activation.
template <bool SILU>
__device__ __forceinline__ float before_act(float dy, float z)
{
    if constexpr (!SILU)
        return dy;
    const float s = sigmoid(z);
    return dy * s * fmaf(z, 1.f - s, 1.f);
}

// A vector of values in fp32, as pairs (the last alone where VEC is odd, i.e. 1).
template <typename T, int VEC>
__device__ __forceinline__ void widened(const Vec<T, VEC> &v, float (&f)[VEC])
{
    if constexpr (VEC % 2 == 0 && sizeof(T) == 2) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(v.v);
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            const float2 p = widen2<T>(w[e]);
            f[2 * e] = p.x, f[2 * e + 1] = p.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            f[e] = widen(v.v[e]);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> narrowed(const float (&f)[VEC])
{
    Vec<T, VEC> v;
    if constexpr (VEC % 2 == 0 && sizeof(T) == 2) {
        uint32_t *w = reinterpret_cast<uint32_t *>(v.v);
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e)
            w[e] = narrow2<T>(make_float2(f[2 * e], f[2 * e + 1]));
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            v.v[e] = narrow<T>(f[e]);
    }
    return v;
}
// d = a b + c by pairs.
template <int VEC>
__device__ __forceinline__ void fma_all(float (&d)[VEC], const float (&a)[VEC], const float (&b)[VEC], const float (&c)[VEC])
{
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const float2 r = fma2(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]), make_float2(c[e], c[e + 1]));
            d[e] = r.x, d[e + 1] = r.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            d[e] = fmaf(a[e], b[e], c[e]);
    }
}
template <int VEC>
__device__ __forceinline__ void add_to(float (&d)[VEC], const float (&a)[VEC])
{
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const float2 r = add2(make_float2(d[e], d[e + 1]), make_float2(a[e], a[e + 1]));
            d[e] = r.x, d[e + 1] = r.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            d[e] += a[e];
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int m = 16; m; m /= 2)
        v += __shfl_xor_sync(~0u, v, m);
    return v;
}

// Lanes that share a group's join where a CTA has so many groups: as many as let all groups join at once.
__device__ __forceinline__ int team_of(int groups)
{
    int t = 32;
    while (t > 1 && t * groups > kThreads)
        t /= 2;
    return t;
}
__device__ __forceinline__ float team_sum(float v, int team)
{
    for (int m = team / 2; m; m /= 2)
        v += __shfl_xor_sync(~0u, v, m);
    return v;
}

// Joins means and sums of squares about them, `many` parts by a team of lanes: the mean first, then what the parts' means
// spread about it (part(i): count, mean, squares).  -> count, mean, squares.  All lanes of a warp call it.
template <typename F>
__device__ __forceinline__ float3 join_parts(int many, int team, F part)
{
    const int lane = threadIdx.x % team;
    float n = 0.f, sum = 0.f, sq = 0.f;
#pragma unroll 4
    for (int i = lane; i < many; i += team) {
        const float3 p = part(i);
        n += p.x;
        sum = fmaf(p.x, p.y, sum);
    }
    n = team_sum(n, team);
    const float mean = team_sum(sum, team) / n;
#pragma unroll 4
    for (int i = lane; i < many; i += team) {
        const float3 p = part(i);
        const float d = p.y - mean;
        sq += p.x > 0.f ? fmaf(p.x * d, d, p.z) : 0.f;
    }
    return make_float3(n, mean, team_sum(sq, team));
}

// Sum of two values over the lanes of a group: L lanes of a warp, or L / 32 warps by way of shared memory.
__device__ __forceinline__ float2 group_sum(float2 v, int L, float2 *part)
{
    const int in = L < 32 ? L : 32;
    for (int m = in / 2; m; m /= 2) {
        v.x += __shfl_xor_sync(~0u, v.x, m);
        v.y += __shfl_xor_sync(~0u, v.y, m);
    }
    if (L > 32) {
        const int warp = threadIdx.x / 32, first = warp & ~(L / 32 - 1);
        __syncthreads();
        if (threadIdx.x % 32 == 0)
            part[warp] = v;
        __syncthreads();
        v = part[first];
        for (int i = 1; i < L / 32; ++i) {
            v.x += part[first + i].x;
            v.y += part[first + i].y;
        }
    }
    return v;
}

// ---------------------------------------------------------------------------------------------------------
// Tokens: one position a sample.  Unit u is group u % G of sample u / G; a CTA holds kThreads / L units, and the grid's
// units are a multiple of G, so that a lane's next unit has the same channels.
// ---------------------------------------------------------------------------------------------------------
// UNITS: of a lane's group at a time, so that enough loads are under way.
template <typename T, int VEC, int NV, int UNITS, bool SILU>
__global__ void __launch_bounds__(kThreads) tokens_kernel(GroupNormArgs a, int L)
{
    __shared__ float2 part[kThreads / 32];
    tc::grid_dep_wait();
    const int W = a.W, lane = threadIdx.x % L, per = kThreads / L;
    const int64_t units = a.N * a.G, stride = (int64_t)gridDim.x * per;
    const int64_t u0 = (int64_t)blockIdx.x * per + threadIdx.x / L;
    const int c0 = (int)(u0 % a.G) * W;
    const float inv = 1.f / W;
    typedef Vec<T, VEC> V;
    float w[NV][VEC], b[NV][VEC];
    bool on[NV];
    V x[UNITS][NV] = {};
    auto ask = [&](int64_t u) {
#pragma unroll
        for (int k = 0; k < UNITS; ++k)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (on[i] && u + k * stride < units)
                    x[k][i] = *reinterpret_cast<const V *>(static_cast<const T *>(a.x) + (u + k * stride) * W + (lane + L * i) * VEC);
    };
#pragma unroll
    for (int i = 0; i < NV; ++i)
        on[i] = (lane + L * i) * VEC < W;
    ask(u0);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = c0 + (lane + L * i) * VEC + e;
            w[i][e] = a.w && on[i] ? a.w[c] : 1.f;
            b[i][e] = a.b && on[i] ? a.b[c] : 0.f;
        }
    // all of a CTA's units take the same turns, as they may share its barriers
    for (int64_t base = (int64_t)blockIdx.x * per; base < units; base += UNITS * stride) {
        const int64_t u = base + threadIdx.x / L;
        float f[UNITS][NV][VEC], mean[UNITS], rstd[UNITS];
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            float sum[VEC] = {};   // lanes without values hold zeros
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                widened(x[k][i], f[k][i]);
                add_to(sum, f[k][i]);
            }
            mean[k] = 0.f;
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                mean[k] += sum[e];
        }
        ask(u + UNITS * stride);
#pragma unroll
        for (int k = 0; k < UNITS; ++k)
            mean[k] = group_sum(make_float2(mean[k], 0.f), L, part).x * inv;
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            rstd[k] = 0.f;
            float minus[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                minus[e] = -mean[k];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float sq[VEC] = {};
                add_to(f[k][i], minus);
                fma_all(sq, f[k][i], f[k][i], sq);
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    sum += sq[e];
                rstd[k] += on[i] ? sum : 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < UNITS; ++k)
            rstd[k] = rsqrtf(fmaf(group_sum(make_float2(rstd[k], 0.f), L, part).x, inv, a.eps));
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const int64_t at = u + k * stride;
            if (at >= units)
                continue;
            float r[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                r[e] = rstd[k];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!on[i])
                    continue;
                float y[VEC], zero[VEC] = {};
                fma_all(y, f[k][i], r, zero);
                fma_all(y, y, w[i], b[i]);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    y[e] = activated<SILU>(y[e]);
                *reinterpret_cast<V *>(static_cast<T *>(a.y) + at * W + (lane + L * i) * VEC) = narrowed<T, VEC>(y);
            }
            if (lane == 0) {
                a.mean[at] = mean[k];
                a.rstd[at] = rstd[k];
            }
        }
    }
}

template <typename T, int VEC, int NV, bool SILU>
__global__ void __launch_bounds__(kThreads) tokens_grad_kernel(GroupNormArgs a, int L)
{
    __shared__ float2 part[kThreads / 32];
    tc::grid_dep_wait();
    const int W = a.W, lane = threadIdx.x % L, per = kThreads / L;
    const int64_t units = a.N * a.G, stride = (int64_t)gridDim.x * per;
    const int64_t u0 = (int64_t)blockIdx.x * per + threadIdx.x / L;
    const int c0 = (int)(u0 % a.G) * W;
    const float inv = 1.f / W;
    typedef Vec<T, VEC> V;
    float w[NV][VEC], b[NV][VEC], dw[NV][VEC], db[NV][VEC];
    bool on[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + L * i) * VEC;
        on[i] = c < W;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            w[i][e] = a.w && on[i] ? a.w[c0 + c + e] : 1.f;
            b[i][e] = a.b && on[i] ? a.b[c0 + c + e] : 0.f;
            dw[i][e] = db[i][e] = 0.f;
        }
    }
    auto ask = [&](const void *p, int64_t u, V (&r)[NV]) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (on[i] && u < units)
                r[i] = *reinterpret_cast<const V *>(static_cast<const T *>(p) + u * W + (lane + L * i) * VEC);
    };
    V next[NV] = {}, next_dy[NV] = {};
    ask(a.x, u0, next);
    ask(a.dy, u0, next_dy);
    // all of a CTA's units take the same turns, as they may share its barriers
    for (int64_t base = (int64_t)blockIdx.x * per; base < units; base += stride) {
        const int64_t u = base + threadIdx.x / L;
        const bool live = u < units;
        V x[NV], dy[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i] = next[i];
            dy[i] = next_dy[i];
        }
        ask(a.x, u + stride, next);
        ask(a.dy, u + stride, next_dy);
        const float mean = live ? a.mean_in[u] : 0.f, rstd = live ? a.rstd_in[u] : 0.f;
        float xh[NV][VEC], g[NV][VEC];
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                if (!on[i] || !live)
                    continue;
                const float n = (widen(x[i].v[e]) - mean) * rstd;
                const float dz = before_act<SILU>(widen(dy[i].v[e]), fmaf(n, w[i][e], b[i][e]));
                db[i][e] += dz;
                dw[i][e] = fmaf(dz, n, dw[i][e]);
                xh[i][e] = n;
                g[i][e] = dz * w[i][e];
                sum = make_float2(sum.x + g[i][e], fmaf(g[i][e], n, sum.y));
            }
        sum = group_sum(sum, L, part);
        if (!live)
            continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!on[i])
                continue;
            V dx;
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                dx.v[e] = narrow<T>(rstd * (g[i][e] - inv * fmaf(xh[i][e], sum.y, sum.x)));
            *reinterpret_cast<V *>(static_cast<T *>(a.dx) + u * W + (lane + L * i) * VEC) = dx;
        }
    }
    if (!a.part_dw)
        return;
    float *pw = a.part_dw + (size_t)u0 * W, *pb = a.part_db + (size_t)u0 * W;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (on[i]) {
                pw[(lane + L * i) * VEC + e] = dw[i][e];
                pb[(lane + L * i) * VEC + e] = db[i][e];
            }
}

// ---------------------------------------------------------------------------------------------------------
// Maps.  CTA (sample, slice of positions, chunk of channels): TX threads on adjacent vectors, TY rows at a time.
// ---------------------------------------------------------------------------------------------------------
struct Slice {
    int64_t n, row0, rows;     // sample, first position and positions
    int slice, chunk, c0, cc;  // channels [c0, c0 + cc)
};
__device__ __forceinline__ Slice slice_of(const GroupNormArgs &a, const GroupNormSplit &s)
{
    Slice r;
    r.chunk = blockIdx.x % s.chunks;
    const int64_t i = blockIdx.x / s.chunks;
    r.slice = (int)(i % s.slices);
    r.n = i / s.slices;
    r.row0 = r.slice * s.rows;
    r.rows = min(s.rows, a.S - r.row0);
    r.c0 = r.chunk * s.chunk;
    r.cc = min(s.chunk, a.C - r.c0);
    return r;
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) maps_sums_kernel(GroupNormArgs a, GroupNormSplit sp)
{
    __shared__ float2 held[kThreads * VEC];
    tc::grid_dep_wait();
    const Slice s = slice_of(a, sp);
    const int tx = threadIdx.x % sp.tx, ty = threadIdx.x / sp.tx;
    const bool on = ty < sp.ty && tx * VEC < s.cc;
    typedef Vec<T, VEC> V;
    const T *x = static_cast<const T *>(a.x) + (s.n * a.S + s.row0) * a.C + s.c0 + tx * VEC;
    auto rows_of = [&](int y) { return y < s.rows ? (float)((s.rows - y + sp.ty - 1) / sp.ty) : 0.f; };
    const bool whole = a.W % VEC == 0;   // a vector's channels are of one group
    if (on) {
        const float many = rows_of(ty), inv = many > 0.f ? 1.f / many : 0.f;
        float mean[VEC] = {}, m2[VEC] = {};
        if (many > 0.f) {
            float minus[VEC], s1[VEC] = {}, s2[VEC] = {};
            widened(*reinterpret_cast<const V *>(x + (int64_t)ty * a.C), minus);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                minus[e] = -minus[e];
#pragma unroll 4
            for (int64_t r = ty + sp.ty; r < s.rows; r += sp.ty) {
                float d[VEC];
                widened(*reinterpret_cast<const V *>(x + r * a.C), d);
                add_to(d, minus);
                add_to(s1, d);
                fma_all(s2, d, d, s2);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                mean[e] = fmaf(s1[e], inv, -minus[e]);
                m2[e] = s2[e] - s1[e] * (s1[e] * inv);
                m2[e] = m2[e] < 0.f ? 0.f : m2[e];   // a NaN stays
            }
        }
        if (whole) {   // of equal counts: the mean of the means, and what they spread
            float sum = 0.f, sq = 0.f;
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                sum += mean[e];
            const float at = sum * (1.f / VEC);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                sq += fmaf(many * (mean[e] - at), mean[e] - at, m2[e]);
            held[ty * sp.tx + tx] = make_float2(at, sq);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                held[ty * sp.chunk + tx * VEC + e] = make_float2(mean[e], m2[e]);
        }
    }
    __syncthreads();
    const int unit = whole ? VEC : 1, pitch = sp.chunk / unit;   // channels of an entry, entries of a row
    const int g0 = s.c0 / a.W, groups = (s.c0 + s.cc - 1) / a.W - g0 + 1, team = team_of(groups);
    for (int first = 0; first < groups; first += kThreads / team) {
        const int k = first + threadIdx.x / team, g = g0 + min(k, groups - 1);
        const int lo = max(g * a.W, s.c0) - s.c0, width = (min((g + 1) * a.W, s.c0 + s.cc) - s.c0 - lo) / unit;
        const float3 m = join_parts(width * sp.ty, team, [&](int i) {
            const int y = i / width;
            const float2 h = held[y * pitch + lo / unit + i - y * width];
            return make_float3(rows_of(y) * unit, h.x, h.y);
        });
        if (k < groups && threadIdx.x % team == 0)
            a.part[(s.n * sp.slices + s.slice) * sp.entries + g + s.chunk] = make_float4(m.x, m.y, m.z, 0.f);
    }
}

// The statistics of the groups of a CTA's chunk, joined over the slices, to shared memory.
__device__ __forceinline__ void join_slices(const GroupNormArgs &a, const GroupNormSplit &sp, const Slice &s, float2 *stat)
{
    const int g0 = s.c0 / a.W, groups = (s.c0 + s.cc - 1) / a.W - g0 + 1, team = team_of(groups);
    for (int first = 0; first < groups; first += kThreads / team) {
        const int at = first + threadIdx.x / team, g = g0 + min(at, groups - 1);
        const int k0 = g * a.W / sp.chunk, chunks = ((g + 1) * a.W - 1) / sp.chunk - k0 + 1;   // chunks with its channels
        const float4 *from = a.part + s.n * sp.slices * sp.entries + g + k0;
        const float3 m = join_parts(sp.slices * chunks, team, [&](int i) {
            const int sl = chunks == 1 ? i : i / chunks;
            const float4 p = from[sl * sp.entries + i - sl * chunks];
            return make_float3(p.x, p.y, p.z);
        });
        const float rstd = rsqrtf(m.z / m.x + a.eps);
        if (at < groups && threadIdx.x % team == 0) {
            stat[at] = make_float2(m.y, rstd);
            if (s.slice == 0 && k0 == s.chunk) {   // one CTA writes them
                a.mean[s.n * a.G + g] = m.y;
                a.rstd[s.n * a.G + g] = rstd;
            }
        }
    }
    __syncthreads();
}

template <typename T, int VEC, bool SILU>
__global__ void __launch_bounds__(kThreads) maps_apply_kernel(GroupNormArgs a, GroupNormSplit sp)
{
    extern __shared__ float2 stat[];
    tc::grid_dep_wait();
    const Slice s = slice_of(a, sp);
    join_slices(a, sp, s, stat);
    const int tx = threadIdx.x % sp.tx, ty = threadIdx.x / sp.tx, g0 = s.c0 / a.W;
    if (ty >= sp.ty || tx * VEC >= s.cc)
        return;
    float minus[VEC], f[VEC], b[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int c = s.c0 + tx * VEC + e;
        const float2 st = stat[c / a.W - g0];
        minus[e] = -st.x;
        f[e] = a.w ? st.y * a.w[c] : st.y;
        b[e] = a.b ? a.b[c] : 0.f;
    }
    typedef Vec<T, VEC> V;
    const int64_t at = (s.n * a.S + s.row0) * a.C + s.c0 + tx * VEC;
    const T *x = static_cast<const T *>(a.x) + at;
    T *y = static_cast<T *>(a.y) + at;
#pragma unroll 4
    for (int64_t r = ty; r < s.rows; r += sp.ty) {
        float v[VEC];
        widened(*reinterpret_cast<const V *>(x + r * a.C), v);
        add_to(v, minus);
        fma_all(v, v, f, b);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            v[e] = activated<SILU>(v[e]);
        *reinterpret_cast<V *>(y + r * a.C) = narrowed<T, VEC>(v);
    }
}

// Backward, first pass: dz and dz xh summed per channel over a slice, and w times them by group.
template <typename T, int VEC, bool SILU>
__global__ void __launch_bounds__(kThreads) maps_grad_sums_kernel(GroupNormArgs a, GroupNormSplit sp)
{
    __shared__ float2 held[kThreads * VEC];
    tc::grid_dep_wait();
    const Slice s = slice_of(a, sp);
    const int tx = threadIdx.x % sp.tx, ty = threadIdx.x / sp.tx;
    if (ty < sp.ty && tx * VEC < s.cc) {
        float minus[VEC], rstd[VEC], w[VEC], b[VEC], zero[VEC] = {}, sum_z[VEC] = {}, sum_zn[VEC] = {};
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = s.c0 + tx * VEC + e;
            const int64_t g = s.n * a.G + c / a.W;
            minus[e] = -a.mean_in[g];
            rstd[e] = a.rstd_in[g];
            w[e] = a.w ? a.w[c] : 1.f;
            b[e] = a.b ? a.b[c] : 0.f;
        }
        typedef Vec<T, VEC> V;
        const int64_t at = (s.n * a.S + s.row0) * a.C + s.c0 + tx * VEC;
        const T *x = static_cast<const T *>(a.x) + at, *dy = static_cast<const T *>(a.dy) + at;
#pragma unroll 4
        for (int64_t r = ty; r < s.rows; r += sp.ty) {
            float n[VEC], dz[VEC];
            widened(*reinterpret_cast<const V *>(x + r * a.C), n);
            widened(*reinterpret_cast<const V *>(dy + r * a.C), dz);
            add_to(n, minus);
            fma_all(n, n, rstd, zero);
            if constexpr (SILU) {
                float z[VEC];
                fma_all(z, n, w, b);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    dz[e] = before_act<SILU>(dz[e], z[e]);
            }
            add_to(sum_z, dz);
            fma_all(sum_zn, dz, n, sum_zn);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            held[ty * sp.chunk + tx * VEC + e] = make_float2(sum_z[e], sum_zn[e]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < s.cc; c += kThreads) {
        float2 t = held[c];
        for (int y = 1; y < sp.ty; ++y) {
            const float2 h = held[y * sp.chunk + c];
            t = make_float2(t.x + h.x, t.y + h.y);
        }
        if (a.part_dw) {
            const int64_t at = (s.n * sp.slices + s.slice) * a.C + s.c0 + c;
            a.part_db[at] = t.x;
            a.part_dw[at] = t.y;
        }
        const float w = a.w ? a.w[s.c0 + c] : 1.f;
        held[c] = make_float2(w * t.x, w * t.y);
    }
    __syncthreads();
    const int g0 = s.c0 / a.W, groups = (s.c0 + s.cc - 1) / a.W - g0 + 1, team = team_of(groups);
    for (int first = 0; first < groups; first += kThreads / team) {
        const int k = first + threadIdx.x / team, g = g0 + min(k, groups - 1);
        const int lo = max(g * a.W, s.c0) - s.c0, hi = min((g + 1) * a.W, s.c0 + s.cc) - s.c0;
        float2 t = make_float2(0.f, 0.f);
        for (int c = lo + threadIdx.x % team; c < hi; c += team)
            t = make_float2(t.x + held[c].x, t.y + held[c].y);
        t = make_float2(team_sum(t.x, team), team_sum(t.y, team));
        if (k < groups && threadIdx.x % team == 0)
            a.part[(s.n * sp.slices + s.slice) * sp.entries + g + s.chunk] = make_float4(t.x, t.y, 0.f, 0.f);
    }
}

// Backward, second pass: dx.
template <typename T, int VEC, bool SILU>
__global__ void __launch_bounds__(kThreads) maps_grad_kernel(GroupNormArgs a, GroupNormSplit sp)
{
    extern __shared__ float2 stat[];
    tc::grid_dep_wait();
    const Slice s = slice_of(a, sp);
    const int g0 = s.c0 / a.W, groups = (s.c0 + s.cc - 1) / a.W - g0 + 1, team = team_of(groups);
    const float inv = 1.f / ((float)a.W * (float)a.S);
    for (int first = 0; first < groups; first += kThreads / team) {
        const int at = first + threadIdx.x / team, g = g0 + min(at, groups - 1);
        const int k0 = g * a.W / sp.chunk, chunks = ((g + 1) * a.W - 1) / sp.chunk - k0 + 1;
        const float4 *from = a.part + s.n * sp.slices * sp.entries + g + k0;
        float2 t = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int i = threadIdx.x % team; i < sp.slices * chunks; i += team) {
            const int sl = chunks == 1 ? i : i / chunks;
            const float4 p = from[sl * sp.entries + i - sl * chunks];
            t = make_float2(t.x + p.x, t.y + p.y);
        }
        t = make_float2(team_sum(t.x, team), team_sum(t.y, team));
        if (at < groups && threadIdx.x % team == 0)
            stat[at] = make_float2(t.x * inv, t.y * inv);
    }
    __syncthreads();
    const int tx = threadIdx.x % sp.tx, ty = threadIdx.x / sp.tx;
    if (ty >= sp.ty || tx * VEC >= s.cc)
        return;
    float minus[VEC], rstd[VEC], w[VEC], b[VEC], m1[VEC], m2[VEC], zero[VEC] = {};
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int c = s.c0 + tx * VEC + e;
        const int64_t g = s.n * a.G + c / a.W;
        const float2 st = stat[c / a.W - g0];
        m1[e] = -st.x, m2[e] = -st.y;
        minus[e] = -a.mean_in[g];
        rstd[e] = a.rstd_in[g];
        w[e] = a.w ? a.w[c] : 1.f;
        b[e] = a.b ? a.b[c] : 0.f;
    }
    typedef Vec<T, VEC> V;
    const int64_t at = (s.n * a.S + s.row0) * a.C + s.c0 + tx * VEC;
    const T *x = static_cast<const T *>(a.x) + at, *dy = static_cast<const T *>(a.dy) + at;
    T *dx = static_cast<T *>(a.dx) + at;
#pragma unroll 2
    for (int64_t r = ty; r < s.rows; r += sp.ty) {
        float n[VEC], dz[VEC], o[VEC];
        widened(*reinterpret_cast<const V *>(x + r * a.C), n);
        widened(*reinterpret_cast<const V *>(dy + r * a.C), dz);
        add_to(n, minus);
        fma_all(n, n, rstd, zero);
        if constexpr (SILU) {
            float z[VEC];
            fma_all(z, n, w, b);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                dz[e] = before_act<SILU>(dz[e], z[e]);
        }
        fma_all(o, w, dz, m1);
        fma_all(o, n, m2, o);
        fma_all(o, o, rstd, zero);
        *reinterpret_cast<V *>(dx + r * a.C) = narrowed<T, VEC>(o);
    }
}

// dw and db from their partial sums: `many` rows of C, 32 columns a CTA.
__global__ void __launch_bounds__(1024) group_norm_dw_kernel(GroupNormArgs a, int64_t many)
{
    __shared__ float2 held[32][33];
    tc::grid_dep_wait();
    const int lane = threadIdx.x % 32, y = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    float2 t = make_float2(0.f, 0.f);
    if (c < a.C)
#pragma unroll 8
        for (int64_t r = y; r < many; r += 32)
            t = make_float2(t.x + a.part_dw[r * a.C + c], t.y + a.part_db[r * a.C + c]);
    held[y][lane] = t;
    __syncthreads();
    t = held[lane][y];   // a warp joins a column
    t = make_float2(warp_sum(t.x), warp_sum(t.y));
    const int at = blockIdx.x * 32 + y;
    if (lane == 0 && at < a.C) {
        if (a.dw) a.dw[at] = t.x;
        if (a.db) a.db[at] = t.y;
    }
}

// Vector width: whole 16-byte units where the groups of tokens (the rows of maps) are made of them.
int vec_of(const GroupNormArgs &a, int dtype, bool tokens)
{
    const int vec = dtype == GLA_F32 ? 4 : 8;
    return (tokens ? a.W : a.C) % vec ? 1 : vec;
}

// Lanes of a group and vectors of a lane of the tokens' kernel: as few vectors as 32 lanes allow, then more lanes.
void lanes_of(int W, int vec, int &L, int &nv)
{
    const int vectors = (W + vec - 1) / vec, most = 16 / vec;
    L = 1;
    while (L < 32 && L < vectors)
        L *= 2;
    nv = 1;
    while (nv < most && L * nv < vectors)
        nv *= 2;
    while (L * nv < vectors)
        L *= 2;
}

}  // namespace

bool group_norm_tokens(int64_t S, int W) { return S == 1 && W <= 4096; }

int64_t group_norm_token_ctas(const GroupNormArgs &a, int dtype, bool back)
{
    int L, nv;
    lanes_of(a.W, vec_of(a, dtype, true), L, nv);
    const int64_t per = kThreads / L, q = a.G / std::gcd((int64_t)a.G, per), need = (a.N * a.G + per - 1) / per;
    const int64_t cap = (int64_t)sm_count() * (back ? 3 : 6);
    return std::max<int64_t>(1, std::min((need + q - 1) / q, std::max<int64_t>(cap / q, 1))) * q;
}

int64_t group_norm_token_parts(const GroupNormArgs &a, int dtype)   // rows of C of partial sums of dw
{
    int L, nv;
    lanes_of(a.W, vec_of(a, dtype, true), L, nv);
    return group_norm_token_ctas(a, dtype, true) * (kThreads / L) / a.G;
}

// Enough slices that the CTAs fill the GPU four times (two CTAs an SM at least stay busy to the end), as long as each has
// 16 turns of rows, or as many as there are SMs with four turns.
GroupNormSplit group_norm_split(const GroupNormArgs &a, int dtype)
{
    const int vec = vec_of(a, dtype, false), vectors = a.C / vec;
    GroupNormSplit s;
    s.chunk = std::min(vectors, kThreads) * vec;
    s.chunks = (a.C + s.chunk - 1) / s.chunk;
    s.tx = s.chunk / vec;
    s.ty = kThreads / s.tx;
    s.entries = a.G + s.chunks - 1;
    const int64_t want = std::max<int64_t>(1, (4 * (int64_t)sm_count()) / std::max<int64_t>(1, a.N * s.chunks));
    const int64_t most = std::max<int64_t>(1, a.S / (16 * s.ty));
    const int64_t least = std::min<int64_t>(std::max<int64_t>(1, a.S / (4 * s.ty)), std::max<int64_t>(1, sm_count() / std::max<int64_t>(1, a.N * s.chunks)));
    const int64_t slices = std::max(least, std::min(want, most));
    s.rows = (a.S + slices - 1) / slices;
    s.slices = (int)((a.S + s.rows - 1) / s.rows);
    return s;
}

namespace {

template <typename F>
cudaError_t by_norm_type(int dtype, int vec, F f)
{
    auto go = [&](auto t) {
        typedef std::remove_pointer_t<decltype(t)> T;
        return vec == 1 ? f(t, std::integral_constant<int, 1>()) : f(t, std::integral_constant<int, 16 / sizeof(T)>());
    };
    switch (dtype) {
    case GLA_F32: return go((float *)0);
    case GLA_BF16: return go((__nv_bfloat16 *)0);
    case GLA_F16: return go((__half *)0);
    default: return cudaErrorInvalidValue;
    }
}

size_t stat_bytes(const GroupNormArgs &a, const GroupNormSplit &sp)
{
    return sizeof(float2) * std::min<int64_t>(a.G, (sp.chunk - 2) / a.W + 2 + 1);
}

}  // namespace

cudaError_t launch_group_norm_tokens(const GroupNormArgs &a, int dtype, bool back, cudaStream_t s)
{
    const int vec = vec_of(a, dtype, true);
    int L, nv;
    lanes_of(a.W, vec, L, nv);
    const unsigned grid = (unsigned)group_norm_token_ctas(a, dtype, back);
    return by_norm_type(dtype, vec, [&](auto t, auto v) {
        typedef std::remove_pointer_t<decltype(t)> T;
        constexpr int VEC = decltype(v)::value;
        auto go = [&](auto count) {
            constexpr int NV = decltype(count)::value;
            constexpr int kUnits = VEC * NV <= 4 ? 4 : VEC * NV <= 8 ? 2 : 1;
            if (back)
                return a.silu ? launch_early(tokens_grad_kernel<T, VEC, NV, true>, grid, kThreads, s, a, L)
                              : launch_early(tokens_grad_kernel<T, VEC, NV, false>, grid, kThreads, s, a, L);
            return a.silu ? launch_early(tokens_kernel<T, VEC, NV, kUnits, true>, grid, kThreads, s, a, L)
                          : launch_early(tokens_kernel<T, VEC, NV, kUnits, false>, grid, kThreads, s, a, L);
        };
        if (nv == 1) return go(std::integral_constant<int, 1>());
        if (nv == 2) return go(std::integral_constant<int, 2>());
        if constexpr (VEC <= 4)
            if (nv == 4) return go(std::integral_constant<int, 4>());
        if constexpr (VEC == 1) {
            if (nv == 8) return go(std::integral_constant<int, 8>());
            return go(std::integral_constant<int, 16>());
        }
        return cudaErrorInvalidValue;
    });
}

cudaError_t launch_group_norm_maps(const GroupNormArgs &a, const GroupNormSplit &sp, int dtype, bool back, int pass, cudaStream_t s)
{
    const unsigned grid = (unsigned)(a.N * sp.slices * sp.chunks);
    return by_norm_type(dtype, vec_of(a, dtype, false), [&](auto t, auto v) {
        typedef std::remove_pointer_t<decltype(t)> T;
        constexpr int VEC = decltype(v)::value;
        auto by_act = [&](auto silu) {
            constexpr bool SILU = decltype(silu)::value;
            if (back)
                return pass == 0 ? launch_early(maps_grad_sums_kernel<T, VEC, SILU>, grid, kThreads, s, a, sp)
                                 : launch_early_shared(maps_grad_kernel<T, VEC, SILU>, grid, kThreads, stat_bytes(a, sp), s, a, sp);
            return pass == 0 ? launch_early(maps_sums_kernel<T, VEC>, grid, kThreads, s, a, sp)
                             : launch_early_shared(maps_apply_kernel<T, VEC, SILU>, grid, kThreads, stat_bytes(a, sp), s, a, sp);
        };
        return a.silu ? by_act(std::true_type()) : by_act(std::false_type());
    });
}

cudaError_t launch_group_norm_dw(const GroupNormArgs &a, int64_t many, cudaStream_t s)
{
    return launch_early(group_norm_dw_kernel, (unsigned)((a.C + 31) / 32), 1024, s, a, many);
}

}  // namespace gla
