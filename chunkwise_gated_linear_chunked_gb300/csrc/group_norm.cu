// Group norm with an activation, channels last.  For sample n and group j of W = C / G channels, over all its positions:
//
//     mean, var over S x W values,   rstd = 1 / sqrt(var + eps),   xh = (x - mean) rstd,   z = xh w + b,   y = act(z)
//     dz = dy act'(z),   a = w dz,   dx = rstd (a - mean(a) - xh mean(a xh)),   dw = sum dz xh,   db = sum dz
//
// Two ways:
//
// One position a sample (tokens) and at most 4096 channels a group: a group is a run of memory that up to 256 lanes hold
// in registers, so that it is read once; variances are sums of squares about the mean.  A lane keeps its channels from
// sample to sample, with their weights and its share of dw and db in registers.  32768 tokens of 2048 channels in 16 groups,
// bf16: 50 us, 5.4 TB/s, bound by instructions (72 % of the issue slots): two groups a lane at a time and four CTAs an SM
// (five: 63 us, four groups at a time: 66).
//
// Otherwise (maps): samples are cut into slices of positions.  A CTA walks a slice with a vector of channels a thread and
// sums per channel, in blocks of at most 32 rows about the thread's first value and then about the mean of those before (so a
// mean far from zero costs nothing, and the sum of squares loses at most 32 units to the cancellation where that value is an
// outlier), joins the threads' means and squares by group, and a second kernel joins
// the slices and writes y (dx); it reads x again, from L2 where the tensor fits.  8 x 4096 positions of 512 channels with
// SiLU, bf16: 29 us forward, 52 backward with inputs in memory (22 and 45 where the last pass left them in L2), bound by the
// loads under way in kernels of one wave (27 % of the copy rate in the sums), by the latency of two (three) of them and by the
// two special functions of a sigmoid (each pass 7 us of them).  Every join has a fixed order, so results do not depend on timing.
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
constexpr int kSumRows = 32;   // rows of a thread whose squares are summed about one value

template <typename T, int VEC>
struct alignas(VEC * sizeof(T)) Vec {
    T v[VEC];
};

// sigmoid(z); its error is that of ex2 and rcp, about 3 units in the last place, and for negative z that of rounding z log2 e,
// which ex2 turns into 0.4 |z| units (8 at z = -20, 31 at -80) of a value that is small there: |z| sigmoid(z) <= 0.28.
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

// Sums over the lanes of a group: L lanes of a warp, or L / 32 warps by way of shared memory.
__device__ __forceinline__ void lanes_sum(float &v, int L)
{
#pragma unroll
    for (int m = 16; m; m /= 2)
        if (m < L)
            v += __shfl_xor_sync(~0u, v, m);
}
__device__ __forceinline__ float2 group_sum(float2 v, int L, float2 *part)
{
    lanes_sum(v.x, L);
    lanes_sum(v.y, L);
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
__device__ __forceinline__ float group_sum(float v, int L, float2 *part)
{
    if (L > 32)
        return group_sum(make_float2(v, 0.f), L, part).x;
    lanes_sum(v, L);
    return v;
}

// ---------------------------------------------------------------------------------------------------------
// Tokens: one position a sample.  Unit u is group u % G of sample u / G; a CTA holds kThreads / L units, and the grid's
// units are a multiple of G, so that a lane's next unit has the same channels.
// ---------------------------------------------------------------------------------------------------------
// UNITS: of a lane's group at a time, so that enough loads are under way.
template <typename T, int VEC, int NV, int UNITS, bool SILU>
__global__ void __launch_bounds__(kThreads, VEC * NV <= 8 ? 4 : 1) tokens_kernel(GroupNormArgs a, int L)
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
            mean[k] = group_sum(mean[k], L, part) * inv;
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
            rstd[k] = rsqrtf(fmaf(group_sum(rstd[k], L, part), inv, a.eps));
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
    // what is not there counts as zeros: then nothing of it reaches a sum
    V next[NV], next_dy[NV];
    float2 next_stat;
    auto ask = [&](int64_t u) {
        const bool live = u < units;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t at = u * W + (lane + L * i) * VEC;
            next[i] = live && on[i] ? *reinterpret_cast<const V *>(static_cast<const T *>(a.x) + at) : V{};
            next_dy[i] = live && on[i] ? *reinterpret_cast<const V *>(static_cast<const T *>(a.dy) + at) : V{};
        }
        next_stat = live ? make_float2(a.mean_in[u], a.rstd_in[u]) : make_float2(0.f, 0.f);
    };
    ask(u0);
    // all of a CTA's units take the same turns, as they may share its barriers
    for (int64_t base = (int64_t)blockIdx.x * per; base < units; base += stride) {
        const int64_t u = base + threadIdx.x / L;
        V x[NV], dy[NV];
        const float2 stat = next_stat;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i] = next[i];
            dy[i] = next_dy[i];
        }
        ask(u + stride);
        float xh[NV][VEC], g[NV][VEC], minus[VEC], rstd[VEC], s1[VEC] = {}, s2[VEC] = {}, zero[VEC] = {};
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            minus[e] = -stat.x, rstd[e] = stat.y;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float dz[VEC];
            widened(x[i], xh[i]);
            widened(dy[i], dz);
            add_to(xh[i], minus);
            fma_all(xh[i], xh[i], rstd, zero);
            if constexpr (SILU) {
                float z[VEC];
                fma_all(z, xh[i], w[i], b[i]);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    dz[e] = before_act<SILU>(dz[e], z[e]);
            }
            add_to(db[i], dz);
            fma_all(dw[i], dz, xh[i], dw[i]);
            fma_all(g[i], dz, w[i], zero);
            add_to(s1, g[i]);
            fma_all(s2, g[i], xh[i], s2);
        }
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            sum = make_float2(sum.x + s1[e], sum.y + s2[e]);
        sum = group_sum(sum, L, part);
        if (u >= units)
            continue;
        float m1[VEC], m2[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            m1[e] = -inv * sum.x, m2[e] = -inv * sum.y;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!on[i])
                continue;
            add_to(g[i], m1);
            fma_all(g[i], xh[i], m2, g[i]);
            fma_all(g[i], g[i], rstd, zero);
            *reinterpret_cast<V *>(static_cast<T *>(a.dx) + u * W + (lane + L * i) * VEC) = narrowed<T, VEC>(g[i]);
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
    int64_t n, at;             // sample, and first value of this thread's first row of the slice
    int rows;                  // positions
    int slice, chunk, c0, cc;  // channels [c0, c0 + cc)
    int tx, ty;                // this thread's vector and first row
    bool on;
};
template <int VEC>
__device__ __forceinline__ Slice slice_of(const GroupNormArgs &a, const GroupNormSplit &s)
{
    Slice r;
    const unsigned i = blockIdx.x / s.chunks, n = i / s.slices;
    r.chunk = blockIdx.x - i * s.chunks;
    r.slice = i - n * s.slices;
    r.n = n;
    const int64_t row0 = (int64_t)r.slice * s.rows;
    r.rows = (int)min((int64_t)s.rows, a.S - row0);
    r.c0 = r.chunk * s.chunk;
    r.cc = min(s.chunk, a.C - r.c0);
    r.ty = threadIdx.x / s.tx;
    r.tx = threadIdx.x - r.ty * s.tx;
    r.on = r.ty < s.ty && r.tx * VEC < r.cc;
    r.at = (r.n * a.S + row0 + r.ty) * a.C + r.c0 + r.tx * VEC;
    return r;
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) maps_sums_kernel(GroupNormArgs a, GroupNormSplit sp)
{
    __shared__ float2 held[kThreads * VEC];
    tc::grid_dep_wait();
    const Slice s = slice_of<VEC>(a, sp);
    const int64_t step = (int64_t)sp.ty * a.C;   // between a thread's rows
    typedef Vec<T, VEC> V;
    const T *x = static_cast<const T *>(a.x) + s.at;
    const int turns = s.rows / sp.ty, more = s.rows - turns * sp.ty;   // rows of a thread: one more of the first
    auto rows_of = [&](int y) { return (float)(turns + (y < more)); };
    const bool whole = a.W % VEC == 0;   // a vector's channels are of one group
    if (s.on) {
        const float many = rows_of(s.ty);
        float mean[VEC] = {}, m2[VEC] = {};
        if (many > 0.f) {
            // sums about `about`, at first the first value, behind each block of rows the mean so far but for `rest`
            float about[VEC], rest[VEC] = {}, n = 1.f;
            widened(*reinterpret_cast<const V *>(x), about);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                mean[e] = about[e];
            for (int r = s.ty + sp.ty; r < s.rows;) {
                const int end = min(s.rows, r + kSumRows * sp.ty);
                float minus[VEC], s1[VEC] = {}, s2[VEC] = {};
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    minus[e] = -about[e];
#pragma unroll 4
                for (; r < end; r += sp.ty) {
                    float d[VEC];
                    x += step;
                    widened(*reinterpret_cast<const V *>(x), d);
                    add_to(d, minus);
                    add_to(s1, d);
                    fma_all(s2, d, d, s2);
                }
                const float all = fminf(n + kSumRows, many), inv = 1.f / all;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float sum = fmaf(n, rest[e], s1[e]), by = sum * inv;   // the rows before are n times `rest` off
                    mean[e] = fmaf(sum, inv, about[e]);
                    m2[e] += s2[e] - sum * by;
                    const float to = about[e] + by, moved = to - about[e];
                    rest[e] = (about[e] - (to - moved)) + (by - moved);   // what the sum has lost
                    about[e] = to;
                }
                n = all;
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                m2[e] = m2[e] < 0.f ? 0.f : m2[e];   // a NaN stays
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
            held[s.ty * sp.tx + s.tx] = make_float2(at, sq);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                held[s.ty * sp.chunk + s.tx * VEC + e] = make_float2(mean[e], m2[e]);
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
    constexpr int kAhead = 4;
    extern __shared__ float2 stat[];
    tc::grid_dep_wait();
    const Slice s = slice_of<VEC>(a, sp);
    const int64_t step = (int64_t)sp.ty * a.C;   // between a thread's rows
    const int g0 = s.c0 / a.W;
    typedef Vec<T, VEC> V;
    const T *x = static_cast<const T *>(a.x) + s.at;
    T *y = static_cast<T *>(a.y) + s.at;
    V next[kAhead] = {};
    auto ask = [&](int r) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (s.on && r + k * sp.ty < s.rows)
                next[k] = *reinterpret_cast<const V *>(x);
            x += step;
        }
    };
    ask(s.ty);   // while the statistics are joined
    join_slices(a, sp, s, stat);
    if (!s.on)
        return;
    float minus[VEC], f[VEC], b[VEC];
    const bool whole = a.W % VEC == 0;
    int g = (s.c0 + s.tx * VEC) / a.W - g0;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int c = s.c0 + s.tx * VEC + e;
        if (!whole)
            g = c / a.W - g0;
        const float2 st = stat[g];
        minus[e] = -st.x;
        f[e] = a.w ? st.y * a.w[c] : st.y;
        b[e] = a.b ? a.b[c] : 0.f;
    }
    for (int r = s.ty; r < s.rows; r += kAhead * sp.ty) {
        V now[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            now[k] = next[k];
        ask(r + kAhead * sp.ty);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (r + k * sp.ty >= s.rows)
                break;
            float v[VEC];
            widened(now[k], v);
            add_to(v, minus);
            fma_all(v, v, f, b);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                v[e] = activated<SILU>(v[e]);
            *reinterpret_cast<V *>(y) = narrowed<T, VEC>(v);
            y += step;
        }
    }
}

// Backward, first pass: dz and dz xh summed per channel over a slice, and w times them by group.
template <typename T, int VEC, bool SILU>
__global__ void __launch_bounds__(kThreads) maps_grad_sums_kernel(GroupNormArgs a, GroupNormSplit sp)
{
    __shared__ float2 held[kThreads * VEC];
    tc::grid_dep_wait();
    const Slice s = slice_of<VEC>(a, sp);
    const int64_t step = (int64_t)sp.ty * a.C;   // between a thread's rows
    if (s.on) {
        float minus[VEC], rstd[VEC], w[VEC], b[VEC], zero[VEC] = {}, sum_z[VEC] = {}, sum_zn[VEC] = {};
        const bool whole = a.W % VEC == 0;
        int64_t g = s.n * a.G + (s.c0 + s.tx * VEC) / a.W;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = s.c0 + s.tx * VEC + e;
            if (!whole)
                g = s.n * a.G + c / a.W;
            minus[e] = -a.mean_in[g];
            rstd[e] = a.rstd_in[g];
            w[e] = a.w ? a.w[c] : 1.f;
            b[e] = a.b ? a.b[c] : 0.f;
        }
        typedef Vec<T, VEC> V;
        const T *x = static_cast<const T *>(a.x) + s.at, *dy = static_cast<const T *>(a.dy) + s.at;
#pragma unroll 4
        for (int r = s.ty; r < s.rows; r += sp.ty) {
            float n[VEC], dz[VEC];
            widened(*reinterpret_cast<const V *>(x), n);
            widened(*reinterpret_cast<const V *>(dy), dz);
            x += step, dy += step;
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
            held[s.ty * sp.chunk + s.tx * VEC + e] = make_float2(sum_z[e], sum_zn[e]);
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
    constexpr int kAhead = VEC == 8 ? 2 : 4;
    extern __shared__ float2 stat[];
    tc::grid_dep_wait();
    const Slice s = slice_of<VEC>(a, sp);
    const int64_t step = (int64_t)sp.ty * a.C;   // between a thread's rows
    typedef Vec<T, VEC> V;
    const T *x = static_cast<const T *>(a.x) + s.at, *dy = static_cast<const T *>(a.dy) + s.at;
    T *dx = static_cast<T *>(a.dx) + s.at;
    V next[kAhead] = {}, next_dy[kAhead] = {};
    auto ask = [&](int r) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (s.on && r + k * sp.ty < s.rows) {
                next[k] = *reinterpret_cast<const V *>(x);
                next_dy[k] = *reinterpret_cast<const V *>(dy);
            }
            x += step, dy += step;
        }
    };
    ask(s.ty);   // while the sums are joined
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
    if (!s.on)
        return;
    float minus[VEC], rstd[VEC], w[VEC], b[VEC], m1[VEC], m2[VEC], zero[VEC] = {};
    const bool whole = a.W % VEC == 0;
    int in = (s.c0 + s.tx * VEC) / a.W;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int c = s.c0 + s.tx * VEC + e;
        if (!whole)
            in = c / a.W;
        const int64_t g = s.n * a.G + in;
        const float2 st = stat[in - g0];
        m1[e] = -st.x, m2[e] = -st.y;
        minus[e] = -a.mean_in[g];
        rstd[e] = a.rstd_in[g];
        w[e] = a.w ? a.w[c] : 1.f;
        b[e] = a.b ? a.b[c] : 0.f;
    }
    for (int r = s.ty; r < s.rows; r += kAhead * sp.ty) {
        V now[kAhead], now_dy[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            now[k] = next[k], now_dy[k] = next_dy[k];
        ask(r + kAhead * sp.ty);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (r + k * sp.ty >= s.rows)
                break;
            float n[VEC], dz[VEC], o[VEC];
            widened(now[k], n);
            widened(now_dy[k], dz);
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
            *reinterpret_cast<V *>(dx) = narrowed<T, VEC>(o);
            dx += step;
        }
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
    const int64_t cap = (int64_t)sm_count() * (back ? 3 : 4);
    return std::max<int64_t>(1, std::min((need + q - 1) / q, std::max<int64_t>(cap / q, 1))) * q;
}

int64_t group_norm_token_parts(const GroupNormArgs &a, int dtype)   // rows of C of partial sums of dw
{
    int L, nv;
    lanes_of(a.W, vec_of(a, dtype, true), L, nv);
    return group_norm_token_ctas(a, dtype, true) * (kThreads / L) / a.G;
}

// Enough slices for two CTAs an SM (8 x 4096 x 512 in bf16 in L2, both kernels: 22.4 us; three 25.7, four 30, one 26: a CTA's start
// and its joins take about 3 us), as long as each has 16 turns of rows, or as many as there are SMs with four turns.
GroupNormSplit group_norm_split(const GroupNormArgs &a, int dtype)
{
    const int vec = vec_of(a, dtype, false), vectors = a.C / vec;
    GroupNormSplit s;
    s.chunk = std::min(vectors, kThreads) * vec;
    s.chunks = (a.C + s.chunk - 1) / s.chunk;
    s.tx = s.chunk / vec;
    s.ty = kThreads / s.tx;
    s.entries = a.G + s.chunks - 1;
    const int64_t want = std::max<int64_t>(1, (2 * (int64_t)sm_count()) / std::max<int64_t>(1, a.N * s.chunks));
    const int64_t most = std::max<int64_t>(1, a.S / (16 * s.ty));
    const int64_t least = std::min<int64_t>(std::max<int64_t>(1, a.S / (4 * s.ty)), std::max<int64_t>(1, sm_count() / std::max<int64_t>(1, a.N * s.chunks)));
    const int64_t slices = std::max(least, std::min(want, most));
    const int64_t rows = std::min<int64_t>((a.S + slices - 1) / slices, 1 << 30);
    s.rows = (int)rows;
    s.slices = (int)((a.S + rows - 1) / rows);
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
