// Gated delta rule token by token, for every type and head size up to 256 x 256 (the chunked kernels take 16-bit inputs
// of 64 or 128 key channels).  With a = exp(g_t), b = beta_t, per sequence and value head:
//
//     S~ = a S_{t-1},   n_t = b (v_t - k_t S~),   S_t = S~ + k_t^T n_t,   o_t = scale q_t S_t
//
// and for the gradients, with dS_t what reaches S_t from o_t and from later tokens:
//
//     dS_t += scale q_t^T do_t,   x_t = k_t dS_t,   dS_{t-1} = a (dS_t - b k_t^T x_t)
//     dv = b x,   dq = scale S do,   e = -S~ x,   f = dS n,   dk = b e + f,   dbeta = x.v + k.e
//     dg_t = sum over i >= t of (q.dq + b k.e - k.f)_i + <ht, dht>
//
// The columns of S and dS do not meet in n and x (delta_cols), nor their rows in dq, e and f (delta_rows), so each CTA
// walks all tokens for 16 columns (rows) of one head with its part of the state in registers: eight lanes hold a column,
// four adjacent values of every 32 each, so that a warp's loads of a token's vector from shared memory are one line that
// all its columns share.  Tokens arrive in blocks through registers and two buffers, one block ahead.  The whole is bound
// by the chain of a token's dot product (eight lanes: three shuffles) where there are few heads.
#include <type_traits>

#include "delta_internal.h"
#include "io.cuh"

namespace gla {
namespace {

constexpr int kThreads = 128, kLanes = 8, kTile = kThreads / kLanes;

__device__ __forceinline__ float group_sum(float v)   // over the eight lanes of a column
{
    v += __shfl_xor_sync(~0u, v, 4);
    v += __shfl_xor_sync(~0u, v, 2);
    return v + __shfl_xor_sync(~0u, v, 1);
}

// Dot product of a lane's share of two vectors, four partial sums.
template <int P>
__device__ __forceinline__ float dot(const float4 (&s)[P / 32], const float *x, int lane)
{
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < P / 32; ++i) {
        const float4 w = *reinterpret_cast<const float4 *>(x + i * 32 + lane * 4);
        sum = make_float4(fmaf(s[i].x, w.x, sum.x), fmaf(s[i].y, w.y, sum.y), fmaf(s[i].z, w.z, sum.z), fmaf(s[i].w, w.w, sum.w));
    }
    return (sum.x + sum.y) + (sum.z + sum.w);
}

// s = c s + x y
template <int P>
__device__ __forceinline__ void advance(float4 (&s)[P / 32], float c, const float *x, float y, int lane)
{
#pragma unroll
    for (int i = 0; i < P / 32; ++i) {
        const float4 w = *reinterpret_cast<const float4 *>(x + i * 32 + lane * 4);
        s[i] = make_float4(fmaf(c, s[i].x, w.x * y), fmaf(c, s[i].y, w.y * y), fmaf(c, s[i].z, w.z * y), fmaf(c, s[i].w, w.w * y));
    }
}

template <int P>
__device__ __forceinline__ void scale_by(float4 (&s)[P / 32], float c)
{
#pragma unroll
    for (int i = 0; i < P / 32; ++i)
        s[i] = make_float4(c * s[i].x, c * s[i].y, c * s[i].z, c * s[i].w);
}

// Reads (or writes) a lane's share of the state: values d = 0.. of P at p + d * pitch.
template <int P>
__device__ __forceinline__ void take(float4 (&s)[P / 32], const float *p, size_t pitch, int D, int lane, bool on)
{
#pragma unroll
    for (int i = 0; i < P / 32; ++i) {
        const int d = i * 32 + lane * 4;
        auto at = [&](int e) { return on && d + e < D ? p[(size_t)(d + e) * pitch] : 0.f; };
        s[i] = make_float4(at(0), at(1), at(2), at(3));
    }
}

template <int P>
__device__ __forceinline__ void put(const float4 (&s)[P / 32], float *p, size_t pitch, int D, int lane)
{
#pragma unroll
    for (int i = 0; i < P / 32; ++i) {
        const int d = i * 32 + lane * 4;
        if (d < D) p[(size_t)d * pitch] = s[i].x;
        if (d + 1 < D) p[(size_t)(d + 1) * pitch] = s[i].y;
        if (d + 2 < D) p[(size_t)(d + 2) * pitch] = s[i].z;
        if (d + 3 < D) p[(size_t)(d + 3) * pitch] = s[i].w;
    }
}

// What a CTA walks: sequence, head, tile of columns or rows, and the tokens' rows.
struct Walk {
    int n, hv, tile, bos, len;
    size_t head;   // n * HV + hv
};

__device__ __forceinline__ bool walk_of(const DeltaArgs &a, int tiles, Walk &w)
{
    w.tile = blockIdx.x % tiles;
    w.head = blockIdx.x / tiles;
    w.n = (int)(w.head / a.HV);
    w.hv = (int)(w.head - (size_t)w.n * a.HV);
    if (delta_sequence(a, w.n, w.bos, w.len))
        return true;
    if (threadIdx.x == 0)
        report(a.status, GLA_ERR_INVALID_ARG);
    return false;
}

// Columns of the state.  Forward: n, and o where it is asked for; backward: x and dv.
template <typename Tx, typename To, int P, bool BACK>
__global__ void __launch_bounds__(kThreads) delta_cols_kernel(DeltaArgs a, int tiles)
{
    constexpr int kBlock = 2048 / P, kEach = kBlock * P / kThreads, kVals = (kBlock * kTile + kThreads - 1) / kThreads;
    __shared__ __align__(16) float ks[2][kBlock][P], qs[2][kBlock][P], vs[2][kBlock][kTile];
    __shared__ float2 ab[2][kBlock];
    Walk w;
    if (!walk_of(a, tiles, w))
        return;
    const int tid = threadIdx.x, lane = tid % kLanes, mine = tid / kLanes, col = w.tile * kTile + mine;
    const int hk = w.hv / (a.HV / a.H);
    const Tx *q = static_cast<const Tx *>(a.q), *k = static_cast<const Tx *>(a.k);
    const Tx *v = static_cast<const Tx *>(BACK ? a.dout : a.v);
    const float *start = BACK ? a.dht : a.h0;
    const size_t state = w.head * a.K * a.V + col;
    float4 s[P / 32];
    take<P>(s, start ? start + state : nullptr, a.V, a.K, lane, start && col < a.V);

    float kr[kEach], qr[kEach], vr[kVals];
    float2 abr = make_float2(0.f, 0.f);
    auto row_of = [&](int t) { return w.bos + (BACK ? w.len - 1 - t : t); };
    auto fetch = [&](int block) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int e = i * kThreads + tid, j = e / P, d = e % P, t = block * kBlock + j;
            const bool on = t < w.len && d < a.K;
            const size_t at = on ? ((size_t)row_of(t) * a.H + hk) * a.K + d : 0;
            kr[i] = on ? widen(k[at]) : 0.f;
            qr[i] = on ? widen(q[at]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kVals; ++i) {
            const int e = i * kThreads + tid, j = e / kTile, c = w.tile * kTile + e % kTile, t = block * kBlock + j;
            vr[i] = j < kBlock && t < w.len && c < a.V ? widen(v[((size_t)row_of(t) * a.HV + w.hv) * a.V + c]) : 0.f;
        }
        if (tid < kBlock && block * kBlock + tid < w.len) {
            const size_t at = (size_t)row_of(block * kBlock + tid) * a.HV + w.hv;
            abr = make_float2(a.g[at], a.beta[at]);
        }
    };
    auto keep = [&](int b) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int e = i * kThreads + tid;
            ks[b][e / P][e % P] = kr[i];
            qs[b][e / P][e % P] = qr[i];
        }
#pragma unroll
        for (int i = 0; i < kVals; ++i) {
            const int e = i * kThreads + tid;
            if (e / kTile < kBlock)
                vs[b][e / kTile][e % kTile] = vr[i];
        }
        if (tid < kBlock)
            ab[b][tid] = make_float2(expf(abr.x), abr.y);
    };
    const int blocks = (w.len + kBlock - 1) / kBlock;
    if (blocks) {
        fetch(0);
        keep(0);
    }
    __syncthreads();
    for (int block = 0; block < blocks; ++block) {
        const int b = block & 1;
        if (block + 1 < blocks)
            fetch(block + 1);
        const int many = min(kBlock, w.len - block * kBlock);
        for (int j = 0; j < many; ++j) {
            const float2 c = ab[b][j];
            const size_t at = ((size_t)row_of(block * kBlock + j) * a.HV + w.hv) * a.V + col;
            const bool out = lane == 0 && col < a.V;
            if constexpr (!BACK) {
                const float n = c.y * (vs[b][j][mine] - c.x * group_sum(dot<P>(s, ks[b][j], lane)));
                advance<P>(s, c.x, ks[b][j], n, lane);
                if (a.upd && out)
                    a.upd[at] = n;
                if (a.o) {
                    const float o = a.scale * group_sum(dot<P>(s, qs[b][j], lane));
                    if (out)
                        static_cast<To *>(a.o)[at] = narrow<To>(o);
                }
            } else {
                advance<P>(s, 1.f, qs[b][j], a.scale * vs[b][j][mine], lane);
                const float x = group_sum(dot<P>(s, ks[b][j], lane)), back = c.y * x;
                advance<P>(s, 1.f, ks[b][j], -back, lane);
                scale_by<P>(s, c.x);
                if (out) {
                    a.dx[at] = x;
                    static_cast<Tx *>(a.dv)[at] = narrow<Tx>(back);
                }
            }
        }
        if (block + 1 < blocks)
            keep(b ^ 1);
        __syncthreads();
    }
    float *end = BACK ? a.dh0 : a.ht;
    if (end && col < a.V)
        put<P>(s, end + state, a.V, a.K, lane);
}

// Rows of the state, with n and x known.  Forward: dq and e; backward: f.
template <typename Tx, int P, bool BACK>
__global__ void __launch_bounds__(kThreads) delta_rows_kernel(DeltaArgs a, int tiles)
{
    constexpr int kBlock = 1024 / P, kEach = kBlock * P / kThreads, kVals = (kBlock * kTile + kThreads - 1) / kThreads;
    __shared__ __align__(16) float ns[2][kBlock][P], xs[2][kBlock][P], ds[2][kBlock][P];
    __shared__ float ks[2][kBlock][kTile], qs[2][kBlock][kTile];
    __shared__ float2 ab[2][kBlock];
    Walk w;
    if (!walk_of(a, tiles, w))
        return;
    const int tid = threadIdx.x, lane = tid % kLanes, mine = tid / kLanes, row = w.tile * kTile + mine;
    const int hk = w.hv / (a.HV / a.H);
    const Tx *q = static_cast<const Tx *>(a.q), *k = static_cast<const Tx *>(a.k), *d = static_cast<const Tx *>(a.dout);
    const float *start = BACK ? a.dht : a.h0;
    const size_t state = (w.head * a.K + row) * a.V;
    float4 s[P / 32];
    take<P>(s, start ? start + state : nullptr, 1, a.V, lane, start && row < a.K);

    float nr[kEach], xr[kEach], dr[kEach], kr[kVals], qr[kVals];
    float2 abr = make_float2(0.f, 0.f);
    auto row_of = [&](int t) { return w.bos + (BACK ? w.len - 1 - t : t); };
    auto fetch = [&](int block) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int e = i * kThreads + tid, j = e / P, c = e % P, t = block * kBlock + j;
            const bool on = t < w.len && c < a.V;
            const size_t at = on ? ((size_t)row_of(t) * a.HV + w.hv) * a.V + c : 0;
            nr[i] = on ? a.upd[at] : 0.f;
            xr[i] = on ? a.dx[at] : 0.f;
            dr[i] = on ? a.scale * widen(d[at]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kVals; ++i) {
            const int e = i * kThreads + tid, j = e / kTile, r = w.tile * kTile + e % kTile, t = block * kBlock + j;
            const bool on = j < kBlock && t < w.len && r < a.K;
            const size_t at = on ? ((size_t)row_of(t) * a.H + hk) * a.K + r : 0;
            kr[i] = on ? widen(k[at]) : 0.f;
            qr[i] = on ? widen(q[at]) : 0.f;
        }
        if (tid < kBlock && block * kBlock + tid < w.len) {
            const size_t at = (size_t)row_of(block * kBlock + tid) * a.HV + w.hv;
            abr = make_float2(a.g[at], a.beta[at]);
        }
    };
    auto keep = [&](int b) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int e = i * kThreads + tid;
            ns[b][e / P][e % P] = nr[i];
            xs[b][e / P][e % P] = xr[i];
            ds[b][e / P][e % P] = dr[i];
        }
#pragma unroll
        for (int i = 0; i < kVals; ++i) {
            const int e = i * kThreads + tid;
            if (e / kTile < kBlock) {
                ks[b][e / kTile][e % kTile] = kr[i];
                qs[b][e / kTile][e % kTile] = qr[i];
            }
        }
        if (tid < kBlock)
            ab[b][tid] = make_float2(expf(abr.x), abr.y);
    };
    const int blocks = (w.len + kBlock - 1) / kBlock;
    if (blocks) {
        fetch(0);
        keep(0);
    }
    __syncthreads();
    for (int block = 0; block < blocks; ++block) {
        const int b = block & 1;
        if (block + 1 < blocks)
            fetch(block + 1);
        const int many = min(kBlock, w.len - block * kBlock);
        for (int j = 0; j < many; ++j) {
            const float2 c = ab[b][j];
            const size_t at = ((size_t)row_of(block * kBlock + j) * a.HV + w.hv) * a.K + row;
            const bool out = lane == 0 && row < a.K;
            if constexpr (!BACK) {
                scale_by<P>(s, c.x);
                const float e = -group_sum(dot<P>(s, xs[b][j], lane));
                advance<P>(s, 1.f, ns[b][j], ks[b][j][mine], lane);
                const float dq = group_sum(dot<P>(s, ds[b][j], lane));
                if (out) {
                    a.eh[at] = e;
                    a.dqh[at] = dq;
                }
            } else {
                advance<P>(s, 1.f, ds[b][j], qs[b][j][mine], lane);
                const float f = group_sum(dot<P>(s, ns[b][j], lane));
                advance<P>(s, 1.f, xs[b][j], -c.y * ks[b][j][mine], lane);
                scale_by<P>(s, c.x);
                if (out)
                    a.fh[at] = f;
            }
        }
        if (block + 1 < blocks)
            keep(b ^ 1);
        __syncthreads();
    }
    if (!BACK && a.hd) {   // this row of <ht, dht>
        float4 t[P / 32];
        take<P>(t, a.dht + state, 1, a.V, lane, row < a.K);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < P / 32; ++i)
            sum += (s[i].x * t[i].x + s[i].y * t[i].y) + (s[i].z * t[i].z + s[i].w * t[i].w);
        sum = group_sum(sum);
        if (lane == 0 && row < a.K)
            a.hd[w.head * a.K + row] = sum;
    }
}

// Joins the value heads of a key head: dq, dk, dbeta, and the gradient of the running sum of gates.  A warp a row.
template <typename Tx>
__global__ void __launch_bounds__(kThreads) delta_join_kernel(DeltaArgs a)
{
    const int slot = blockIdx.x / a.H, h = blockIdx.x - slot * a.H, per = a.HV / a.H, lane = threadIdx.x % 32;
    int n, c, first, rows;
    if (!delta_chunk(a, slot, n, c, first, rows))
        return;
    const Tx *q = static_cast<const Tx *>(a.q), *k = static_cast<const Tx *>(a.k), *v = static_cast<const Tx *>(a.v);
    for (int r = threadIdx.x / 32; r < rows; r += kThreads / 32) {
        const size_t row = first + r, key = (row * a.H + h) * a.K;
        for (int j = 0; j < per; ++j) {   // the sums of each value head
            const size_t head = row * a.HV + h * per + j;
            float ke = 0.f, kf = 0.f, qd = 0.f, xv = 0.f;
            for (int d = lane; d < a.K; d += 32) {
                const float kd = widen(k[key + d]);
                ke = fmaf(kd, a.eh[head * a.K + d], ke);
                kf = fmaf(kd, a.fh[head * a.K + d], kf);
                qd = fmaf(widen(q[key + d]), a.dqh[head * a.K + d], qd);
            }
            for (int d = lane; d < a.V; d += 32)
                xv = fmaf(a.dx[head * a.V + d], widen(v[head * a.V + d]), xv);
#pragma unroll
            for (int m = 16; m; m /= 2) {
                ke += __shfl_xor_sync(~0u, ke, m);
                kf += __shfl_xor_sync(~0u, kf, m);
                qd += __shfl_xor_sync(~0u, qd, m);
                xv += __shfl_xor_sync(~0u, xv, m);
            }
            if (lane == 0) {
                a.dbeta[head] = xv + ke;
                a.dG[head] = qd + a.beta[head] * ke - kf;
            }
        }
        for (int d = lane; d < a.K; d += 32) {
            float dq = 0.f, dk = 0.f;
            for (int j = 0; j < per; ++j) {
                const size_t head = row * a.HV + h * per + j;
                dq += a.dqh[head * a.K + d];
                dk += fmaf(a.beta[head], a.eh[head * a.K + d], a.fh[head * a.K + d]);
            }
            static_cast<Tx *>(a.dq)[key + d] = narrow<Tx>(dq);
            static_cast<Tx *>(a.dk)[key + d] = narrow<Tx>(dk);
        }
    }
}

// dg: sums of dG from the end of each sequence, held in 64 bits as they run over all its tokens.
__global__ void __launch_bounds__(256) delta_gates_kernel(DeltaArgs a)
{
    __shared__ double part[8];
    const size_t head = blockIdx.x;
    const int n = (int)(head / a.HV), hv = (int)(head - (size_t)n * a.HV), tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    int bos, len;
    if (!delta_sequence(a, n, bos, len))
        return;
    double carry = 0.;
    if (a.hd)
        for (int d = 0; d < a.K; ++d)
            carry += a.hd[head * a.K + d];
    for (int base = 0; base < len; base += 256) {
        const int t = base + tid;   // from the end
        const size_t at = (size_t)(bos + len - 1 - t) * a.HV + hv;
        double v = t < len ? (double)a.dG[at] : 0.;
#pragma unroll
        for (int m = 1; m < 32; m *= 2) {
            const double u = __shfl_up_sync(~0u, v, m);
            if (lane >= m)
                v += u;
        }
        if (lane == 31)
            part[warp] = v;
        __syncthreads();
        double before = carry;
        for (int i = 0; i < 8; ++i) {
            if (i == warp && t < len)
                a.dg[at] = (float)(before + v);
            before += part[i];
        }
        carry = before;
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_delta_cols(const DeltaArgs &a, int dtype, bool backward, cudaStream_t s)
{
    const int tiles = (a.V + kTile - 1) / kTile;
    const unsigned grid = (unsigned)((size_t)a.N * a.HV * tiles);
    return delta_types(dtype, [&](auto x, auto o) {
        typedef std::remove_pointer_t<decltype(x)> Tx;
        typedef std::remove_pointer_t<decltype(o)> To;
        auto go = [&](auto p) {
            constexpr int P = decltype(p)::value;
            if (!backward)
                delta_cols_kernel<Tx, To, P, false><<<grid, kThreads, 0, s>>>(a, tiles);
            else if constexpr (std::is_same_v<To, float>)   // the backward has no outputs of another type
                delta_cols_kernel<Tx, float, P, true><<<grid, kThreads, 0, s>>>(a, tiles);
            return cudaGetLastError();
        };
        return a.K <= 64 ? go(std::integral_constant<int, 64>()) : a.K <= 128 ? go(std::integral_constant<int, 128>())
                                                                              : go(std::integral_constant<int, 256>());
    });
}

cudaError_t launch_delta_rows(const DeltaArgs &a, int dtype, bool backward, cudaStream_t s)
{
    const int tiles = (a.K + kTile - 1) / kTile;
    const unsigned grid = (unsigned)((size_t)a.N * a.HV * tiles);
    return delta_types(dtype, [&](auto x, auto o) {
        typedef std::remove_pointer_t<decltype(x)> Tx;
        if constexpr (std::is_same_v<std::remove_pointer_t<decltype(o)>, float>) {
            auto go = [&](auto p) {
                constexpr int P = decltype(p)::value;
                if (backward)
                    delta_rows_kernel<Tx, P, true><<<grid, kThreads, 0, s>>>(a, tiles);
                else
                    delta_rows_kernel<Tx, P, false><<<grid, kThreads, 0, s>>>(a, tiles);
                return cudaGetLastError();
            };
            return a.V <= 64 ? go(std::integral_constant<int, 64>()) : a.V <= 128 ? go(std::integral_constant<int, 128>())
                                                                                  : go(std::integral_constant<int, 256>());
        } else {
            return cudaErrorInvalidValue;
        }
    });
}

cudaError_t launch_delta_join(const DeltaArgs &a, int dtype, cudaStream_t s)
{
    const unsigned grid = (unsigned)((size_t)a.slots * a.H);
    return delta_types(dtype, [&](auto x, auto) {
        delta_join_kernel<std::remove_pointer_t<decltype(x)>><<<grid, kThreads, 0, s>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t launch_delta_gates(const DeltaArgs &a, cudaStream_t s)
{
    delta_gates_kernel<<<(unsigned)((size_t)a.N * a.HV), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace gla
