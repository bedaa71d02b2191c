// Gated delta rule token by token, for every type and head size up to 256 x 256 (the chunked kernels take 16-bit inputs
// of 64 or 128 key channels).  With a = exp(g_t), b = beta_t, per sequence and value head:
//
//     S~ = a S_{t-1},   n_t = b (v_t - k_t S~),   S_t = S~ + k_t^T n_t,   o_t = scale q_t S_t
//
// and for the gradients, with dS_t what reaches S_t from o_t and from later tokens:
//
//     dS_t += scale q_t^T do_t,   x_t = k_t dS_t,   dS_{t-1} = a (dS_t - b k_t^T x_t)
//     dv = b x,   dq = scale S do,   e = -S~ x,   f = dS n,   dk = b e + f,   dbeta = x.v + k.e
//     dg_t = sum over i >= t of (q.dq - dv.v)_i + <S, dS> at the sum's end
//
// The terms of a gate's sum cancel but for what a few tokens have of one another, so that it starts again at the end of every
// 64 tokens, from a state that the rows' pass forward keeps for the one backward.  Heads of 64 x 64 in fp32 are off by at most
// 1.6e-6 of dg whatever the length, where sums to the sequence's end, in 64 bits but with all later tokens' roundings in their
// terms, left 1.4e-5 at 16384 tokens (2.5e-5 in the first 256), for K V floats of workspace a chunk and head and the same time
// (4 x 2048 tokens, 8 heads of 128 x 128: 3.71 ms of fp32, 3.75 before).
//
// The columns of S and dS do not meet in n and x (delta_cols), nor their rows in dq, e and f (delta_rows), so each CTA
// walks all tokens for 8 columns (rows) of one head with its part of the state in registers: 16 lanes hold a column,
// four adjacent values of every 64 each, so that a warp's loads of a token's vector from shared memory are two lines that
// its columns share.  Tokens arrive in blocks through registers and two buffers, one block ahead.
//
// Where there are few heads the chain from token to token bounds it, and of that the sums over the lanes.  So
// four tokens go together: their products with the state that enters the four are summed at once, what they add to one
// another comes from products of their keys and queries (found once a block of tokens, times the decays between them), and
// the state advances by four at a time.  3 x 1001 tokens, 5 heads of 96 x 80 in fp32: 165 us (660 ns a four, of which the
// products and the update take some 370 instructions a warp); 264 us token by token with eight lanes a column.
#include <type_traits>

#include "api_common.h"
#include "delta_internal.h"

namespace gla {
namespace {

constexpr int kThreads = 128, kLanes = 16, kTile = kThreads / kLanes;

// Vectors of four values of a lane, of P values in all; where the lane's i-th starts.
template <int P>
constexpr int kHeld = P / (4 * kLanes);
__device__ __forceinline__ int held_at(int i, int lane) { return (i * kLanes + lane) * 4; }

__device__ __forceinline__ float group_sum(float v)   // over the lanes of a column
{
    v += __shfl_xor_sync(~0u, v, 8);
    v += __shfl_xor_sync(~0u, v, 4);
    v += __shfl_xor_sync(~0u, v, 2);
    return v + __shfl_xor_sync(~0u, v, 1);
}

// Sums over the 16 lanes of a column of N values each (4 or 8): lane l is left with that of value l / 2 (N = 4: l / 4).
template <int N>
__device__ __forceinline__ float sums_by_lane(float (&v)[N], int lane)
{
    int bit = 8;
#pragma unroll
    for (int half = N / 2; half; half /= 2, bit /= 2)
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float keep = lane & bit ? v[half + i] : v[i], send = lane & bit ? v[i] : v[half + i];
            v[i] = keep + __shfl_xor_sync(~0u, send, bit);
        }
    float sum = v[0];
#pragma unroll
    for (; bit; bit /= 2)
        sum += __shfl_xor_sync(~0u, sum, bit);
    return sum;
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float sum)
{
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, sum))));
}
__device__ __forceinline__ float4 add4(float4 s, float4 x, float y)
{
    return make_float4(fmaf(x.x, y, s.x), fmaf(x.y, y, s.y), fmaf(x.z, y, s.z), fmaf(x.w, y, s.w));
}

__device__ __forceinline__ float4 times(float4 s, float c) { return make_float4(c * s.x, c * s.y, c * s.z, c * s.w); }

// Reads (or writes) a lane's share of the state: values d = 0.. of P at p + d * pitch.
template <int P>
__device__ __forceinline__ void take(float4 (&s)[kHeld<P>], const float *p, size_t pitch, int D, int lane, bool on)
{
#pragma unroll
    for (int i = 0; i < kHeld<P>; ++i) {
        const int d = held_at(i, lane);
        auto at = [&](int e) { return on && d + e < D ? p[(size_t)(d + e) * pitch] : 0.f; };
        s[i] = make_float4(at(0), at(1), at(2), at(3));
    }
}

template <int P>
__device__ __forceinline__ void put(const float4 (&s)[kHeld<P>], float *p, size_t pitch, int D, int lane)
{
#pragma unroll
    for (int i = 0; i < kHeld<P>; ++i) {
        const int d = held_at(i, lane);
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

// What four tokens in their order of processing have to do with one another; a = decay, b = strength.
struct Four {
    float m[4][4];   // forward: scale q_i.k_j, backward: scale k_i.q_j (j <= i), times the decays in between
    float l[4][4];   // k_i.k_j (j < i), likewise
    float start[4], end[4], b[4];   // decays from the start to a token, and from it to the end
    float all;
};

// Columns of the state.  Forward: n, and o where it is asked for; backward: x and dv.
//     forward:   n_i = b_i (v_i - start_i k_i.S - sum over j < i of l_ij n_j),   o_i = scale start_i q_i.S + sum of m_ij n_j
//     backward:  x_i = start_i k_i.dS + sum over j <= i of m_ij do_j - sum over j < i of l_ij b_j x_j
template <typename Tx, typename To, int P, bool BACK>
__global__ void __launch_bounds__(kThreads) delta_cols_kernel(DeltaArgs a, int tiles)
{
    constexpr int kBlock = 2048 / P, kEach = kBlock * P / kThreads, kVals = (kBlock * kTile + kThreads - 1) / kThreads;
    __shared__ __align__(16) float ks[2][kBlock][P], qs[2][kBlock][P], vs[2][kBlock][kTile];
    __shared__ float2 ab[2][kBlock];
    __shared__ Four fours[kBlock / 4];
    Walk w;
    if (!walk_of(a, tiles, w))
        return;
    const int tid = threadIdx.x, lane = tid % kLanes, mine = tid / kLanes, col = w.tile * kTile + mine;
    const int hk = w.hv / (a.HV / a.H);
    const Tx *q = static_cast<const Tx *>(a.q), *k = static_cast<const Tx *>(a.k);
    const Tx *v = static_cast<const Tx *>(BACK ? a.dout : a.v);
    const float *start = BACK ? a.dht : a.h0;
    const size_t state = w.head * a.K * a.V + col;
    float4 s[kHeld<P>];
    take<P>(s, start ? start + state : nullptr, a.V, a.K, lane, start && col < a.V);

    constexpr int kEachQuads = kEach / 4;
    const bool quads = a.K % 4 == 0;   // rows of keys arrive by fours
    struct alignas(4 * sizeof(Tx)) Quad {
        Tx v[4];
    };
    float kr[kEach], qr[kEach], vr[kVals];
    float2 abr;
    auto row_of = [&](int t) { return w.bos + (BACK ? w.len - 1 - t : t); };
    auto fetch = [&](int block) {   // behind the last token: nothing that changes the state
        if (quads) {
#pragma unroll
            for (int i = 0; i < kEachQuads; ++i) {
                const int e = (i * kThreads + tid) * 4, j = e / P, d = e % P, t = block * kBlock + j;
                const bool on = t < w.len && d < a.K;
                const size_t at = on ? ((size_t)row_of(t) * a.H + hk) * a.K + d : 0;
                const Quad none = {}, kq = on ? *reinterpret_cast<const Quad *>(k + at) : none, qq = on ? *reinterpret_cast<const Quad *>(q + at) : none;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    kr[4 * i + x] = widen(kq.v[x]);
                    qr[4 * i + x] = widen(qq.v[x]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int e = i * kThreads + tid, j = e / P, d = e % P, t = block * kBlock + j;
                const bool on = t < w.len && d < a.K;
                const size_t at = on ? ((size_t)row_of(t) * a.H + hk) * a.K + d : 0;
                kr[i] = on ? widen(k[at]) : 0.f;
                qr[i] = on ? widen(q[at]) : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < kVals; ++i) {
            const int e = i * kThreads + tid, j = e / kTile, c = w.tile * kTile + e % kTile, t = block * kBlock + j;
            vr[i] = j < kBlock && t < w.len && c < a.V ? widen(v[((size_t)row_of(t) * a.HV + w.hv) * a.V + c]) : 0.f;
        }
        abr = make_float2(0.f, 0.f);
        if (tid < kBlock && block * kBlock + tid < w.len) {
            const size_t at = (size_t)row_of(block * kBlock + tid) * a.HV + w.hv;
            abr = make_float2(a.g[at], a.beta[at]);
        }
    };
    auto keep = [&](int b) {
        if (quads) {
#pragma unroll
            for (int i = 0; i < kEachQuads; ++i) {
                const int e = (i * kThreads + tid) * 4;
                *reinterpret_cast<float4 *>(&ks[b][e / P][e % P]) = make_float4(kr[4 * i], kr[4 * i + 1], kr[4 * i + 2], kr[4 * i + 3]);
                *reinterpret_cast<float4 *>(&qs[b][e / P][e % P]) = make_float4(qr[4 * i], qr[4 * i + 1], qr[4 * i + 2], qr[4 * i + 3]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int e = i * kThreads + tid;
                ks[b][e / P][e % P] = kr[i];
                qs[b][e / P][e % P] = qr[i];
            }
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
    // a block's fours: kShare threads a product, which start at different places of their rows (they lie in the same banks)
    auto join = [&](int b) {
        constexpr int kShare = kThreads * P / 8192, kQuads = 2048 / kThreads;   // threads of a product, fours of a thread
        const int d = tid / kShare % 16, f = tid / kShare / 16, t0 = 4 * f;
        const bool inner = d < 10;   // m, else l
        const int e = inner ? d : d - 10, i = inner ? (e >= 6 ? 3 : e >= 3 ? 2 : e >= 1 ? 1 : 0) : (e >= 3 ? 3 : e >= 1 ? 2 : 1);
        const int j = inner ? e - i * (i + 1) / 2 : e - i * (i - 1) / 2;
        const float *x = inner && !BACK ? qs[b][t0 + i] : ks[b][t0 + i], *y = inner && BACK ? qs[b][t0 + j] : ks[b][t0 + j];
        float sums[4] = {};
#pragma unroll
        for (int n = 0; n < kQuads; ++n) {
            const int at = ((n + d) % kQuads * kShare + tid % kShare) * 4;
            sums[n % 4] = dot4(*reinterpret_cast<const float4 *>(x + at), *reinterpret_cast<const float4 *>(y + at), sums[n % 4]);
        }
        float sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
#pragma unroll
        for (int m = kShare / 2; m; m /= 2)
            sum += __shfl_xor_sync(~0u, sum, m);
        for (int m = BACK ? j : j + 1; m < (BACK ? i : i + 1); ++m)
            sum *= ab[b][t0 + m].x;
        if (tid % kShare == 0)
            (inner ? fours[f].m : fours[f].l)[i][j] = inner ? a.scale * sum : sum;
        if (tid < kBlock) {   // a token's own
            const int f0 = tid / 4, n = tid % 4;
            float before = 1.f, behind = 1.f;
            for (int m = 0; m < 4; ++m) {
                const float c = ab[b][4 * f0 + m].x;
                if (BACK ? m < n : m <= n) before *= c;
                if (BACK ? m >= n : m > n) behind *= c;
            }
            fours[f0].start[n] = before;
            fours[f0].end[n] = behind;
            fours[f0].b[n] = ab[b][tid].y;
            if (n == 3)
                fours[f0].all = BACK ? before * ab[b][tid].x : before;
        }
    };
    const int blocks = (w.len + kBlock - 1) / kBlock;
    if (blocks) {
        fetch(0);
        keep(0);
    }
    for (int block = 0; block < blocks; ++block) {
        const int b = block & 1;
        __syncthreads();
        join(b);
        if (block + 1 < blocks)
            fetch(block + 1);
        __syncthreads();
        const int many = min(kBlock, w.len - block * kBlock);
        for (int t0 = 0; t0 < many; t0 += 4) {
            const Four &f = fours[t0 / 4];
            constexpr int kSums = BACK ? 4 : 8;
            float part[kSums] = {};
#pragma unroll
            for (int i = 0; i < kHeld<P>; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    part[j] = dot4(*reinterpret_cast<const float4 *>(&ks[b][t0 + j][held_at(i, lane)]), s[i], part[j]);
                    if constexpr (!BACK)
                        part[4 + j] = dot4(*reinterpret_cast<const float4 *>(&qs[b][t0 + j][held_at(i, lane)]), s[i], part[4 + j]);
                }
            const float sum = sums_by_lane<kSums>(part, lane);
            float u[4], n[4], x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[i] = __shfl_sync(~0u, sum, (tid % 32 & ~(kLanes - 1)) | (BACK ? 4 * i : 2 * i));
                x[i] = vs[b][t0 + i][mine];
            }
            // lanes 0, 2, 4, 6 put n, lanes 8, 10, 12, 14 put o (lanes 0, 4, 8, 12: x and dv)
            const int token = BACK ? lane / 4 : lane / 2 % 4;
            const bool out = col < a.V && t0 + token < many && lane % (BACK ? 4 : 2) == 0;
            const size_t at = ((size_t)row_of(block * kBlock + t0 + token) * a.HV + w.hv) * a.V + col;
            if constexpr (!BACK) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float r = fmaf(-f.start[i], u[i], x[i]);
#pragma unroll
                    for (int j = 0; j < i; ++j)
                        r = fmaf(-f.l[i][j], n[j], r);
                    n[i] = f.b[i] * r;
                }
                if (a.upd && out && lane < 8)
                    a.upd[at] = token == 0 ? n[0] : token == 1 ? n[1] : token == 2 ? n[2] : n[3];
                if (a.o && out && lane >= 8) {
                    float o = a.scale * f.start[token] * sum;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j <= token)
                            o = fmaf(f.m[token][j], n[j], o);
                    static_cast<To *>(a.o)[at] = narrow<To>(o);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    n[j] *= f.end[j];
#pragma unroll
                for (int i = 0; i < kHeld<P>; ++i) {
                    s[i] = times(s[i], f.all);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[i] = add4(s[i], *reinterpret_cast<const float4 *>(&ks[b][t0 + j][held_at(i, lane)]), n[j]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float r = f.start[i] * u[i];
#pragma unroll
                    for (int j = 0; j <= i; ++j)
                        r = fmaf(f.m[i][j], x[j], r);
#pragma unroll
                    for (int j = 0; j < i; ++j)
                        r = fmaf(-f.l[i][j], f.b[j] * n[j], r);
                    n[i] = r;
                }
                if (out) {
                    const float mine_x = token == 0 ? n[0] : token == 1 ? n[1] : token == 2 ? n[2] : n[3];
                    a.dx[at] = mine_x;
                    static_cast<Tx *>(a.dv)[at] = narrow<Tx>(f.b[token] * mine_x);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    n[j] *= -f.end[j] * f.b[j];
                    x[j] *= f.end[j] * a.scale;
                }
#pragma unroll
                for (int i = 0; i < kHeld<P>; ++i) {
                    s[i] = times(s[i], f.all);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[i] = add4(s[i], *reinterpret_cast<const float4 *>(&ks[b][t0 + j][held_at(i, lane)]), n[j]);
                        s[i] = add4(s[i], *reinterpret_cast<const float4 *>(&qs[b][t0 + j][held_at(i, lane)]), x[j]);
                    }
                }
            }
        }
        if (block + 1 < blocks)
            keep(b ^ 1);
    }
    float *end = BACK ? a.dh0 : a.ht;
    if (end && col < a.V)
        put<P>(s, end + state, a.V, a.K, lane);
}

// Rows of the state, with n and x known.  Forward: dq and e; backward: f.  Four CTAs an SM, with 16 bytes of spills: left to
// itself the compiler takes 139 and 168 registers and orders the loads so that bf16 rows of 96 take 858 us (709).
template <typename Tx, int P, bool BACK>
__global__ void __launch_bounds__(kThreads, 4) delta_rows_kernel(DeltaArgs a, int tiles)
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
    float4 s[kHeld<P>];
    take<P>(s, start ? start + state : nullptr, 1, a.V, lane, start && row < a.K);

    float nr[kEach], xr[kEach], dr[kEach], kr[kVals], qr[kVals];
    float2 abr;
    // backward, blocks begin behind the end, so that chunks end between blocks there too
    static_assert(kDeltaChunk % kBlock == 0, "chunks are whole blocks");
    const int pad = BACK ? (kBlock - w.len % kBlock) % kBlock : 0, all = w.len + pad;
    auto row_of = [&](int t) { return w.bos + (BACK ? all - 1 - t : t); };
    auto there = [&](int t) { return t >= pad && t < all; };
    // this row of the state at the end of the chunk with token e
    const size_t first = (size_t)delta_first_slot(a, w.n) * a.HV + w.hv;
    auto kept_at = [&](int e) { return (first + (size_t)(e / kDeltaChunk) * a.HV) * a.K + row; };
    auto fetch = [&](int block) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int e = i * kThreads + tid, j = e / P, c = e % P, t = block * kBlock + j;
            const bool on = there(t) && c < a.V;
            const size_t at = on ? ((size_t)row_of(t) * a.HV + w.hv) * a.V + c : 0;
            nr[i] = on ? a.upd[at] : 0.f;
            xr[i] = on ? a.dx[at] : 0.f;
            dr[i] = on ? a.scale * widen(d[at]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kVals; ++i) {
            const int e = i * kThreads + tid, j = e / kTile, r = w.tile * kTile + e % kTile, t = block * kBlock + j;
            const bool on = j < kBlock && there(t) && r < a.K;
            const size_t at = on ? ((size_t)row_of(t) * a.H + hk) * a.K + r : 0;
            kr[i] = on ? widen(k[at]) : 0.f;
            qr[i] = on ? widen(q[at]) : 0.f;
        }
        abr = make_float2(0.f, 0.f);
        if (tid < kBlock && there(block * kBlock + tid)) {
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
    const int blocks = (all + kBlock - 1) / kBlock;
    if (blocks) {
        fetch(0);
        keep(0);
    }
    __syncthreads();
    constexpr int kPer = kDeltaChunk / kBlock;   // blocks of a chunk
    for (int block = 0, end; block < blocks; block = end) {
        end = min(blocks, BACK ? block + (blocks - block - 1) % kPer + 1 : block + kPer);
        if constexpr (BACK) {   // this row of <S, dS> at a chunk's end
            const size_t at = kept_at(all - 1 - block * kBlock);
            float4 kept[kHeld<P>];
            take<P>(kept, a.kept + at * a.V, 1, a.V, lane, row < a.K);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < kHeld<P>; ++i)
                sum += (s[i].x * kept[i].x + s[i].y * kept[i].y) + (s[i].z * kept[i].z + s[i].w * kept[i].w);
            sum = group_sum(sum);
            if (lane == 0 && row < a.K)
                a.hd[at] = sum;
        }
        const size_t ends = kept_at(block * kBlock) * a.V;
        for (; block < end; ++block) {
            const int b = block & 1;
            if (block + 1 < blocks)
                fetch(block + 1);
            const int many = min(kBlock, all - block * kBlock);
            for (int t0 = 0; t0 < many; t0 += 4) {   // four tokens' sums over the lanes together
                float part[BACK ? 4 : 8] = {};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 c = ab[b][t0 + j];
                    const float kj = ks[b][t0 + j][mine], qj = qs[b][t0 + j][mine];
#pragma unroll
                    for (int i = 0; i < kHeld<P>; ++i) {
                        const float4 n = *reinterpret_cast<const float4 *>(&ns[b][t0 + j][held_at(i, lane)]);
                        const float4 x = *reinterpret_cast<const float4 *>(&xs[b][t0 + j][held_at(i, lane)]);
                        const float4 d = *reinterpret_cast<const float4 *>(&ds[b][t0 + j][held_at(i, lane)]);
                        if constexpr (!BACK) {
                            s[i] = times(s[i], c.x);
                            part[j] = dot4(s[i], x, part[j]);
                            s[i] = add4(s[i], n, kj);
                            part[4 + j] = dot4(s[i], d, part[4 + j]);
                        } else {
                            s[i] = add4(s[i], d, qj);
                            part[j] = dot4(s[i], n, part[j]);
                            s[i] = times(add4(s[i], x, -c.y * kj), c.x);
                        }
                    }
                }
                const float sum = sums_by_lane<BACK ? 4 : 8>(part, lane);
                const int token = BACK ? lane / 4 : lane / 2 % 4;
                if (row < a.K && t0 + token < many && block * kBlock + t0 + token >= pad && lane % (BACK ? 4 : 2) == 0) {
                    const size_t at = ((size_t)row_of(block * kBlock + t0 + token) * a.HV + w.hv) * a.K + row;
                    if constexpr (!BACK)
                        (lane < 8 ? a.eh : a.dqh)[at] = lane < 8 ? -sum : sum;
                    else
                        a.fh[at] = sum;
                }
            }
            if (block + 1 < blocks)
                keep(b ^ 1);
            __syncthreads();
        }
        if (!BACK && row < a.K)   // rows behind the sequence's end have changed nothing
            put<P>(s, a.kept + ends, 1, a.V, lane);
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
            float ke = 0.f, qd = 0.f, xv = 0.f;
            for (int d = lane; d < a.K; d += 32) {
                const float kd = widen(k[key + d]);
                ke = fmaf(kd, a.eh[head * a.K + d], ke);
                qd = fmaf(widen(q[key + d]), a.dqh[head * a.K + d], qd);
            }
            for (int d = lane; d < a.V; d += 32)
                xv = fmaf(a.dx[head * a.V + d], widen(v[head * a.V + d]), xv);
#pragma unroll
            for (int m = 16; m; m /= 2) {
                ke += __shfl_xor_sync(~0u, ke, m);
                qd += __shfl_xor_sync(~0u, qd, m);
                xv += __shfl_xor_sync(~0u, xv, m);
            }
            if (lane == 0) {
                a.dbeta[head] = xv + ke;
                a.dG[head] = qd - a.beta[head] * xv;   // (o.dO - dv.v: a decay scales what later rows read, not what they add)
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

// dg: sums of dG from the end of each chunk, and <S, dS> there; a thread a token.
__global__ void __launch_bounds__(kDeltaChunk) delta_gates_kernel(DeltaArgs a)
{
    __shared__ double part[2], ends[2];
    const int slot = blockIdx.x / a.HV, hv = blockIdx.x - slot * a.HV, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    int n, c, first, rows;
    if (!delta_chunk(a, slot, n, c, first, rows))
        return;
    const size_t at = (size_t)(first + tid) * a.HV + hv;
    double sum = tid < rows ? (double)a.dG[at] : 0., end = 0.;
    for (int d = tid; d < a.K; d += kDeltaChunk)
        end += a.hd[((size_t)slot * a.HV + hv) * a.K + d];
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
        const double u = __shfl_down_sync(~0u, sum, m);
        if (lane + m < 32)
            sum += u;
        end += __shfl_xor_sync(~0u, end, m);
    }
    if (lane == 0)
        part[warp] = sum, ends[warp] = end;
    __syncthreads();
    if (tid < rows)
        a.dg[at] = (float)(sum + (warp == 0 ? part[1] : 0.) + (ends[0] + ends[1]));
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
    delta_gates_kernel<<<(unsigned)((size_t)a.slots * a.HV), kDeltaChunk, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace gla
