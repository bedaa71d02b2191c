// Gradients of q and k of the gated delta rule, chunk by chunk, from what the two chains have left (16-bit values; the
// outputs have 16 bits too, and nothing else passes these products).  Per (chunk, key head), summed over its value heads:
//
//     p_ij = scale D_ij dO_i.N_j (j <= i),   b_ij = -beta_i D_ij x_i.N_j (j < i),   D_ij = e^(G_i - G_j)
//     dq = scale e^G dO S' + p k,   dk = -beta e^G x S' + e^(G_end - G) N dS' + p' q + (b + b') k
//
// Persistent CTAs of 16 warps: warp (r, h) has 16 rows and a quarter of the keys, with dq and dk in registers over all value
// heads.  The values come 64 columns at a time in two stages (one ahead, across heads and chunks): products over them of
// 16-row blocks into dO S', x S', N dS' and, by halves of columns, p (h < 2) or b, which pass shared memory once to be left
// operands both as they are and transposed.  4 x 2048 tokens of 8 heads 67 us, 150 MB: bound by shared memory (the right
// operands of every warp) and the steps of an item that do not overlap; eight warps with half of the keys each took 69.
#include <algorithm>

#include "delta_chain.cuh"

namespace gla {
namespace {

constexpr int kThreads = 512;

template <int KD>
struct GradShared {
    struct Rows {
        uint16_t k[KD / 64][64][64], q[KD / 64][64][64];
    } rows[2];
    struct alignas(1024) Stage {
        uint16_t d[64][64];                        // dO, swizzled: on 1024 bytes
        uint32_t n[8][8][32], x[8][8][32];         // blocks of 8 x 8: columns by tokens
        uint32_t s[8][KD / 8][32], ds[8][KD / 8][32];   // columns by keys
        float4 row[kDeltaChunk];
        float2 gate[kDeltaChunk];
        float power[16][8];                        // fp16: of the head's groups of 16 columns (DeltaTrace)
    } stage[2];
    uint16_t p[64][72], b[64][72];
    uint64_t full[2];
};

// What a CTA works on: 64 columns of a value head of a chunk.
struct GradPiece {
    int item;   // slot * H + key head
    int first, rows, slot, h, v, c;   // first row and rows of the chunk; value head of the key head; piece of its columns
    int turn, items;                  // pieces and items so far
};

// Whether `p.item` or one after it (a grid apart) is a chunk with rows; p becomes its first piece.
__device__ __forceinline__ bool find_item(const DeltaArgs &a, GradPiece &p)
{
    const int end = a.slots * a.H;
    for (; p.item < end; p.item += gridDim.x) {
        int n, c;
        p.slot = p.item / a.H;
        p.h = p.item - p.slot * a.H;
        if (delta_chunk(a, p.slot, n, c, p.first, p.rows)) {
            p.v = p.c = 0;
            return true;
        }
    }
    return false;
}
__device__ __forceinline__ bool next_piece(const DeltaArgs &a, GradPiece &p)
{
    ++p.turn;
    if (++p.c * 64 < a.V)
        return true;
    p.c = 0;
    if (++p.v < a.HV / a.H)
        return true;
    ++p.items;
    p.item += gridDim.x;
    return find_item(a, p);
}

// Four blocks of 8 x 8: rows of blocks r and r + 1 (BY_ROW: the first two matrices differ in the row), columns c and c + 1.
template <bool BY_ROW>
__device__ __forceinline__ void blocks_t(uint32_t (&f)[4], const uint32_t *base, int across, int r, int c, int lane)
{
    const int m = lane / 8, dr = BY_ROW ? m & 1 : m >> 1, dc = BY_ROW ? m >> 1 : m & 1;
    ldsm_t(f, tc::smem_u32(base + ((r + dr) * across + c + dc) * 32 + (lane & 7) * 4));
}

template <typename T, int KD>
__global__ void __launch_bounds__(kThreads, 1) delta_grads_kernel(const __grid_constant__ ChainMaps maps, DeltaArgs a)
{
    typedef GradShared<KD> Shared;
    constexpr int NT = KD / 32;   // tiles of 8 keys of a warp
    extern __shared__ __align__(1024) char raw[];
    Shared &sh = *reinterpret_cast<Shared *>(raw);
    const int tid = threadIdx.x, lane = tid % 32, r = tid / 32 % 4, h = tid / 128, two = 2 * (lane % 4), i0 = 16 * r + lane / 4;
    const int per = a.HV / a.H;
    bars_init(sh.full);
    tc::grid_dep_wait();
    // the first lanes of eight warps ask for a part each: a copy takes its thread some 200 cycles to issue
    auto ask = [&](const GradPiece &p) {
        if (lane)
            return;
        auto &st = sh.stage[p.turn & 1];
        uint64_t *bar = &sh.full[p.turn & 1];
        const int hv = p.h * per + p.v, blocks = min(8, (a.V - 64 * p.c) / 8);   // rows of blocks
        const bool begins = p.v == 0 && p.c == 0;
        const uint32_t narrow_bytes = blocks * 8 * 128, wide_bytes = blocks * (KD / 8) * 128, power_bytes = a.V / 16 * sizeof st.power[0];
        const size_t cell = (size_t)p.slot * a.HV + hv;
        const size_t narrow_at = cell * a.trace.n_size + (size_t)p.c * 8 * 8 * 32, wide_at = cell * a.trace.s_size + (size_t)p.c * 8 * (KD / 8) * 32;
        const char *from = a.chunk + cell * sizeof(DeltaCellBack);
        switch (tid / 32) {
        case 0:
            tc::bar_expect_tx(bar, (uint32_t)(sizeof st.d + 2 * narrow_bytes + 2 * wide_bytes + sizeof st.row + sizeof st.gate +
                                              (kScaled<T> ? power_bytes : 0) + (begins ? sizeof sh.rows[0] : 0)));
            copy_bulk(st.s, a.trace.s + wide_at, wide_bytes, bar);
            break;
        case 1: copy_bulk(st.ds, a.trace.ds + wide_at, wide_bytes, bar); break;
        case 2: tc::tma_load_3d(st.d, &maps.d, 64 * p.c, hv, p.first, bar); break;
        case 3: copy_bulk(st.n, a.trace.n + narrow_at, narrow_bytes, bar); break;
        case 4: copy_bulk(st.x, a.trace.x + narrow_at, narrow_bytes, bar); break;
        case 5:
            copy_bulk(st.row, from + kCellRows, sizeof st.row, bar);
            copy_bulk(st.gate, from + sizeof(DeltaCellBack) - sizeof st.gate, sizeof st.gate, bar);
            if constexpr (kScaled<T>)
                copy_bulk(st.power, a.trace.power + cell * (a.V / 16) * 8, power_bytes, bar);
            break;
        case 6:
            if (begins)
#pragma unroll
                for (int i = 0; i < KD / 64; ++i)
                    tc::tma_load_3d(sh.rows[p.items & 1].k[i], &maps.k, 64 * i, p.h, p.first, bar);
            break;
        case 7:
            if (begins)
#pragma unroll
                for (int i = 0; i < KD / 64; ++i)
                    tc::tma_load_3d(sh.rows[p.items & 1].q[i], &maps.q, 64 * i, p.h, p.first, bar);
            break;
        }
    };
    GradPiece now = {}, ahead;
    now.item = blockIdx.x;
    if (!find_item(a, now))
        return;
    ahead = now;
    ask(now);
    float dq[NT][4], dk[NT][4], m[4][4], ds[NT][4], xs[NT][4], nd[NT][4];
    auto clear = [](auto &x) {
        for (auto &t : x)
            t[0] = t[1] = t[2] = t[3] = 0.f;
    };
    clear(m), clear(ds), clear(xs), clear(nd), clear(dq), clear(dk);
    for (;;) {
        auto &st = sh.stage[now.turn & 1];
        auto &rows = sh.rows[now.items & 1];
        const bool ok = tc::bar_wait(&sh.full[now.turn & 1], (now.turn >> 1) & 1);
        if (__syncthreads_or(!ok)) {
            give_up(a.status, &sh.full[now.turn & 1], (now.turn >> 1) & 1);
            return;
        }
        const bool more = next_piece(a, ahead);
        if (more)
            ask(ahead);
        if (now.rows < kDeltaChunk) {   // rows behind the sequence's end may hold anything
            const uint4 zero = make_uint4(0, 0, 0, 0);
            for (int i = now.rows * 8 + tid; i < 512; i += kThreads) {
                reinterpret_cast<uint4 *>(st.d)[i] = zero;
                if (now.v == 0 && now.c == 0)
#pragma unroll
                    for (int x = 0; x < KD / 64; ++x) {
                        reinterpret_cast<uint4 *>(rows.k[x])[i] = zero;
                        reinterpret_cast<uint4 *>(rows.q[x])[i] = zero;
                    }
            }
            tc::fence_proxy_async();   // before a later copy to the same place
            __syncthreads();
        }
        const int steps = min(4, (a.V - 64 * now.c) / 16);
        // fp16: the largest powers of the head's columns.  Products are sums over columns: each group's operands are taken
        // over the largest, and what comes of them times it
        float most[6] = {};
        auto over = [](uint32_t (&f)[4], float p) {
            if constexpr (kScaled<T>)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    f[e] = times_power(f[e], p);
        };
        if constexpr (kScaled<T>)
            for (int g = 0; g < a.V / 16; ++g)
#pragma unroll
                for (int e = 0; e < 6; ++e)
                    if (e != 3)
                        most[e] = fmaxf(most[e], st.power[g][e]);
        for (int s = 0; s < steps; ++s) {
            uint32_t fd[4], fx[4], fn[4];
            float p_s = 1.f, p_n = 1.f, p_ds = 1.f;
            ldsm(fd, tc::smem_u32(st.d) + unit_at(16 * r + lane % 16, 2 * s + lane / 16));
            blocks_t<false>(fx, &st.x[0][0][0], 8, 2 * s, 2 * r, lane);
            blocks_t<false>(fn, &st.n[0][0][0], 8, 2 * s, 2 * r, lane);
            if constexpr (kScaled<T>) {
                const float *p = st.power[4 * now.c + s];
                p_s = p[0] * inverse_power(most[0]), p_n = p[1] * inverse_power(most[1]), p_ds = p[4] * inverse_power(most[4]);
                over(fx, p[5] * inverse_power(most[5]));
                over(fn, p_n);
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {   // columns of p, or of b, in this block of rows
                if (2 * (h & 1) + p > r)
                    break;
                uint32_t f[4];
                blocks_t<true>(f, &st.n[0][0][0], 8, 2 * s, 4 * (h & 1) + 2 * p, lane);
                over(f, p_n);
                mma<T>(m[2 * p], h > 1 ? fx : fd, f[0], f[1]);
                mma<T>(m[2 * p + 1], h > 1 ? fx : fd, f[2], f[3]);
            }
#pragma unroll
            for (int p = 0; p < NT / 2; ++p) {
                uint32_t f[4], g[4];
                blocks_t<true>(f, &st.s[0][0][0], KD / 8, 2 * s, h * NT + 2 * p, lane);
                blocks_t<true>(g, &st.ds[0][0][0], KD / 8, 2 * s, h * NT + 2 * p, lane);
                over(f, p_s);
                over(g, p_ds);
                mma<T>(ds[2 * p], fd, f[0], f[1]);
                mma<T>(ds[2 * p + 1], fd, f[2], f[3]);
                mma<T>(xs[2 * p], fx, f[0], f[1]);
                mma<T>(xs[2 * p + 1], fx, f[2], f[3]);
                mma<T>(nd[2 * p], fn, g[0], g[1]);
                mma<T>(nd[2 * p + 1], fn, g[2], g[3]);
            }
        }
        if ((now.c + 1) * 64 >= a.V) {   // the value head's last columns
            const float4 c0 = st.row[i0], c1 = st.row[i0 + 8];
            const float2 g0 = st.gate[i0], g1 = st.gate[i0 + 8];
            // fp16: p over scale and the powers of dO and N, b over those of beta x and N
            const float by = h > 1 ? -1.f : inverse_power(most[2]);
            const float f0 = kScaled<T> ? by : h > 1 ? -c0.x : a.scale, f1 = kScaled<T> ? by : h > 1 ? -c1.x : a.scale;
            const float of_p = a.scale * most[1] * most[2], of_b = most[1] * most[5];
            uint16_t(*to)[72] = h > 1 ? sh.b : sh.p;
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int j = 32 * (h & 1) + 16 * p + 8 * y + two;
                    const float2 ga = st.gate[j], gb = st.gate[j + 1];
                    auto take_if = [&](int i, int jj, float f, float2 gi, float2 gj, float v) {
                        return i < now.rows && (h > 1 ? jj < i : jj <= i) ? f * exp2_fast((gi.x - gj.x) + (gi.y - gj.y)) * v : 0.f;
                    };
                    const float(&v)[4] = m[2 * p + y];
                    *reinterpret_cast<uint32_t *>(&to[i0][j]) =
                        narrow2<T>(make_float2(take_if(i0, j, f0, g0, ga, v[0]), take_if(i0, j + 1, f0, g0, gb, v[1])));
                    *reinterpret_cast<uint32_t *>(&to[i0 + 8][j]) =
                        narrow2<T>(make_float2(take_if(i0 + 8, j, f1, g1, ga, v[2]), take_if(i0 + 8, j + 1, f1, g1, gb, v[3])));
                }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 &c = e < 2 ? c0 : c1;
                    if constexpr (kScaled<T>) {
                        dq[j][e] = fmaf(c.w * most[0], ds[j][e], dq[j][e]);
                        dk[j][e] = fmaf(c.z * (most[1] * most[4]), nd[j][e], fmaf(-c.y * (most[5] * most[0]), xs[j][e], dk[j][e]));
                    } else {
                        dq[j][e] = fmaf(c.w, ds[j][e], dq[j][e]);
                        dk[j][e] = fmaf(c.z, nd[j][e], fmaf(-c.x * c.y, xs[j][e], dk[j][e]));
                    }
                }
            clear(m), clear(ds), clear(xs), clear(nd);
            float(&pk)[NT][4] = kScaled<T> ? ds : dq, (&bk)[NT][4] = kScaled<T> ? xs : dk, (&pq)[NT][4] = kScaled<T> ? nd : dk;
            __syncthreads();
            const int m8 = lane / 8;
            for (int s = 0; s < 4; ++s) {
                uint32_t fp[4], fb[4], ft[4], fu[4];
                if (s <= r) {   // as left operands: rows of this block, columns of step s
                    ldsm(fp, tc::smem_u32(&sh.p[16 * r + lane % 16][16 * s + (lane / 16) * 8]));
                    ldsm(fb, tc::smem_u32(&sh.b[16 * r + lane % 16][16 * s + (lane / 16) * 8]));
                }
                if (s >= r) {   // transposed: columns of this block, rows of step s
                    ldsm_t(ft, tc::smem_u32(&sh.p[16 * s + (m8 >> 1) * 8 + (lane & 7)][16 * r + (m8 & 1) * 8]));
                    ldsm_t(fu, tc::smem_u32(&sh.b[16 * s + (m8 >> 1) * 8 + (lane & 7)][16 * r + (m8 & 1) * 8]));
                }
#pragma unroll
                for (int p = 0; p < NT / 2; ++p) {
                    uint32_t f[4];
                    const int key = h * (KD / 4) + 16 * p;   // first of 16 keys
                    const uint32_t at = unit_at(16 * s + (lane & 15), key % 64 / 8 + lane / 16);
                    ldsm_t(f, tc::smem_u32(rows.k[key / 64]) + at);
                    if (s <= r) {
                        mma<T>(pk[2 * p], fp, f[0], f[1]);
                        mma<T>(pk[2 * p + 1], fp, f[2], f[3]);
                        mma<T>(bk[2 * p], fb, f[0], f[1]);
                        mma<T>(bk[2 * p + 1], fb, f[2], f[3]);
                    }
                    if (s >= r) {
                        mma<T>(bk[2 * p], fu, f[0], f[1]);
                        mma<T>(bk[2 * p + 1], fu, f[2], f[3]);
                        ldsm_t(f, tc::smem_u32(rows.q[key / 64]) + at);
                        mma<T>(pq[2 * p], ft, f[0], f[1]);
                        mma<T>(pq[2 * p + 1], ft, f[2], f[3]);
                    }
                }
            }
            if constexpr (kScaled<T>) {
                bool bad = false;
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        dq[j][e] = fmaf(of_p, pk[j][e], dq[j][e]);
                        dk[j][e] = fmaf(of_b, bk[j][e], fmaf(of_p, pq[j][e], dk[j][e]));
                        bad |= lost(dq[j][e]) || lost(dk[j][e]);
                    }
                if (bad)
                    report(a.status, GLA_ERR_RANGE);
                clear(pk), clear(bk), clear(pq);
            }
            if (now.v + 1 == per) {   // by way of the keys' and queries' place, to rows of whole units
                __syncthreads();
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int key = h * (KD / 4) + 8 * j;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t at = unit_at(i0 + 8 * e, key % 64 / 8) + 2 * two;
                        *reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(rows.k[key / 64]) + at) = narrow2<T>(make_float2(dq[j][2 * e], dq[j][2 * e + 1]));
                        *reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(rows.q[key / 64]) + at) = narrow2<T>(make_float2(dk[j][2 * e], dk[j][2 * e + 1]));
                    }
                }
                __syncthreads();
                for (int u = tid; u < now.rows * (KD / 8); u += kThreads) {
                    const int t = u / (KD / 8), unit = u % (KD / 8);
                    const uint32_t at = unit_at(t, unit % 8);
                    const size_t to = ((size_t)(now.first + t) * a.H + now.h) * KD + 8 * unit;
                    *reinterpret_cast<uint4 *>(static_cast<T *>(a.dq) + to) = *reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(rows.k[unit / 8]) + at);
                    *reinterpret_cast<uint4 *>(static_cast<T *>(a.dk) + to) = *reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(rows.q[unit / 8]) + at);
                }
                tc::fence_proxy_async();
                clear(dq), clear(dk);
            }
        }
        if (!more)
            return;
        now = ahead;
    }
}

}  // namespace

cudaError_t launch_delta_grads(const DeltaArgs &a, bool half, int sms, cudaStream_t s)
{
    ChainMaps maps;
    if (!make_maps(maps, a, 64, half))
        return cudaErrorInvalidValue;
    auto go = [&](auto kernel, size_t shared) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
        if (e != cudaSuccess)
            return e;
        return launch_early_shared(kernel, (unsigned)std::min<int64_t>((int64_t)a.slots * a.H, sms), kThreads, shared, s, maps, a);
    };
    auto by_keys = [&](auto t) {
        typedef std::remove_pointer_t<decltype(t)> T;
        return a.K == 128 ? go(delta_grads_kernel<T, 128>, sizeof(GradShared<128>)) : go(delta_grads_kernel<T, 64>, sizeof(GradShared<64>));
    };
    return half ? by_keys((__half *)0) : by_keys((__nv_bfloat16 *)0);
}

}  // namespace gla
