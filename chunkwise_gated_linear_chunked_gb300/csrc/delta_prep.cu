// Gated delta rule in chunks of 64 tokens, what does not depend on the state: of each (chunk, value head) the decays, the
// scores P and the inverse that turns the values' remainders into update rows (see DeltaCell).  One CTA a (chunk, key
// head): k k^T and q k^T once for the value heads that share the key head.
//
// With L_ij = e^(G_i - G_j) k_i.k_j (j < i) and N the rows that update the state, N = beta Y and Y = R - L N for
// R = V - e^G K S, so Y = (I + L diag(beta))^-1 R.  The inverse is I + W diag(beta), and the one that the gradients take,
// (I + diag(beta) L)^-1, is I + diag(beta) W, with W_ij = -(L_ij + sum over j < m < i of L_im beta_m W_mj): found by
// substitution, a lane a column, in two blocks of 32 side by side, then the block below them by two products.  A sum of
// powers of L would need none of it and is not taken: for keys that look alike its terms grow like binomials.
//
// Differences of G decide the decays, and G may run far from zero, so it is summed in 64 bits and kept in two floats.
// Gates count as at least -1000 (a decay of 0), which keeps differences of two cleared rows finite.
#include "delta_mma.cuh"

namespace gla {
namespace {

constexpr int kThreads = 128;
constexpr int kPitch = 68;   // floats of a row of L and W

template <int KD>
struct PrepShared {
    uint16_t k[64][KD + 8], q[64][KD + 8];
    float l[64][kPitch], w[64][kPitch], b[32][36];
    float g_hi[64], g_lo[64], beta[64];
};

__device__ __forceinline__ float decay_between(float hi_i, float lo_i, float hi_j, float lo_j)
{
    return exp2_fast((hi_i - hi_j) + (lo_i - lo_j));   // G is held times log2 e
}

template <typename T, int KD, bool BACK>
__global__ void __launch_bounds__(kThreads) delta_prep_kernel(DeltaArgs a)
{
    typedef std::conditional_t<BACK, DeltaCellBack, DeltaCell> Cell;
    extern __shared__ __align__(16) char raw[];
    PrepShared<KD> &sh = *reinterpret_cast<PrepShared<KD> *>(raw);
    const int slot = blockIdx.x / a.H, h = blockIdx.x - slot * a.H, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    int n, c, first, rows;
    if (!delta_chunk(a, slot, n, c, first, rows))
        return;
    const size_t key = ((size_t)first * a.H + h) * KD, pitch = (size_t)a.H * KD;
    copy_rows<KD, kThreads>(tc::smem_u32(sh.k), static_cast<const T *>(a.k) + key, pitch, rows, KD);
    copy_rows<KD, kThreads>(tc::smem_u32(sh.q), static_cast<const T *>(a.q) + key, pitch, rows, KD);
    copies_end();
    copies_wait<0>();
    __syncthreads();

    // rows 16 warp up of k k^T and q k^T, columns up to the diagonal block
    float kk[8][4] = {}, qk[8][4] = {};
    {
        const uint32_t row = (16 * warp + lane % 16) * (KD + 8) * 2 + (lane / 16) * 16;
        const uint32_t ka = tc::smem_u32(sh.k) + row, qa = tc::smem_u32(sh.q) + row;
        const uint32_t kb = tc::smem_u32(sh.k) + ((lane & 7) + (lane / 16) * 8) * (KD + 8) * 2 + ((lane / 8) & 1) * 16;
#pragma unroll
        for (int s = 0; s < KD / 16; ++s) {
            uint32_t fk[4], fq[4];
            ldsm(fk, ka + s * 32);
            ldsm(fq, qa + s * 32);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                if (p > warp)
                    break;
                uint32_t b[4];   // columns 16 p up: two tiles of 8
                ldsm(b, kb + p * 16 * (KD + 8) * 2 + s * 32);
                mma<T>(kk[2 * p], fk, b[0], b[1]);
                mma<T>(kk[2 * p + 1], fk, b[2], b[3]);
                mma<T>(qk[2 * p], fq, b[0], b[1]);
                mma<T>(qk[2 * p + 1], fq, b[2], b[3]);
            }
        }
    }

    const int per = a.HV / a.H;
    for (int v = 0; v < per; ++v) {
        const int hv = h * per + v;
        Cell &cell = reinterpret_cast<Cell *>(a.chunk)[(size_t)slot * a.HV + hv];
        __syncthreads();   // the last head's sums are read
        if (warp == 0) {   // two rows a lane
            double g[2];
            float bt[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e;
                const size_t at = (size_t)(first + t) * a.HV + hv;
                const float gate = t < rows ? a.g[at] : 0.f;
                bt[e] = t < rows ? a.beta[at] : 0.f;
                g[e] = (gate < -1000.f ? -1000.0 : (double)gate) * 1.4426950408889634;
            }
            g[1] += g[0];
            double sum = g[1];
#pragma unroll
            for (int m = 1; m < 32; m *= 2) {
                const double u = __shfl_up_sync(~0u, sum, m);
                if (lane >= m)
                    sum += u;
            }
            const double before = sum - g[1], end = __shfl_sync(~0u, sum, 31);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e;
                const double G = before + g[e];
                sh.g_hi[t] = (float)G;
                sh.g_lo[t] = (float)(G - (double)(float)G);
                sh.beta[t] = bt[e];
                const float start = exp2_fast((float)G);
                cell.row[t] = make_float4(bt[e], start, exp2_fast((float)(end - G)), a.scale * start);
            }
        }
        __syncthreads();
        // L to shared memory, P to the cell: a result's rows are a right operand's columns, so P goes as it lies
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = 16 * warp + lane / 4 + 8 * half;
            const float hi = sh.g_hi[i], lo = sh.g_lo[i];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                uint32_t word[4];
                float pv[4];
#pragma unroll
                for (int tile = 0; tile < 2; ++tile)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int j = 16 * p + 8 * tile + 2 * (lane % 4) + e;
                        const float d = j <= i ? decay_between(hi, lo, sh.g_hi[j], sh.g_lo[j]) : 0.f;
                        sh.l[i][j] = j < i ? d * kk[2 * p + tile][2 * half + e] : 0.f;
                        pv[2 * tile + e] = j <= i ? a.scale * d * qk[2 * p + tile][2 * half + e] : 0.f;
                        if constexpr (BACK)
                            sh.w[i][j] = pv[2 * tile + e];   // for its transpose, before W lies there
                    }
                if (p > warp)
                    continue;
                split2<T>(pv[0], pv[1], word[0], word[2]);
                split2<T>(pv[2], pv[3], word[1], word[3]);
                cell.score[triangle_at(2 * warp + half, p) * 32 + lane] = make_uint4(word[0], word[1], word[2], word[3]);
            }
        }
        __syncthreads();
        // fragments of a transposed matrix: tile j, step i, entry (column 8 j + lane / 4, row 16 i + 2 (lane % 4) ..)
        auto store_t = [&](uint4 *to, auto value) {
            for (int f = warp; f < kTriangle; f += kThreads / 32) {
                int j = 7, i = 3;
                while (triangle_at_t(j, i) != f)   // tiles from the last, steps from the last
                    if (--i < j / 2)
                        --j, i = 3;
                const int t = 8 * j + lane / 4, r = 16 * i + 2 * (lane % 4);
                uint32_t word[4];
                split2<T>(value(r, t), value(r + 1, t), word[0], word[2]);
                split2<T>(value(r + 8, t), value(r + 9, t), word[1], word[3]);
                to[f * 32 + lane] = make_uint4(word[0], word[1], word[2], word[3]);
            }
        };
        if constexpr (BACK) {
            store_t(static_cast<DeltaCellBack &>(cell).score_t, [&](int r, int t) { return sh.w[r][t]; });
            __syncthreads();
        }
        // W: the blocks on the diagonal, a warp each, a lane a column
        if (warp < 2) {
            const int o = 32 * warp;
            float w[32];   // beta W of the rows so far, 1 on the diagonal
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int m = 0; m < i; m += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(&sh.l[o + i][o + m]);
                    s0 = fmaf(x.x, w[m], s0);
                    if (m + 1 < i) s1 = fmaf(x.y, w[m + 1], s1);
                    if (m + 2 < i) s0 = fmaf(x.z, w[m + 2], s0);
                    if (m + 3 < i) s1 = fmaf(x.w, w[m + 3], s1);
                }
                const float value = -(s0 + s1);
                sh.w[o + i][o + lane] = i > lane ? value : 0.f;
                w[i] = i == lane ? 1.f : i > lane ? sh.beta[o + i] * value : 0.f;
            }
        }
        __syncthreads();
        // below them: B = L21 (beta W + I)11, W21 = -(W diag(beta) + I)22 B; four adjacent columns of two rows a thread
        {
            const int r = tid / 8 * 2, x = tid % 8 * 4;
            float acc[2][4] = {};
#pragma unroll 4
            for (int m = 0; m < 32; ++m) {
                const float4 w = *reinterpret_cast<const float4 *>(&sh.w[m][x]);
                const float f = sh.beta[m];
                const float u[4] = {m == x ? 1.f : f * w.x, m == x + 1 ? 1.f : f * w.y, m == x + 2 ? 1.f : f * w.z,
                                    m == x + 3 ? 1.f : f * w.w};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float l = sh.l[32 + r + e][m];
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        acc[e][d] = fmaf(l, u[d], acc[e][d]);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float4 *>(&sh.b[r + e][x]) = make_float4(acc[e][0], acc[e][1], acc[e][2], acc[e][3]);
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 b = *reinterpret_cast<const float4 *>(&sh.b[r + e][x]);
                acc[e][0] = b.x, acc[e][1] = b.y, acc[e][2] = b.z, acc[e][3] = b.w;
            }
#pragma unroll 4
            for (int m = 0; m < 32; ++m) {
                const float4 b = *reinterpret_cast<const float4 *>(&sh.b[m][x]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f = sh.w[32 + r + e][32 + m] * sh.beta[32 + m];   // 0 from the diagonal on
                    acc[e][0] = fmaf(f, b.x, acc[e][0]);
                    acc[e][1] = fmaf(f, b.y, acc[e][1]);
                    acc[e][2] = fmaf(f, b.z, acc[e][2]);
                    acc[e][3] = fmaf(f, b.w, acc[e][3]);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float4 *>(&sh.w[32 + r + e][x]) = make_float4(-acc[e][0], -acc[e][1], -acc[e][2], -acc[e][3]);
        }
        __syncthreads();
        for (int f = warp; f < kTriangle; f += kThreads / 32) {
            int j = 0, i = 0;
            while (triangle_at(j, i) != f)
                if (++i > j / 2)
                    ++j, i = 0;
            const int t = 8 * j + lane / 4, s = 16 * i + 2 * (lane % 4);
            auto value = [&](int u) { return u == t ? 1.f : u < t ? sh.w[t][u] * sh.beta[u] : 0.f; };
            uint32_t word[4];
            split2<T>(value(s), value(s + 1), word[0], word[2]);
            split2<T>(value(s + 8), value(s + 9), word[1], word[3]);
            cell.inverse[f * 32 + lane] = make_uint4(word[0], word[1], word[2], word[3]);
        }
        if constexpr (BACK)
            store_t(static_cast<DeltaCellBack &>(cell).inverse_t,
                    [&](int r, int t) { return r == t ? 1.f : r > t ? sh.beta[r] * sh.w[r][t] : 0.f; });
    }
}

}  // namespace

size_t delta_cell_bytes(bool backward) { return backward ? sizeof(DeltaCellBack) : sizeof(DeltaCell); }

cudaError_t launch_delta_prep(const DeltaArgs &a, bool half, bool backward, cudaStream_t s)
{
    auto go = [&](auto kernel, size_t shared) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
        if (e != cudaSuccess)
            return e;
        kernel<<<(unsigned)((size_t)a.slots * a.H), kThreads, shared, s>>>(a);
        return cudaGetLastError();
    };
    auto by_back = [&](auto t, auto kd) {
        typedef std::remove_pointer_t<decltype(t)> T;
        constexpr int KD = decltype(kd)::value;
        return backward ? go(delta_prep_kernel<T, KD, true>, sizeof(PrepShared<KD>)) : go(delta_prep_kernel<T, KD, false>, sizeof(PrepShared<KD>));
    };
    auto by_type = [&](auto kd) { return half ? by_back((__half *)0, kd) : by_back((__nv_bfloat16 *)0, kd); };
    return a.K == 128 ? by_type(Int<128>()) : by_type(Int<64>());
}

}  // namespace gla
