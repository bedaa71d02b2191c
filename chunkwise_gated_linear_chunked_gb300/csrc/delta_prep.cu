// Gated delta rule in chunks of 64 tokens, what does not depend on the state: of each (chunk, value head) the decays, the
// scores P and the inverse that turns the values' remainders into update rows (see DeltaCell).  One CTA a (chunk, key
// head): k k^T and q k^T once for the value heads that share the key head.
//
// With L_ij = e^(G_i - G_j) k_i.k_j (j < i) and N the rows that update the state, N = beta Y and Y = R - L N for
// R = V - e^G K S, so Y = (I + L diag(beta))^-1 R.  The inverse is T^ = I + W diag(beta), and the one that the gradients
// take, (I + diag(beta) L)^-1, is T = I + diag(beta) W, with one W below the diagonal.  Warp w holds rows 16 w up.  Its block
// on the diagonal is found by substitution in fp32, a lane a column (W_ij = -(L_ij + sum over j < m < i of L_im beta_m
// W_mj)); what lies left of it by warp products, W_wp = -sum over p <= m < w of (T^_ww L_wm) T_mp, rows of blocks one after
// the other.  A sum of powers of L would need no substitution and is not taken: for keys that look alike its terms grow
// like binomials.  Products of two rounded matrices take three terms, so that blocks are within 2^-16 of their size.  Both
// inverses are stored without their diagonal of ones, which the chains add in fp32.
//
// Differences of G decide the decays, and G may run far from zero, so it is summed in 64 bits and kept in two floats.
// Gates count as at least -1000 (a decay of 0), which keeps differences of two cleared rows finite.
//
// Bound by the latency of a CTA's steps: 4 x 2048 tokens of 8 heads take 25 us (1024 CTAs, four an SM; three: 30, five, with
// spills: 36; eight warps a CTA in two paths: 41), 65536 tokens of 32 heads 555 us for 1.7 GB.  Substitution over 32 rows
// in place of blocks of 16 took 46 us.
#include "delta_mma.cuh"

namespace gla {
namespace {

constexpr int kThreads = 128;

template <bool BACK>
struct PrepShared {
    uint16_t t_hi[64][72], t_lo[64][72];   // L, then T (16 bits and remainders), by blocks up to the diagonal
    uint16_t d_hi[4][16][24], d_lo[4][16][24];   // T^ on the diagonal
    float l[4][16][20];                    // L on the diagonal
    float g_hi[64], g_lo[64], beta[64];
    float most[4];                         // largest q.k of each warp's rows (fp16)
    uint16_t p_hi[BACK ? 64 : 1][72], p_lo[BACK ? 64 : 1][72];
};
template <int KD, bool BACK>
union PrepMemory {
    struct {
        uint16_t k[64][KD + 8], q[64][KD + 8];
    } rows;   // until the products are formed
    PrepShared<BACK> s;
};

// c += (a_hi + a_lo) (b_hi + b_lo) but for the remainders' product; two tiles, b as ldsm_t of the two planes gives it.
template <typename T>
__device__ __forceinline__ void mma3(float (&c)[2][4], const uint32_t (&a_hi)[4], const uint32_t (&a_lo)[4], const uint32_t (&b_hi)[4],
                                     const uint32_t (&b_lo)[4])
{
#pragma unroll
    for (int y = 0; y < 2; ++y)
        mma<T>(c[y], a_hi, b_hi[2 * y], b_hi[2 * y + 1]);
#pragma unroll
    for (int y = 0; y < 2; ++y)
        mma<T>(c[y], a_lo, b_hi[2 * y], b_hi[2 * y + 1]);
#pragma unroll
    for (int y = 0; y < 2; ++y)
        mma<T>(c[y], a_hi, b_lo[2 * y], b_lo[2 * y + 1]);
}

// Words of a 16 x 16 block (two tiles of a result) to two planes of 16-bit values.
template <int PITCH>
__device__ __forceinline__ void put_block(uint16_t (*hi)[PITCH], uint16_t (*lo)[PITCH], int row, int col, const uint32_t (&h)[4], const uint32_t (&l)[4])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {   // (rows, rows + 8) of the first tile, then of the second
        *reinterpret_cast<uint32_t *>(&hi[row + (e & 1) * 8][col + (e >> 1) * 8]) = h[e];
        *reinterpret_cast<uint32_t *>(&lo[row + (e & 1) * 8][col + (e >> 1) * 8]) = l[e];
    }
}

template <typename T, int KD, bool BACK>
__global__ void __launch_bounds__(kThreads, BACK ? 3 : 4) delta_prep_kernel(DeltaArgs a)
{
    typedef std::conditional_t<BACK, DeltaCellBack, DeltaCell> Cell;
    extern __shared__ __align__(16) char raw[];
    PrepMemory<KD, BACK> &mem = *reinterpret_cast<PrepMemory<KD, BACK> *>(raw);
    PrepShared<BACK> &sh = mem.s;
    const int slot = blockIdx.x / a.H, h = blockIdx.x - slot * a.H, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    int n, c, first, rows;
    tc::grid_dep_wait();
    if (!delta_chunk(a, slot, n, c, first, rows))
        return;
    const int per = a.HV / a.H;
    const size_t key = ((size_t)first * a.H + h) * KD, pitch = (size_t)a.H * KD;
    copy_rows<KD, kThreads>(tc::smem_u32(mem.rows.k), static_cast<const T *>(a.k) + key, pitch, rows, KD);
    copy_rows<KD, kThreads>(tc::smem_u32(mem.rows.q), static_cast<const T *>(a.q) + key, pitch, rows, KD);
    copies_end();
    float gate[2], strength[2];   // of two rows a lane of the first warp, one head ahead
    auto ask = [&](int v) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            const bool on = warp == 0 && v < per && t < rows;
            const size_t at = (size_t)(first + t) * a.HV + h * per + v;
            gate[e] = on ? a.g[at] : 0.f;
            strength[e] = on ? a.beta[at] : 0.f;
        }
    };
    ask(0);
    copies_wait<0>();
    __syncthreads();

    // rows 16 warp up of k k^T and q k^T, columns up to the diagonal block
    float kk[8][4] = {}, qk[8][4] = {};
    {
        const uint32_t row = (16 * warp + lane % 16) * (KD + 8) * 2 + (lane / 16) * 16;
        const uint32_t ka = tc::smem_u32(mem.rows.k) + row, qa = tc::smem_u32(mem.rows.q) + row;
        const uint32_t kb = tc::smem_u32(mem.rows.k) + ((lane & 7) + (lane / 16) * 8) * (KD + 8) * 2 + ((lane / 8) & 1) * 16;
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

    // fp16: P goes in over the power of two of the largest q.k, and without `scale`
    float most = 0.f;
    Power power = {1.f, 1.f};
    if constexpr (kScaled<T>) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            if (p > warp)
                break;
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (16 * p + 8 * y + 2 * (lane % 4) + (e & 1) <= 16 * warp + lane / 4 + (e >> 1) * 8)
                        most = fmaxf(most, fabsf(qk[2 * p + y][e]));
        }
        most = warp_largest(most);
    }

    // a block of 16-bit values [rows][columns] as a right operand: rows are its steps (ldsm_t), or its columns (ldsm)
    const int step_row = (lane & 7) + ((lane / 8) & 1) * 8, step_col = (lane / 16) * 8;
    const int t0 = 16 * warp + lane / 4, two = 2 * (lane % 4);
    for (int v = 0; v < per; ++v) {
        Cell &cell = reinterpret_cast<Cell *>(a.chunk)[(size_t)slot * a.HV + h * per + v];
        __syncthreads();   // the rows' products (the last head's blocks) are read
        if (warp == 0) {
            double g[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                g[e] = (gate[e] < -1000.f ? -1000.0 : (double)gate[e]) * 1.4426950408889634;
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
                sh.beta[t] = strength[e];
                const float start = exp2_fast((float)G);
                cell.row[t] = make_float4(strength[e], start, exp2_fast((float)(end - G)), a.scale * start);
                if constexpr (BACK)
                    cell.gate[t] = make_float2(sh.g_hi[t], sh.g_lo[t]);
            }
        }
        ask(v + 1);
        if (kScaled<T> && lane == 0)
            sh.most[warp] = most;
        __syncthreads();
        if constexpr (kScaled<T>) {
            power = power_of<kOperand>(fmaxf(fmaxf(sh.most[0], sh.most[1]), fmaxf(sh.most[2], sh.most[3])));
            if (tid == 0)
                a.score[(size_t)slot * a.HV + h * per + v] = a.scale * power.from;
        }
        const float by = kScaled<T> ? power.to : a.scale;
        // decays of this lane's rows t0 and t0 + 8 times k k^T and q k^T: P goes to the cell as it lies (a result's rows
        // are a right operand's columns), L to shared memory
        const float hi0 = sh.g_hi[t0], lo0 = sh.g_lo[t0], hi1 = sh.g_hi[t0 + 8], lo1 = sh.g_lo[t0 + 8];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            if (p > warp)
                break;
            float l[2][4], s[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = 16 * p + 8 * y + two + e;
                    const float hj = sh.g_hi[j], lj = sh.g_lo[j];
                    const float d0 = j <= t0 ? exp2_fast((hi0 - hj) + (lo0 - lj)) : 0.f;
                    const float d1 = j <= t0 + 8 ? exp2_fast((hi1 - hj) + (lo1 - lj)) : 0.f;
                    s[y][e] = j <= t0 ? by * (d0 * qk[2 * p + y][e]) : 0.f;
                    s[y][2 + e] = j <= t0 + 8 ? by * (d1 * qk[2 * p + y][2 + e]) : 0.f;
                    l[y][e] = j < t0 ? d0 * kk[2 * p + y][e] : 0.f;
                    l[y][2 + e] = j < t0 + 8 ? d1 * kk[2 * p + y][2 + e] : 0.f;
                }
            uint32_t hi[4], lo[4];
            split_pair<T>(s[0], s[1], hi, lo);   // rows t0 and t0 + 8 of the first tile, then of the second
            cell.score[triangle_at(2 * warp, p) * 32 + lane] = make_uint4(hi[0], hi[2], lo[0], lo[2]);
            cell.score[triangle_at(2 * warp + 1, p) * 32 + lane] = make_uint4(hi[1], hi[3], lo[1], lo[3]);
            if constexpr (BACK)
                put_block<72>(sh.p_hi, sh.p_lo, t0, 16 * p + two, hi, lo);
            if (p < warp) {
                split_pair<T>(l[0], l[1], hi, lo);
                put_block<72>(sh.t_hi, sh.t_lo, t0, 16 * p + two, hi, lo);
            } else {
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sh.l[warp][lane / 4 + (e >> 1) * 8][8 * y + two + (e & 1)] = l[y][e];
            }
        }
        __syncwarp();
        {   // the block on the diagonal; both halves of the warp find it, one stores T^, the other T
            const int x = lane % 16;
            const float bx = sh.beta[16 * warp + x];
            float w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int m = 0; m < i; m += 4) {
                    const float4 l = *reinterpret_cast<const float4 *>(&sh.l[warp][i][m]);
                    s0 = fmaf(l.x, w[m], s0);
                    if (m + 1 < i) s1 = fmaf(l.y, w[m + 1], s1);
                    if (m + 2 < i) s0 = fmaf(l.z, w[m + 2], s0);
                    if (m + 3 < i) s1 = fmaf(l.w, w[m + 3], s1);
                }
                const float value = -(s0 + s1);
                w[i] = i == x ? 1.f : i > x ? sh.beta[16 * warp + i] * value : 0.f;
                const float out = lane < 16 && i > x ? bx * value : w[i];
                uint32_t hi, lo;
                split2<T>(out, 0.f, hi, lo);
                if (lane < 16)
                    sh.d_hi[warp][i][x] = (uint16_t)hi, sh.d_lo[warp][i][x] = (uint16_t)lo;
                else
                    sh.t_hi[16 * warp + i][16 * warp + x] = (uint16_t)hi, sh.t_lo[16 * warp + i][16 * warp + x] = (uint16_t)lo;
            }
        }
        __syncwarp();
        const uint32_t below = lane / 4 == two ? 0xffff0000u : lane / 4 == two + 1 ? 0xffffu : ~0u;   // clears ones on a diagonal
        uint32_t m_hi[3][4], m_lo[3][4];   // -T^ L of this row of blocks
        {
            uint32_t d_hi[4], d_lo[4], f_hi[4], f_lo[4];
            ldsm(d_hi, tc::smem_u32(&sh.d_hi[warp][lane % 16][(lane / 16) * 8]));
            ldsm(d_lo, tc::smem_u32(&sh.d_lo[warp][lane % 16][(lane / 16) * 8]));
            // as a right operand its rows are the columns: words 0, 2 hold rows up to 8, words 1, 3 the others
            cell.inverse[triangle_at(2 * warp, warp) * 32 + lane] = make_uint4(d_hi[0] & below, d_hi[2], d_lo[0], d_lo[2]);
            cell.inverse[triangle_at(2 * warp + 1, warp) * 32 + lane] = make_uint4(d_hi[1], d_hi[3] & below, d_lo[1], d_lo[3]);
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                if (p >= warp)
                    break;
                float f[2][4] = {};
                ldsm_t(f_hi, tc::smem_u32(&sh.t_hi[16 * warp + step_row][16 * p + step_col]));
                ldsm_t(f_lo, tc::smem_u32(&sh.t_lo[16 * warp + step_row][16 * p + step_col]));
                mma3<T>(f, d_hi, d_lo, f_hi, f_lo);
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        f[y][e] = -f[y][e];
                split_pair<T>(f[0], f[1], m_hi[p], m_lo[p]);
            }
        }
        const float b0 = sh.beta[t0], b1 = sh.beta[t0 + 8];
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            __syncthreads();   // the rows of blocks before this one are there
            if (warp != w)
                continue;
#pragma unroll
            for (int p = 0; p < w; ++p) {
                float f[2][4] = {};
#pragma unroll
                for (int m = p; m < w; ++m) {
                    uint32_t f_hi[4], f_lo[4];
                    ldsm_t(f_hi, tc::smem_u32(&sh.t_hi[16 * m + step_row][16 * p + step_col]));
                    ldsm_t(f_lo, tc::smem_u32(&sh.t_lo[16 * m + step_row][16 * p + step_col]));
                    mma3<T>(f, m_hi[m], m_lo[m], f_hi, f_lo);
                }
                uint32_t hi[4], lo[4];
                float t[2][4], i[2][4];
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        t[y][e] = (e < 2 ? b0 : b1) * f[y][e];
                        i[y][e] = sh.beta[16 * p + 8 * y + two + (e & 1)] * f[y][e];
                    }
                split_pair<T>(t[0], t[1], hi, lo);
                put_block<72>(sh.t_hi, sh.t_lo, t0, 16 * p + two, hi, lo);
                split_pair<T>(i[0], i[1], hi, lo);
                cell.inverse[triangle_at(2 * w, p) * 32 + lane] = make_uint4(hi[0], hi[2], lo[0], lo[2]);
                cell.inverse[triangle_at(2 * w + 1, p) * 32 + lane] = make_uint4(hi[1], hi[3], lo[1], lo[3]);
            }
        }
        if constexpr (BACK) {   // T' and P': blocks (step i, column tiles 2 p and 2 p + 1), i >= p
            __syncthreads();
            DeltaCellBack &back = static_cast<DeltaCellBack &>(cell);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i < warp)
                    continue;
                uint32_t hi[4], lo[4];
                ldsm_t(hi, tc::smem_u32(&sh.t_hi[16 * i + step_row][16 * warp + step_col]));
                ldsm_t(lo, tc::smem_u32(&sh.t_lo[16 * i + step_row][16 * warp + step_col]));
                if (i == warp)
                    hi[0] &= below, hi[3] &= below;
                back.inverse_t[triangle_at_t(2 * warp, i) * 32 + lane] = make_uint4(hi[0], hi[1], lo[0], lo[1]);
                back.inverse_t[triangle_at_t(2 * warp + 1, i) * 32 + lane] = make_uint4(hi[2], hi[3], lo[2], lo[3]);
                ldsm_t(hi, tc::smem_u32(&sh.p_hi[16 * i + step_row][16 * warp + step_col]));
                ldsm_t(lo, tc::smem_u32(&sh.p_lo[16 * i + step_row][16 * warp + step_col]));
                back.score_t[triangle_at_t(2 * warp, i) * 32 + lane] = make_uint4(hi[0], hi[1], lo[0], lo[1]);
                back.score_t[triangle_at_t(2 * warp + 1, i) * 32 + lane] = make_uint4(hi[2], hi[3], lo[2], lo[3]);
            }
        }
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
        return launch_early_shared(kernel, (unsigned)((size_t)a.slots * a.H), kThreads, shared, s, a);
    };
    auto by_back = [&](auto t, auto kd) {
        typedef std::remove_pointer_t<decltype(t)> T;
        constexpr int KD = decltype(kd)::value;
        return backward ? go(delta_prep_kernel<T, KD, true>, sizeof(PrepMemory<KD, true>))
                        : go(delta_prep_kernel<T, KD, false>, sizeof(PrepMemory<KD, false>));
    };
    auto by_type = [&](auto kd) { return half ? by_back((__half *)0, kd) : by_back((__nv_bfloat16 *)0, kd); };
    return a.K == 128 ? by_type(Int<128>()) : by_type(Int<64>());
}

}  // namespace gla
