// Gated delta rule in chunks of 64 tokens, the chain over a sequence's chunks (see DeltaCell for what the cells hold):
//
//     R = V - e^G K S,   Y = T^ R,   N = beta Y,   o = scale e^G q S + P N,   S <- e^G_end S + (e^(G_end - G) K)^T N
//
// The columns of S do not meet, and 16 of them make one warp's rows: transposed, S' (16 x keys) is the left operand of
// S' K', whose result is the left operand of (T^ R)' = R' T^', whose result is that of S' += N' K.  So the whole chain
// of a chunk's products stays in registers, and no value of it passes shared memory.  Two warps share 16 columns, half of
// the keys (and of the tokens' steps in R' T^' and N' P') each, and add their partial results through shared memory: three
// exchanges a chunk, each behind products that do not wait for it, where one warp alone would have twice the chain (316
// products of 16 x 8 x 16, at 8 cycles each, on the way from one state to the next).
//
// Inputs are exact operands; S, R, N and the cells' matrices go in as a rounded value and its remainder, two products for
// an exact partner and three for another such (the product of two remainders, 2^-18, is left out).
//
// Warp matrix instructions and not tcgen05: the chain is bound by its latency, with 16 to 64 columns a CTA, and there a
// product's way through tensor memory and shared memory (a commit, a load, a conversion and a store between any two) costs
// more than the products; 587 TFLOP/s are there for them (measured) against the chain's 250 or so.
#include "delta_mma.cuh"

namespace gla {
namespace {

// Shared memory of a CTA of VG groups of 16 columns.
template <int KD, int VG, bool SAVE>
struct ChainShared {
    static constexpr int kStages = VG <= 2 ? 3 : 2;
    struct Stage {
        uint16_t k[64][KD + 8], q[64][KD + 8], v[64][16 * VG + 8];
        uint16_t d[SAVE ? 64 : 1][16 * VG + 8];
        DeltaCell cell;
    } stage[kStages];
    float4 part[2 * VG][16][32];   // a warp's partial results for its partner: 4 tiles of k S, 8 of N, 4 of o
};

__device__ __forceinline__ void pair_sync(int pair) { asm volatile("bar.sync %0, 64;" ::"r"(pair + 1) : "memory"); }

__device__ __forceinline__ float4 as_float4(const float (&c)[4]) { return make_float4(c[0], c[1], c[2], c[3]); }

// Steps of 16 tokens that a warp of the pair takes: 0 and 3, or 1 and 2 (ten tiles of a triangle each).
__device__ __forceinline__ constexpr int step_of(int warp, int x) { return x ? (warp ? 2 : 3) : warp; }

// c (64 tokens) += left operands of this warp's two steps times a triangle of the cell, lower or upper.
template <typename T, int W, bool UPPER>
__device__ __forceinline__ void triangle(float (&c)[8][4], const uint32_t (&hi)[2][4], const uint32_t (&lo)[2][4], const uint4 *m, int lane)
{
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int i = step_of(W, x);
        uint4 b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (UPPER ? i >= j / 2 : i <= j / 2)
                b[j] = m[(UPPER ? triangle_at_t(j, i) : triangle_at(j, i)) * 32 + lane];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (UPPER ? i >= j / 2 : i <= j / 2)
                mma<T>(c[j], hi[x], b[j].x, b[j].y);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (UPPER ? i >= j / 2 : i <= j / 2)
                mma<T>(c[j], lo[x], b[j].x, b[j].y);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (UPPER ? i >= j / 2 : i <= j / 2)
                mma<T>(c[j], hi[x], b[j].z, b[j].w);
    }
}

// c (64 tokens) += S' rows', for rows of keys in shared memory at `at` (this lane's address for its part of the keys).
template <typename T, int KD>
__device__ __forceinline__ void state_by_rows(float (&c)[8][4], const uint32_t (&hi)[KD / 32][4], const uint32_t (&lo)[KD / 32][4], uint32_t at)
{
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int m = 0; m < KD / 64; ++m) {
            uint32_t b[4][4];   // four tiles of 8 tokens, two steps of 16 keys
#pragma unroll
            for (int j = 0; j < 4; ++j)
                ldsm(b[j], at + (half * 4 + j) * 8 * (KD + 8) * 2 + m * 64);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma<T>(c[half * 4 + j], hi[2 * m + e], b[j][2 * e], b[j][2 * e + 1]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma<T>(c[half * 4 + j], lo[2 * m + e], b[j][2 * e], b[j][2 * e + 1]);
            }
        }
}

// S' (this warp's keys) += left operands over the 64 tokens times rows of keys in shared memory.
template <typename T, int KD>
__device__ __forceinline__ void state_add(float (&s)[KD / 16][4], const uint32_t (&hi)[4][4], const uint32_t (&lo)[4][4], uint32_t at)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int p = 0; p < KD / 64; ++p) {
            uint32_t b[2][4];   // two pairs of tiles of 8 keys
#pragma unroll
            for (int x = 0; x < 2; ++x)
                ldsm_t(b[x], at + i * 16 * (KD + 8) * 2 + (2 * p + x) * 32);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                mma<T>(s[4 * p + 2 * x], hi[i], b[x][0], b[x][1]);
                mma<T>(s[4 * p + 2 * x + 1], hi[i], b[x][2], b[x][3]);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                mma<T>(s[4 * p + 2 * x], lo[i], b[x][0], b[x][1]);
                mma<T>(s[4 * p + 2 * x + 1], lo[i], b[x][2], b[x][3]);
            }
        }
}

// What a CTA walks.
struct ChainWalk {
    int n, hv, hk, bos, len, chunks, slot, v0;
    size_t head;
};
__device__ __forceinline__ bool chain_walk(const DeltaArgs &a, int tiles, int width, ChainWalk &w)
{
    w.v0 = blockIdx.x % tiles * width;
    w.head = blockIdx.x / tiles;
    w.n = (int)(w.head / a.HV);
    w.hv = (int)(w.head - (size_t)w.n * a.HV);
    w.hk = w.hv / (a.HV / a.H);
    if (!delta_sequence(a, w.n, w.bos, w.len)) {
        if (threadIdx.x == 0)
            report(a.status, GLA_ERR_INVALID_ARG);
        return false;
    }
    w.chunks = (w.len + kDeltaChunk - 1) / kDeltaChunk;
    w.slot = delta_first_slot(a, w.n);
    return true;
}

// This warp's part of the state: columns v0 + lane / 4 (and 8 on), keys k0 + 8 tile + 2 (lane % 4) (and 1 on).
template <int KD>
__device__ __forceinline__ void state_io(float (&s)[KD / 16][4], float *p, const float *from, size_t at, int V, int col, bool on, bool out)
{
#pragma unroll
    for (int j = 0; j < KD / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const size_t i = at + (size_t)(8 * j + (e & 1)) * V + col + (e >> 1) * 8;
            if (out) {
                if (on)
                    p[i] = s[j][e];
            } else {
                s[j][e] = on && from ? from[i] : 0.f;
            }
        }
}

template <typename T, typename To, int KD, int VG, bool SAVE>
__global__ void __launch_bounds__(64 * VG, 1) delta_chain_kernel(DeltaArgs a, int tiles)
{
    typedef ChainShared<KD, VG, SAVE> Shared;
    constexpr int kThreads = 64 * VG, kStages = Shared::kStages, kWidth = 16 * VG, kRow = (KD + 8) * 2;
    extern __shared__ __align__(16) char raw[];
    Shared &sh = *reinterpret_cast<Shared *>(raw);
    ChainWalk w;
    if (!chain_walk(a, tiles, kWidth, w))
        return;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, pair = warp / 2, half = warp % 2;
    const int col = w.v0 + 16 * pair + lane / 4, two = 2 * (lane % 4);
    const bool on = w.v0 + 16 * pair < a.V;   // whole groups of 16 columns
    const size_t cell_bytes = sizeof(DeltaCell);

    float s[KD / 16][4];
    const size_t state = (w.head * a.K + half * (KD / 2) + two) * a.V;
    state_io<KD>(s, nullptr, a.h0, state, a.V, col, on, false);

    auto issue = [&](int c) {
        if (c < w.chunks) {
            typename Shared::Stage &st = sh.stage[c % kStages];
            const int rows = min(kDeltaChunk, w.len - c * kDeltaChunk);
            const size_t row = (size_t)w.bos + (size_t)c * kDeltaChunk, key = (row * a.H + w.hk) * KD, val = (row * a.HV + w.hv) * a.V + w.v0;
            copy_rows<KD, kThreads>(tc::smem_u32(st.k), static_cast<const T *>(a.k) + key, (size_t)a.H * KD, rows, KD);
            copy_rows<KD, kThreads>(tc::smem_u32(st.q), static_cast<const T *>(a.q) + key, (size_t)a.H * KD, rows, KD);
            copy_rows<kWidth, kThreads>(tc::smem_u32(st.v), static_cast<const T *>(a.v) + val, (size_t)a.HV * a.V, rows, a.V - w.v0);
            const char *cell = a.chunk + ((size_t)(w.slot + c) * a.HV + w.hv) * cell_bytes;
#pragma unroll
            for (int i = 0; i < (int)(sizeof(DeltaCell) / 16 + kThreads - 1) / kThreads; ++i) {
                const int e = i * kThreads + tid;
                if (e < (int)sizeof(DeltaCell) / 16)
                    copy16(tc::smem_u32(&st.cell) + e * 16, cell + e * 16, true);
            }
        }
        copies_end();
    };
    float o[2][2][4];   // own two steps of o, two tiles each
    auto store_o = [&](int c) {
        const int rows = min(kDeltaChunk, w.len - c * kDeltaChunk);
        To *out = static_cast<To *>(a.o) + (((size_t)w.bos + (size_t)c * kDeltaChunk) * a.HV + w.hv) * a.V + col;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const float4 p = sh.part[warp ^ 1][12 + 2 * x + y][lane];
                const float r[4] = {o[x][y][0] + p.x, o[x][y][1] + p.y, o[x][y][2] + p.z, o[x][y][3] + p.w};
                const int t = 16 * step_of(half, x) + 8 * y + two;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (on && t + (e & 1) < rows)
                        out[(size_t)(t + (e & 1)) * a.HV * a.V + (e >> 1) * 8] = narrow<To>(r[e]);
            }
    };
    auto body = [&](auto which, int c) {
        constexpr int W = decltype(which)::value;
        typename Shared::Stage &st = sh.stage[c % kStages];
        const float4 *row = st.cell.row;
        const uint32_t rows_at = (lane & 7) * kRow + (lane / 8) * 16 + W * KD;   // of ldsm: 8 tokens, 32 keys of this half
        const uint32_t keys_at = ((lane & 7) + ((lane / 8) & 1) * 8) * kRow + (lane / 16) * 16 + W * KD;   // of ldsm_t: 16 tokens, 16 keys
        uint32_t sh_hi[KD / 32][4], sh_lo[KD / 32][4];
#pragma unroll
        for (int i = 0; i < KD / 32; ++i)
            split_pair<T>(s[2 * i], s[2 * i + 1], sh_hi[i], sh_lo[i]);
        float ks[8][4] = {};
        state_by_rows<T, KD>(ks, sh_hi, sh_lo, tc::smem_u32(st.k) + rows_at);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y)
                sh.part[warp][2 * x + y][lane] = as_float4(ks[2 * step_of(1 - W, x) + y]);
        float qs[8][4] = {};
        state_by_rows<T, KD>(qs, sh_hi, sh_lo, tc::smem_u32(st.q) + rows_at);
        pair_sync(pair);
        // R of this warp's steps
        uint32_t r_hi[2][4], r_lo[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int i = step_of(W, x);
            uint32_t v[4];
            ldsm_t(v, tc::smem_u32(st.v) + (16 * i + (lane & 7) + (lane / 16) * 8) * (kWidth + 8) * 2 + pair * 32 + ((lane / 8) & 1) * 16);
            float r[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const float4 p = sh.part[warp ^ 1][2 * x + y][lane];
                const float f0 = row[16 * i + 8 * y + two].y, f1 = row[16 * i + 8 * y + two + 1].y;
                const float2 v0 = widen2<T>(v[2 * y]), v1 = widen2<T>(v[2 * y + 1]);
                const float(&k)[4] = ks[2 * i + y];
                r[y][0] = fmaf(-f0, k[0] + p.x, v0.x);
                r[y][1] = fmaf(-f1, k[1] + p.y, v0.y);
                r[y][2] = fmaf(-f0, k[2] + p.z, v1.x);
                r[y][3] = fmaf(-f1, k[3] + p.w, v1.y);
            }
            split_pair<T>(r[0], r[1], r_hi[x], r_lo[x]);
        }
        float n[8][4] = {};
        triangle<T, W, false>(n, r_hi, r_lo, st.cell.inverse, lane);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sh.part[warp][4 + j][lane] = as_float4(n[j]);
        // meanwhile: q S scaled by its rows' decays
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f0 = row[8 * j + two].w, f1 = row[8 * j + two + 1].w;
            qs[j][0] *= f0, qs[j][1] *= f1, qs[j][2] *= f0, qs[j][3] *= f1;
        }
        pair_sync(pair);
        uint32_t n_hi[4][4], n_lo[4][4], p_hi[2][4], p_lo[2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float u[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int j = 2 * i + y;
                const float4 p = sh.part[warp ^ 1][4 + j][lane], c0 = row[8 * j + two], c1 = row[8 * j + two + 1];
                n[j][0] = c0.x * (n[j][0] + p.x);
                n[j][1] = c1.x * (n[j][1] + p.y);
                n[j][2] = c0.x * (n[j][2] + p.z);
                n[j][3] = c1.x * (n[j][3] + p.w);
                u[y][0] = c0.z * n[j][0], u[y][1] = c1.z * n[j][1], u[y][2] = c0.z * n[j][2], u[y][3] = c1.z * n[j][3];
            }
            split_pair<T>(u[0], u[1], n_hi[i], n_lo[i]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
            split_pair<T>(n[2 * step_of(W, x)], n[2 * step_of(W, x) + 1], p_hi[x], p_lo[x]);
        const float last = row[kDeltaChunk - 1].y;
#pragma unroll
        for (int j = 0; j < KD / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[j][e] *= last;
        state_add<T, KD>(s, n_hi, n_lo, tc::smem_u32(st.k) + keys_at);
        triangle<T, W, false>(qs, p_hi, p_lo, st.cell.score, lane);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                sh.part[warp][12 + 2 * x + y][lane] = as_float4(qs[2 * step_of(1 - W, x) + y]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[x][y][e] = qs[2 * step_of(W, x) + y][e];
            }
    };

    for (int c = 0; c < kStages - 1; ++c)
        issue(c);
    for (int c = 0; c < w.chunks; ++c) {
        copies_wait<kStages - 2>();
        __syncthreads();
        if (c)
            store_o(c - 1);
        issue(c + kStages - 1);
        if (half == 0)
            body(Int<0>(), c);
        else
            body(Int<1>(), c);
    }
    __syncthreads();
    if (w.chunks)
        store_o(w.chunks - 1);
    if (a.ht)
        state_io<KD>(s, a.ht, nullptr, state, a.V, col, on, true);
}

template <typename F>
cudaError_t with_shared(F kernel, size_t shared, unsigned grid, int threads, const DeltaArgs &a, int tiles, cudaStream_t s)
{
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
    if (e != cudaSuccess)
        return e;
    kernel<<<grid, threads, shared, s>>>(a, tiles);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_chain(const DeltaArgs &a, int dtype, int sms, cudaStream_t s)
{
    return delta_types(dtype, [&](auto x, auto o) {
        typedef std::remove_pointer_t<decltype(x)> T;
        typedef std::remove_pointer_t<decltype(o)> To;
        if constexpr (std::is_same_v<T, float>) {
            return cudaErrorInvalidValue;
        } else {
            auto go = [&](auto kd, auto vg) {
                constexpr int KD = decltype(kd)::value, VG = decltype(vg)::value;
                const int tiles = (a.V + 16 * VG - 1) / (16 * VG);
                return with_shared(delta_chain_kernel<T, To, KD, VG, false>, sizeof(ChainShared<KD, VG, false>),
                                   (unsigned)((size_t)a.N * a.HV * tiles), 64 * VG, a, tiles, s);
            };
            const bool few = (size_t)a.N * a.HV * ((a.V + 31) / 32) <= (size_t)sms;
            auto by_keys = [&](auto vg) { return a.K == 128 ? go(Int<128>(), vg) : go(Int<64>(), vg); };
            return few ? by_keys(Int<2>()) : by_keys(Int<4>());
        }
    });
}

}  // namespace gla
