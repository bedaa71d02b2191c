// Gated delta rule in chunks of 64 tokens, the chain over a sequence's chunks (see DeltaCell for what the cells hold):
//
//     R = V - e^G K S,   Y = T^ R,   N = beta Y,   o = scale e^G q S + P N,   S <- e^G_end S + (e^(G_end - G) K)^T N
//
// The columns of S do not meet, and 16 of them make one warp's rows: transposed, S' (16 x keys) is the left operand of
// S' K', whose result is the left operand of (T^ R)' = R' T^', whose result is that of S' += N' K.  So the chain of a
// chunk's products stays in the registers of one warp.  A second warp has what is not on the way from one state to the
// next: the output o' = S' q' + N' P' from the first one's rounded S and its Y, and before that the remainders' share of
// S' K'.  Each has 252 of a chunk's 504 products of 16 x 8 x 16 (8 cycles each on a quarter of an SM).
//
// Inputs are exact operands; S, R, N and the cells' matrices go in as a rounded value and its remainder, two products for
// an exact partner and three for another such (the product of two remainders, 2^-18, is left out).
//
// A CTA takes 32 columns where those make fewer CTAs than the GPU has SMs: its four warps have a quarter of the SM each.
// Otherwise 64: shared memory, which every warp's right operands pass, and the quarters are then about equally busy.  (Two
// warps that share 16 columns by keys, and add their partial sums through shared memory, were bound by it: 2.7 us a chunk
// of 32 columns where the products take 1.0.)
//
// Warp matrix instructions and not tcgen05: the chain is bound by its latency, with 32 columns a CTA, and there a
// product's way through tensor memory and shared memory (a commit, a load, a conversion and a store between any two) costs
// more than the products.
#include <atomic>
#include <cstring>

#include <cudaTypedefs.h>

#include "api_common.h"
#include "delta_mma.cuh"

namespace gla {
namespace {

// Shared memory of a CTA of VG groups of 16 columns; ROWS: matrices of 64 rows of values (v, and dO for the gradients).
template <int KD, int VG, int ROWS, typename Cell>
struct ChainShared {
    struct Stage {
        uint16_t k[KD / 64][64][64], q[KD / 64][64][64], v[ROWS][64][16 * VG];   // as the tensor copies swizzle them
        Cell cell;
    } stage[2];
    static_assert(sizeof(Stage) % 1024 == 0, "swizzled tiles start on 1024 bytes");
    uint4 state[VG][KD / 16][2][32];     // the chain's rounded S and its remainders, as left operands
    float4 ks[VG][8][32], n[VG][8][32];  // the remainders' share of k S; Y
    uint64_t full[2];
};

// Barriers of the two warps of a group of 16 columns.
enum { kBarState = 1, kBarShare = 5, kBarRows = 9 };
__device__ __forceinline__ void bar_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void bar_tell(int id) { asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory"); }

__device__ __forceinline__ void copy_bulk(void *to, const void *from, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(tc::smem_u32(to)),
                 "l"(from), "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ float4 as_float4(const float (&c)[4]) { return make_float4(c[0], c[1], c[2], c[3]); }
__device__ __forceinline__ uint4 as_uint4(const uint32_t (&c)[4]) { return make_uint4(c[0], c[1], c[2], c[3]); }
__device__ __forceinline__ void take(uint32_t (&r)[4], uint4 v) { r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w; }

// c (64 tokens) += left operands of the four steps of 16 tokens times a triangle of the cell, lower or upper.
template <typename T, bool UPPER>
__device__ __forceinline__ void triangle(float (&c)[8][4], const uint32_t (&hi)[4][4], const uint32_t (&lo)[4][4], const uint4 *m, int lane)
{
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int i = UPPER ? 3 - x : x;   // the longest first
        uint4 b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (UPPER ? i >= j / 2 : i <= j / 2)
                b[j] = m[(UPPER ? triangle_at_t(j, i) : triangle_at(j, i)) * 32 + lane];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (UPPER ? i >= j / 2 : i <= j / 2)
                mma<T>(c[j], hi[i], b[j].x, b[j].y);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (UPPER ? i >= j / 2 : i <= j / 2)
                mma<T>(c[j], lo[i], b[j].x, b[j].y);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (UPPER ? i >= j / 2 : i <= j / 2)
                mma<T>(c[j], hi[i], b[j].z, b[j].w);
    }
}

// Offset of 16-byte unit u (eight keys) of row r in a tile of 64 keys of 64 rows.
__device__ __forceinline__ uint32_t unit_at(int r, int u) { return r * 128 + ((u ^ (r & 7)) << 4); }

// c (64 tokens) += S' rows', for rows of keys in shared memory.  TWO: S' is a sum of two operands.
template <typename T, int KD, bool TWO>
__device__ __forceinline__ void state_by_rows(float (&c)[8][4], const uint32_t (&x)[KD / 16][4], const uint32_t (&y)[KD / 16][4],
                                              const uint16_t (*rows)[64][64], int lane)
{
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int m = 0; m < KD / 32; ++m) {
            uint32_t b[4][4];   // four tiles of 8 tokens, two steps of 16 keys
#pragma unroll
            for (int j = 0; j < 4; ++j)
                ldsm(b[j], tc::smem_u32(rows[m / 2]) + (half * 4 + j) * 1024 + unit_at(lane & 7, 4 * (m % 2) + lane / 8));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma<T>(c[half * 4 + j], x[2 * m + e], b[j][2 * e], b[j][2 * e + 1]);
                if constexpr (TWO)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma<T>(c[half * 4 + j], y[2 * m + e], b[j][2 * e], b[j][2 * e + 1]);
            }
        }
}

// S' += left operands over the 64 tokens times rows of keys in shared memory.
template <typename T, int KD>
__device__ __forceinline__ void state_add(float (&s)[KD / 8][4], const uint32_t (&hi)[4][4], const uint32_t (&lo)[4][4],
                                          const uint16_t (*rows)[64][64], int lane)
{
#pragma unroll
    for (int p = 0; p < KD / 32; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t b[2][4];   // two pairs of tiles of 8 keys
#pragma unroll
            for (int x = 0; x < 2; ++x)
                ldsm_t(b[x], tc::smem_u32(rows[p / 2]) + unit_at(16 * i + (lane & 15), 4 * (p % 2) + 2 * x + lane / 16));
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

// Transposed values of 16 tokens from row 16 i on and a group's 16 columns: words (tile, columns + 8) as results have them.
template <int VG>
__device__ __forceinline__ void values_t(uint32_t (&v)[4], const void *rows, int i, int group, int lane)
{
    const int r = 16 * i + (lane & 7) + (lane / 16) * 8, u = 2 * group + ((lane / 8) & 1);
    ldsm_t(v, tc::smem_u32(rows) + (VG == 4 ? unit_at(r, u) : r * 64 + ((u ^ ((r >> 1) & 3)) << 4)));
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

// The state's columns `col` (and 8 on), keys 8 tile + 2 (lane % 4) (and 1 on); `at`: the first of these keys in p or from.
template <int KD>
__device__ __forceinline__ void state_io(float (&s)[KD / 8][4], float *p, const float *from, size_t at, int V, int col, bool on, bool out)
{
#pragma unroll
    for (int j = 0; j < KD / 8; ++j)
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

__device__ __forceinline__ void bars_init(uint64_t (&full)[2])
{
    if (threadIdx.x == 0) {
        tc::bar_init(&full[0], 1);
        tc::bar_init(&full[1], 1);
        tc::bar_fence_init();
    }
    __syncthreads();
}

// Tensor maps of q, k, v and dO: boxes of 64 rows of one head.
struct ChainMaps {
    CUtensorMap q, k, v, d;
};

// Asks for a chunk's cell and rows (one thread; a bulk copy for each row took 3400 cycles a chunk to issue, 16-byte copies
// by all threads 2300 and slowed the loads of the chain).
template <int KD, int VG, int ROWS, typename Cell>
__device__ __forceinline__ void ask_chunk(const DeltaArgs &a, const ChainMaps &maps, const ChainWalk &w, ChainShared<KD, VG, ROWS, Cell> &sh, int c,
                                          int turn)
{
    auto &st = sh.stage[turn & 1];
    uint64_t *bar = &sh.full[turn & 1];
    const int row = w.bos + c * kDeltaChunk;
    tc::bar_expect_tx(bar, (uint32_t)sizeof st);
#pragma unroll
    for (int i = 0; i < KD / 64; ++i) {
        tc::tma_load_3d(st.k[i], &maps.k, 64 * i, w.hk, row, bar);
        tc::tma_load_3d(st.q[i], &maps.q, 64 * i, w.hk, row, bar);
    }
    copy_bulk(&st.cell, a.chunk + ((size_t)(w.slot + c) * a.HV + w.hv) * sizeof(Cell), sizeof(Cell), bar);
    tc::tma_load_3d(st.v[0], &maps.v, w.v0, w.hv, row, bar);
    if constexpr (ROWS > 1)
        tc::tma_load_3d(st.v[1], &maps.d, w.v0, w.hv, row, bar);
}

// Rows behind a sequence's end belong to others: zeros in their place, as what they hold may be NaN.
template <int VG, typename Stage>
__device__ __forceinline__ void clear_tail(Stage &st, int rows)
{
    constexpr int kThreads = 64 * VG, kWide = sizeof st.k / 8192, kTile = 64 * 16 * VG * 2, kRows = sizeof st.v / kTile;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int i = rows * 8 + threadIdx.x; i < 512; i += kThreads)
#pragma unroll
        for (int x = 0; x < kWide; ++x) {
            reinterpret_cast<uint4 *>(st.k[x])[i] = zero;
            reinterpret_cast<uint4 *>(st.q[x])[i] = zero;
        }
    for (int i = rows * 2 * VG + threadIdx.x; i < kTile / 16; i += kThreads)
#pragma unroll
        for (int x = 0; x < kRows; ++x)
            reinterpret_cast<uint4 *>(st.v[x])[i] = zero;
}

template <typename T, typename To, int KD, int VG>
__global__ void __launch_bounds__(64 * VG, 1) delta_chain_kernel(const __grid_constant__ ChainMaps maps, DeltaArgs a, int tiles)
{
    typedef ChainShared<KD, VG, 1, DeltaCell> Shared;
    constexpr int kThreads = 64 * VG;
    extern __shared__ __align__(1024) char raw[];
    Shared &sh = *reinterpret_cast<Shared *>(raw);
    ChainWalk w;
    if (!chain_walk(a, tiles, 16 * VG, w))
        return;
    const int tid = threadIdx.x, lane = tid % 32, group = tid / 32 % VG;
    const bool output = tid >= kThreads / 2;
    const int col = w.v0 + 16 * group + lane / 4, two = 2 * (lane % 4);
    const bool on = w.v0 + 16 * group < a.V;   // whole groups of 16 columns
    const size_t state = (w.head * a.K + two) * a.V;
    bars_init(sh.full);

    auto chain = [&](typename Shared::Stage &st, float (&s)[KD / 8][4]) {
        const float4 *row = st.cell.row;
        float n[8][4] = {};
        {
            uint32_t s_hi[KD / 16][4];
#pragma unroll
            for (int i = 0; i < KD / 16; ++i) {
                uint32_t s_lo[4];
                split_pair<T>(s[2 * i], s[2 * i + 1], s_hi[i], s_lo);
                sh.state[group][i][0][lane] = as_uint4(s_hi[i]);
                sh.state[group][i][1][lane] = as_uint4(s_lo);
            }
            bar_tell(kBarState + group);
            state_by_rows<T, KD, false>(n, s_hi, s_hi, st.k, lane);
        }
        bar_sync(kBarShare + group);
        uint32_t hi[4][4], lo[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // R
            uint32_t v[4];
            values_t<VG>(v, st.v[0], i, group, lane);
            float r[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int j = 2 * i + y;
                const float4 p = sh.ks[group][j][lane];
                const float f0 = row[8 * j + two].y, f1 = row[8 * j + two + 1].y;
                const float2 v0 = widen2<T>(v[2 * y]), v1 = widen2<T>(v[2 * y + 1]);
                r[y][0] = fmaf(-f0, n[j][0] + p.x, v0.x);
                r[y][1] = fmaf(-f1, n[j][1] + p.y, v0.y);
                r[y][2] = fmaf(-f0, n[j][2] + p.z, v1.x);
                r[y][3] = fmaf(-f1, n[j][3] + p.w, v1.y);
                n[j][0] = n[j][1] = n[j][2] = n[j][3] = 0.f;
            }
            split_pair<T>(r[0], r[1], hi[i], lo[i]);
        }
        triangle<T, false>(n, hi, lo, st.cell.inverse, lane);
        const float last = row[kDeltaChunk - 1].y;
#pragma unroll
        for (int j = 0; j < KD / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[j][e] *= last;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float u[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int j = 2 * i + y;
                sh.n[group][j][lane] = as_float4(n[j]);
                const float4 c0 = row[8 * j + two], c1 = row[8 * j + two + 1];
                const float f0 = c0.z * c0.x, f1 = c1.z * c1.x;
                u[y][0] = f0 * n[j][0], u[y][1] = f1 * n[j][1], u[y][2] = f0 * n[j][2], u[y][3] = f1 * n[j][3];
            }
            split_pair<T>(u[0], u[1], hi[i], lo[i]);
        }
        bar_tell(kBarRows + group);
        state_add<T, KD>(s, hi, lo, st.k, lane);
    };
    auto put_out = [&](typename Shared::Stage &st, int c) {
        const float4 *row = st.cell.row;
        float o[8][4] = {};
        bar_sync(kBarState + group);
        {
            uint32_t s_hi[KD / 16][4], s_lo[KD / 16][4];
#pragma unroll
            for (int i = 0; i < KD / 16; ++i)
                take(s_lo[i], sh.state[group][i][1][lane]);
            state_by_rows<T, KD, false>(o, s_lo, s_lo, st.k, lane);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sh.ks[group][j][lane] = as_float4(o[j]);
                o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
            }
            bar_tell(kBarShare + group);
#pragma unroll
            for (int i = 0; i < KD / 16; ++i)
                take(s_hi[i], sh.state[group][i][0][lane]);
            state_by_rows<T, KD, true>(o, s_hi, s_lo, st.q, lane);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f0 = row[8 * j + two].w, f1 = row[8 * j + two + 1].w;
            o[j][0] *= f0, o[j][1] *= f1, o[j][2] *= f0, o[j][3] *= f1;
        }
        bar_sync(kBarRows + group);
        uint32_t hi[4][4], lo[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float n[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int j = 2 * i + y;
                const float4 p = sh.n[group][j][lane];
                const float b0 = row[8 * j + two].x, b1 = row[8 * j + two + 1].x;
                n[y][0] = b0 * p.x, n[y][1] = b1 * p.y, n[y][2] = b0 * p.z, n[y][3] = b1 * p.w;
            }
            split_pair<T>(n[0], n[1], hi[i], lo[i]);
        }
        triangle<T, false>(o, hi, lo, st.cell.score, lane);
        const int rows = min(kDeltaChunk, w.len - c * kDeltaChunk);
        To *out = static_cast<To *>(a.o) + (((size_t)w.bos + (size_t)c * kDeltaChunk) * a.HV + w.hv) * a.V + col;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 8 * j + two + (e & 1);
                if (on && t < rows)
                    out[(size_t)t * a.HV * a.V + (e >> 1) * 8] = narrow<To>(o[j][e]);
            }
    };

    // the warps of a role go their own ways through a chunk and meet at its end
    auto walk = [&](auto work) {
        if (tid == kThreads / 2 && w.chunks)
            ask_chunk(a, maps, w, sh, 0, 0);
        for (int c = 0; c < w.chunks; ++c) {
            const bool ok = tc::bar_wait(&sh.full[c & 1], (c >> 1) & 1);
            if (__syncthreads_or(!ok)) {
                if (tid == 0)
                    report(a.status, GLA_ERR_TIMEOUT);
                return;
            }
            if (tid == kThreads / 2 && c + 1 < w.chunks)
                ask_chunk(a, maps, w, sh, c + 1, c + 1);
            if (w.len - c * kDeltaChunk < kDeltaChunk) {
                clear_tail<VG>(sh.stage[c & 1], w.len - c * kDeltaChunk);
                __syncthreads();
            }
            work(sh.stage[c & 1], c);
        }
    };
    if (!output) {
        float s[KD / 8][4];
        state_io<KD>(s, nullptr, a.h0, state, a.V, col, on, false);
        walk([&](auto &st, int) { chain(st, s); });
        if (a.ht)
            state_io<KD>(s, a.ht, nullptr, state, a.V, col, on, true);
    } else {
        walk([&](auto &st, int c) { put_out(st, c); });
    }
}

PFN_cuTensorMapEncodeTiled_v12000 map_encoder()
{
    static std::atomic<void *> known{nullptr};
    void *p = known.load(std::memory_order_acquire);
    if (!p) {
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        known.store(p, std::memory_order_release);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
}

// Map of [rows, heads, D]: boxes of 64 rows of `width` values of one head (64 or 32: 128 or 64 bytes, swizzled).
bool map_rows(CUtensorMap *m, const void *p, int D, int heads, int64_t rows, int width, bool half)
{
    const auto encode = map_encoder();
    if (!encode)
        return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows}, strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * heads * 2};
    const cuuint32_t box[3] = {(cuuint32_t)width, 1, kDeltaChunk}, step[3] = {1, 1, 1};
    return encode(m, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box,
                  step, CU_TENSOR_MAP_INTERLEAVE_NONE, width == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_maps(ChainMaps &maps, const DeltaArgs &a, int width, bool half)
{
    std::memset(&maps, 0, sizeof maps);
    if (a.rows == 0)   // no chunks: nothing is read by way of them
        return true;
    return map_rows(&maps.q, a.q, a.K, a.H, a.rows, 64, half) && map_rows(&maps.k, a.k, a.K, a.H, a.rows, 64, half) &&
           map_rows(&maps.v, a.v, a.V, a.HV, a.rows, width, half) &&
           (!a.dout || map_rows(&maps.d, a.dout, a.V, a.HV, a.rows, width, half));
}

template <typename F>
cudaError_t launch_chain(F kernel, size_t shared, int groups, bool half, const DeltaArgs &a, cudaStream_t s)
{
    ChainMaps maps;
    if (!make_maps(maps, a, 16 * groups, half))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
    if (e != cudaSuccess)
        return e;
    const int tiles = (a.V + 16 * groups - 1) / (16 * groups);
    kernel<<<(unsigned)((size_t)a.N * a.HV * tiles), 64 * groups, shared, s>>>(maps, a, tiles);
    return cudaGetLastError();
}

// Whether CTAs of 32 columns have an SM each.
bool few_columns(const DeltaArgs &a) { return (size_t)a.N * a.HV * ((a.V + 31) / 32) <= (size_t)sm_count(); }

}  // namespace

cudaError_t launch_delta_chain(const DeltaArgs &a, int dtype, cudaStream_t s)
{
    return delta_types(dtype, [&](auto x, auto o) {
        typedef std::remove_pointer_t<decltype(x)> T;
        typedef std::remove_pointer_t<decltype(o)> To;
        if constexpr (std::is_same_v<T, float>) {
            return cudaErrorInvalidValue;
        } else {
            auto go = [&](auto kd, auto vg) {
                constexpr int KD = decltype(kd)::value, VG = decltype(vg)::value;
                return launch_chain(delta_chain_kernel<T, To, KD, VG>, sizeof(ChainShared<KD, VG, 1, DeltaCell>), VG, std::is_same_v<T, __half>, a, s);
            };
            auto by_keys = [&](auto vg) { return a.K == 128 ? go(Int<128>(), vg) : go(Int<64>(), vg); };
            return few_columns(a) ? by_keys(Int<2>()) : by_keys(Int<4>());
        }
    });
}

}  // namespace gla
