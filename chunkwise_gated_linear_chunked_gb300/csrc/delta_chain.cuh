// Shared by the two chains of the gated delta rule (delta_chain.cu, delta_back.cu): a CTA's shared memory, products of the
// state and of triangles, the copies of a chunk, and the launch.
#pragma once

#include <atomic>
#include <cstring>

#include <cudaTypedefs.h>

#include "api_common.h"
#include "delta_mma.cuh"

namespace gla {

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
    float power[VG][16];                 // fp16: what the columns of the rounded state were divided by
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

// c (64 tokens) += the products of 16 tokens' values (two tiles of results, v0 and v1, as left operands of TERMS terms) with
// their step i of a triangle of the cell, lower or upper.  Steps taken from 3 down (lower) or from 0 up (upper) add to no
// tile of c that a later step still has to read, so that c's own tiles can be where the values come from.  hi: the first terms.
// ALL: with the second term's product with the matrix's remainders too.
template <typename T, bool UPPER, int TERMS, bool ALL = false>
__device__ __forceinline__ void triangle_step(float (&c)[8][4], const float (&v0)[4], const float (&v1)[4], uint32_t (&hi)[4], int i,
                                              const uint4 *m, int lane)
{
    uint32_t mid[4], lo[4];
    if constexpr (TERMS == 3)
        split_pair<T>(v0, v1, hi, mid, lo);
    else
        split_pair<T>(v0, v1, hi, mid);
    uint4 b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (UPPER ? i >= j / 2 : i <= j / 2)
            b[j] = m[(UPPER ? triangle_at_t(j, i) : triangle_at(j, i)) * 32 + lane];
#pragma unroll
    for (int term = 0; term < 5; ++term)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (UPPER ? i >= j / 2 : i <= j / 2) {
                if (term < 2)
                    mma<T>(c[j], term == 0 ? hi : mid, b[j].x, b[j].y);
                else if (term == 2)
                    mma<T>(c[j], hi, b[j].z, b[j].w);
                else if (term == 3 && TERMS == 3)
                    mma<T>(c[j], lo, b[j].x, b[j].y);
                else if (term == 4 && ALL)
                    mma<T>(c[j], mid, b[j].z, b[j].w);
            }
}

// The same over all steps (fp16), times the powers of c's rows: c += c (the triangle).
template <typename T, bool UPPER, int TERMS>
__device__ __forceinline__ void triangle_rows(float (&c)[8][4], const uint4 *m, int lane)
{
    Power by[2];
    rows_power<kOperand>(c, by);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        times_rows(c[j], c[j], by[0].to, by[1].to);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int i = UPPER ? x : 3 - x;
        uint32_t hi[4];
        const float v0[4] = {c[2 * i][0], c[2 * i][1], c[2 * i][2], c[2 * i][3]};
        const float v1[4] = {c[2 * i + 1][0], c[2 * i + 1][1], c[2 * i + 1][2], c[2 * i + 1][3]};
        triangle_step<T, UPPER, TERMS>(c, v0, v1, hi, i, m, lane);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        times_rows(c[j], c[j], by[0].from, by[1].from);
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

// The same with one term more.
template <typename T, int KD>
__device__ __forceinline__ void state_add(float (&s)[KD / 8][4], const uint32_t (&x)[4][4], const uint16_t (*rows)[64][64], int lane)
{
#pragma unroll
    for (int p = 0; p < KD / 16; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t b[4];
            ldsm_t(b, tc::smem_u32(rows[p / 4]) + unit_at(16 * i + (lane & 15), 2 * (p % 4) + lane / 16));
            mma<T>(s[2 * p], x[i], b[0], b[1]);
            mma<T>(s[2 * p + 1], x[i], b[2], b[3]);
        }
}

// Transposed values of 16 tokens from row 16 i on and a group's 16 columns: words (tile, columns + 8) as results have them.
template <int VG>
__device__ __forceinline__ void values_t(uint32_t (&v)[4], const void *rows, int i, int group, int lane)
{
    const int r = 16 * i + (lane & 7) + (lane / 16) * 8, u = 2 * group + ((lane / 8) & 1);
    ldsm_t(v, tc::smem_u32(rows) + (VG == 4 ? unit_at(r, u) : r * 64 + ((u ^ ((r >> 1) & 3)) << 4)));
}

// 16 rows of rounded values (left operands, STEPS of 16 columns) as blocks of 8 x 8 in rows of 16 bytes: 128 bytes that
// a warp stores at once and that ldmatrix takes as they are.  Blocks of a row of blocks are adjacent, `across` of them.
template <int STEPS>
__device__ __forceinline__ void put_blocks(uint32_t *to, const uint32_t (&r)[STEPS][4], int block_row, int across, int lane)
{
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)   // rows + 8 (e & 1), columns + 8 (e >> 1)
            to[((block_row + (e & 1)) * across + 2 * i + (e >> 1)) * 32 + lane] = r[i][e];
}

// The largest over a group's 16 columns of values of which each lane has those of its two rows.
__device__ __forceinline__ float group_largest(const float (&p)[2])
{
    float most = fmaxf(p[0], p[1]);
#pragma unroll
    for (int m = 4; m < 32; m *= 2)
        most = fmaxf(most, __shfl_xor_sync(~0u, most, m));
    return most;
}
// Rounded values (left operands) of columns over their own powers p, over one of the group's that is no smaller; in place.
template <int STEPS>
__device__ __forceinline__ void to_group(uint32_t (&r)[STEPS][4], const float (&p)[2], float group)
{
    const float f0 = p[0] * inverse_power(group), f1 = p[1] * inverse_power(group);
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            r[i][e] = times_power(r[i][e], e & 1 ? f1 : f0);
}

// Sums over the eight lanes that share lane % 4 of N values each: lane is left with those from N / 8 (lane / 4) on.
template <int N>
__device__ __forceinline__ void sum_over_columns(float (&v)[N], int lane)
{
#pragma unroll
    for (int bit = 2; bit >= 0; --bit) {
        const int half = N >> (3 - bit);   // values that stay
        const bool up = (lane >> (2 + bit)) & 1;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float keep = up ? v[half + i] : v[i], send = up ? v[i] : v[half + i];
            v[i] = keep + __shfl_xor_sync(~0u, send, 4 << bit);
        }
    }
}

// Whether a value is not finite.  With fp16 operands (GLA_F16) such a result is reported: a value on the way may have left
// their range, where bf16 has fp32's.
__device__ __forceinline__ bool lost(float v) { return !(fabsf(v) <= 3.402823466e38f); }
template <typename T, int N>
__device__ __forceinline__ void report_lost(const DeltaArgs &a, const float (&s)[N][4], bool already)
{
    if constexpr (std::is_same_v<T, __half>) {
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                already |= lost(s[j][e]);
        if (already)
            report(a.status, GLA_ERR_RANGE);
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

// Where a wait for copies ran out, before the CTA ends: the copies under way get as long again, since a CTA's shared memory goes
// to the next one.  All threads call it; nothing but what this barrier counts is under way.  (Inlined, it costs the forward
// chain 3 % by the order of the instructions around it.)
__device__ __noinline__ static void give_up(int *status, uint64_t *bar, uint32_t parity)
{
    if (threadIdx.x == 0) {
        report(status, GLA_ERR_TIMEOUT);
        tc::bar_wait(bar, parity);
    }
    __syncthreads();
}

// Tensor maps of q, k, v and dO: boxes of 64 rows of one head.
struct ChainMaps {
    CUtensorMap q, k, v, d;
};

// Asks for a chunk's rows, and for its cell from `from` bytes on (one thread; a bulk copy for each row took 3400 cycles a
// chunk to issue, 16-byte copies by all threads 2300 and slowed the loads of the chain).
template <int KD, int VG, int ROWS, typename Cell>
__device__ __forceinline__ void ask_chunk(const DeltaArgs &a, const ChainMaps &maps, const ChainWalk &w, ChainShared<KD, VG, ROWS, Cell> &sh, int c,
                                          int turn, size_t cell_bytes, size_t from)
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
    copy_bulk(&st.cell, a.chunk + ((size_t)(w.slot + c) * a.HV + w.hv) * cell_bytes + from, sizeof st.cell, bar);
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
    tc::fence_proxy_async();   // before a later copy to the same place
}

inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder()
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
inline bool map_rows(CUtensorMap *m, const void *p, int D, int heads, int64_t rows, int width, bool half)
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

inline bool make_maps(ChainMaps &maps, const DeltaArgs &a, int width, bool half)
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
    return launch_early_shared(kernel, (unsigned)((size_t)a.N * a.HV * tiles), 64 * groups, shared, s, maps, a, tiles);
}

// Whether CTAs of 32 columns have an SM each.
inline bool few_columns(const DeltaArgs &a) { return (size_t)a.N * a.HV * ((a.V + 31) / 32) <= (size_t)sm_count(); }

}  // namespace gla
