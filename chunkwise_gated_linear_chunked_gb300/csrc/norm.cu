// Residual addition and root-mean-square norm: forward (fp32 / 16-bit or e4m3 output) and backward.
//
// Up to 8192 columns (shifted rows: 8185 in 16 bits, 8189 in fp32) a row lives in registers, 16 values a thread: it is
// read once, reduced, and written.  A warp holds 512 adjacent columns, up to 16 warps a row; rows of at most 256 columns
// share a warp.  A CTA keeps its share of the weights in registers, walks rows a grid apart, and asks for its next row
// before it reduces the present one.  Wider rows are read again from cache instead, value by value by one CTA a row.
//
// Memory is read and written in whole 16-byte units whatever D is.  A row starts k values into such a unit; a thread's
// vectors lie on units, so vector v holds columns VEC v - k and up, and the two vectors that hang over the row's ends
// go value by value.  Rows a multiple of VEC apart have the same k, so a thread keeps its columns (and its weights).
//
// Bound by HBM: 65536 rows of 4096 columns in 16 bits with a residual 335 us (6.4 TB/s), e4m3 in groups of 128 with an
// fp32 residual, 16384 x 2048, 57 us (6.5), the backward of 32768 x 2048 84 us (6.4), 65536 rows of 1001 columns 85 us
// (6.2), their backward 101 us (5.2).  Groups of 128 of shifted rows are bound by instructions: 146 us at 65536 x 1001,
// where 65536 x 1000 takes 72 us.  The wide rows' kernels are bound by instructions and latency: 4096 rows of 16384 columns
// in 16 bits, forward 207 us, e4m3 228, in groups of 128 (one after the other) 622, backward (its sums of dw in global
// memory) 622, where a copy takes 69 to 79.  The forward takes three CTAs of 256 threads an SM; four, at 64 registers, ran slower
// (86 -> 93 us at 65536 x 1024).
#include <algorithm>
#include <atomic>

#include "api_common.h"
#include "layer_internal.h"
#include "tc_ptx.cuh"

namespace gla {
namespace {

constexpr int kThreads = 256;        // threads of a CTA (more where a row needs them)
constexpr int kHeld = 16;            // values of a row in a thread
constexpr int kMaxHeld = 8192;       // columns of a row that 16 warps hold, with what hangs over where rows are shifted
constexpr float kE4m3Max = 448.f, kScaleMin = 1e-30f;

// Maximum that keeps a NaN of either side.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// 1 / v to a unit in the last place.
__device__ __forceinline__ float reciprocal(float v)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// The scale of values of which the largest is `most`.
__device__ __forceinline__ float scale_of(float most) { return max_nan(most * (1.f / kE4m3Max), kScaleMin); }

// Threads of a row and rows of a CTA.
struct Split {
    int lanes, rows, threads;
};
int held_columns(int D, int vec) { return D % vec ? D + vec - 1 : D; }   // with what hangs over
Split split_of(int D, int vec)
{
    const int held = held_columns(D, vec);
    Split s;
    if (held <= 256) {
        s.lanes = 1;
        while (s.lanes * kHeld < held)
            s.lanes *= 2;
    } else {
        s.lanes = (held + 32 * kHeld - 1) / (32 * kHeld) * 32;
    }
    s.rows = s.lanes < kThreads ? kThreads / s.lanes : 1;
    s.threads = s.rows * s.lanes;
    return s;
}

// BYTES of global memory to shared memory, or zeros.  CACHED: by way of L1, for a thread whose next copy is the other
// half of a sector (fp32 beside 16-bit values: 65536 x 1000 from 225 to 171 us).
template <int BYTES, bool CACHED = false>
__device__ __forceinline__ void copy_async(void *dst, const void *src, bool ok)
{
    if constexpr (CACHED)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0)
                     : "memory");
    else if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(ok ? 4 : 0)
                     : "memory");
}

// A row's place: its first value's number in the tensor, its columns, and the tensor's values.
struct Place {
    int64_t at;
    int D;
    int64_t end;
};

template <int VEC, bool SHIFTED>
__device__ __forceinline__ bool over(int c, int D) { return SHIFTED && (c < 0 || c + VEC > D); }   // the vector at c

// Stores the values of a vector of eight (E; two of them a P, four a Q) at column c that lie in [0, D), in at most three
// pieces: those past its first k are a piece of one where k is odd, then one of two, then the last four.
template <typename E, typename P, typename Q>
__device__ __forceinline__ void put_end(E *p, Q lo, Q hi, int c, int D)
{
    auto from = [&](int i) { return (i < 4 ? lo : hi) >> (8 * sizeof(E) * (i & 3)); };
    if (c < 0 && c + 8 > D) {
        for (int i = -c; i < D - c; ++i)
            p[i] = (E)from(i);
    } else if (c < 0) {
        int k = -c;
        if (k & 1) {
            p[k] = (E)from(k);
            ++k;
        }
        if (k & 2) {
            *reinterpret_cast<P *>(p + k) = (P)from(k);
            k += 2;
        }
        if (k == 4)
            *reinterpret_cast<Q *>(p + 4) = hi;
    } else if (c < D) {
        const int e = D - c;
        if (e & 4)
            *reinterpret_cast<Q *>(p) = lo;
        if (e & 2)
            *reinterpret_cast<P *>(p + (e & 4)) = (P)from(e & 4);
        if (e & 1)
            p[e - 1] = (E)from(e - 1);
    }
}

// A thread's part of a row as it lies in memory: N vectors of VEC values.  SHIFTED: some vectors hang over the row's
// ends.  Of 32-bit values they are loaded one by one.  Of 16-bit values, two a register, that would make every load wait
// to be put together; they are loaded like the others (their other values are the neighbouring rows') and masked when
// they are used, and what would reach over the tensor's end is loaded only then.  Masks kept in registers and ends
// stored in pieces of one, two and four took 65536 x 1001 from 93 to 85 us, its backward from 138 to 101, against a
// test for each value.
template <typename T, int VEC, bool SHIFTED>
struct Part {
    static constexpr int N = kHeld / VEC;
    static constexpr bool kOneByOne = SHIFTED && sizeof(T) == 4;
    alignas(16) T v[kHeld];
    __device__ __forceinline__ void load(const T *p, const Place &at, const int (&col)[N])
    {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (kOneByOne && over<VEC, SHIFTED>(col[j], at.D)) {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    v[j * VEC + i] = (unsigned)(col[j] + i) < (unsigned)at.D ? p[at.at + col[j] + i] : T(0.f);
                continue;
            }
            const bool ok = col[j] < at.D && (!SHIFTED || kOneByOne || at.at + col[j] + VEC <= at.end);
#pragma unroll
            for (int i = 0; i < VEC * (int)sizeof(T) / 16; ++i)
                reinterpret_cast<uint4 *>(v + j * VEC)[i] =
                    ok ? reinterpret_cast<const uint4 *>(p + at.at + col[j])[i] : make_uint4(0, 0, 0, 0);
        }
    }
    // Zeros for what is not the row's (`keep`: see keep_own), and the values that `load` left out at the tensor's end.
    __device__ __forceinline__ void mend(const T *p, const Place &at, const int (&col)[N], const uint32_t (&keep)[kHeld / 2])
    {
        if constexpr (!kOneByOne) {
#pragma unroll
            for (int i = 0; i < kHeld / 2; ++i)
                reinterpret_cast<uint32_t *>(v)[i] &= keep[i];
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (col[j] < at.D && at.at + col[j] + VEC > at.end)
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if ((unsigned)(col[j] + i) < (unsigned)at.D)
                            v[j * VEC + i] = p[at.at + col[j] + i];
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kHeld * (int)sizeof(T) / 16; ++i)
            reinterpret_cast<uint4 *>(v)[i] = make_uint4(0, 0, 0, 0);
    }
    // The same by way of shared memory, into units of the thread's own, `step` apart: ask starts the copies (and zeros
    // what lies outside), take reads them once they have arrived.
    static constexpr int kUnits = kHeld * (int)sizeof(T) / 16;
    static __device__ __forceinline__ void ask(uint4 *slot, int step, const T *p, const Place &at, const int (&col)[N])
    {
        constexpr int kEach = VEC * (int)sizeof(T) / 16;   // units of a vector
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (kOneByOne && over<VEC, SHIFTED>(col[j], at.D)) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const bool ok = (unsigned)(col[j] + i) < (unsigned)at.D;
                    copy_async<4>(reinterpret_cast<T *>(slot + (j * kEach + i / 4) * step) + i % 4, ok ? p + at.at + col[j] + i : p,
                                  ok);
                }
                continue;
            }
            const bool ok = col[j] < at.D && (!SHIFTED || kOneByOne || at.at + col[j] + VEC <= at.end);
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                copy_async<16, (kEach > 1)>(slot + (j * kEach + i) * step, ok ? p + at.at + col[j] + i * (16 / (int)sizeof(T)) : p, ok);
        }
    }
    __device__ __forceinline__ void take(const uint4 *slot, int step)
    {
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
            reinterpret_cast<uint4 *>(v)[i] = slot[i * step];
    }
    __device__ __forceinline__ float2 pair(int i) const   // values 2 i and 2 i + 1
    {
        if constexpr (sizeof(T) == 4)
            return make_float2(v[2 * i], v[2 * i + 1]);
        else
            return widen2<T>(reinterpret_cast<const uint32_t *>(v)[i]);
    }
    __device__ __forceinline__ void set(int i, float2 f)
    {
        if constexpr (sizeof(T) == 4) {
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        } else {
            reinterpret_cast<uint32_t *>(v)[i] = narrow2<T>(f);
        }
    }
    __device__ __forceinline__ void store(T *p, const Place &at, const int (&col)[N]) const
    {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (over<VEC, SHIFTED>(col[j], at.D)) {
                if constexpr (sizeof(T) == 2 && VEC == 8) {
                    const uint64_t *half = reinterpret_cast<const uint64_t *>(v + j * VEC);
                    put_end<uint16_t, uint32_t>(reinterpret_cast<uint16_t *>(p + at.at + col[j]), half[0], half[1], col[j], at.D);
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if ((unsigned)(col[j] + i) < (unsigned)at.D)
                            p[at.at + col[j] + i] = v[j * VEC + i];
                }
            } else if (col[j] < at.D) {
#pragma unroll
                for (int i = 0; i < VEC * (int)sizeof(T) / 16; ++i)
                    reinterpret_cast<uint4 *>(p + at.at + col[j])[i] = reinterpret_cast<const uint4 *>(v + j * VEC)[i];
            }
        }
    }
};

// The first column of each vector of a row's lane l, for rows that start k values into a 16-byte unit.
template <int VEC>
__device__ __forceinline__ void columns(int (&col)[kHeld / VEC], int l, int lanes, int k)
{
    constexpr int N = kHeld / VEC;
#pragma unroll
    for (int j = 0; j < N; ++j)
        col[j] = (lanes < 32 ? j * lanes + l : (l / 32 * N + j) * 32 + l % 32) * VEC - k;
}

// Masks of a thread's 16-bit values, two a word, that are its row's own.
template <int VEC>
__device__ __forceinline__ void keep_own(uint32_t (&keep)[kHeld / 2], const int (&col)[kHeld / VEC], int D)
{
    auto own = [&](int i) { return (unsigned)(col[i / VEC] + i % VEC) < (unsigned)D; };
#pragma unroll
    for (int i = 0; i < kHeld / 2; ++i)
        keep[i] = (own(2 * i) ? 0xffffu : 0u) | (own(2 * i + 1) ? 0xffff0000u : 0u);
}

template <int VEC>
__device__ __forceinline__ void load_weights(float2 (&w)[kHeld / 2], const float *p, const int (&col)[kHeld / VEC], int D)
{
    auto one = [&](int i) {
        const int c = col[i / VEC] + i % VEC;
        return (unsigned)c >= (unsigned)D ? 0.f : p ? p[c] : 1.f;
    };
#pragma unroll
    for (int i = 0; i < kHeld / 2; ++i)
        w[i] = make_float2(one(2 * i), one(2 * i + 1));
}

// Over a warp, in one instruction: 92 -> 87 us for e4m3 rows of 65536 x 1001 against five exchanges.
__device__ __forceinline__ float max_warp(float m)
{
    asm volatile("redux.sync.max.NaN.f32 %0, %0, -1;" : "+f"(m));
    return m;
}

__device__ __forceinline__ float max_lanes(float m, int lanes)   // over groups of so many adjacent lanes
{
    for (int d = lanes / 2; d; d >>= 1)
        m = max_nan(m, __shfl_xor_sync(~0u, m, d));
    return m;
}

// What a warp tells the other warps of its row: its sum and maximum, and of the groups of 128 columns that it shares
// with them the maxima of its first (`head`: the columns before its first whole group) and of its last.
struct Told {
    float sum, most, head, last;
};

// Sum (and maximum) over the lanes of a row.  `told` has a slot per warp; a CTA's rows come here together, and two
// calls in a row use different slots.
template <bool MAX>
__device__ __forceinline__ void reduce_row(Told &t, int lanes, Told *told)
{
    for (int m = min(lanes, 32) / 2; m; m >>= 1)
        t.sum += __shfl_xor_sync(~0u, t.sum, m);
    if (MAX)
        t.most = lanes >= 32 ? max_warp(t.most) : max_lanes(t.most, min(lanes, 32));
    if (lanes <= 32)
        return;
    const int warp = threadIdx.x / 32, count = lanes / 32, first = warp / count * count;
    if (threadIdx.x % 32 == 0)
        told[warp] = t;
    __syncthreads();
    t.sum = told[first].sum;
    t.most = told[first].most;
    for (int i = 1; i < count; ++i) {
        t.sum += told[first + i].sum;
        if (MAX)
            t.most = max_nan(t.most, told[first + i].most);
    }
}

// Maxima of |v| over groups of 128 columns.  Where rows share a warp a row has at most two groups, and a value counts by
// its column.  Where a row has whole warps, group g is vectors G g .. G g + G - 1 (G = 128 / VEC lanes) but
// for the k values that the first of them has before the group's first column, plus the k such values of vector
// G (g + 1): those of a neighbouring vector, or of the next warp's first, which reduce_row carries.
template <int VEC>
struct Groups {
    static constexpr int N = kHeld / VEC, G = 128 / VEC;
    static constexpr int kFew = 2;     // most groups of a row that shares a warp
    float m[N];                        // by group, or by vector: of the group that holds vector j's own columns
    float before[N];                   // of the k values of vector j that belong to the group before

    __device__ __forceinline__ void find(const float2 (&v)[kHeld / 2], const int (&col)[N], int lanes, int k, Told &t)
    {
        auto size = [&](int i) { return fabsf(i % 2 ? v[i / 2].y : v[i / 2].x); };
        const int lane = threadIdx.x % 32;
        if (lanes < 32) {
#pragma unroll
            for (int g = 0; g < kFew; ++g) {
                m[g] = 0.f;
#pragma unroll
                for (int i = 0; i < kHeld; ++i)
                    m[g] = (col[i / VEC] + i % VEC) >> 7 == g ? max_nan(m[g], size(i)) : m[g];
                m[g] = max_lanes(m[g], lanes);
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            m[j] = before[j] = 0.f;
            const bool first = lane % G == 0;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if (first && i < k)
                    before[j] = max_nan(before[j], size(j * VEC + i));
                else
                    m[j] = max_nan(m[j], size(j * VEC + i));
            }
            m[j] = G == 32 ? max_warp(m[j]) : max_lanes(m[j], G);
        }
        t.head = before[0];                                   // lane 0's is what counts
        t.last = __shfl_sync(~0u, m[N - 1], 31);
        if (k) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float up = __shfl_sync(~0u, before[j], G % 32);            // of this block's second group
                const float next = j + 1 < N ? __shfl_sync(~0u, before[j + 1 < N ? j + 1 : j], 0) : 0.f;
                m[j] = max_nan(m[j], G < 32 && lane < G ? up : next);
            }
        }
    }

    // After the reduction: scales from the maxima, written by one lane a group; `m` and `before` become the scales'
    // reciprocals, of the vectors' own columns and of the k before.
    __device__ __forceinline__ void scale(float *out, int groups, float rstd, int l, int lanes, int k, const Told *told)
    {
        auto of = [&](float most) { return scale_of(most * rstd); };
        if (lanes < 32) {
#pragma unroll
            for (int g = 0; g < kFew; ++g) {
                m[g] = of(m[g]);
                if (l == 0 && g < groups)
                    out[g] = m[g];
                m[g] = reciprocal(m[g]);
            }
            return;
        }
        const int lane = l % 32, warp = threadIdx.x / 32, in_row = l / 32;
        float prior = 0.f;   // the group that the warp's first k columns belong to
        if (k && lanes > 32) {
            if (in_row + 1 < lanes / 32 && lane >= 32 - G)   // the last group goes on in the next warp
                m[N - 1] = max_nan(m[N - 1], told[warp + 1].head);
            if (in_row > 0)
                prior = max_nan(told[warp - 1].last, told[warp].head);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            m[j] = of(m[j]);
            const int g = (in_row * N + j) * (32 / G) + lane / G;
            if (lane % G == 0 && g < groups)
                out[g] = m[j];
            m[j] = reciprocal(m[j]);
        }
        if (k) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float down = __shfl_sync(~0u, m[j], 0);   // first group of this block
                const float back = j ? __shfl_sync(~0u, m[j ? j - 1 : 0], 31) : reciprocal(of(prior));   // last before it
                before[j] = lane >= G ? down : back;
            }
        }
    }
    __device__ __forceinline__ float inverse(int i, const int (&col)[N], int lanes, int k) const   // for value i
    {
        if (lanes < 32)
            return col[i / VEC] + i % VEC < 128 ? m[0] : m[1];
        return i % VEC < k && threadIdx.x % G == 0 ? before[i / VEC] : m[i / VEC];
    }
};

// A vector of e4m3 values.
template <int VEC, bool SHIFTED>
__device__ __forceinline__ void put_e4m3(uint8_t *p, const Place &at, int c, const float2 *v)
{
    alignas(8) __nv_fp8x2_storage_t b[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i)
        b[i] = __nv_cvt_float2_to_fp8x2(v[i], __NV_SATFINITE, __NV_E4M3);
    if (over<VEC, SHIFTED>(c, at.D)) {
        if constexpr (VEC == 8) {
            const uint32_t *half = reinterpret_cast<const uint32_t *>(b);
            put_end<uint8_t, uint16_t>(p + at.at + c, half[0], half[1], c, at.D);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if ((unsigned)(c + i) < (unsigned)at.D)
                    p[at.at + c + i] = reinterpret_cast<const uint8_t *>(b)[i];
        }
    } else if (c < at.D) {
        if constexpr (VEC == 8)
            *reinterpret_cast<uint2 *>(p + at.at + c) = *reinterpret_cast<const uint2 *>(b);
        else
            *reinterpret_cast<uint32_t *>(p + at.at + c) = *reinterpret_cast<const uint32_t *>(b);
    }
}

enum Quant { kPlain, kByRow, kByGroup };

// Registers: as many as hold the row and the next one (12 bytes spill of e4m3 rows by row, shifted, of 16 bits with an fp32
// residual).  Groups of unshifted 16-bit rows go faster with
// three CTAs of 256 threads, at 80, than with two, at 96 (81 -> 72 us at 65536 x 1000, though 78 -> 81 at 29127 x 2304);
// those of shifted rows do not (146 -> 152 us at 65536 x 1001).
template <typename Tx, typename Tr, Quant Q, bool SHIFTED>
__global__ void __maxnreg__(sizeof(Tr) == 2 ? (Q == kByGroup && SHIFTED ? 96 : 80) : Q == kByRow ? 128 : 112)
norm_fwd_rows(NormArgs a, Split sp)
{
    constexpr int VEC = 16 / sizeof(Tx), N = kHeld / VEC;
    __shared__ Told told[2][16];
    tc::grid_dep_wait();
    const int l = threadIdx.x % sp.lanes;
    const Tx *x_in = static_cast<const Tx *>(a.x);
    const Tr *res_in = static_cast<const Tr *>(a.res);
    const int64_t stride = (int64_t)gridDim.x * sp.rows;
    int64_t row = (int64_t)blockIdx.x * sp.rows + threadIdx.x / sp.lanes;
    const int k = SHIFTED ? (int)(row * a.D % VEC) : 0;
    Place at = {row * a.D, a.D, a.rows * a.D};
    int col[N];
    columns<VEC>(col, l, sp.lanes, k);
    uint32_t keep[kHeld / 2];
    keep_own<VEC>(keep, col, a.D);
    Part<Tx, VEC, SHIFTED> x;
    Part<Tr, VEC, SHIFTED> res;
    res.zero();
    auto fetch = [&](int64_t r) {
        if (r < a.rows) {
            const Place to = {r * a.D, a.D, at.end};
            x.load(x_in, to, col);
            if (res_in)
                res.load(res_in, to, col);
        } else {
            x.zero();
        }
    };
    fetch(row);
    float2 w[kHeld / 2];
    load_weights<VEC>(w, a.w, col, a.D);
    const float part = 1.f / a.D;
    // every thread of the CTA takes the same number of turns (they meet in the reduction)
    for (int64_t first = (int64_t)blockIdx.x * sp.rows, turn = 0; first < a.rows; first += stride, ++turn) {
        const bool on = row < a.rows;
        at.at = row * a.D;
        if (SHIFTED && on) {
            x.mend(x_in, at, col, keep);
            if (res_in)
                res.mend(res_in, at, col, keep);
        }
        float2 v[kHeld / 2], sq = make_float2(0.f, 0.f);
        Told t = {};
#pragma unroll
        for (int i = 0; i < kHeld / 2; ++i) {
            v[i] = add2(x.pair(i), res.pair(i));
            sq = fma2(v[i], v[i], sq);
        }
        t.sum = sq.x + sq.y;
        if (on && a.s) {
            Part<Tr, VEC, SHIFTED> s;
#pragma unroll
            for (int i = 0; i < kHeld / 2; ++i)
                s.set(i, v[i]);
            s.store(static_cast<Tr *>(a.s), at, col);
        }
        row += stride;
        fetch(row);
#pragma unroll
        for (int i = 0; i < kHeld / 2; ++i) {
            v[i] = mul2(v[i], w[i]);
            if (Q == kByRow)
                t.most = max_nan(t.most, max_nan(fabsf(v[i].x), fabsf(v[i].y)));
        }
        Groups<VEC> groups;
        if (Q == kByGroup)
            groups.find(v, col, sp.lanes, k, t);
        reduce_row<Q == kByRow>(t, sp.lanes, told[turn & 1]);
        const float rstd = rsqrtf(t.sum * part + a.eps);
        if (on && a.rstd && l == 0)
            a.rstd[row - stride] = rstd;
#pragma unroll
        for (int i = 0; i < kHeld / 2; ++i)
            v[i] = mul2(v[i], make_float2(rstd, rstd));
        if constexpr (Q == kPlain) {
            Part<Tx, VEC, SHIFTED> y;
#pragma unroll
            for (int i = 0; i < kHeld / 2; ++i)
                y.set(i, v[i]);
            if (on)
                y.store(static_cast<Tx *>(a.y), at, col);
        } else {
            if constexpr (Q == kByRow) {
                const float scale = scale_of(t.most * rstd), inv = reciprocal(scale);
                if (on && l == 0)
                    a.scales[row - stride] = scale;
#pragma unroll
                for (int i = 0; i < kHeld / 2; ++i)
                    v[i] = mul2(v[i], make_float2(inv, inv));
            } else {
                const int count = (a.D + 127) / 128;
                groups.scale(a.scales + (on ? (row - stride) * count : 0), on ? count : 0, rstd, l, sp.lanes, k, told[turn & 1]);
#pragma unroll
                for (int i = 0; i < kHeld / 2; ++i)
                    v[i] = mul2(v[i], make_float2(groups.inverse(2 * i, col, sp.lanes, k),
                                                  groups.inverse(2 * i + 1, col, sp.lanes, k)));
            }
            if (on)
#pragma unroll
                for (int j = 0; j < N; ++j)
                    put_e4m3<VEC, SHIFTED>(static_cast<uint8_t *>(a.y), at, col[j], v + j * VEC / 2);
        }
    }
}

// How many rows a thread asks for before their turn by way of shared memory, and the units of 16 bytes that it holds of
// each.
template <typename Tr>
constexpr int kAhead = sizeof(Tr) == 2 ? 2 : 1;
template <typename Tx, typename Tr>
constexpr int kRowUnits = kHeld * (2 * (int)sizeof(Tr) + (int)sizeof(Tx)) / 16;

// Whether rows go by way of shared memory: where a CTA has several turns of rows so wide that few are under way, and, of
// 16-bit rows of more than 256 threads (one CTA an SM), only those in whole 32-byte sectors.  In us by registers and by
// shared memory, 67 million values: 16 bits 2048 columns 87 and 82, 4096: 89 and 85, 5120: 110 and 99, 8000: 96 and 88, but
// 4500: 139 and 145, 7000: 100 and 106, 8184: 95 and 103; fp32 2048: 159 and 153, 4500: 213 and 177, 8184: 173 and 165; 16
// bits with an fp32 residual 3000: 188 and 188, 3600: 181 and 166, 4500: 283 and 210, 8184: 206 and 169 (4096 alone goes the
// other way, 171 and 184).  65536 x 1000 in 16 bits 89 and 92; one row of 2880: 4.0 and 4.6.
template <typename Tx, typename Tr>
bool by_shared(const NormArgs &a, const Split &sp)
{
    const bool sectors = sizeof(Tr) == 4 || sp.lanes <= 256 || a.D % 16 == 0;
    return sectors && sp.lanes >= (sizeof(Tx) == sizeof(Tr) ? 128 : 256) && a.rows > (int64_t)a.ctas * sp.rows;
}

// 128 registers a thread for up to 512 threads (24 bytes spill of fp16 rows by registers).
template <typename Tx, typename Tr, bool SHIFTED, bool SHARED>
__global__ void __launch_bounds__(512) norm_bwd_rows(NormArgs a, Split sp)
{
    constexpr int VEC = 16 / sizeof(Tx), N = kHeld / VEC;
    // rows asked for before their turn; by registers one, where there are registers for it beside the present one
    constexpr int AHEAD = SHARED ? kAhead<Tr> : sizeof(Tr) == 2 ? 1 : 0;
    typedef Part<Tr, VEC, SHIFTED> PR;
    typedef Part<Tx, VEC, SHIFTED> PX;
    __shared__ Told told[2][16];
    extern __shared__ uint4 staged[];   // SHARED: by row asked for, unit and thread; after the rows the sums of dw
    tc::grid_dep_wait();
    const int l = threadIdx.x % sp.lanes, D = a.D, threads = sp.threads;
    const Tr *s_in = static_cast<const Tr *>(a.s_in), *ds_in = static_cast<const Tr *>(a.ds);
    const Tx *dy_in = static_cast<const Tx *>(a.dy);
    // a CTA's rows: adjacent ones, or (SHIFTED) a grid apart, a multiple of 8, so that all of them have the same shift
    // and a column's sum is one lane's for each
    const int64_t stride = (int64_t)gridDim.x * sp.rows, base = SHIFTED ? blockIdx.x : (int64_t)blockIdx.x * sp.rows;
    int64_t row = base + threadIdx.x / sp.lanes * (SHIFTED ? (int64_t)gridDim.x : 1);
    Place at = {row * D, D, a.rows * D};
    int col[N];
    columns<VEC>(col, l, sp.lanes, SHIFTED ? (int)(row * D % VEC) : 0);
    uint32_t keep[kHeld / 2];
    keep_own<VEC>(keep, col, D);
    PR s, ds;
    PX dy;
    float rstd = 0.f;
    ds.zero();
    auto slot = [&](int turn, int unit) {
        return staged + (turn % (AHEAD ? AHEAD : 1) * kRowUnits<Tx, Tr> + unit) * threads + threadIdx.x;
    };
    auto rstd_of = [&](int turn) {
        return reinterpret_cast<float *>(staged + AHEAD * kRowUnits<Tx, Tr> * threads) + turn % (AHEAD ? AHEAD : 1) * threads +
               threadIdx.x;
    };
    auto fetch = [&](int64_t r, int turn) {
        const Place to = {r * D, D, at.end};
        if constexpr (SHARED) {
            if (r < a.rows) {
                PR::ask(slot(turn, 0), threads, s_in, to, col);
                PX::ask(slot(turn, PR::kUnits), threads, dy_in, to, col);
                if (ds_in)
                    PR::ask(slot(turn, PR::kUnits + PX::kUnits), threads, ds_in, to, col);
                copy_async<4>(rstd_of(turn), a.rstd_in + r, true);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else if (r < a.rows) {
            s.load(s_in, to, col);
            dy.load(dy_in, to, col);
            if (ds_in)
                ds.load(ds_in, to, col);
            rstd = a.rstd_in[r];
        } else {
            s.zero();
            dy.zero();
        }
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        fetch(row + i * stride, i);
    float2 w[kHeld / 2], dw[kHeld / 2];
    load_weights<VEC>(w, a.w, col, D);
#pragma unroll
    for (int i = 0; i < kHeld / 2; ++i)
        dw[i] = make_float2(0.f, 0.f);
    const float part = 1.f / D;
    int turn = 0;
    for (int64_t first = base; first < a.rows; first += stride, row += stride, ++turn) {
        if (AHEAD == 0)
            fetch(row, turn);
        const bool on = row < a.rows;
        at.at = row * D;
        if constexpr (SHARED) {   // the thread's own copies: nobody else waits for them
            asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
            s.zero();
            dy.zero();
            ds.zero();
            if (on) {
                s.take(slot(turn, 0), threads);
                dy.take(slot(turn, PR::kUnits), threads);
                if (ds_in)
                    ds.take(slot(turn, PR::kUnits + PX::kUnits), threads);
                rstd = *rstd_of(turn);
            }
        }
        if (SHIFTED && on) {
            s.mend(s_in, at, col, keep);
            dy.mend(dy_in, at, col, keep);
            if (ds_in)
                ds.mend(ds_in, at, col, keep);
        }
        const float r = rstd;
        float2 n[kHeld / 2], g[kHeld / 2], up[kHeld / 2], c = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kHeld / 2; ++i) {
            n[i] = mul2(s.pair(i), make_float2(r, r));
            g[i] = dy.pair(i);
            up[i] = ds.pair(i);
            dw[i] = fma2(g[i], n[i], dw[i]);
            g[i] = mul2(g[i], w[i]);
            c = fma2(g[i], n[i], c);
        }
        if (AHEAD > 0)
            fetch(row + AHEAD * stride, turn);
        Told t = {};
        t.sum = c.x + c.y;
        reduce_row<false>(t, sp.lanes, told[turn & 1]);
        const float mean = -t.sum * part;
#pragma unroll
        for (int i = 0; i < kHeld / 2; ++i)
            up[i] = fma2(make_float2(r, r), fma2(n[i], make_float2(mean, mean), g[i]), up[i]);
        if (on && a.dx) {
            PX out;
#pragma unroll
            for (int i = 0; i < kHeld / 2; ++i)
                out.set(i, up[i]);
            out.store(static_cast<Tx *>(a.dx), at, col);
        }
        if (on && a.dres) {
            PR out;
#pragma unroll
            for (int i = 0; i < kHeld / 2; ++i)
                out.set(i, up[i]);
            out.store(static_cast<Tr *>(a.dres), at, col);
        }
    }
    if (!a.dw)
        return;
    // the CTA's sum of dw: over the rows of a warp, then over the warps (or the rows of whole warps) in order
    for (int m = sp.lanes; m < 32; m *= 2)
#pragma unroll
        for (int i = 0; i < kHeld / 2; ++i)
            dw[i] = add2(dw[i], make_float2(__shfl_xor_sync(~0u, dw[i].x, m), __shfl_xor_sync(~0u, dw[i].y, m)));
    float *out = a.ctas == 1 ? a.dw : a.part + (size_t)blockIdx.x * D;
    float *acc = reinterpret_cast<float *>(staged);
    __syncthreads();   // every thread is done with its copies
    const int width = max(sp.lanes, 32), parts = sp.threads / width, mine = threadIdx.x / width;
    if (threadIdx.x % width < sp.lanes)
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int d = col[i / VEC] + i % VEC;
            if ((unsigned)d < (unsigned)D)
                (parts > 1 ? acc + mine * D : out)[d] = i % 2 ? dw[i / 2].y : dw[i / 2].x;
        }
    if (parts == 1)
        return;
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += sp.threads) {
        float sum = acc[d];
        for (int i = 1; i < parts; ++i)
            sum += acc[i * D + d];
        out[d] = sum;
    }
}

// --- rows wider than kMaxHeld: one CTA a row, read again from cache -----------------------------------------------

template <typename F>
__device__ __forceinline__ float block_reduce(float v, float *sh, F f)
{
    for (int m = 16; m; m >>= 1)
        v = f(v, __shfl_xor_sync(~0u, v, m));
    __syncthreads();
    if (threadIdx.x % 32 == 0)
        sh[threadIdx.x / 32] = v;
    __syncthreads();
    v = sh[0];
    for (int i = 1; i < kThreads / 32; ++i)
        v = f(v, sh[i]);
    return v;
}

__device__ __forceinline__ float block_sum(float v, float *sh)
{
    return block_reduce(v, sh, [](float a, float b) { return a + b; });
}

template <typename Tx, typename Tr>
__global__ void __launch_bounds__(kThreads) norm_fwd_wide(NormArgs a)
{
    __shared__ float sh[kThreads / 32];
    const Tx *x = static_cast<const Tx *>(a.x);
    const Tr *res = static_cast<const Tr *>(a.res);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t at = row * a.D;
        auto total = [&](int d) { return widen(x[at + d]) + (res ? widen(res[at + d]) : 0.f); };
        float sq = 0.f;
        for (int d = threadIdx.x; d < a.D; d += kThreads)
            sq = fmaf(total(d), total(d), sq);
        const float rstd = rsqrtf(block_sum(sq, sh) / a.D + a.eps);
        if (a.rstd && threadIdx.x == 0)
            a.rstd[row] = rstd;
        auto normed = [&](int d) { return total(d) * (a.w ? a.w[d] : 1.f) * rstd; };
        const int group = a.group ? a.group : a.D, groups = (a.D + group - 1) / group;
        for (int c = 0; c < (a.scales ? groups : 1); ++c) {
            const int lo = a.scales ? c * group : 0, hi = a.scales ? min(a.D, lo + group) : a.D;
            float inv = 1.f;
            if (a.scales) {
                float m = 0.f;
                for (int d = lo + threadIdx.x; d < hi; d += kThreads)
                    m = max_nan(m, fabsf(normed(d)));
                const float scale = scale_of(block_reduce(m, sh, max_nan));
                inv = reciprocal(scale);
                if (threadIdx.x == 0)
                    a.scales[row * groups + c] = scale;
            }
            for (int d = lo + threadIdx.x; d < hi; d += kThreads) {
                const float y = normed(d), s = total(d);
                if (a.scales)
                    static_cast<__nv_fp8_storage_t *>(a.y)[at + d] =
                        __nv_cvt_float_to_fp8(y * inv, __NV_SATFINITE, __NV_E4M3);
                else
                    static_cast<Tx *>(a.y)[at + d] = narrow<Tx>(y);
                if (a.s)   // last: s may be res itself
                    static_cast<Tr *>(a.s)[at + d] = narrow<Tr>(s);
            }
        }
    }
}

template <typename Tx, typename Tr>
__global__ void __launch_bounds__(kThreads) norm_bwd_wide(NormArgs a)
{
    __shared__ float sh[kThreads / 32];
    const Tr *s = static_cast<const Tr *>(a.s_in), *ds = static_cast<const Tr *>(a.ds);
    const Tx *dy = static_cast<const Tx *>(a.dy);
    float *part = a.ctas == 1 && a.dw ? a.dw : a.part + (size_t)blockIdx.x * a.D;
    for (int d = threadIdx.x; d < a.D; d += kThreads)
        part[d] = 0.f;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t at = row * a.D;
        const float r = a.rstd_in[row];
        float c = 0.f;
        for (int d = threadIdx.x; d < a.D; d += kThreads)
            c = fmaf((a.w ? a.w[d] : 1.f) * widen(dy[at + d]), widen(s[at + d]) * r, c);
        c = block_sum(c, sh) / a.D;
        for (int d = threadIdx.x; d < a.D; d += kThreads) {
            const float n = widen(s[at + d]) * r, g = widen(dy[at + d]);
            const float grad = fmaf(r, (a.w ? a.w[d] : 1.f) * g - n * c, ds ? widen(ds[at + d]) : 0.f);
            part[d] = fmaf(g, n, part[d]);
            if (a.dx)
                static_cast<Tx *>(a.dx)[at + d] = narrow<Tx>(grad);
            if (a.dres)
                static_cast<Tr *>(a.dres)[at + d] = narrow<Tr>(grad);
        }
    }
}

// dw from the CTAs' partial sums: 32 columns a CTA, 32 threads a column, in a fixed order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(NormArgs a)
{
    __shared__ float sh[32][33];
    tc::grid_dep_wait();
    const int c = threadIdx.x % 32, k = threadIdx.x / 32, d = blockIdx.x * 32 + c;
    float sum = 0.f;
    if (d < a.D)
        for (int i = k; i < a.ctas; i += 32)
            sum += a.part[(size_t)i * a.D + d];
    sh[k][c] = sum;
    __syncthreads();
    sum = sh[c][k];
    for (int m = 16; m; m >>= 1)
        sum += __shfl_xor_sync(~0u, sum, m);
    if (c == 0 && blockIdx.x * 32 + k < a.D)
        a.dw[blockIdx.x * 32 + k] = sum;
}

template <typename F>
cudaError_t by_norm_types(int dtype, bool res_f32, F f)
{
    typedef __nv_bfloat16 bf;
    if (dtype == GLA_F32)
        return f((float *)0, (float *)0);
    if (dtype == GLA_BF16)
        return res_f32 ? f((bf *)0, (float *)0) : f((bf *)0, (bf *)0);
    return res_f32 ? f((__half *)0, (float *)0) : f((__half *)0, (__half *)0);
}

// Persistent CTAs, `per_sm` of them, or one for each of its rows where there are fewer.  Where a CTA takes several
// turns its rows stay a multiple of 8 apart, so that they keep their shift.
int grid_of(int64_t rows, const Split &sp, int per_sm)
{
    const int64_t need = (rows + sp.rows - 1) / sp.rows, most = (int64_t)per_sm * sm_count() / 8 * 8;
    return (int)std::min(need, most);
}

// The backward's: a multiple of 8 where rows are shifted and several to a CTA.
int bwd_grid(int64_t rows, int D, int vec)
{
    const Split sp = split_of(D, vec);
    const int ctas = grid_of(rows, sp, std::max(1, 512 / sp.threads));   // 128 registers a thread
    return D % vec && sp.rows > 1 ? (ctas + 7) / 8 * 8 : ctas;
}

template <typename Tx, typename Tr, Quant Q, bool SHIFTED>
cudaError_t fwd_rows(const NormArgs &a, cudaStream_t s)
{
    auto kernel = norm_fwd_rows<Tx, Tr, Q, SHIFTED>;
    const Split sp = split_of(a.D, 16 / sizeof(Tx));
    static std::atomic<int> fit[17];   // CTAs an SM holds, by warps of a CTA (0: not asked yet)
    std::atomic<int> &known = fit[sp.threads / 32];
    int per_sm = known.load(std::memory_order_relaxed);
    if (per_sm == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, sp.threads, 0) != cudaSuccess || per_sm < 1)
            per_sm = 1;
        known.store(per_sm, std::memory_order_relaxed);
    }
    return launch_early(kernel, grid_of(a.rows, sp, per_sm), sp.threads, s, a, sp);
}

template <typename Tx, typename Tr, Quant Q>
cudaError_t fwd(const NormArgs &a, cudaStream_t s)
{
    return a.D % (16 / (int)sizeof(Tx)) ? fwd_rows<Tx, Tr, Q, true>(a, s) : fwd_rows<Tx, Tr, Q, false>(a, s);
}

template <typename Tx, typename Tr, bool SHIFTED>
cudaError_t bwd_rows(const NormArgs &a, cudaStream_t s)
{
    const Split sp = split_of(a.D, 16 / sizeof(Tx));
    if (!by_shared<Tx, Tr>(a, sp))
        return launch_early_shared(norm_bwd_rows<Tx, Tr, SHIFTED, false>, a.ctas, sp.threads,
                                   sp.rows > 1 || sp.lanes < 32 ? sp.threads * kHeld * sizeof(float) : 0, s, a, sp);
    auto shared = [](int threads) { return kAhead<Tr> * threads * (kRowUnits<Tx, Tr> * 16 + (int)sizeof(float)); };
    auto kernel = norm_bwd_rows<Tx, Tr, SHIFTED, true>;
    static std::atomic<bool> sized[128];   // by device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev >= 128)
        return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    if (!sized[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, shared(512));
        if (e != cudaSuccess)
            return e;
        sized[dev].store(true, std::memory_order_relaxed);
    }
    return launch_early_shared(kernel, a.ctas, sp.threads, shared(sp.threads), s, a, sp);
}

bool wide(int D, int vec) { return held_columns(D, vec) > kMaxHeld; }

}  // namespace

int norm_bwd_ctas(int64_t rows, int D, int dtype)
{
    const int vec = dtype == GLA_F32 ? 4 : 8;
    if (wide(D, vec))
        return (int)std::min<int64_t>(rows, 2 * sm_count());
    return bwd_grid(rows, D, vec);
}

cudaError_t launch_norm_fwd(const NormArgs &a, int dtype, bool res_f32, cudaStream_t s)
{
    return by_norm_types(dtype, res_f32, [&](auto x, auto r) {
        typedef std::remove_pointer_t<decltype(x)> Tx;
        typedef std::remove_pointer_t<decltype(r)> Tr;
        if (wide(a.D, 16 / sizeof(Tx))) {
            norm_fwd_wide<Tx, Tr><<<(unsigned)std::min<int64_t>(a.rows, 16 * sm_count()), kThreads, 0, s>>>(a);
            return cudaGetLastError();
        }
        return !a.scales ? fwd<Tx, Tr, kPlain>(a, s)
               : a.group && a.group < a.D ? fwd<Tx, Tr, kByGroup>(a, s) : fwd<Tx, Tr, kByRow>(a, s);
    });
}

cudaError_t launch_norm_bwd(const NormArgs &a, int dtype, bool res_f32, cudaStream_t s)
{
    return by_norm_types(dtype, res_f32, [&](auto x, auto r) {
        typedef std::remove_pointer_t<decltype(x)> Tx;
        typedef std::remove_pointer_t<decltype(r)> Tr;
        if (wide(a.D, 16 / sizeof(Tx)))
            norm_bwd_wide<Tx, Tr><<<a.ctas, kThreads, 0, s>>>(a);
        else if (a.D % (16 / (int)sizeof(Tx)))
            return bwd_rows<Tx, Tr, true>(a, s);
        else
            return bwd_rows<Tx, Tr, false>(a, s);
        return cudaGetLastError();
    });
}

cudaError_t launch_norm_dw(const NormArgs &a, cudaStream_t s)
{
    return launch_early(norm_dw_kernel, (a.D + 31) / 32, 1024, s, a);
}

}  // namespace gla
