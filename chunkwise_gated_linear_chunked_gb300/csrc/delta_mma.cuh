// Pieces shared by the chunked kernels of the gated delta rule: the layout of a chunk's cell in the workspace, and warp
// matrix instructions (m16n8k16 of 16-bit operands, fp32 sums) with their fragments.
//
// Fragments of a warp's product: lane l holds of a 16 x 8 result c[0..1] at row l / 4, columns 2 (l % 4) and + 1, and
// c[2..3] eight rows further.  Two adjacent results are, rounded to 16 bits, the left operand (16 x 16) of a next product,
// which is what lets the chain of a chunk's products stay in registers.
#pragma once

#include <type_traits>

#include "delta_internal.h"
#include "tc_ptx.cuh"

namespace gla {

// One (chunk, value head): per row (beta, e^G, e^(G_end - G), scale e^G), G the running sum of gates in the chunk, and the
// lower triangles of two 64 x 64 matrices in fragments of right operands, 16 bytes a lane: two words of rounded values and
// two of the remainders.  Result tile j (rows 8 j up) takes steps i (columns 16 i up) with 16 i <= 8 j + 7: 20 in all.
constexpr int kTriangle = 20, kFragments = kTriangle * 32;
struct DeltaCell {
    uint4 inverse[kFragments];   // T^ - I, T^ = (I + L diag(beta))^-1, L_ij = e^(G_i - G_j) k_i.k_j below the diagonal
    uint4 score[kFragments];     // P_ij = scale e^(G_i - G_j) q_i.k_j up to the diagonal (fp16: over DeltaArgs::score)
    float4 row[kDeltaChunk];
};
struct DeltaCellBack : DeltaCell {   // and transposed: rows and columns of the tiles' numbers run from the other end
    uint4 inverse_t[kFragments];     // T' - I, T' = (I + L' diag(beta))^-1
    uint4 score_t[kFragments];       // P'
    float2 gate[kDeltaChunk];        // G times log2 e in two floats
};
struct DeltaCellRows {               // the part of it that the gradients' chain copies, from `row` on
    float4 row[kDeltaChunk];
    uint4 inverse[kFragments], score[kFragments];   // T' - I, P'
};
constexpr size_t kCellRows = 2 * kFragments * sizeof(uint4);   // where `row` lies in a cell
__host__ __device__ constexpr int triangle_at(int j, int i) { return (j / 2) * (j / 2 + 1) + (j % 2) * (j / 2 + 1) + i; }
__host__ __device__ constexpr int triangle_at_t(int j, int i) { return triangle_at(7 - j, 3 - i); }

template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same_v<T, __half>)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8 x 8 matrices of 16-bit values from shared memory, lane l giving the address of row l % 8 of matrix l / 8.  In
// order with barriers (volatile), but other loads and stores may pass it: what it reads is written before a barrier.
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}

// Two values as 16-bit ones and their remainders: bf16 keeps 2^-18 of the value, fp16 2^-22 (down to 2^-25 in all: Power).
template <typename T>
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo)
{
    hi = narrow2<T>(make_float2(x, y));
    const float2 h = widen2<T>(hi);
    lo = narrow2<T>(make_float2(x - h.x, y - h.y));
}

// Powers of two for operands of fp16, whose remainders end at 2^-25 whatever the value is: a row of a left operand (a column of
// the state, of the rows that update it, of their gradients) goes in times `to`, which brings its largest value up to fp16's
// upper end, and what comes of it is taken times `from`.  Both are exact, so that operands are within 2^-22 of their own size,
// however small, down to 2^-37 of the row's largest (of a state 2^-26).  What is large already stays as it is, and costs the
// small ones beside it nothing.  bf16 has fp32's range: kScaled is false, and nothing of this is compiled.  The price in fp16
// (times of operands as they are, where values of 1e-4 leave 1e-2 in the gradients): 4 x 2048 tokens of 8 heads forward
// 131 us (100), backward 379 (309); packs of 16 and 8 sequences of 16 heads 1088 (971) and 1019 (911).
template <typename T>
constexpr bool kScaled = std::is_same_v<T, __half>;
struct Power {
    float to, from;
};
// Where the largest value goes: [2^at, 2^(at + 1)).  kOperand: values from there to 2^15 stay, larger ones come down to it.
// kState: to a state a chunk's rows add at most 64 times the largest of them and the keys' length, which may be 250, and it
// does not come down, so that one which leaves fp16's range is seen.  kTerm: values of one term, whose products are operands again.
enum { kTerm = 0, kState = 1, kOperand = 12 };
template <int AT>
__device__ __forceinline__ Power power_of(float largest)   // from 2^-100 to 2^100
{
    const int exponent = (int)(__float_as_uint(largest) >> 23);
    int e = 254 + AT - exponent;
    if (AT == kState)
        e = max(e, 127);
    if (AT == kOperand)
        e = max(e, min(127, 254 + 14 - exponent));
    e = min(max(e, 27), 227);
    return {__uint_as_float((uint32_t)e << 23), __uint_as_float((uint32_t)(254 - e) << 23)};
}
__device__ __forceinline__ float inverse_power(float p) { return __uint_as_float((254u << 23) - __float_as_uint(p)); }

// Largest magnitudes of a lane's two rows (of the result's, over the four lanes that share them).
template <int N>
__device__ __forceinline__ void rows_largest(const float (&c)[N][4], float (&most)[2])
{
#pragma unroll
    for (int j = 0; j < N; ++j) {
        most[0] = fmaxf(most[0], fmaxf(fabsf(c[j][0]), fabsf(c[j][1])));
        most[1] = fmaxf(most[1], fmaxf(fabsf(c[j][2]), fabsf(c[j][3])));
    }
}
template <int AT>
__device__ __forceinline__ void rows_power(float (&most)[2], Power (&p)[2])
{
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        most[x] = fmaxf(most[x], __shfl_xor_sync(~0u, most[x], 1));
        most[x] = fmaxf(most[x], __shfl_xor_sync(~0u, most[x], 2));
        p[x] = power_of<AT>(most[x]);
    }
}
template <int AT, int N>
__device__ __forceinline__ void rows_power(const float (&c)[N][4], Power (&p)[2])
{
    float most[2] = {};
    rows_largest(c, most);
    rows_power<AT>(most, p);
}
__device__ __forceinline__ float warp_largest(float v)
{
#pragma unroll
    for (int m = 16; m; m /= 2)
        v = fmaxf(v, __shfl_xor_sync(~0u, v, m));
    return v;
}
// d = a result's tile times its rows' factors.
__device__ __forceinline__ void times_rows(float (&d)[4], const float (&c)[4], float f0, float f1)
{
    d[0] = f0 * c[0], d[1] = f0 * c[1], d[2] = f1 * c[2], d[3] = f1 * c[3];
}
// Two fp16 values times a power of two of at most 1 (what falls below 2^-25 is lost).
__device__ __forceinline__ uint32_t times_power(uint32_t v, float p)
{
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&v), __float2half2_rn(p));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// A left operand's 16 columns from two adjacent results.
template <typename T>
__device__ __forceinline__ void split_pair(const float (&c0)[4], const float (&c1)[4], uint32_t (&hi)[4], uint32_t (&lo)[4])
{
    split2<T>(c0[0], c0[1], hi[0], lo[0]);
    split2<T>(c0[2], c0[3], hi[1], lo[1]);
    split2<T>(c1[0], c1[1], hi[2], lo[2]);
    split2<T>(c1[2], c1[3], hi[3], lo[3]);
}
// The same times the rows' powers (fp16 alone).
template <typename T>
__device__ __forceinline__ void split_rows(const float (&c0)[4], const float (&c1)[4], const Power (&p)[2], uint32_t (&hi)[4], uint32_t (&lo)[4])
{
    if constexpr (kScaled<T>) {
        float d0[4], d1[4];
        times_rows(d0, c0, p[0].to, p[1].to);
        times_rows(d1, c1, p[0].to, p[1].to);
        split_pair<T>(d0, d1, hi, lo);
    } else {
        split_pair<T>(c0, c1, hi, lo);
    }
}

// The sum of the two terms that split2 leaves.
template <typename T>
__device__ __forceinline__ float2 in_two(float x, float y)
{
    uint32_t hi, lo;
    split2<T>(x, y, hi, lo);
    const float2 h = widen2<T>(hi), l = widen2<T>(lo);
    return make_float2(h.x + l.x, h.y + l.y);
}

// The same of a row that goes in times its power (fp16).
template <typename T>
__device__ __forceinline__ float2 in_two(float x, float y, const Power &p)
{
    if constexpr (!kScaled<T>)
        return in_two<T>(x, y);
    const float2 r = in_two<T>(x * p.to, y * p.to);
    return make_float2(r.x * p.from, r.y * p.from);
}

// The same in three terms, which hold all of an fp32 value (bf16; fp16's range ends with the second).
template <typename T>
__device__ __forceinline__ void split3(float x, float y, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    hi = narrow2<T>(make_float2(x, y));
    const float2 h = widen2<T>(hi);
    split2<T>(x - h.x, y - h.y, mid, lo);
}
template <typename T>
__device__ __forceinline__ void split_pair(const float (&c0)[4], const float (&c1)[4], uint32_t (&hi)[4], uint32_t (&mid)[4], uint32_t (&lo)[4])
{
    split3<T>(c0[0], c0[1], hi[0], mid[0], lo[0]);
    split3<T>(c0[2], c0[3], hi[1], mid[1], lo[1]);
    split3<T>(c1[0], c1[1], hi[2], mid[2], lo[2]);
    split3<T>(c1[2], c1[3], hi[3], mid[3], lo[3]);
}

__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool on)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// 64 rows of WIDTH 16-bit values, `pitch` apart in memory, to shared rows of WIDTH + 8 values (an odd number of 16-byte
// units, so that eight rows' units lie in different banks); rows from `rows` on, and columns from `cols` on, are zeros.
template <int WIDTH, int THREADS, typename T>
__device__ __forceinline__ void copy_rows(uint32_t to, const T *from, size_t pitch, int rows, int cols)
{
    constexpr int kUnits = WIDTH / 8;
    static_assert(64 * kUnits % THREADS == 0 || 64 * kUnits < THREADS, "whole turns");
#pragma unroll
    for (int i = 0; i < (64 * kUnits + THREADS - 1) / THREADS; ++i) {
        const int e = i * THREADS + threadIdx.x % THREADS, r = e / kUnits, u = e % kUnits;
        if (64 * kUnits < THREADS && e >= 64 * kUnits)
            break;
        const bool on = r < rows && u * 8 < cols;
        copy16(to + (r * (kUnits + 1) + u) * 16, from + (on ? r * pitch + u * 8 : 0), on);
    }
}

template <int I>
using Int = std::integral_constant<int, I>;

}  // namespace gla
