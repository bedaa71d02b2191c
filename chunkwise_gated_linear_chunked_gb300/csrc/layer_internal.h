// Internal declarations of the operators beside the chunkwise kernels: the vector-state gated linear recurrence
// (scan.cu), the one-token state updates (step.cu) and the residual norm (norm.cu); entry points in layer_api.cu.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "gla.h"

namespace gla {

// Recurrence forward and backward (passed by value).  Row r of a strided tensor starts at r * ld elements.
struct ScanArgs {
    const void *x, *g, *h_in, *dh;     // forward: x, g; backward: g, h_in (the forward's output), dh
    const float *h0, *dht;
    void *h, *dx, *dg;
    float *ht, *dh0;
    const int32_t *cu;                 // device offsets or nullptr
    int N, T, D;                       // sequences, rows of one sequence (dense) or of the pack, channels
    int64_t ldx, ldg, lddx, lddg;
    int alone;                         // sequences of at most so many rows go to threads that walk alone (-1: none)
    int *status;
};

// One-token updates (passed by value).
struct StepArgs {
    const void *x, *g;                 // scan: x, g;  GLA: q in x
    const void *k, *v;
    void *h;
    const float *h0;
    float *ht;
    const int32_t *slots;              // or nullptr: sequence b uses state b
    float scale;
    int B, S, D, H, K, V;
    int64_t ldx, ldg;
    int *status;
};

// Norm forward and backward (passed by value).
struct NormArgs {
    const void *x, *res, *s_in, *dy, *ds;
    const float *w, *rstd_in;
    void *y, *s, *dx, *dres;           // y: x's type, or e4m3 with scales
    float *rstd, *scales, *dw, *part;  // part: partial sums of dw, one row per CTA (a single CTA writes dw itself)
    int64_t rows;
    int D, group, ctas;
    float eps;
};

// A recurrence's sequences of at most `rows` rows go to the kernel whose threads walk alone (none: -1), and what is left
// (if any can be) to the one that cuts the time axis into tiles.
struct ScanShare {
    int rows;
    bool tiles;
};
ScanShare scan_share(const ScanArgs &a);
cudaError_t launch_scan_fwd(const ScanArgs &a, int dtype, bool alone, cudaStream_t s);
cudaError_t launch_scan_bwd(const ScanArgs &a, int dtype, bool alone, cudaStream_t s);
cudaError_t launch_scan_step(const StepArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_gla_step(const StepArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_norm_fwd(const NormArgs &a, int dtype, bool res_f32, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormArgs &a, int dtype, bool res_f32, cudaStream_t s);
cudaError_t launch_norm_dw(const NormArgs &a, cudaStream_t s);
int norm_bwd_ctas(int64_t rows, int D, int dtype);   // CTAs (and partial sums of dw) of the norm's backward

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }

// Two adjacent 16-bit values in a word.
template <typename T>
__device__ __forceinline__ float2 widen2(uint32_t w);
template <>
__device__ __forceinline__ float2 widen2<__nv_bfloat16>(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 widen2<__half>(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t narrow2(float2 v);
template <>
__device__ __forceinline__ uint32_t narrow2<__nv_bfloat16>(float2 v)
{
    const __nv_bfloat162 b = __float22bfloat162_rn(v);
    return *reinterpret_cast<const uint32_t *>(&b);
}
template <>
__device__ __forceinline__ uint32_t narrow2<__half>(float2 v)
{
    const __half2 b = __float22half2_rn(v);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// Two fp32 operations in one instruction (the same roundings as one by one).
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\t"
        "mov.b64 {%0, %1}, d;}" : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\t"
        "mov.b64 {%0, %1}, d;}" : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// 2^t (subnormal results are 0).
__device__ __forceinline__ float exp2_fast(float t)
{
    float a;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(t));
    return a;
}

// exp(g) as 2^(g log2 e): two instructions for the eight of expf.  Measured against fp64 on 2^20 gates a range: off by
// at most 2.6 u (mean -0.4 u, u = 2^-24) for -1 < g < 0, where expf is off by 2.3 u (mean 0.2 u).  Further out the
// rounding of g log2 e adds about |g| u relative, of a decay that is small by then: |g| exp(g) <= 0.37 for g <= 0.  Below
// g = -87.3 the result, subnormal, is 0.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float decay(float g) { return exp2_fast(g * kLog2e); }

// Launches a kernel that may be put on the SMs while the one before it on the stream ends, whose end every one of its
// threads waits for first thing (grid_dep_wait): about 0.4 us less a kernel in a chain of short ones (gla_step of one
// sequence and 8 heads in a CUDA graph: 2.05 -> 1.63 us).
template <typename... P, typename... A>
cudaError_t launch_early_shared(void (*kernel)(P...), unsigned grid, unsigned block, size_t shared, cudaStream_t s, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, unsigned block, cudaStream_t s, A... args)
{
    return launch_early_shared(kernel, grid, block, 0, s, args...);
}

// Calls f with null pointers of the (x, gate, output) types of a recurrence dtype code.
template <typename F>
cudaError_t by_types(int dtype, F f)
{
    typedef __nv_bfloat16 bf;
    switch (dtype) {
    case GLA_F32: return f((float *)0, (float *)0, (float *)0);
    case GLA_BF16: return f((bf *)0, (bf *)0, (float *)0);
    case GLA_BF16_OBF16: return f((bf *)0, (bf *)0, (bf *)0);
    case GLA_F16: return f((__half *)0, (__half *)0, (float *)0);
    case GLA_F16_OF16: return f((__half *)0, (__half *)0, (__half *)0);
    case GLA_BF16_GF32: return f((bf *)0, (float *)0, (float *)0);
    case GLA_F16_GF32: return f((__half *)0, (float *)0, (float *)0);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace gla
