// C ABI of the operators beside the chunkwise kernels: argument checks and launches of the vector-state gated
// linear recurrence, the one-token state updates and the residual norm.  Contracts: include/gla.h.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "api_checks.h"
#include "layer_internal.h"

namespace gla {
namespace {

constexpr size_t kStatusBytes = 256;
constexpr int kMaxNormD = 16384;
constexpr int64_t kMaxStride = int64_t(1) << 40;

__device__ __align__(256) char g_shared_status[kStatusBytes];   // one a device, zero from the start

struct TypeSizes {
    size_t x, g, o;
};

bool type_sizes(int dtype, TypeSizes &t)
{
    switch (dtype) {
    case GLA_F32: t = {4, 4, 4}; return true;
    case GLA_BF16: case GLA_F16: t = {2, 2, 4}; return true;
    case GLA_BF16_OBF16: case GLA_F16_OF16: t = {2, 2, 2}; return true;
    case GLA_BF16_GF32: case GLA_F16_GF32: t = {2, 4, 4}; return true;
    default: return false;
    }
}

// (sequence, channel tile, time slice) numbers are 32-bit
bool tiles_ok(int n, int D) { return (long long)n * (D / 32 + 1) <= INT_MAX / 16; }

int check_scan_shape(int N, int B, int T, int D, bool varlen, std::initializer_list<int64_t> lds)
{
    if (B < 0 || T < 0 || N < 0 || D <= 0 || (varlen ? B != 1 : N != B))
        return GLA_ERR_INVALID_ARG;
    for (int64_t ld : lds)
        if (ld < D || ld > kMaxStride)
            return GLA_ERR_INVALID_ARG;
    if ((long long)B * T > INT_MAX - (1 << 16) || !tiles_ok(N, D))   // row and CTA numbers are 32-bit, slices included
        return GLA_ERR_UNSUPPORTED;
    return GLA_OK;
}

}  // namespace
}  // namespace gla

using namespace gla;

extern "C" size_t gla_scan_workspace_size(void) { return kStatusBytes; }

extern "C" void *gla_scan_shared_workspace(void)
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_shared_status) == cudaSuccess ? p : nullptr;
}

extern "C" int gla_scan_fwd(const void *x, const void *g, void *h, const float *h0, float *ht,
                            const int32_t *cu_seqlens, int N, int B, int T, int D, int64_t ldx, int64_t ldg, int dtype,
                            void *workspace, size_t workspace_bytes, void *stream)
{
    const bool varlen = cu_seqlens != nullptr;
    TypeSizes ts;
    if (!type_sizes(dtype, ts))
        return GLA_ERR_UNSUPPORTED;
    if (int rc = check_scan_shape(N, B, T, D, varlen, {ldx, ldg}))
        return rc;
    const size_t rows = (size_t)B * T;
    if (rows > 0 && (!x || !g || !h))
        return GLA_ERR_INVALID_ARG;
    if (any_misaligned({x, g, h, h0, ht, cu_seqlens}))
        return GLA_ERR_ALIGNMENT;
    if (int rc = check_workspace(workspace, workspace_bytes, kStatusBytes))
        return rc;
    const size_t state = (size_t)N * D * 4;
    const Rows out[] = {flat(h, rows * D * ts.o), flat(ht, ht ? state : 0), flat(workspace, kStatusBytes)};
    const Rows in[] = {rows_of(x, rows, D * ts.x, ldx * ts.x), rows_of(g, rows, D * ts.g, ldg * ts.g),
                       flat(h0, h0 && h0 != ht ? state : 0), flat(cu_seqlens, varlen ? 4 * (size_t)(N + 1) : 0)};
    if (outputs_clash(out, in))
        return GLA_ERR_INVALID_ARG;
    g_prof.launches = 0;
    if (N == 0)
        return GLA_OK;
    ScanArgs a;
    std::memset(&a, 0, sizeof a);
    a.x = x; a.g = g; a.h = h; a.h0 = h0; a.ht = ht; a.cu = cu_seqlens;
    a.N = N; a.T = T; a.D = D; a.ldx = ldx; a.ldg = ldg;
    a.status = static_cast<int *>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const ScanShare share = scan_share(a);
    a.alone = share.rows;
    if (share.rows >= 0 &&
        profiled(K_SCAN_FWD_ROWS, s, [&] { return launch_scan_fwd(a, dtype, true, s); }) != cudaSuccess)
        return GLA_ERR_CUDA;
    if (share.tiles && profiled(K_SCAN_FWD, s, [&] { return launch_scan_fwd(a, dtype, false, s); }) != cudaSuccess)
        return GLA_ERR_CUDA;
    return GLA_OK;
}

extern "C" int gla_scan_bwd(const void *g, const void *h, const void *dh, const float *h0, const float *dht, void *dx,
                            void *dg, float *dh0, const int32_t *cu_seqlens, int N, int B, int T, int D, int64_t ldg,
                            int64_t lddx, int64_t lddg, int dtype, void *workspace, size_t workspace_bytes,
                            void *stream)
{
    const bool varlen = cu_seqlens != nullptr;
    TypeSizes ts;
    if (!type_sizes(dtype, ts))
        return GLA_ERR_UNSUPPORTED;
    if (int rc = check_scan_shape(N, B, T, D, varlen, {ldg, lddx, lddg}))
        return rc;
    const size_t rows = (size_t)B * T;
    if (rows > 0 && (!g || !h || !dh || !dx || !dg))
        return GLA_ERR_INVALID_ARG;
    if (any_misaligned({g, h, dh, h0, dht, dx, dg, dh0, cu_seqlens}))
        return GLA_ERR_ALIGNMENT;
    if (int rc = check_workspace(workspace, workspace_bytes, kStatusBytes))
        return rc;
    const size_t state = (size_t)N * D * 4;
    const Rows out[] = {rows_of(dx, rows, D * ts.x, lddx * ts.x), rows_of(dg, rows, D * ts.g, lddg * ts.g),
                        flat(dh0, dh0 ? state : 0), flat(workspace, kStatusBytes)};
    const Rows in[] = {rows_of(g, rows, D * ts.g, ldg * ts.g), flat(h, rows * D * ts.o), flat(dh, rows * D * ts.o),
                       flat(h0, h0 ? state : 0), flat(dht, dht ? state : 0),
                       flat(cu_seqlens, varlen ? 4 * (size_t)(N + 1) : 0)};
    if (outputs_clash(out, in))
        return GLA_ERR_INVALID_ARG;
    g_prof.launches = 0;
    if (N == 0)
        return GLA_OK;
    ScanArgs a;
    std::memset(&a, 0, sizeof a);
    a.g = g; a.h_in = h; a.dh = dh; a.h0 = h0; a.dht = dht; a.dx = dx; a.dg = dg; a.dh0 = dh0; a.cu = cu_seqlens;
    a.N = N; a.T = T; a.D = D; a.ldg = ldg; a.lddx = lddx; a.lddg = lddg;
    a.status = static_cast<int *>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const ScanShare share = scan_share(a);
    a.alone = share.rows;
    if (share.rows >= 0 &&
        profiled(K_SCAN_BWD_ROWS, s, [&] { return launch_scan_bwd(a, dtype, true, s); }) != cudaSuccess)
        return GLA_ERR_CUDA;
    if (share.tiles && profiled(K_SCAN_BWD, s, [&] { return launch_scan_bwd(a, dtype, false, s); }) != cudaSuccess)
        return GLA_ERR_CUDA;
    return GLA_OK;
}

extern "C" int gla_scan_step(const void *x, const void *g, void *h, const float *h0, float *ht, const int32_t *slots,
                             int B, int S, int D, int64_t ldx, int64_t ldg, int dtype, void *workspace,
                             size_t workspace_bytes, void *stream)
{
    TypeSizes ts;
    if (!type_sizes(dtype, ts))
        return GLA_ERR_UNSUPPORTED;
    if (B < 0 || S < 0 || D <= 0 || (!slots && S != B) || ldx < D || ldg < D || ldx > kMaxStride || ldg > kMaxStride)
        return GLA_ERR_INVALID_ARG;
    if (!tiles_ok(B, D))
        return GLA_ERR_UNSUPPORTED;
    if (B > 0 && (!x || !g || !h || (S > 0 && (!h0 || !ht))))
        return GLA_ERR_INVALID_ARG;
    if (any_misaligned({x, g, h, h0, ht, slots}))
        return GLA_ERR_ALIGNMENT;
    if (int rc = check_workspace(workspace, workspace_bytes, kStatusBytes))
        return rc;
    const size_t pool = (size_t)S * D * 4;
    const Rows out[] = {flat(h, (size_t)B * D * ts.o), flat(ht, pool), flat(workspace, kStatusBytes)};
    const Rows in[] = {rows_of(x, B, D * ts.x, ldx * ts.x), rows_of(g, B, D * ts.g, ldg * ts.g),
                       flat(h0, h0 != ht ? pool : 0), flat(slots, slots ? 4 * (size_t)B : 0)};
    if (outputs_clash(out, in))
        return GLA_ERR_INVALID_ARG;
    g_prof.launches = 0;
    if (B == 0)
        return GLA_OK;
    StepArgs a;
    std::memset(&a, 0, sizeof a);
    a.x = x; a.g = g; a.h = h; a.h0 = h0; a.ht = ht; a.slots = slots;
    a.B = B; a.S = S; a.D = D; a.ldx = ldx; a.ldg = ldg;
    a.status = static_cast<int *>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return profiled(K_SCAN_STEP, s, [&] { return launch_scan_step(a, dtype, s); }) == cudaSuccess ? GLA_OK
                                                                                                 : GLA_ERR_CUDA;
}

extern "C" int gla_step(const void *q, const void *k, const void *v, const void *g, void *o, float scale,
                        const float *h0, float *ht, const int32_t *slots, int B, int S, int H, int K, int V, int dtype,
                        void *workspace, size_t workspace_bytes, void *stream)
{
    TypeSizes ts;
    if (!type_sizes(dtype, ts))
        return GLA_ERR_UNSUPPORTED;
    if (B < 0 || S < 0 || H <= 0 || K <= 0 || V <= 0 || (!slots && S != B))
        return GLA_ERR_INVALID_ARG;
    if ((K != 64 && K != 128) || (V != 64 && V != 128 && V != 256))
        return GLA_ERR_UNSUPPORTED;
    if ((long long)B * H > INT_MAX / 16)   // (sequence, head, column tile) numbers are 32-bit
        return GLA_ERR_UNSUPPORTED;
    if (!(scale > 0.f) || !std::isfinite(scale))
        return GLA_ERR_INVALID_ARG;
    if (B > 0 && (!q || !k || !v || !g || !o || (S > 0 && (!h0 || !ht))))
        return GLA_ERR_INVALID_ARG;
    if (any_misaligned({q, k, v, g, o, h0, ht, slots}))
        return GLA_ERR_ALIGNMENT;
    if (int rc = check_workspace(workspace, workspace_bytes, kStatusBytes))
        return rc;
    const size_t heads = (size_t)B * H, pool = (size_t)S * H * K * V * 4;
    const Rows out[] = {flat(o, heads * V * ts.o), flat(ht, pool), flat(workspace, kStatusBytes)};
    const Rows in[] = {flat(q, heads * K * ts.x), flat(k, heads * K * ts.x), flat(v, heads * V * ts.x),
                       flat(g, heads * K * ts.g), flat(h0, h0 != ht ? pool : 0),
                       flat(slots, slots ? 4 * (size_t)B : 0)};
    if (outputs_clash(out, in))
        return GLA_ERR_INVALID_ARG;
    g_prof.launches = 0;
    if (B == 0)
        return GLA_OK;
    StepArgs a;
    std::memset(&a, 0, sizeof a);
    a.x = q; a.k = k; a.v = v; a.g = g; a.h = o; a.scale = scale; a.h0 = h0; a.ht = ht; a.slots = slots;
    a.B = B; a.S = S; a.H = H; a.K = K; a.V = V;
    a.status = static_cast<int *>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return profiled(K_GLA_STEP, s, [&] { return launch_gla_step(a, dtype, s); }) == cudaSuccess ? GLA_OK
                                                                                               : GLA_ERR_CUDA;
}

// ---------------------------------------------------------------------------------------------------
// Residual norm
// ---------------------------------------------------------------------------------------------------
namespace {

bool norm_sizes(int dtype, size_t &x, size_t &r)
{
    const bool res_f32 = (dtype & GLA_RES_F32) != 0;
    dtype &= ~GLA_RES_F32;
    if (dtype != GLA_F32 && dtype != GLA_BF16 && dtype != GLA_F16)
        return false;
    x = dtype == GLA_F32 ? 4 : 2;
    r = res_f32 ? 4 : x;
    return true;
}

bool norm_rows_ok(int64_t rows, int D) { return rows <= (int64_t(1) << 62) / (16 * (int64_t)D); }

int norm_forward(const void *x, const void *res, const float *w, void *y, float *scales, void *s, float *rstd,
                 int64_t rows, int D, float eps, int group, int dtype, bool quant, void *stream)
{
    size_t xs, rs;
    if (!norm_sizes(dtype, xs, rs))
        return GLA_ERR_UNSUPPORTED;
    if (rows < 0 || D <= 0 || !(eps >= 0.f) || !std::isfinite(eps) || group < 0)
        return GLA_ERR_INVALID_ARG;
    if (D > kMaxNormD || (group != 0 && group != 128) || !norm_rows_ok(rows, D))
        return GLA_ERR_UNSUPPORTED;
    if (rows > 0 && (!x || !y || (quant && !scales)))
        return GLA_ERR_INVALID_ARG;
    if (any_misaligned({x, res, w, y, scales, s, rstd}))
        return GLA_ERR_ALIGNMENT;
    const size_t n = (size_t)rows * D, groups = group ? (D + group - 1) / group : 1;
    const Rows out[] = {flat(y, n * (quant ? 1 : xs)), flat(scales, scales ? rows * groups * 4 : 0),
                        flat(s, s ? n * rs : 0), flat(rstd, rstd ? (size_t)rows * 4 : 0)};
    const Rows in[] = {flat(x, n * xs), flat(res, res && res != s ? n * rs : 0), flat(w, w ? (size_t)D * 4 : 0)};
    if (outputs_clash(out, in))
        return GLA_ERR_INVALID_ARG;
    g_prof.launches = 0;
    if (rows == 0)
        return GLA_OK;
    NormArgs a;
    std::memset(&a, 0, sizeof a);
    a.x = x; a.res = res; a.w = w; a.y = y; a.s = s; a.rstd = rstd; a.scales = scales;
    a.rows = rows; a.D = D; a.eps = eps; a.group = group;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool res_f32 = (dtype & GLA_RES_F32) != 0;
    return profiled(quant ? K_NORM_QUANT : K_NORM_FWD, st, [&] {
               return launch_norm_fwd(a, dtype & ~GLA_RES_F32, res_f32, st);
           }) == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

}  // namespace

extern "C" int gla_norm_fwd(const void *x, const void *res, const float *w, void *y, void *s, float *rstd,
                            int64_t rows, int D, float eps, int dtype, void *stream)
{
    return norm_forward(x, res, w, y, nullptr, s, rstd, rows, D, eps, 0, dtype, false, stream);
}

extern "C" int gla_norm_quant_fwd(const void *x, const void *res, const float *w, void *q, float *scales, void *s,
                                  float *rstd, int64_t rows, int D, float eps, int group, int dtype, void *stream)
{
    return norm_forward(x, res, w, q, scales, s, rstd, rows, D, eps, group, dtype, true, stream);
}

extern "C" size_t gla_norm_bwd_workspace_size(int64_t rows, int D)
{
    if (rows < 0 || D <= 0 || D > kMaxNormD)
        return 0;
    const int ctas = std::max(norm_bwd_ctas(rows, D, GLA_F32), norm_bwd_ctas(rows, D, GLA_BF16));
    return kAlign + align_up((size_t)ctas * D * 4);
}

extern "C" int gla_norm_bwd(const void *s, const float *rstd, const float *w, const void *dy, const void *ds, void *dx,
                            void *dres, float *dw, int64_t rows, int D, int dtype, void *workspace,
                            size_t workspace_bytes, void *stream)
{
    size_t xs, rs;
    if (!norm_sizes(dtype, xs, rs))
        return GLA_ERR_UNSUPPORTED;
    if (rows < 0 || D <= 0 || (!dx && !dres && rows > 0))
        return GLA_ERR_INVALID_ARG;
    if (D > kMaxNormD || !norm_rows_ok(rows, D))
        return GLA_ERR_UNSUPPORTED;
    if (rows > 0 && (!s || !rstd || !dy))
        return GLA_ERR_INVALID_ARG;
    if (any_misaligned({s, rstd, w, dy, ds, dx, dres, dw}))
        return GLA_ERR_ALIGNMENT;
    const size_t need = gla_norm_bwd_workspace_size(rows, D);
    if (int rc = check_workspace(workspace, workspace_bytes, need))
        return rc;
    const size_t n = (size_t)rows * D;
    const Rows out[] = {flat(dx, dx ? n * xs : 0), flat(dres, dres ? n * rs : 0), flat(dw, dw ? (size_t)D * 4 : 0),
                        flat(workspace, need)};
    const Rows in[] = {flat(s, n * rs), flat(rstd, (size_t)rows * 4), flat(w, w ? (size_t)D * 4 : 0),
                       flat(dy, dy != dx ? n * xs : 0), flat(ds, ds && ds != dres ? n * rs : 0)};
    if (outputs_clash(out, in))
        return GLA_ERR_INVALID_ARG;
    // an output that may replace one input must still not overlap the others
    if ((dy == dx && share(flat(dy, n * xs), flat(dres, dres ? n * rs : 0))) ||
        (ds && ds == dres && share(flat(ds, n * rs), flat(dx, dx ? n * xs : 0))))
        return GLA_ERR_INVALID_ARG;
    g_prof.launches = 0;
    if (rows == 0 && !dw)
        return GLA_OK;
    NormArgs a;
    std::memset(&a, 0, sizeof a);
    a.s_in = s; a.rstd_in = rstd; a.w = w; a.dy = dy; a.ds = ds; a.dx = dx; a.dres = dres; a.dw = dw;
    a.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + kAlign);
    a.rows = rows; a.D = D;
    a.ctas = norm_bwd_ctas(rows, D, dtype & ~GLA_RES_F32);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool res_f32 = (dtype & GLA_RES_F32) != 0;
    if (rows > 0 && profiled(K_NORM_BWD, st, [&] {
            return launch_norm_bwd(a, dtype & ~GLA_RES_F32, res_f32, st);
        }) != cudaSuccess)
        return GLA_ERR_CUDA;
    if (dw && a.ctas != 1 && profiled(K_NORM_DW, st, [&] { return launch_norm_dw(a, st); }) != cudaSuccess)
        return GLA_ERR_CUDA;
    return GLA_OK;
}
