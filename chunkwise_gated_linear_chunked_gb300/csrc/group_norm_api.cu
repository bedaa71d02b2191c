// C ABI of the group norm: argument checks and launches.  Contracts: include/gla.h.
#include <climits>
#include <cmath>
#include <cstring>

#include "api_checks.h"
#include "group_norm.h"

namespace gla {
namespace {

size_t type_size(int dtype) { return dtype == GLA_F32 ? 4 : dtype == GLA_BF16 || dtype == GLA_F16 ? 2 : 0; }

int check_shape(GroupNormArgs &a, int64_t N, int64_t S, int C, int G, int act, int dtype)
{
    if (!type_size(dtype))
        return GLA_ERR_UNSUPPORTED;
    if (N < 0 || S < 1 || C < 1 || G < 1 || C % G || (act != GLA_ACT_NONE && act != GLA_ACT_SILU))
        return GLA_ERR_INVALID_ARG;
    if (N > (int64_t(1) << 58) / C / S)
        return GLA_ERR_UNSUPPORTED;
    std::memset(&a, 0, sizeof a);
    a.N = N; a.S = S; a.C = C; a.G = G; a.W = C / G;
    a.silu = act == GLA_ACT_SILU;
    if (N > 0 && !group_norm_tokens(S, a.W)) {   // CTA numbers are 32-bit
        const GroupNormSplit sp = group_norm_split(a, dtype);
        if (N > INT_MAX / sp.slices / sp.chunks)
            return GLA_ERR_UNSUPPORTED;
    }
    return GLA_OK;
}

// Places the partial sums in the workspace (without one: counts its bytes).
size_t place(GroupNormArgs &a, int dtype, bool backward, bool sums, char *base)
{
    size_t at = 0;
    auto put = [&](auto *&p, size_t count) {
        p = base ? reinterpret_cast<std::remove_reference_t<decltype(p)>>(base + at) : nullptr;
        at += align_up(count * sizeof *p);
    };
    if (a.N == 0)
        return 0;
    if (group_norm_tokens(a.S, a.W)) {
        if (!backward)
            return 0;
        const size_t parts = (size_t)group_norm_token_parts(a, dtype) * a.C;
        put(a.part_dw, parts);
        put(a.part_db, parts);
    } else {
        const GroupNormSplit sp = group_norm_split(a, dtype);
        const size_t slices = (size_t)a.N * sp.slices;
        put(a.part, slices * sp.entries);
        if (backward) {
            put(a.part_dw, slices * a.C);
            put(a.part_db, slices * a.C);
        }
    }
    if (!sums)
        a.part_dw = a.part_db = nullptr;
    return at;
}

}  // namespace
}  // namespace gla

using namespace gla;

extern "C" size_t gla_group_norm_workspace_size(int64_t N, int64_t S, int C, int G, int dtype, int backward)
{
    GroupNormArgs a;
    if (check_shape(a, N, S, C, G, GLA_ACT_NONE, dtype))
        return 0;
    return place(a, dtype, backward != 0, true, nullptr);
}

extern "C" int gla_group_norm_fwd(const void *x, const float *w, const float *b, void *y, float *mean, float *rstd,
                                  int64_t N, int64_t S, int C, int G, float eps, int act, int dtype, void *workspace,
                                  size_t workspace_bytes, void *stream)
{
    GroupNormArgs a;
    if (int rc = check_shape(a, N, S, C, G, act, dtype))
        return rc;
    if (!(eps >= 0.f) || !std::isfinite(eps) || (N > 0 && (!x || !y || !mean || !rstd)))
        return GLA_ERR_INVALID_ARG;
    if (any_misaligned({x, w, b, y, mean, rstd}))
        return GLA_ERR_ALIGNMENT;
    const size_t need = place(a, dtype, false, false, nullptr);
    if (need)
        if (int rc = check_workspace(workspace, workspace_bytes, need))
            return rc;
    const size_t n = (size_t)N * S * C * type_size(dtype), stats = (size_t)N * G * 4;
    const Rows out[] = {flat(y, n), flat(mean, stats), flat(rstd, stats), flat(workspace, need)};
    const Rows in[] = {flat(x, n), flat(w, w ? (size_t)C * 4 : 0), flat(b, b ? (size_t)C * 4 : 0)};
    if (outputs_clash(out, in))
        return GLA_ERR_INVALID_ARG;
    g_prof.launches = 0;
    if (N == 0)
        return GLA_OK;
    a.x = x; a.w = w; a.b = b; a.y = y; a.mean = mean; a.rstd = rstd; a.eps = eps;
    place(a, dtype, false, false, static_cast<char *>(workspace));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (group_norm_tokens(S, a.W))
        return profiled(K_GN_TOKENS, s, [&] { return launch_group_norm_tokens(a, dtype, false, s); }) == cudaSuccess
                   ? GLA_OK : GLA_ERR_CUDA;
    const GroupNormSplit sp = group_norm_split(a, dtype);
    if (profiled(K_GN_SUMS, s, [&] { return launch_group_norm_maps(a, sp, dtype, false, 0, s); }) != cudaSuccess ||
        profiled(K_GN_APPLY, s, [&] { return launch_group_norm_maps(a, sp, dtype, false, 1, s); }) != cudaSuccess)
        return GLA_ERR_CUDA;
    return GLA_OK;
}

extern "C" int gla_group_norm_bwd(const void *x, const float *mean, const float *rstd, const float *w, const float *b,
                                  const void *dy, void *dx, float *dw, float *db, int64_t N, int64_t S, int C, int G,
                                  int act, int dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    GroupNormArgs a;
    if (int rc = check_shape(a, N, S, C, G, act, dtype))
        return rc;
    if (N > 0 && (!x || !mean || !rstd || !dy || !dx))
        return GLA_ERR_INVALID_ARG;
    if (any_misaligned({x, mean, rstd, w, b, dy, dx, dw, db}))
        return GLA_ERR_ALIGNMENT;
    const size_t need = place(a, dtype, true, true, nullptr);
    if (need)
        if (int rc = check_workspace(workspace, workspace_bytes, need))
            return rc;
    const size_t n = (size_t)N * S * C * type_size(dtype), stats = (size_t)N * G * 4, width = (size_t)C * 4;
    const Rows out[] = {flat(dx, n), flat(dw, dw ? width : 0), flat(db, db ? width : 0), flat(workspace, need)};
    const Rows in[] = {flat(x, n), flat(dy, n), flat(mean, stats), flat(rstd, stats), flat(w, w ? width : 0),
                       flat(b, b ? width : 0)};
    if (outputs_clash(out, in))
        return GLA_ERR_INVALID_ARG;
    g_prof.launches = 0;
    a.x = x; a.dy = dy; a.w = w; a.b = b; a.mean_in = mean; a.rstd_in = rstd; a.dx = dx; a.dw = dw; a.db = db;
    const bool sums = dw || db;
    place(a, dtype, true, sums, static_cast<char *>(workspace));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int64_t parts = 0;
    if (N > 0 && group_norm_tokens(S, a.W)) {
        parts = group_norm_token_parts(a, dtype);
        if (profiled(K_GN_TOKENS_BACK, s, [&] { return launch_group_norm_tokens(a, dtype, true, s); }) != cudaSuccess)
            return GLA_ERR_CUDA;
    } else if (N > 0) {
        const GroupNormSplit sp = group_norm_split(a, dtype);
        parts = N * sp.slices;
        if (profiled(K_GN_GRAD_SUMS, s, [&] { return launch_group_norm_maps(a, sp, dtype, true, 0, s); }) != cudaSuccess ||
            profiled(K_GN_GRAD, s, [&] { return launch_group_norm_maps(a, sp, dtype, true, 1, s); }) != cudaSuccess)
            return GLA_ERR_CUDA;
    }
    if (sums && profiled(K_GN_DW, s, [&] { return launch_group_norm_dw(a, parts, s); }) != cudaSuccess)
        return GLA_ERR_CUDA;
    return GLA_OK;
}
