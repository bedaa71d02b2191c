// C ABI of the gated delta rule: argument checks and launches.  Contracts: include/gla.h.
#include <climits>
#include <cmath>
#include <cstring>

#include "api_checks.h"
#include "delta_internal.h"

namespace gla {
namespace {

constexpr size_t kStatusBytes = 256;
constexpr int kMaxHead = 256;

bool delta_sizes(int dtype, bool backward, size_t &x, size_t &o)
{
    switch (dtype) {
    case GLA_F32: x = o = 4; return true;
    case GLA_BF16: case GLA_F16: x = 2; o = 4; return true;
    case GLA_BF16_OBF16: case GLA_F16_OF16: x = o = 2; return !backward;
    default: return false;
    }
}

int check_shape(int N, int B, int T, int H, int HV, int K, int V, bool varlen)
{
    if (B < 0 || T < 0 || N < 0 || H <= 0 || HV <= 0 || K <= 0 || V <= 0 || (varlen ? B != 1 : N != B) || HV % H)
        return GLA_ERR_INVALID_ARG;
    // rows, and (sequence, head, tile) and (chunk, head) numbers, are 32-bit
    const long long rows = (long long)B * T;
    if (K > kMaxHead || V > kMaxHead || rows > INT_MAX - (1 << 16) || (long long)N * HV > INT_MAX / 64 ||
        (rows / kDeltaChunk + N + 1) * HV > INT_MAX / 16)
        return GLA_ERR_UNSUPPORTED;
    return GLA_OK;
}

void plan(DeltaArgs &a, int N, int B, int T, int H, int HV, int K, int V, bool varlen)
{
    a.N = N; a.B = B; a.T = T; a.H = H; a.HV = HV; a.K = K; a.V = V;
    a.rows = (int64_t)B * T;
    a.slots = varlen ? T / kDeltaChunk + N : B * ((T + kDeltaChunk - 1) / kDeltaChunk);
}

// Places an array in the workspace (without one: counts its bytes).
template <typename E>
void place(E *&p, char *base, size_t &at, size_t count)
{
    p = base ? reinterpret_cast<E *>(base + at) : nullptr;
    at += align_up(count * sizeof(E));
}

// The chunked forward's workspace.
size_t place_fwd(DeltaArgs &a, int dtype, char *base)
{
    size_t at = 0;
    if (delta_chunked(dtype, a.K, a.V)) {
        const size_t cells = (size_t)a.slots * a.HV;
        place(a.chunk, base, at, cells * delta_cell_bytes(false));
        if (delta_half(dtype))
            place(a.score, base, at, cells);
    }
    return at;
}

// The backward's workspace.
size_t place_bwd(DeltaArgs &a, int dtype, char *base)
{
    size_t at = 0;
    if (delta_chunked(dtype, a.K, a.V)) {
        const size_t cells = (size_t)a.slots * a.HV, columns = a.V / 16;
        constexpr int kRows = kDeltaChunk * kDeltaKept;
        const size_t kept = (size_t)(a.cu ? a.T / kRows + a.N : a.B * ((a.T + kRows - 1) / kRows)) * a.HV * columns;
        DeltaTrace &t = a.trace;
        t.s_size = (size_t)a.V * a.K / 2;
        t.n_size = (size_t)a.V * kDeltaChunk / 2;
        place(a.chunk, base, at, cells * delta_cell_bytes(true));
        place(t.s, base, at, cells * t.s_size);
        place(t.ds, base, at, cells * t.s_size);
        place(t.n, base, at, cells * t.n_size);
        place(t.x, base, at, cells * t.n_size);
        place(t.y, base, at, cells * columns * 256);
        place(t.dots, base, at, cells * columns * 3 * kDeltaChunk);
        place(t.kept, base, at, kept * (a.K / 8) * 32);
        place(t.across, base, at, kept);
        if (delta_half(dtype)) {
            place(t.power, base, at, cells * columns * 8);
            place(a.score, base, at, cells);
        }
        return at;
    }
    const size_t heads = (size_t)a.rows * a.HV;
    place(a.upd, base, at, heads * a.V);
    place(a.dx, base, at, heads * a.V);
    place(a.dqh, base, at, heads * a.K);
    place(a.eh, base, at, heads * a.K);
    place(a.fh, base, at, heads * a.K);
    place(a.dG, base, at, heads);
    place(a.kept, base, at, (size_t)a.slots * a.HV * a.K * a.V);
    place(a.hd, base, at, (size_t)a.slots * a.HV * a.K);
    return at;
}

}  // namespace
}  // namespace gla

using namespace gla;

extern "C" size_t gla_delta_fwd_workspace_size(int N, int B, int T, int H, int HV, int K, int V, int dtype, int varlen)
{
    size_t x, o;
    if (!delta_sizes(dtype, false, x, o) || check_shape(N, B, T, H, HV, K, V, varlen != 0))
        return 0;
    DeltaArgs a;
    std::memset(&a, 0, sizeof a);
    plan(a, N, B, T, H, HV, K, V, varlen != 0);
    return place_fwd(a, dtype, nullptr);
}

extern "C" size_t gla_delta_bwd_workspace_size(int N, int B, int T, int H, int HV, int K, int V, int dtype, int varlen)
{
    size_t x, o;
    if (!delta_sizes(dtype, true, x, o) || check_shape(N, B, T, H, HV, K, V, varlen != 0))
        return 0;
    DeltaArgs a;
    std::memset(&a, 0, sizeof a);
    plan(a, N, B, T, H, HV, K, V, varlen != 0);
    static const int32_t offsets = 0;
    a.cu = varlen ? &offsets : nullptr;   // only whether there are any
    return place_bwd(a, dtype, nullptr);
}

extern "C" int gla_delta_fwd(const void *q, const void *k, const void *v, const float *g, const float *beta, void *o,
                             float scale, const float *h0, float *ht, const int32_t *cu_seqlens, int N, int B, int T,
                             int H, int HV, int K, int V, int dtype, void *status, void *workspace,
                             size_t workspace_bytes, void *stream)
{
    const bool varlen = cu_seqlens != nullptr;
    size_t xs, os;
    if (!delta_sizes(dtype, false, xs, os))
        return GLA_ERR_UNSUPPORTED;
    if (int rc = check_shape(N, B, T, H, HV, K, V, varlen))
        return rc;
    if (!(scale > 0.f) || !std::isfinite(scale))
        return GLA_ERR_INVALID_ARG;
    DeltaArgs a;
    std::memset(&a, 0, sizeof a);
    plan(a, N, B, T, H, HV, K, V, varlen);
    const size_t rows = (size_t)a.rows, state = (size_t)N * HV * K * V * 4;
    if (rows > 0 && (!q || !k || !v || !g || !beta || !o))
        return GLA_ERR_INVALID_ARG;
    if (any_misaligned({q, k, v, g, beta, o, h0, ht, cu_seqlens}))
        return GLA_ERR_ALIGNMENT;
    if (int rc = check_workspace(status, kStatusBytes, kStatusBytes))
        return rc;
    const size_t need = gla_delta_fwd_workspace_size(N, B, T, H, HV, K, V, dtype, varlen);
    if (need)
        if (int rc = check_workspace(workspace, workspace_bytes, need))
            return rc;
    const Rows out[] = {flat(o, rows * HV * V * os), flat(ht, ht ? state : 0), flat(status, kStatusBytes), flat(workspace, need)};
    const Rows in[] = {flat(q, rows * H * K * xs), flat(k, rows * H * K * xs), flat(v, rows * HV * V * xs),
                       flat(g, rows * HV * 4), flat(beta, rows * HV * 4), flat(h0, h0 && h0 != ht ? state : 0),
                       flat(cu_seqlens, varlen ? 4 * (size_t)(N + 1) : 0)};
    if (outputs_clash(out, in))
        return GLA_ERR_INVALID_ARG;
    g_prof.launches = 0;
    if (N == 0)
        return GLA_OK;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.o = o; a.h0 = h0; a.ht = ht; a.cu = cu_seqlens; a.scale = scale;
    a.status = static_cast<int *>(status);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!delta_chunked(dtype, K, V))
        return profiled(K_DELTA_COLS, s, [&] { return launch_delta_cols(a, dtype, false, s); }) == cudaSuccess
                   ? GLA_OK : GLA_ERR_CUDA;
    place_fwd(a, dtype, static_cast<char *>(workspace));
    const bool half = delta_half(dtype);
    if (a.slots && profiled(K_DELTA_PREP, s, [&] { return launch_delta_prep(a, half, false, s); }) != cudaSuccess)
        return GLA_ERR_CUDA;
    if (profiled(K_DELTA_CHAIN, s, [&] { return launch_delta_chain(a, dtype, false, s); }) != cudaSuccess)
        return GLA_ERR_CUDA;
    return GLA_OK;
}

extern "C" int gla_delta_bwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                             const void *dout, float scale, const float *h0, const float *dht, void *dq, void *dk,
                             void *dv, float *dg, float *dbeta, float *dh0, const int32_t *cu_seqlens, int N, int B,
                             int T, int H, int HV, int K, int V, int dtype, void *status, void *workspace,
                             size_t workspace_bytes, void *stream)
{
    const bool varlen = cu_seqlens != nullptr;
    size_t xs, os;
    if (!delta_sizes(dtype, true, xs, os))
        return GLA_ERR_UNSUPPORTED;
    if (int rc = check_shape(N, B, T, H, HV, K, V, varlen))
        return rc;
    if (!(scale > 0.f) || !std::isfinite(scale))
        return GLA_ERR_INVALID_ARG;
    DeltaArgs a;
    std::memset(&a, 0, sizeof a);
    plan(a, N, B, T, H, HV, K, V, varlen);
    const size_t rows = (size_t)a.rows, state = (size_t)N * HV * K * V * 4, qk = rows * H * K * xs, vb = rows * HV * V * xs;
    if (rows > 0 && (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta))
        return GLA_ERR_INVALID_ARG;
    if (any_misaligned({q, k, v, g, beta, dout, h0, dht, dq, dk, dv, dg, dbeta, dh0, cu_seqlens}))
        return GLA_ERR_ALIGNMENT;
    if (int rc = check_workspace(status, kStatusBytes, kStatusBytes))
        return rc;
    const size_t need = gla_delta_bwd_workspace_size(N, B, T, H, HV, K, V, dtype, varlen);
    if (need)
        if (int rc = check_workspace(workspace, workspace_bytes, need))
            return rc;
    const Rows out[] = {flat(dq, qk), flat(dk, qk), flat(dv, vb), flat(dg, rows * HV * 4), flat(dbeta, rows * HV * 4),
                        flat(dh0, dh0 ? state : 0), flat(status, kStatusBytes), flat(workspace, need)};
    const Rows in[] = {flat(q, qk), flat(k, qk), flat(v, vb), flat(g, rows * HV * 4), flat(beta, rows * HV * 4),
                       flat(dout, vb), flat(h0, h0 ? state : 0), flat(dht, dht ? state : 0),
                       flat(cu_seqlens, varlen ? 4 * (size_t)(N + 1) : 0)};
    if (outputs_clash(out, in))
        return GLA_ERR_INVALID_ARG;
    g_prof.launches = 0;
    if (N == 0)
        return GLA_OK;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.dout = dout; a.h0 = h0; a.dht = dht; a.cu = cu_seqlens;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.dh0 = dh0; a.scale = scale;
    a.status = static_cast<int *>(status);
    place_bwd(a, dtype, static_cast<char *>(workspace));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (delta_chunked(dtype, K, V)) {
        const bool half = delta_half(dtype);
        if (a.slots && (profiled(K_DELTA_PREP, s, [&] { return launch_delta_prep(a, half, true, s); }) != cudaSuccess ||
                        profiled(K_DELTA_CHAIN, s, [&] { return launch_delta_chain(a, dtype, true, s); }) != cudaSuccess))
            return GLA_ERR_CUDA;
        if (profiled(K_DELTA_CHAIN_BACK, s, [&] { return launch_delta_chain_back(a, half, s); }) != cudaSuccess)
            return GLA_ERR_CUDA;
        if (rows && (profiled(K_DELTA_GRADS, s, [&] { return launch_delta_grads(a, half, sm_count(), s); }) != cudaSuccess ||
                     profiled(K_DELTA_GATES, s, [&] { return launch_delta_chunk_gates(a, s); }) != cudaSuccess))
            return GLA_ERR_CUDA;
        return GLA_OK;
    }
    if (profiled(K_DELTA_COLS, s, [&] { return launch_delta_cols(a, dtype, false, s); }) != cudaSuccess ||
        profiled(K_DELTA_COLS_BACK, s, [&] { return launch_delta_cols(a, dtype, true, s); }) != cudaSuccess)
        return GLA_ERR_CUDA;
    if (rows == 0)
        return GLA_OK;
    if (profiled(K_DELTA_ROWS, s, [&] { return launch_delta_rows(a, dtype, false, s); }) != cudaSuccess ||
        profiled(K_DELTA_ROWS_BACK, s, [&] { return launch_delta_rows(a, dtype, true, s); }) != cudaSuccess ||
        profiled(K_DELTA_JOIN, s, [&] { return launch_delta_join(a, dtype, s); }) != cudaSuccess ||
        profiled(K_DELTA_GATES, s, [&] { return launch_delta_gates(a, s); }) != cudaSuccess)
        return GLA_ERR_CUDA;
    return GLA_OK;
}

extern "C" int gla_delta_step(const void *q, const void *k, const void *v, const float *g, const float *beta, void *o,
                              float scale, const float *h0, float *ht, const int32_t *slots, int B, int S, int H, int HV,
                              int K, int V, int dtype, void *status, void *stream)
{
    size_t xs, os;
    if (!delta_sizes(dtype, false, xs, os))
        return GLA_ERR_UNSUPPORTED;
    if (B < 0 || S < 0 || H <= 0 || HV <= 0 || K <= 0 || V <= 0 || HV % H || (!slots && S != B))
        return GLA_ERR_INVALID_ARG;
    if (K > kMaxHead || V > kMaxHead || (long long)B * HV > INT_MAX / 16)   // (sequence, head, tile) numbers are 32-bit
        return GLA_ERR_UNSUPPORTED;
    if (!(scale > 0.f) || !std::isfinite(scale))
        return GLA_ERR_INVALID_ARG;
    if (B > 0 && (!q || !k || !v || !g || !beta || !o || (S > 0 && (!h0 || !ht))))
        return GLA_ERR_INVALID_ARG;
    if (any_misaligned({q, k, v, g, beta, o, h0, ht, slots}))
        return GLA_ERR_ALIGNMENT;
    if (int rc = check_workspace(status, kStatusBytes, kStatusBytes))
        return rc;
    const size_t heads = (size_t)B * HV, keys = (size_t)B * H * K * xs, pool = (size_t)S * HV * K * V * 4;
    const Rows out[] = {flat(o, heads * V * os), flat(ht, pool), flat(status, kStatusBytes)};
    const Rows in[] = {flat(q, keys), flat(k, keys), flat(v, heads * V * xs), flat(g, heads * 4), flat(beta, heads * 4),
                       flat(h0, h0 != ht ? pool : 0), flat(slots, slots ? 4 * (size_t)B : 0)};
    if (outputs_clash(out, in))
        return GLA_ERR_INVALID_ARG;
    g_prof.launches = 0;
    if (B == 0)
        return GLA_OK;
    DeltaStepArgs a;
    std::memset(&a, 0, sizeof a);
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.o = o; a.scale = scale; a.h0 = h0; a.ht = ht; a.slots = slots;
    a.B = B; a.S = S; a.H = H; a.HV = HV; a.K = K; a.V = V;
    a.status = static_cast<int *>(status);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return profiled(K_DELTA_STEP, s, [&] { return launch_delta_step(a, dtype, s); }) == cudaSuccess ? GLA_OK
                                                                                                    : GLA_ERR_CUDA;
}
