// Internal declarations of the gated delta rule: entry points in delta_api.cu, the token-by-token kernels for any type
// and head size in delta_scan.cu, the chunked tensor-core kernels in delta_mma.cu and delta_grads.cu, one token in
// delta_step.cu.
#pragma once

#include "gla_internal.h"
#include "layer_internal.h"

namespace gla {

// What the chunked forward leaves for the gradients, and the reverse pass for them; a cell is a (slot, value head).
struct DeltaTrace {
    uint32_t *s, *ds, *n, *x;          // cells of s_size (s, ds) or n_size (n, x) words: S' at the chunk's start and its
                                       // gradient at the end, N' and the gradient of N, in blocks of 8 x 8 rounded values
    float4 *y;                         // [cell][V / 16][8][32] Y as a warp's results have it
    float *dots;                       // [cell][V / 16][3][64] o.dO, x.Y and dv.v over 16 columns
    float4 *kept;                      // [kept group][HV][V / 16][K / 8][32] states at the ends of groups of chunks
    float *across;                     // [kept group][HV][V / 16] their products with their gradients
    float *power;                      // fp16: [cell][V / 16][8] powers of two that the 16 columns of S, N, dO (0 .. 2), dS and
                                       // beta x (4, 5) were divided by
    size_t s_size, n_size;
};

// Forward and backward (passed by value).  Rows are tokens of all sequences; key head of value head hv: hv / (HV / H).
struct DeltaArgs {
    const void *q, *k, *v, *dout;      // [rows, H, K], [rows, H, K], [rows, HV, V], [rows, HV, V]
    const float *g, *beta;             // [rows, HV]
    const float *h0, *dht;             // [N, HV, K, V] or nullptr
    const int32_t *cu;                 // device offsets or nullptr
    void *o, *dq, *dk, *dv;
    float *ht, *dg, *dbeta, *dh0;
    float scale;
    int N, B, T, H, HV, K, V;
    int64_t rows;                      // B * T
    int slots;                         // (sequence, chunk of 64 rows) pairs, an upper bound in packs
    int *status;
    // workspace of the backward's token-by-token kernels, fp32
    float *upd, *dx;                   // [rows, HV, V]: update rows of the state, and their gradients over beta
    float *dqh, *eh, *fh;              // [rows, HV, K]: gradients of q, and of k by way of k S and of k^T n
    float *dG;                         // [rows, HV]: gradient of the running sum of gates
    float *kept;                       // [slots, HV, K, V]: states at the chunks' ends
    float *hd;                         // [slots, HV, K]: rows of their products with their gradients
    // workspace of the chunked kernels
    char *chunk;                       // cells (DeltaCell, or DeltaCellBack)
    float *score;                      // fp16: [cell] factor of P, which is stored over a power of two and `scale`
    DeltaTrace trace;
};

// One token (passed by value).
struct DeltaStepArgs {
    const void *q, *k, *v;             // [B, H, K], [B, H, K], [B, HV, V]
    const float *g, *beta, *h0;
    void *o;
    float *ht;
    const int32_t *slots;
    float scale;
    int B, S, H, HV, K, V;
    int *status;
};

constexpr int kDeltaChunk = 64;        // rows of a chunk
constexpr int kDeltaKept = 2;          // chunks between two states that are kept in fp32

// Rows of sequence n, [bos, bos + len).  False for offsets outside [0, T] or decreasing.
__device__ __forceinline__ bool delta_sequence(const DeltaArgs &a, int n, int &bos, int &len)
{
    if (!a.cu) {
        bos = n * a.T;
        len = a.T;
        return true;
    }
    bos = a.cu[n];
    const int eos = a.cu[n + 1];
    len = eos - bos;
    return bos >= 0 && len >= 0 && eos <= a.T;
}

// Slots of a pack's sequence n start at cu[n] / 64 + n: at least as many as it has chunks before the next one's first.
__device__ __forceinline__ int delta_first_slot(const DeltaArgs &a, int n)
{
    return a.cu ? a.cu[n] / kDeltaChunk + n : n * ((a.T + kDeltaChunk - 1) / kDeltaChunk);
}

// Groups of kDeltaKept chunks, numbered likewise; the place of a group's state at the end of chunk c.
__device__ __forceinline__ int delta_first_group(const DeltaArgs &a, int n)
{
    constexpr int kRows = kDeltaChunk * kDeltaKept;
    return a.cu ? a.cu[n] / kRows + n : n * ((a.T + kRows - 1) / kRows);
}
__device__ __forceinline__ size_t delta_kept_at(const DeltaArgs &a, int n, int c, int hv, int g16)
{
    return ((size_t)(delta_first_group(a, n) + c / kDeltaKept) * a.HV + hv) * (a.V / 16) + g16;
}

// The chunk of a slot: its sequence, its number in it, its first row and its rows.  False for a slot without rows.
__device__ __forceinline__ bool delta_chunk(const DeltaArgs &a, int slot, int &n, int &c, int &row, int &rows)
{
    if (!a.cu) {
        const int per = (a.T + kDeltaChunk - 1) / kDeltaChunk;
        n = slot / per;
    } else {
        int lo = 0, hi = a.N - 1;   // the last sequence that starts at or before the slot
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (delta_first_slot(a, mid) <= slot)
                lo = mid;
            else
                hi = mid - 1;
        }
        n = lo;
    }
    int bos, len;
    if (!delta_sequence(a, n, bos, len))
        return false;
    c = slot - delta_first_slot(a, n);
    if (c < 0 || (int64_t)c * kDeltaChunk >= len)
        return false;
    row = bos + c * kDeltaChunk;
    rows = min(kDeltaChunk, len - c * kDeltaChunk);
    return true;
}

inline bool delta_half(int dtype) { return dtype == GLA_F16 || dtype == GLA_F16_OF16; }
// 16-bit inputs whose keys are whole warp products and whose values are whole groups of 16 columns go in chunks.
inline bool delta_chunked(int dtype, int K, int V) { return dtype != GLA_F32 && (K == 64 || K == 128) && V % 16 == 0; }
size_t delta_cell_bytes(bool backward);
cudaError_t launch_delta_prep(const DeltaArgs &a, bool half, bool backward, cudaStream_t s);
cudaError_t launch_delta_chain(const DeltaArgs &a, int dtype, bool save, cudaStream_t s);
cudaError_t launch_delta_chain_back(const DeltaArgs &a, bool half, cudaStream_t s);
cudaError_t launch_delta_grads(const DeltaArgs &a, bool half, int sms, cudaStream_t s);
cudaError_t launch_delta_chunk_gates(const DeltaArgs &a, cudaStream_t s);

cudaError_t launch_delta_cols(const DeltaArgs &a, int dtype, bool backward, cudaStream_t s);
cudaError_t launch_delta_rows(const DeltaArgs &a, int dtype, bool backward, cudaStream_t s);
cudaError_t launch_delta_join(const DeltaArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_delta_gates(const DeltaArgs &a, cudaStream_t s);
cudaError_t launch_delta_step(const DeltaStepArgs &a, int dtype, cudaStream_t s);

// Calls f with null pointers of the (input, output) types of a dtype code.
template <typename F>
cudaError_t delta_types(int dtype, F f)
{
    typedef __nv_bfloat16 bf;
    switch (dtype) {
    case GLA_F32: return f((float *)0, (float *)0);
    case GLA_BF16: return f((bf *)0, (float *)0);
    case GLA_BF16_OBF16: return f((bf *)0, (bf *)0);
    case GLA_F16: return f((__half *)0, (float *)0);
    case GLA_F16_OF16: return f((__half *)0, (__half *)0);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace gla
