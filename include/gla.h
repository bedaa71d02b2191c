/*
 * gla.h — C ABI of libgla: the chunkwise-parallel forward pass of gated linear attention (GLA) on one
 * NVIDIA GB300 (sm_103a).
 *
 * The method (page "fla/ops/gla/fused_chunk.py": fused_chunk_gla_fwd_kernel, fwd_inner_chunk,
 * prepare_qg_kg, FusedChunkGLAFunction.forward) is the recurrence, per sequence n and head h,
 *
 *     S_0 = h0[n,h] (or 0),   S_t = diag(exp(g_t)) S_{t-1} + k_t^T v_t,   o_t = scale * q_t S_t,
 *     ht[n,h] = S_{last}
 *
 * with a per-key-dimension log-decay g_t <= 0 and a K x V state.  The library computes it chunkwise: a
 * chunk-local cumsum of g, per-segment state contributions, a decayed scan over segments, and a fused
 * output kernel that adds the inter-chunk term q~ S to the causally masked intra-chunk term.
 *
 * Conventions shared by every entry point
 *   - Layout: time-major with interleaved heads, contiguous, no strides (page
 *     "fla/ops/ttt/fused_chunk.py", fused_chunk_ttt_linear: [B, T, H, K] inputs).
 *       q, k, g : [B, T, H, K]        v, o : [B, T, H, V]        h0, ht : [N, H, K, V] fp32, row-major
 *     (K rows, V columns: the state layout of fused_chunk_gla_fwd_kernel's h0/ht blocks).
 *   - Varlen packing: cu_seqlens != NULL is a DEVICE array of N+1 int32 offsets (page
 *     "fla/ops/ttt/fused_chunk.py", fused_chunk_ttt_linear_fwd_kernel: bos/eos from cu_seqlens); then
 *     B must be 1, T is the packed total and cu_seqlens must run non-decreasing from 0 to T.  Because the
 *     offsets live on the device they are checked there; a violation is reported through
 *     gla_get_status() as GLA_ERR_INVALID_ARG and no output is written.  Zero-length sequences are
 *     allowed (their ht is h0, or 0).  Without cu_seqlens, N must equal B.
 *   - Pointers: every device pointer must be 16-byte aligned (GLA_ERR_ALIGNMENT otherwise).  The
 *     caller owns every buffer, including o, ht and the workspace; the library allocates nothing.
 *     No input may alias an output, except h0 == ht (in-place state streaming), which is allowed.
 *   - Streams: `stream` is a cudaStream_t (NULL = the legacy default stream).  Every call is
 *     stream-ordered and returns once its kernels are enqueued; nothing synchronises the host.
 *   - Errors: synchronous validation returns a gla_status code and enqueues nothing.  Device-side
 *     conditions (bad cu_seqlens, a bounded wait that ran out) are recorded in the workspace's status
 *     word, read with gla_get_status().
 */
#ifndef GLA_H
#define GLA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gla_status {
    GLA_OK = 0,
    GLA_ERR_INVALID_ARG = 1,   /* NULL/negative/inconsistent argument, bad cu_seqlens, bad scale   */
    GLA_ERR_UNSUPPORTED = 2,   /* shape or dtype outside the supported set                          */
    GLA_ERR_ALIGNMENT = 3,     /* a device pointer is not 16-byte aligned                           */
    GLA_ERR_WORKSPACE = 4,     /* workspace NULL or smaller than gla_fwd_workspace_size()           */
    GLA_ERR_CUDA = 5,          /* a CUDA runtime call or kernel launch failed                       */
    GLA_ERR_TIMEOUT = 6,       /* (device) a bounded wait inside a kernel ran out; outputs invalid  */
    GLA_ERR_RANGE = 7          /* (device) a value left the fp16 operand range of the tensor-core
                                  path (see gla_fwd); outputs invalid, use GLA_F32 inputs instead  */
} gla_status;

typedef enum gla_dtype {
    GLA_F32 = 0,        /* q, k, v, g fp32; o fp32                                                  */
    GLA_BF16 = 1,       /* q, k, v, g bf16; o fp32 (default for bf16 inputs, see below)             */
    GLA_BF16_OBF16 = 2, /* q, k, v, g bf16; o bf16 (the pages' o.to(v) convention)                  */
    GLA_F16 = 3,        /* q, k, v, g fp16; o fp32 (same paths and bounds as GLA_BF16)                */
    GLA_BF16_GF32 = 4,  /* q, k, v bf16, g fp32; o fp32 (forward: the tensor-core path for K == 128)  */
    GLA_F16_GF32 = 5,   /* q, k, v fp16, g fp32; o fp32 (as GLA_BF16_GF32)                             */
    GLA_F16_OF16 = 6    /* q, k, v, g fp16; o fp16 (gla_step and the gla_scan_* functions only)        */
} gla_dtype;

/* OR-ed into the dtype argument of gla_fwd / gla_bwd (and their workspace queries): q, k, v, g, o (and the
 * gradients) are head-first [B, H, T, *] instead of [B, T, H, *]; with cu_seqlens (B == 1) that is [1, H, T, *]
 * over the packed rows.  h0 / ht keep [N, H, K, V].  Same paths, kernels and results otherwise. */
#define GLA_HEAD_FIRST 0x100
/* o is fp32 for bf16 inputs by default: at the benchmark magnitudes (|o| up to ~20) a bf16-rounded o
 * alone carries up to 0.06 of rounding error, above the 2e-2 max-abs parity bound.  State h0/ht is fp32
 * for every dtype (fused_chunk_gla_fwd_kernel keeps the state in fp32 and stores ht as fp32). */

/*
 * gla_fwd — GLA forward over a batch (or a varlen pack) of sequences.
 *
 *   q, k, g     [B,T,H,K] input dtype (device).  g is the per-step log-decay (expected <= 0).
 *   v           [B,T,H,V] input dtype (device).
 *   o           [B,T,H,V] output (device), fp32 for GLA_F32 / GLA_BF16, bf16 for GLA_BF16_OBF16.
 *   scale       multiplies q only (prepare_qg_kg); must be finite and > 0.  ht carries no scale.
 *   h0          [N,H,K,V] fp32 initial state (device) or NULL for zeros.  It is decayed by the first
 *               token's gate like any carried state (fused_chunk_gla_fwd_kernel).
 *   ht          [N,H,K,V] fp32 final state (device) or NULL to skip it.  May equal h0.
 *   cu_seqlens  int32 [N+1] device offsets or NULL (dense: N == B sequences of T rows).
 *   chunk       chunk length: 16, 32, 64 or 128.  The result does not depend on it in exact arithmetic;
 *               the kernels tile at 64 rows whatever the value (so it selects no different rounding here).
 *   K           64 or 128.          V  64, 128 or 256.          B, T, H, N >= 0 (T*H*max(K,V) < 2^31).
 *   workspace   device scratch of at least gla_fwd_workspace_size() bytes, 256-byte aligned, ZEROED
 *               BEFORE ITS FIRST USE and not written by the caller afterwards: its 256-byte header carries
 *               the sticky status word, work counters and a launch epoch between calls (the epoch tags
 *               the segment scan's publication flags, so they need no clearing per call).  One workspace
 *               must not be used by two calls that may run concurrently.
 *
 * Paths: 16-bit q, k, v (g 16-bit or fp32) with K == 128 and V in {128, 256} run on the tcgen05 tensor cores
 * with fp16 operands and fp32 accumulation; everything else runs on fp32 CUDA cores.  Valid domain of the tensor-core path
 * (its intra-chunk scores are factorised around an anchor row in the middle of each chunk): every
 * operand it forms must stay inside the fp16 range, i.e. |q|, |k| * exp(gate sum over up to half a chunk)
 * below 65000, |v| < 65000, |state| < 65000 and intra-chunk scores below 65000 in magnitude; the kernels
 * check this and report GLA_ERR_RANGE through gla_get_status() otherwise.  The fp32 path's domain is the
 * fp32 range of the same factorisation (gate sums over half a chunk above about -80).
 * Returns GLA_OK once enqueued, else a synchronous gla_status.
 */
int gla_fwd(const void *q, const void *k, const void *v, const void *g, void *o, float scale,
            const float *h0, float *ht, const int32_t *cu_seqlens, int N, int B, int T, int H,
            int K, int V, int chunk, int dtype, void *workspace, size_t workspace_bytes,
            void *stream);

/*
 * Bytes of device workspace gla_fwd needs for this problem on the CURRENT device (the segment plan
 * depends on its SM count).  Returns 0 for arguments gla_fwd would reject.  Never fails otherwise.
 */
size_t gla_fwd_workspace_size(int B, int T, int H, int K, int V, int N, int chunk, int dtype);

/*
 * Synchronises `stream`, then returns and clears the sticky device status word of `workspace`
 * (GLA_OK if no enqueued call since the last read reported a device-side error).  Returns
 * GLA_ERR_CUDA if the synchronisation itself failed, GLA_ERR_INVALID_ARG for a NULL workspace.
 */
int gla_get_status(void *workspace, void *stream);

/* Static description of a gla_status code (never NULL). */
const char *gla_strerror(int code);

/*
 * gla_chunk_local_cumsum — the chunk-local inclusive cumsum of the log-decay as a standalone pass
 * (FusedChunkGLAFunction.forward computes it in fp32 before everything else):
 *     G[t] = sum of g[u] for u from the first row of t's chunk to t,
 * chunks of `chunk` rows starting at every sequence start (cu_seqlens, or every T rows when NULL).
 * g [B,T,H,K] in the input dtype (GLA_F32 or GLA_BF16), G [B,T,H,K] fp32, both device.  gla_fwd does
 * not call this: its kernels form the same sums on chip.  Device-side cu_seqlens errors are not
 * checked here (pass valid offsets).  chunk in {16, 32, 64, 128}.
 */
int gla_chunk_local_cumsum(const void *g, float *G, const int32_t *cu_seqlens, int N, int B, int T,
                           int H, int K, int chunk, int dtype, void *stream);

/*
 * gla_fwd_noalloc — gla_fwd without a caller-provided workspace, for callers that cannot allocate device
 * memory: host runtimes that own every device byte through their own pool and forbid other allocations
 * once running, or call paths that must not risk an allocation failure or the device-wide
 * synchronisation a cudaMalloc can cause.  It has no counterpart on the pages.
 *
 * Arguments, layouts, results and synchronous errors are those of gla_fwd.  The scratch comes from one
 * 32 MiB device array inside the library (held by every device that loads it, until exit); problems whose
 * gla_fwd_workspace_size() exceeds 32 MiB are rejected with GLA_ERR_WORKSPACE before anything is enqueued.
 * The array's device address is looked up (cudaGetSymbolAddress) with the device current on the first call
 * in each context, i.e. on the first call on a device and again after a device reset; make such a call
 * before any stream capture.  Nothing is allocated: no cudaMalloc, cudaFree or allocating library routine
 * is called, and the call enqueues only the gla_fwd kernels.  All calls share the one array, which keeps
 * the previous call's contents, so calls that may overlap on the GPU (different streams without ordering)
 * race on it and must not be made.  Device-side conditions (bad cu_seqlens, GLA_ERR_RANGE,
 * GLA_ERR_TIMEOUT) go to a status word inside the array that cannot be read back; callers that need them
 * use gla_fwd with a workspace.
 */
int gla_fwd_noalloc(const void *q, const void *k, const void *v, const void *g, void *o, float scale,
                    const float *h0, float *ht, const int32_t *cu_seqlens, int N, int B, int T, int H,
                    int K, int V, int chunk, int dtype, void *stream);

/*
 * gla_fwd_host — gla_fwd on inputs and outputs in HOST memory (a serving path whose requests arrive in host
 * memory).  It has no counterpart on the pages: the result is gla_fwd's, computed head group by head group.
 *
 * q, k, g [rows, H, K], v [rows, H, V], o [rows, H, V], h0 / ht [N, H, K, V] (fp32, each may be NULL) and
 * cu_seqlens [N + 1] (int32 or NULL) are host pointers, time-major (GLA_HEAD_FIRST is rejected with
 * GLA_ERR_UNSUPPORTED); page-locked host memory lets the copies run asynchronously and at full speed, other
 * host memory works but is copied through staging.  The other arguments are gla_fwd's.  The H heads are
 * processed in head_groups groups of H / head_groups heads (H must be a multiple of it, else
 * GLA_ERR_INVALID_ARG): while one group's kernels run, the next group's inputs are copied to the device and
 * the previous group's o (and ht) copied back, so a call takes about the time of its larger copy direction.
 * Each group runs gla_fwd with H / head_groups heads; its segment plan can differ from that of one call with
 * all H heads, so the two results agree within the arithmetic's rounding, not bit for bit.
 *
 * workspace: device memory of at least gla_fwd_host_workspace_size() bytes, 256-byte aligned, zeroed before
 * its first use (it holds gla_fwd's workspace for one group, a copy of cu_seqlens and up to three groups'
 * device buffers); gla_get_status() reads its status word.  Calls that share a workspace must be ordered on
 * the GPU (for example on one stream).  The call enqueues everything on `stream` and on two side streams of
 * its own (created on the first call from each host thread on each device, with their events, and kept until
 * exit), joined back into `stream`: the host buffers may be read or reused once `stream` has reached that
 * point.  Returns GLA_OK once enqueued, else a synchronous gla_status (GLA_ERR_WORKSPACE for a missing or
 * small workspace, GLA_ERR_CUDA if an enqueue failed; work already enqueued then still runs).
 */
int gla_fwd_host(const void *q, const void *k, const void *v, const void *g, void *o, float scale,
                 const float *h0, float *ht, const int32_t *cu_seqlens, int N, int B, int T, int H, int K,
                 int V, int chunk, int dtype, int head_groups, void *workspace, size_t workspace_bytes,
                 void *stream);

/* Bytes of device workspace gla_fwd_host needs (0 for arguments it would reject). */
size_t gla_fwd_host_workspace_size(int B, int T, int H, int K, int V, int N, int chunk, int dtype,
                                   int head_groups);

/*
 * gla_bwd — gradients of the forward above (page "fla/ops/gla/fused_chunk.py": fused_chunk_gla_bwd_kernel,
 * bwd_inner_chunk, FusedChunkGLAFunction.backward) for the loss L = sum(o * dout) + sum(ht * dht):
 *
 *   dq = dL/dq, dk = dL/dk, dg = dL/dg   [rows, H, K] fp32 (device, written)
 *   dv = dL/dv                           [rows, H, V] fp32 (device, written)
 *   dh0 = dL/dh0                         [N, H, K, V] fp32 (device) or NULL to skip it
 *
 * q, k, v, g, scale, h0, cu_seqlens, N, B, T, H, chunk: as for gla_fwd (the forward is recomputed; pass the
 * same h0 the forward used, or NULL for a zero initial state).  dout [rows, H, V] in the input dtype (the
 * gradient of o); dht [N, H, K, V] fp32 or NULL (no loss on the final state).  dtype GLA_F32 (every input
 * fp32), GLA_BF16 (q, k, v, g, dout bf16), GLA_F16, GLA_BF16_GF32 or GLA_F16_GF32 (fp32 g), optionally OR-ed
 * with GLA_HEAD_FIRST.  Arithmetic is fp32: for bf16 inputs with K == 128 the per-chunk sums and the per-chunk
 * gradients run on the tcgen05 tensor cores (fp32 operands split exactly into three bf16 terms, fp32
 * accumulation), every other step on CUDA cores.  K in {64, 128}, V in {64, 128, 256} (V = 256 runs as two
 * 128-wide value slices: dq, dk and dg are accumulated over them); chunk 16, 32, 64 or 128 (tiled at 64 rows,
 * as for gla_fwd).  workspace: at least gla_bwd_workspace_size() bytes, 256-byte aligned, zeroed before its
 * first use (status word in its first bytes); it holds the chunk-start states and chunk-end adjoints of one
 * value slice (2 * chunks * H * K * min(V, 128) fp32).  Outputs must not overlap any input, the workspace or one another.  The
 * library allocates nothing and is stream-ordered.  Errors as for gla_fwd (GLA_ERR_UNSUPPORTED for other
 * dtypes or head sizes); valid domain: the fp32 range of the same mid-chunk factorisation as the fp32
 * forward path.  Returns GLA_OK once enqueued.
 */
int gla_bwd(const void *q, const void *k, const void *v, const void *g, const void *dout, float scale,
            const float *h0, const float *dht, float *dq, float *dk, float *dv, float *dg, float *dh0,
            const int32_t *cu_seqlens, int N, int B, int T, int H, int K, int V, int chunk, int dtype,
            void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of device workspace gla_bwd needs for this problem (0 for an unsupported shape). */
size_t gla_bwd_workspace_size(int B, int T, int H, int K, int V, int N, int chunk, int dtype);

/*
 * gla_ttt_linear_fwd — TTT-linear forward, the second workload of the same chunked-state machinery (page
 * "fla/ops/ttt/fused_chunk.py": fused_chunk_ttt_linear_fwd_kernel, then the norm_residual step of
 * fused_chunk_ttt_linear).  Per (sequence, head) an inner model h [D][D], hb [D] takes one gradient step of
 * 1/2 |LN(k h + hb) * w + b + k - v|^2 per mini-batch of `chunk` rows (the result depends on `chunk`), and
 * o_i = scale q_i h_i + hb_i (dual form, rows up to i of the mini-batch), followed by o += LN(o) * w + b.
 *
 *   q, k, v     [rows, H, D] device, fp32 / bf16 / fp16 by dtype (GLA_F32, GLA_BF16, GLA_F16); K == V == D
 *   w, b        [H, D] fp32 LayerNorm weight and bias;  eta [rows, H] fp32 per-token learning rate
 *   scale > 0, eps > 0;  h0 [N, H, D, D], hb0 [N, H, D] fp32 or NULL (zeros)
 *   o           [rows, H, D] fp32 (written);  ht [N, H, D, D], hbt [N, H, D] fp32 or NULL
 *   cu_seqlens  int32 [N+1] device offsets or NULL (as gla_fwd);  D in {64, 128};  chunk in {16, 32}
 *   workspace   gla_ttt_workspace_size() bytes, 256-byte aligned, zeroed before first use (status word:
 *               bad cu_seqlens are reported there, read it with gla_get_status; those sequences are skipped)
 *
 * Rows past the end of a sequence take no part in the last mini-batch (the page's kernel adds its zero-padded
 * rows to the hb update).  fp32 CUDA cores, one thread-block cluster of D / 16 CTAs per (sequence, head).
 * Errors as for gla_fwd; a bounded wait inside the kernel that ran out is reported as GLA_ERR_TIMEOUT in
 * the status word (the outputs of that call are then void).
 */
int gla_ttt_linear_fwd(const void *q, const void *k, const void *v, const float *w, const float *b,
                       const float *eta, float scale, float eps, const float *h0, const float *hb0, float *o,
                       float *ht, float *hbt, const int32_t *cu_seqlens, int N, int B, int T, int H, int D,
                       int chunk, int dtype, void *workspace, size_t workspace_bytes, void *stream);
size_t gla_ttt_workspace_size(void);

/*
 * Measurement hook (no counterpart on the pages; it exists so a benchmark can time each kernel of the
 * path with CUDA events on the stream the kernels run on).  While `events` is non-NULL, every later
 * gla_fwd / gla_bwd call made from this host thread records events[2i] right before and events[2i+1] right after
 * its i-th kernel launch (for i < n_events / 2), on the call's stream, and stores that launch's kernel id
 * in kernel_ids[i] (host array of n_events / 2 ints, may be NULL).  `events` are cudaEvent_t handles
 * created by the caller.  Pass events == NULL to stop.  Returns GLA_OK, or GLA_ERR_INVALID_ARG for
 * n_events < 0.  gla_profile_launches() returns how many kernels the last gla_fwd / gla_bwd call on this
 * thread launched, and gla_kernel_name() names a kernel id.
 */
int gla_profile_events(void **events, int n_events, int *kernel_ids);
int gla_profile_launches(void);
const char *gla_kernel_name(int kernel_id);

/*
 * gla_wy_fwd — WY representation forward of the gated delta rule, a third chunked workload (page
 * "fla/ops/gated_delta_rule/backends/triton_ascend/wy_fast.py": recompute_w_u_fwd_kernel_npu and its launcher
 * recompute_w_u_fwd_npu).  Each sequence is cut into chunks of `chunk` rows from its first row (the last one
 * may be partial).  For value head hv, whose key head is hv / (HV / H), and row t of chunk [c0, c1):
 *
 *   u_t = sum_{s in [c0, c1)} A_t[s - c0] beta_s v_s,   w_t = sum_{s in [c0, c1)} A_t[s - c0] beta_s 2^{g_s} k_s
 *
 *   k      [rows, H, K] device, input dtype          v     [rows, HV, V] device, input dtype
 *   beta   [rows, HV]   device, input dtype          A     [rows, HV, chunk] device, input dtype: row t holds
 *                                                           row t - c0 of its chunk's matrix (full square)
 *   g      [rows, HV] fp32 log2-domain gate (the factor is 2^g) or NULL (factor 1)
 *   w      [rows, HV, K], u [rows, HV, V] device, written: fp32, or bf16 for GLA_BF16_OBF16
 *   rows = B * T (dense) or the packed length T (varlen: cu_seqlens int32 [N+1] on the device, B == 1,
 *   cu_seqlens[N] == T; bad offsets are reported in the status word and no row is written)
 *   dtype  GLA_F32, GLA_BF16 (fp32 outputs), GLA_BF16_OBF16 or GLA_F16 (fp32 outputs);  K, V in {64, 128};
 *   HV a multiple of H;  chunk in {16, 32, 64}
 *   workspace  at least gla_wy_workspace_size(T, N, chunk) bytes, 256-byte aligned, zeroed before its first
 *              use (status word, then the varlen chunk table)
 *
 * Rows past the end of a sequence do not exist: the columns of A that would refer to them are not read.
 * bf16 inputs with K == V in {64, 128} run on the tcgen05 tensor cores (the fp32 operand k * beta * 2^g |
 * v * beta split into three bf16 terms, A as it is stored, fp32 accumulation; a bounded wait inside reports
 * GLA_ERR_TIMEOUT in the status word); everything else on fp32 CUDA cores.  Outputs must not overlap any
 * input, the workspace or each other.  Errors as for gla_fwd; returns GLA_OK once enqueued.
 */
int gla_wy_fwd(const void *k, const void *v, const void *beta, const void *A, const float *g, void *w, void *u,
               const int32_t *cu_seqlens, int N, int B, int T, int H, int HV, int K, int V, int chunk, int dtype,
               void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of device workspace gla_wy_fwd needs (dense batches: N is ignored). */
size_t gla_wy_workspace_size(int T, int N, int chunk, int varlen);

/* ---------------------------------------------------------------------------------------------------------
 * Operators beside the chunkwise kernels in a model: a gated linear recurrence with a vector state (forward,
 * backward, one token), the GLA state update for one token, and the root-mean-square norm with the residual's
 * addition.  They have no counterpart on the pages.  The conventions at the top of this file hold (16-byte
 * aligned device pointers, caller-owned memory, stream order, synchronous argument checks), except that row
 * counts and sizes may exceed 2^31 elements.  Sums, states and norms are held in fp32 whatever the input types.
 * ------------------------------------------------------------------------------------------------------ */

/*
 * gla_scan_fwd — gated linear recurrence with a vector state.  Per sequence n and channel d,
 *
 *     h_t = exp(g_t) h_{t-1} + x_t,   h_0 = h0[n] (or 0),   ht[n] = h_last
 *
 *   x, g        [rows, D] device; rows = B * T (dense) or the packed length T (cu_seqlens, B == 1).  Row r starts
 *               at r * ldx (ldg) elements, so x and g may be column ranges of one projection's output
 *   h           [rows, D] device, contiguous, written
 *   h0, ht      [N, D] fp32 device or NULL; ht may equal h0.  A sequence of length zero has ht = h0 (or 0)
 *   D >= 1, ldx >= D, ldg >= D (odd sizes and strides are fine; rows of 16-byte multiples are fastest)
 *   dtype       types of (x, g, h): GLA_F32 (f32, f32, f32), GLA_BF16 (bf16, bf16, f32), GLA_BF16_OBF16 (bf16, bf16,
 *               bf16), GLA_F16 (f16, f16, f32), GLA_F16_OF16 (f16, f16, f16), GLA_BF16_GF32 (bf16, f32, f32),
 *               GLA_F16_GF32 (f16, f32, f32)
 *   workspace   gla_scan_workspace_size() bytes, 256-byte aligned, zeroed before first use: the status word.  A
 *               sequence with bad offsets (cu_seqlens must run from 0 to T without decreasing) is reported there
 *               (gla_get_status) and skipped; a bounded wait that ran out is reported as GLA_ERR_TIMEOUT (the
 *               outputs of that call are then void)
 *
 * g is usually <= 0 but may be any value whose exponential is an fp32 number.  The recurrence is evaluated as written,
 * also where sums of gates leave an exponential's range and come back: h_t is the sum of its rows' shares
 * exp(g_{s+1} + .. + g_t) x_s, and as long as none of them passes fp32's largest value on the way, h_t is right to the
 * roundings of that sum (a share that falls below fp32's normal numbers on the way may count as 0).  Once one has, what
 * follows in that channel is void (infinite, NaN, or finite again where the gates fall).  Infinities and NaN of the inputs spread as they would step by step, except that a segment's total decay
 * multiplies the state that enters it: a state of infinity becomes NaN where that decay is below 2^-252.
 * A decay is within (2^-22 + |g| 2^-24) exp(g) + 2^-126 of exp(g): subnormal decays are 0.  The total decay of up to 16
 * rows is the exponential of the fp32 sum of their gates.
 * Results do not depend on timing (no atomics).
 */
int gla_scan_fwd(const void *x, const void *g, void *h, const float *h0, float *ht, const int32_t *cu_seqlens, int N,
                 int B, int T, int D, int64_t ldx, int64_t ldg, int dtype, void *workspace, size_t workspace_bytes,
                 void *stream);

/*
 * gla_scan_bwd — gradients of gla_scan_fwd for L = sum(h * dh) + sum(ht * dht), from the forward's gate and output:
 *
 *     lam_t = dh_t + mu_{t+1},   mu_t = exp(g_t) lam_t,   mu_{last+1} = dht (or 0)
 *     dx_t = lam_t,   dg_t = mu_t h_{t-1},   dh0 = mu_1
 *
 *   g, h        as the forward read and wrote them (dg carries h's rounding);  dh [rows, D] contiguous, h's type
 *   h0, dht     [N, D] fp32 or NULL (zeros);  dh0 [N, D] fp32 or NULL to skip it
 *   dx, dg      written, the types of x and g; row r at r * lddx (lddg) elements, so both may be column ranges of
 *               one gradient
 * The rest as for gla_scan_fwd.  Outputs must not overlap any input or one another.
 */
int gla_scan_bwd(const void *g, const void *h, const void *dh, const float *h0, const float *dht, void *dx, void *dg,
                 float *dh0, const int32_t *cu_seqlens, int N, int B, int T, int D, int64_t ldg, int64_t lddx,
                 int64_t lddg, int dtype, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of device workspace gla_scan_fwd, gla_scan_bwd, gla_scan_step and gla_step need (the status word). */
size_t gla_scan_workspace_size(void);

/* Such a workspace on the CURRENT device that the library itself holds (static device memory, zero when it is loaded), for
 * callers that keep none; NULL without a device.  May be asked for during a stream capture.  All its users share the
 * status word, whatever their streams and threads: gla_get_status then tells that one of their calls since the last look
 * failed, not which. */
void *gla_scan_shared_workspace(void);

/*
 * gla_scan_step — one token of the recurrence above for each of B sequences, with the states in a pool:
 *
 *     s = slots ? slots[b] : b,   ht[s] = exp(g_b) h0[s] + x_b,   h_b = ht[s] rounded to h's type
 *
 *   x, g        [B, D], row strides ldx, ldg;   h [B, D] contiguous, written
 *   h0, ht      [S, D] fp32 state pools; ht may equal h0 (update in place).  Only the addressed rows are written
 *   slots       int32 [B] device or NULL (then S == B).  A slot of -1 marks an idle sequence: its h is zeros and no
 *               state is read or written.  Any other slot outside [0, S) is treated the same and reported in the
 *               status word as GLA_ERR_INVALID_ARG.  Two sequences must not share a slot
 *   dtype, workspace as for gla_scan_fwd
 */
int gla_scan_step(const void *x, const void *g, void *h, const float *h0, float *ht, const int32_t *slots, int B,
                  int S, int D, int64_t ldx, int64_t ldg, int dtype, void *workspace, size_t workspace_bytes,
                  void *stream);

/*
 * gla_step — one token of the GLA recurrence (gla_fwd) for each of B sequences, with the states in a pool:
 *
 *     s = slots ? slots[b] : b,   ht[s] = diag(exp g_b) h0[s] + k_b^T v_b,   o_b = scale * q_b ht[s]
 *
 *   q, k, g     [B, H, K],  v [B, H, V] device, contiguous;  o [B, H, V] device, written
 *   h0, ht      [S, H, K, V] fp32 state pools; ht may equal h0 (update in place)
 *   slots       as for gla_scan_step (an idle sequence's o is zeros)
 *   K in {64, 128}, V in {64, 128, 256};  scale finite and > 0
 *   dtype       types of (q, k, v; g; o), as the types of (x, g, h) of gla_scan_fwd
 *   workspace   as for gla_scan_fwd
 */
int gla_step(const void *q, const void *k, const void *v, const void *g, void *o, float scale, const float *h0,
             float *ht, const int32_t *slots, int B, int S, int H, int K, int V, int dtype, void *workspace,
             size_t workspace_bytes, void *stream);

/* OR-ed into the dtype argument of the gla_norm_* functions: the residual stream (res, s and its gradients) is fp32
 * whatever the type of x and y. */
#define GLA_RES_F32 0x200

/*
 * gla_norm_fwd — residual addition and root-mean-square norm of each row:
 *
 *     s = x + res,   rstd = 1 / sqrt(mean(s^2) + eps),   y = s * rstd * w
 *
 *   x, y        [rows, D] device, fp32 / bf16 / fp16 by dtype (GLA_F32, GLA_BF16, GLA_F16)
 *   res, s      [rows, D] device, x's type (fp32 with GLA_RES_F32).  res may be NULL (s = x); s may be NULL to skip
 *               it, and may equal res (update in place).  The norm takes s before its rounding to the stored type
 *   w           [D] fp32 or NULL (ones);   rstd [rows] fp32 or NULL to skip it (the backward needs it)
 *   1 <= D <= 16384,  eps finite and >= 0.  A row with a NaN has NaN everywhere; rows are independent
 */
int gla_norm_fwd(const void *x, const void *res, const float *w, void *y, void *s, float *rstd, int64_t rows, int D,
                 float eps, int dtype, void *stream);

/*
 * gla_norm_quant_fwd — gla_norm_fwd with y in 8 bits (e4m3) and fp32 scales, for a product with 8-bit operands:
 *
 *     scale = max(max |y| / 448, 1e-30) over each group of columns,   q = e4m3(y / scale)  (to nearest, ties to even)
 *
 *   q           [rows, D] device, written.  y is not rounded in between; the scale is max |y| times the fp32 value of
 *               1 / 448, and the quotient y times the scale's fp32 reciprocal (one unit in the last place): each within
 *               2^-22 of the exact one, so that a y next to a tie may take the code on its other side
 *   scales      [rows, ceil(D / group)] fp32 device, written (the last group may be partial)
 *   group       0 (one scale per row) or 128
 * The rest as for gla_norm_fwd.  A NaN makes its row's values and scales NaN.
 */
int gla_norm_quant_fwd(const void *x, const void *res, const float *w, void *q, float *scales, void *s, float *rstd,
                       int64_t rows, int D, float eps, int group, int dtype, void *stream);

/*
 * gla_norm_bwd — gradients of gla_norm_fwd for upstream gradients dy of y and ds of the written s:
 *
 *     n = s * rstd,   grad = rstd * (w dy - n mean(w dy n)) + ds,   dw = sum over rows of dy n
 *
 *   s, rstd     as the forward wrote them (s = x where res was NULL);  dy [rows, D], x's type
 *   ds          [rows, D], s's type, or NULL (zeros)
 *   dx          [rows, D] grad in x's type, dres [rows, D] grad in s's type; either may be NULL, not both.  Without
 *               GLA_RES_F32 the two types are the same: pass one of them.  dres may equal ds, dx may equal dy
 *   dw          [D] fp32 or NULL to skip it
 *   workspace   gla_norm_bwd_workspace_size() bytes, 256-byte aligned (no zeroing): partial sums of dw, added in a
 *               fixed order, so that results do not depend on timing
 */
int gla_norm_bwd(const void *s, const float *rstd, const float *w, const void *dy, const void *ds, void *dx, void *dres,
                 float *dw, int64_t rows, int D, int dtype, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of device workspace gla_norm_bwd needs on the CURRENT device (0 for a D it would reject). */
size_t gla_norm_bwd_workspace_size(int64_t rows, int D);

#ifdef __cplusplus
}
#endif
#endif /* GLA_H */
