/*
 * kda.h -- C ABI of the GB300 (sm_103a) KDA recurrence library, libkda_gb300.so.
 *
 * KDA (Kimi Delta Attention) keeps, per head, a dk x dv fp32 state S and for
 * every token t applies the per-channel gated delta rule
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(exp(g_t)) S_{t-1} + beta_t k_t v_t^T
 *     o_t = S_t^T q_t                      (read out from the UPDATED state)
 *
 * Defined by: "Colibri Kimi K3 Metal backend" (architecture section, the
 * state update; section 8.2, the two-pass token step and its readout;
 * section 8.4, alpha = exp(g) per element and beta per head), with the model
 * sizes of "Kimi K3 -> TPU v7x feasibility" (section 2 model table: 96 heads,
 * head width 128, decay gate lower bound -5).
 *
 * Conventions shared by every call
 *   - Pointers are DEVICE pointers unless marked "host"; the caller owns all
 *     memory it passes.  The tensor-core prefill (bf16, chunk 64) also needs
 *     a scratch workspace of 59 KB per (64-token chunk, head):
 *     kda_prefill_chunked takes it from a library-owned stream-ordered memory
 *     pool on the current device, which keeps that memory for later calls;
 *     kda_prefill_chunked_ws runs in a buffer the caller passes, and
 *     kda_prefill_chunked_noalloc in a fixed array in the library's device
 *     image.  That pool, that array and the device error word
 *     (kda_device_error) are the library's only global state.
 *   - Layouts are token-major and dense (C order):
 *         q, k, g : [T, H, dk]      v, o : [T, H, dv]      beta : [T, H]
 *         S       : [N, H, dk, dv]  with S[n][h][i][j], i = key channel,
 *                                   j = value channel (the pages' S[i][j],
 *                                   decayed per row i)
 *   - q, k, v are bf16 (KDA_BF16) or fp32 (KDA_F32); g, beta, S and o are
 *     always fp32.  g is the log-decay (decay = exp(g)); beta is already in
 *     [0, 1] (any sigmoid is applied by the caller); q is used as given (any
 *     1/sqrt(dk) scale is folded in by the caller).
 *   - Supported sizes: dk = dv = 128.  Preconditions: -5 <= g <= 0 (the
 *     model's gate bound; the tensor-core prefill's decay folding relies on
 *     it and raises bit 2 of the device error word when it sees a gate
 *     outside that range, or a NaN, in a prefill's input); for the
 *     tensor-core prefill, |q| |k| and |v| far below 65504 (q and k are
 *     L2-normalised in the model, as the layer's prologue makes them; u is
 *     checked, bit 4 below); finite inputs (not checked elsewhere).
 *   - Every pointer must be 16-byte aligned (KDA_ERR_ALIGN otherwise).
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream); they never synchronise.  Arguments are validated on
 *     the host before any launch; on an argument error nothing is launched.
 *     A launch failure is reported as KDA_ERR_CUDA.  Calls never throw.
 */
#ifndef KDA_GB300_H
#define KDA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_NULL = 1,        /* a required pointer is NULL */
    KDA_ERR_DIM = 2,         /* unsupported or inconsistent sizes */
    KDA_ERR_CHUNK = 3,       /* chunk not in {16, 32, 64} */
    KDA_ERR_ALIGN = 4,       /* a pointer is not 16-byte aligned */
    KDA_ERR_DTYPE = 5,       /* dtype not a kda_dtype_t */
    KDA_ERR_WORKSPACE = 6,   /* the prefill's scratch workspace could not be allocated, or the caller's is too small */
    KDA_ERR_CUDA = 7,        /* the CUDA runtime reported an error at launch */
    KDA_ERR_VALUE = 8        /* a scalar argument is out of range, or buffers alias */
} kda_status_t;

typedef enum {
    KDA_BF16 = 0,            /* q, k, v stored as bfloat16 */
    KDA_F32 = 1              /* q, k, v stored as float32 */
} kda_dtype_t;

/* Library version, major * 10000 + minor * 100 + patch. */
int kda_version(void);

/* Static string naming a status code (never NULL). */
const char *kda_status_string(int status);

/*
 * Chunked prefill over a packed batch of N variable-length sequences.
 *
 * Operation: for every sequence n (tokens cu_seqlens[n] .. cu_seqlens[n+1]-1)
 * and head h, run the recurrence above from S0[n][h] (zeros if S0 == NULL),
 * write o for each token and the final state to S_out[n][h].  The chunked
 * form (chunks of `chunk` tokens, UT transform inside a chunk, fp32 state
 * carried between chunks) computes the same map up to rounding; it follows
 * from unrolling the recurrence inside a chunk.  The varlen packing follows
 * the per-sequence (cu_seqlens) convention of the TPU KDA kernel ("Kimi K3
 * -> TPU v7x feasibility", section 4.2).  Sequences of any length (including
 * 0, and lengths that are not a multiple of `chunk`) are handled in the
 * kernel; an empty sequence copies S0 (or zeros) to S_out.
 *
 *   q, k       [T, H, dk]  bf16 or fp32 (dtype)
 *   v          [T, H, dv]  bf16 or fp32
 *   g          [T, H, dk]  fp32 log-decay
 *   beta       [T, H]      fp32
 *   S0         [N, H, dk, dv] fp32, or NULL for a zero initial state
 *   o          [T, H, dv]  fp32, written
 *   S_out      [N, H, dk, dv] fp32, written; may alias S0 exactly (in place)
 *   cu_seqlens [N + 1]     int32 DEVICE array, cu_seqlens[0] = 0,
 *                          non-decreasing, cu_seqlens[N] = T.  The host
 *                          cannot read it; the kernels check it on the
 *                          device: entries below 0, above T or decreasing
 *                          raise bit 0 of the device error word, and no
 *                          kernel then reads or writes outside the buffers
 *                          sized for T (the outputs are invalid)
 *   N          number of sequences (>= 1); T total tokens (>= 0, < 2^31)
 *   H          heads (>= 1); dk, dv must be 128
 *   chunk      16, 32 or 64.  bf16 inputs with chunk 64 run on the
 *              tensor cores (tcgen05, TMA) in two kernels: an intra-chunk
 *              kernel over every (chunk, head) at once, then an inter-chunk
 *              state pass per (sequence, head); every other combination runs
 *              the fp32 CUDA-core kernel.
 *   dtype      kda_dtype_t of q, k, v
 *   stream     cudaStream_t
 * Returns KDA_OK or a kda_status_t (KDA_ERR_WORKSPACE when the tensor-core
 * path cannot get its workspace).  With T == 0 only S_out is written.
 */
int kda_prefill_chunked(const void *q, const void *k, const void *v,
                        const float *g, const float *beta, const float *S0,
                        float *o, float *S_out, const int32_t *cu_seqlens,
                        int N, int64_t T, int H, int dk, int dv, int chunk,
                        int dtype, void *stream);

/*
 * Measurement form of kda_prefill_chunked for the tensor-core path (bf16,
 * chunk 64, T > 0; KDA_ERR_CHUNK otherwise): the same computation, and it
 * records the caller's four timing events (cudaEvent_t, created by the
 * caller) on `stream` before the chunk-plan kernel, before the intra-chunk
 * kernel, before the state pass and after it, so that each kernel's time can
 * be read with cudaEventElapsedTime.  events: host array of 4 cudaEvent_t.
 */
int kda_prefill_chunked_events(const void *q, const void *k, const void *v,
                               const float *g, const float *beta, const float *S0,
                               float *o, float *S_out, const int32_t *cu_seqlens,
                               int N, int64_t T, int H, int dk, int dv, int chunk,
                               int dtype, void *stream, void *const *events);

/*
 * kda_prefill_chunked without any device allocation during the call.
 *
 * Same operation, arguments, layouts and results as kda_prefill_chunked.
 * The recurrence itself has no such variant (the pages describe no
 * workspace at all); this entry point exists for callers that may not
 * allocate device memory inside a call: runtimes that budget all device
 * memory in a fixed arena up front, where a library pool growing mid-call
 * would break the budget, and latency-critical loops where the first growth
 * of a pool (a driver allocation, which synchronises the device) cannot be
 * afforded.
 *
 * The tensor-core path (bf16, chunk 64, T > 0) takes its workspace from a
 * fixed 64 MiB array in the library's device image instead of the pool.  It
 * needs kda_prefill_workspace_bytes(N, T, H, ...) bytes (about
 * (ceil(T / 64) + N) * H * 60416); larger inputs are rejected with KDA_ERR_WORKSPACE before anything
 * is launched (for H = 96 and one sequence: T <= 640).  Every other dtype /
 * chunk combination runs the CUDA-core kernel, which needs no workspace.
 * Nothing in the array has to be cleared between calls.
 *
 * First call on each device: the library looks up the array's address
 * (cudaGetSymbolAddress, which may load the library's device image); make
 * that first call before any stream capture begins.  The address is cached
 * with the identity of the device's context; after a cudaDeviceReset the
 * next call looks it up again (so that call, too, should come before any
 * capture).  The array is shared by
 * all calls on a device: two calls whose executions overlap (different
 * streams, or different host threads) race on it and must be serialised by
 * the caller.  Returns KDA_OK or a kda_status_t.
 */
int kda_prefill_chunked_noalloc(const void *q, const void *k, const void *v,
                                const float *g, const float *beta, const float *S0,
                                float *o, float *S_out, const int32_t *cu_seqlens,
                                int N, int64_t T, int H, int dk, int dv, int chunk,
                                int dtype, void *stream);

/*
 * Bytes of caller-owned workspace that kda_prefill_chunked_ws needs for these
 * sizes on the tensor-core path (bf16, chunk 64, T > 0): with
 * C = ceil(T / 64) + N chunks (one spare per sequence for a partial tail),
 * 1024 * ceil(4 (N + 2) / 1024) + 1024 * ceil(8 C / 1024) + C * H * 60416
 * (the chunk offsets and a job counter, the chunk table, one record per
 * (chunk, head)); 0 for
 * every other combination (the CUDA-core kernel needs none) and for invalid sizes.
 * Host-only, no CUDA call.
 */
size_t kda_prefill_workspace_bytes(int N, int64_t T, int H, int dk, int dv, int chunk, int dtype);

/*
 * kda_prefill_chunked with a workspace the caller owns (for instance a
 * buffer from the caller's own allocator), so that the library allocates
 * nothing.  Same operation, arguments, layouts and results as
 * kda_prefill_chunked, plus:
 *   workspace  device memory of ws_bytes bytes, 256-byte aligned
 *              (KDA_ERR_ALIGN otherwise), read and written by the call's
 *              kernels on `stream` (the caller keeps it alive and unshared
 *              until they finish); NULL is accepted where
 *              kda_prefill_workspace_bytes gives 0
 *   ws_bytes   at least kda_prefill_workspace_bytes(...) (KDA_ERR_WORKSPACE
 *              otherwise, before anything is launched)
 * Nothing in the workspace has to be initialised or cleared between calls.
 * Returns KDA_OK or a kda_status_t.
 */
int kda_prefill_chunked_ws(const void *q, const void *k, const void *v,
                           const float *g, const float *beta, const float *S0,
                           float *o, float *S_out, const int32_t *cu_seqlens,
                           int N, int64_t T, int H, int dk, int dv, int chunk,
                           int dtype, void *workspace, size_t ws_bytes, void *stream);

/*
 * One decode token for each of B sequences, state updated IN PLACE.
 *
 * Operation: the recurrence above applied once per (b, h) with
 * S = S_inout[b][h]: decay the rows by exp(g), u = S^T k, w = beta (v - u),
 * S += k w^T, o = S^T q (the two passes of "Colibri Kimi K3 Metal backend",
 * section 8.2, fused into one kernel that reads and writes each state once).
 *
 *   q, k      [B, H, dk]  bf16 or fp32 (dtype)
 *   v         [B, H, dv]  bf16 or fp32
 *   g         [B, H, dk]  fp32 log-decay
 *   beta      [B, H]      fp32
 *   S_inout   [B, H, dk, dv] fp32, read and overwritten in place
 *   o         [B, H, dv]  fp32, written (must not alias S_inout)
 *   B, H      >= 1 (B = 0 is a no-op returning KDA_OK); dk, dv must be 128
 * Returns KDA_OK or a kda_status_t.
 */
int kda_decode_step(const void *q, const void *k, const void *v,
                    const float *g, const float *beta, float *S_inout, float *o,
                    int B, int H, int dk, int dv, int dtype, void *stream);

/*
 * One decode token for each of B sequences whose states live in a pool:
 * sequence b reads and updates pool row state_indices[b] in place (the
 * decode-side interface of continuous batching: the TPU KDA decode kernel
 * indexes its state the same way, "Kimi K3 -> TPU v7x feasibility", section
 * 4.2), and the pool may be stored in bf16 to halve the state traffic (the
 * pages list a bf16 state as not yet evaluated for stability, same review,
 * section 6; the recurrence is computed in fp32 and each state value is
 * rounded to nearest-even bf16 when it is stored).
 *
 *   q, k, v, g, beta, o   as for kda_decode_step ([B, H, ...])
 *   S_pool        [P, H, dk, dv], fp32 (state_dtype KDA_F32) or bf16
 *                 (KDA_BF16), read and overwritten in place
 *   state_indices [B] int32 DEVICE array of pool rows, or NULL for the
 *                 identity (then P >= B).  A negative entry marks a padding
 *                 row: its o is written as zeros and no state is touched.
 *                 Entries must be distinct (two sequences on one row race);
 *                 an entry >= P is skipped like padding and sets bit 1 of
 *                 the device error word.
 *   P             pool rows (>= 0)
 * Returns KDA_OK or a kda_status_t; B = 0 is a no-op.
 */
int kda_decode_step_pool(const void *q, const void *k, const void *v,
                         const float *g, const float *beta, void *S_pool,
                         int state_dtype, const int32_t *state_indices, int P,
                         float *o, int B, int H, int dk, int dv, int dtype,
                         void *stream);

/* ---------------------------------------------------------------------------
 * The layer around the recurrence.  "Colibri Kimi K3 Metal backend",
 * section 8 introduction: per token the KDA layer runs conv1d + SiLU on its
 * q, k, v projections, L2-normalises q and k per head, steps the state, then
 * applies a per-head RMSNorm and a sigmoid of its full-rank gate projection
 * to o.  Section 8.3 gives the conv (a per-channel window of the last four
 * raw inputs, shifted left by one per token with the new input in the last
 * slot, dotted with the channel's four taps, then SiLU(x) = x / (1 + e^-x))
 * and the L2 norm (n = 1 / sqrt(sum x^2 + eps) over a head's 128 channels,
 * eps = 1e-6; q is scaled by n * q_scale, the pages' q_scale being
 * 1/sqrt(128); k by n; v is not normalised).  Section 8.4 gives the gated
 * norm: out = o / sqrt(mean_j o_j^2 + eps) * norm_w_j * sigmoid(gate_j).
 *
 * Conv windows ("conv states") are bf16 [rows, 3, 3, H, 128]: index 1 is the
 * projection (0 = q, 1 = k, 2 = v), index 2 the window slot, oldest first
 * (slot 2 = the input just before the next token).  They hold raw bf16
 * projections, so they are exact.  Conv taps are fp32 [3, H, 128, 4]: tap m
 * multiplies window slot m, tap 3 the newest input (y_t = sum_m w_m
 * x_{t-3+m}).
 * ------------------------------------------------------------------------- */

/*
 * conv1d + SiLU + L2-norm prologue of a packed varlen prefill: turns the raw
 * projections into the q, k, v that kda_prefill_chunked takes.
 *
 *   xq, xk, xv [T, H, 128] bf16 raw projections
 *   conv_w     [3, H, 128, 4] fp32 taps
 *   conv_in    [N, 3, 3, H, 128] bf16 window before each sequence, or NULL
 *              (zeros: every sequence starts fresh)
 *   conv_out   [N, 3, 3, H, 128] bf16, written: the window after each
 *              sequence's last token (conv_in's, or zeros, for an empty
 *              sequence), to carry into a later call or the decode step; or
 *              NULL.  Must not be conv_in (KDA_ERR_VALUE).
 *   q, k, v    [T, H, 128] bf16, written (rounded to nearest even)
 *   cu_seqlens [N + 1] int32 device array as for kda_prefill_chunked
 *   d          must be 128; q_scale finite; eps >= 0 (the pages' 1e-6)
 * Returns KDA_OK or a kda_status_t.
 */
int kda_conv_prologue(const void *xq, const void *xk, const void *xv, const float *conv_w,
                      const void *conv_in, void *conv_out, void *q, void *k, void *v,
                      const int32_t *cu_seqlens, int N, int64_t T, int H, int d,
                      float q_scale, float eps, void *stream);

/*
 * kda_prefill_chunked with the layer's gated RMSNorm applied to o: writes
 * out = o / sqrt(mean_j o_j^2 + eps) * norm_w_j * sigmoid(gate_j) per
 * (token, head) instead of o.  On the tensor-core path (bf16, chunk 64) the
 * norm runs inside the inter-chunk state pass on each chunk of o before it
 * is stored; other configurations run the CUDA-core prefill into `out`, then
 * the norm in place.
 *
 *   gate     [T, H, 128] bf16 gate projection (before its sigmoid)
 *   norm_w   [128] fp32 RMSNorm weight, shared by the heads
 *   eps      >= 0
 *   out      [T, H, 128] fp32, written
 *   every other argument as for kda_prefill_chunked (S_out gets the final
 *   states, unchanged by the norm)
 * Returns KDA_OK or a kda_status_t.
 */
int kda_prefill_chunked_gated(const void *q, const void *k, const void *v, const float *g,
                              const float *beta, const float *S0, const void *gate,
                              const float *norm_w, float eps, float *out, float *S_out,
                              const int32_t *cu_seqlens, int N, int64_t T, int H, int dk, int dv,
                              int chunk, int dtype, void *stream);

/*
 * The whole layer's prefill in one call ("Colibri Kimi K3 Metal backend",
 * sections 8.3 and 8.4: the conv + L2-norm prologue feeds the recurrence, the
 * gated RMSNorm follows it): kda_conv_prologue followed by
 * kda_prefill_chunked_gated on the tensor-core path, with q, k, v kept in the
 * call's workspace, so a caller needs no buffers for them.  The results are
 * those two calls' bit for bit.
 *
 *   xq, xk, xv [T, H, 128] bf16 raw projections
 *   conv_w     [3, H, 128, 4] fp32 taps
 *   conv_in    [N, 3, 3, H, 128] bf16 windows before each sequence, or NULL
 *   conv_out   [N, 3, 3, H, 128] bf16, written, or NULL; not conv_in
 *   g, beta, S0, S_out, cu_seqlens   as for kda_prefill_chunked
 *   gate       [T, H, 128] bf16; norm_w [128] fp32
 *   out        [T, H, 128] fp32, written: the gated RMSNorm of o
 *   q_scale    finite; l2_eps, norm_eps >= 0
 *   dk, dv     must be 128
 * The workspace (q, k, v in bf16, 768 bytes per token-head, and the records
 * of kda_prefill_chunked) comes from the library's pool (KDA_ERR_WORKSPACE if
 * it cannot grow).  Returns KDA_OK or a kda_status_t.
 */
int kda_layer_prefill(const void *xq, const void *xk, const void *xv, const float *conv_w,
                      const void *conv_in, void *conv_out, const float *g, const float *beta,
                      const float *S0, const void *gate, const float *norm_w, float q_scale,
                      float l2_eps, float norm_eps, float *out, float *S_out,
                      const int32_t *cu_seqlens, int N, int64_t T, int H, int dk, int dv,
                      void *stream);

/*
 * One token of the whole layer for each of B sequences on slot-indexed
 * pools, in one kernel: conv1d + SiLU + L2 norm of the raw projections (the
 * window of pool row state_indices[b] is read and shifted in place), the
 * state step of kda_decode_step_pool (its q, k, v kept in fp32, not rounded
 * to bf16), and the gated RMSNorm of o.
 *
 *   xq, xk, xv    [B, H, 128] bf16 raw projections of the token
 *   conv_w        [3, H, 128, 4] fp32 taps
 *   conv_pool     [P, 3, 3, H, 128] bf16 windows, read and updated in place
 *   g, beta       [B, H, 128] / [B, H] fp32 as for kda_decode_step
 *   gate          [B, H, 128] bf16; norm_w [128] fp32
 *   S_pool        [P, H, 128, 128] fp32 (state_dtype KDA_F32) or bf16
 *                 (KDA_BF16), updated in place
 *   state_indices [B] int32 device array of pool rows, or NULL (rows 0..B-1;
 *                 then P >= B).  Negative = padding: out row zero, neither
 *                 pool touched.  Entries must be distinct; an entry >= P is
 *                 skipped like padding and sets bit 1 of the device error
 *                 word.
 *   out           [B, H, 128] fp32, written
 *   q_scale       finite; l2_eps, norm_eps >= 0
 * Returns KDA_OK or a kda_status_t; B = 0 is a no-op.
 */
int kda_decode_layer_step(const void *xq, const void *xk, const void *xv, const float *conv_w,
                          void *conv_pool, const float *g, const float *beta, const void *gate,
                          const float *norm_w, void *S_pool, int state_dtype,
                          const int32_t *state_indices, int P, float *out, int B, int H,
                          int dk, int dv, float q_scale, float l2_eps, float norm_eps,
                          void *stream);

/* ---------------------------------------------------------------------------
 * Latent attention over a paged cache: the hybrid model's other token mixer
 * ("Kimi K3 -> TPU v7x feasibility", section 2: latent-attention layers
 * without rotary positions between the KDA layers; section 4.2 lists its
 * ragged paged kernel).  Per token the layer keeps one row of 576 bf16 for
 * all heads,
 *     row = [c (512, the latent) | r (64, a key part shared by the heads)],
 * and head h's keys and values are expansions of it: k = [c Wk_h | r]
 * (128 + 64), v = c Wv_h (128).  Two equal forms:
 *   absorbed   q' = [q_nope Wk_h^T | q_pe] (576) attends to the rows as they
 *              are, and o' (512) is multiplied by Wv_h afterwards
 *              (kda_latent_decode: each cached row is read once for all heads)
 *   expanded   keys and values are multiplied out first (kda_latent_prefill:
 *              320 instead of 1,088 multiply-adds per query, key and head)
 * The products with Wk and Wv are the caller's.
 *
 * The cache is [P, page, 576] bf16; page is a power of two, 16 to 1024, and
 * P * page < 2^31.  block_table [N, max_pages] int32: entry i of row b is the
 * page of sequence b's positions i * page .. (i + 1) * page - 1; entries
 * behind the last needed one are not read into any result and may hold
 * anything.  The device arrays seq_lens, cu_seqlens and block_table are not
 * seen by the host; the kernels check them: a length below 0 or above
 * max_pages * page, or offsets that decrease or leave [0, T], raise bit 0 of
 * the device error word, a page index outside [0, P) raises bit 1 (its rows
 * read as zeros, writes to it are dropped), and nothing outside the buffers
 * is touched.  Rows of x, q and o that no sequence holds (t >= cu_seqlens[N])
 * are neither read into a result nor written.
 * ------------------------------------------------------------------------- */

/*
 * Write the rows of new tokens into the cache.  Token i of sequence b's n new
 * ones (packed rows cu_seqlens[b] ..) goes to position seq_lens[b] - n + i.
 *
 *   x          [T, 576] bf16
 *   cache      [P, page, 576] bf16, the new tokens' rows written
 *   seq_lens   [N] int32: lengths with the new tokens counted in
 *   cu_seqlens [N + 1] int32, or NULL: one new token a sequence (then T = N)
 *   norm_w     [512] fp32, or NULL: with it the latent part is stored as
 *              c / sqrt(mean_j c_j^2 + eps) * norm_w_j, rounded once; without
 *              it, and for the shared part always, the bits of x are kept
 *   eps        >= 0
 * No two new tokens may have the same place.  Returns KDA_OK or a
 * kda_status_t; T = 0 is a no-op.
 */
int kda_latent_append(const void *x, void *cache, const int32_t *block_table, const int32_t *seq_lens,
                      const int32_t *cu_seqlens, const float *norm_w, float eps, int N, int64_t T,
                      int64_t P, int page, int max_pages, int d_latent, int d_pe, void *stream);

/*
 * Read the first cu_seqlens[b + 1] - cu_seqlens[b] rows of every sequence b
 * into out [T, 576] bf16, packed in order (the input of the expansion that
 * kda_latent_prefill's keys and values come from).  Returns KDA_OK or a
 * kda_status_t; T = 0 is a no-op.
 */
int kda_latent_gather(const void *cache, const int32_t *block_table, const int32_t *cu_seqlens,
                      void *out, int N, int64_t T, int64_t P, int page, int max_pages, int d_latent,
                      int d_pe, void *stream);

/*
 * Absorbed attention of one or a few new tokens a sequence over the cache
 * that holds them already.  Token i of sequence b's n new ones sees positions
 * 0 .. seq_lens[b] - n + i; for each of its heads
 *     s_p = scale <q, row_p>,  o = sum_p softmax(s)_p c_p,  lse = ln sum_p e^{s_p}.
 * A token that sees nothing (an empty sequence) gets o = 0 and lse = -inf.
 *
 *   q          [T, H, 576] bf16
 *   seq_lens   [N] int32: lengths with the new tokens counted in
 *   cu_seqlens [N + 1] int32, or NULL: one new token a sequence (then T = N).
 *              For 65 to 512 heads NULL is the faster way to say so: a
 *              sequence's tiles of heads are then taken at the same time
 *              (64 sequences of 2,000-4,096 tokens at 96 heads: 75 us, 91 us
 *              with offsets)
 *   scale      > 0, finite
 *   o          [T, H, 512] bf16, written
 *   lse        [T, H] fp32, written, or NULL
 *   workspace  kda_latent_decode_workspace_bytes(N, T, H, ...) bytes of device
 *              memory, 256-byte aligned, alive and unshared until the call's
 *              kernels finish; nothing in it has to be initialised
 * The rows of the positions that a token sees are finite (what lies behind a
 * sequence's end in its last page may be anything).  A row of q that is not
 * (NaN, infinities) has o = NaN where it sees anything, and lse = NaN, or -inf
 * if each of its scores is; other rows are not touched by it.  Returns KDA_OK
 * or a kda_status_t; T = 0 is a no-op.
 */
int kda_latent_decode(const void *q, const void *cache, const int32_t *block_table,
                      const int32_t *seq_lens, const int32_t *cu_seqlens, float scale, void *o,
                      float *lse, int N, int64_t T, int H, int64_t P, int page, int max_pages,
                      int d_latent, int d_pe, void *workspace, size_t ws_bytes, void *stream);

/* Bytes of workspace of kda_latent_decode (0 for invalid sizes). */
size_t kda_latent_decode_workspace_bytes(int N, int64_t T, int H, int d_latent, int d_pe);

/*
 * Expanded attention of new tokens over their sequence's keys and values.
 * Sequence b has the queries cu_seqlens_q[b] .. and the keys cu_seqlens_k[b]
 * .. (packed); its queries are its last tokens, so with causal = 1 query i of
 * nq sees keys 0 .. nk - nq + i (none where that is negative: o = 0,
 * lse = -inf).  With causal = 0 every query sees all nk keys; two such
 * results over disjoint keys join by their lse.
 *
 *   q          [Tq, H, 192] bf16: 128 channels, then the 64 of the shared part
 *   kv         [Tk, H, 256] bf16: key (128), then value (128), of each head
 *   k_pe       bf16 rows of 64, k_pe_stride elements apart (a multiple of 8:
 *              576 for the shared part of gathered cache rows), one a token
 *   scale      > 0, finite
 *   o          [Tq, H, 128] bf16, written
 *   lse        [Tq, H] fp32, written, or NULL
 *   d_nope, d_pe, dv   must be 128, 64, 128
 *   workspace  kda_latent_prefill_workspace_bytes(...) bytes of device memory,
 *              256-byte aligned, alive and unshared until the call's kernels
 *              finish; nothing in it has to be initialised.  Few queries over
 *              many keys need some (their keys are cut into pieces that are
 *              joined); NULL is accepted where the size is 0
 * The keys and values of every sequence are finite; a row of q that is not
 * gives what kda_latent_decode gives for one.  Returns KDA_OK or a
 * kda_status_t; Tq = 0 is a no-op.
 */
int kda_latent_prefill(const void *q, const void *kv, const void *k_pe, int64_t k_pe_stride,
                       const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, float scale,
                       int causal, void *o, float *lse, int N, int64_t Tq, int64_t Tk, int H,
                       int d_nope, int d_pe, int dv, void *workspace, size_t ws_bytes, void *stream);

/* Bytes of workspace of kda_latent_prefill (0 where it needs none and for
 * invalid sizes). */
size_t kda_latent_prefill_workspace_bytes(int N, int64_t Tq, int64_t Tk, int H, int d_nope, int d_pe, int dv);

/* ---------------------------------------------------------------------------
 * Positions rotated into queries and rows, for latent-attention layers that
 * have them (the model's own do without).  The 64 shared key channels, and the
 * queries' channels against them, are d / 2 pairs; pair i of a token at
 * position p is turned by the angle p f_i:
 *     y_a = amplitude (x_a cos - x_b sin),   y_b = amplitude (x_b cos + x_a sin)
 * with (a, b) = (i, i + d / 2) for KDA_ROTARY_HALF, (2 i, 2 i + 1) for
 * KDA_ROTARY_INTERLEAVED.  The frequencies come as turns[i] = f_i / (2 pi) in
 * whole 2^-64ths of a turn a position (int64, wrapping): p turns[i] is the
 * angle's part of a turn exactly, at any position, so that positions far out
 * lose nothing.  Scaled frequencies and amplitudes (for contexts longer than
 * those trained on) are only other numbers in turns and amplitude.
 *
 * Token i of sequence b's n new ones is at position seq_lens[b] - n + i, the
 * place that kda_latent_append gives its row.  A token before position 0 raises
 * bit 0 of the device error word and is left as it was.
 * ------------------------------------------------------------------------- */

/*
 * Rotate the d channels that x's rows point at.
 *
 *   x, out     T x H rows of d channels, a row's channels side by side; strides
 *              in elements between tokens and heads, multiples of 16 bytes below
 *              2^31, all rows within 2^60 elements.  A part of a head is given by
 *              its first channel's address.  x's strides may be 0 (a row for all
 *              heads); out's rows lie apart, all heads of a token before the next
 *              token's or the other way round.  out may be x (with x's strides)
 *              and does not overlap it otherwise
 *   turns      [d / 2] int64
 *   seq_lens   [N] int32: lengths with the new tokens counted in
 *   cu_seqlens [N + 1] int32, or NULL: one new token a sequence (then T = N)
 *   amplitude  finite
 *   inverse    1: by the opposite angles, with the same amplitude: the
 *              transpose, which takes the gradient of out to that of x
 *   d          a multiple of 16, 16 to 256
 *   dtype      KDA_BF16 or KDA_F32, of x and out; the arithmetic is fp32, with
 *              one rounding
 * Rows that no sequence holds are not written.  Returns KDA_OK or a
 * kda_status_t; T = 0 is a no-op.
 */
#define KDA_ROTARY_HALF 0
#define KDA_ROTARY_INTERLEAVED 1
int kda_latent_rotate(const void *x, int64_t x_token_stride, int64_t x_head_stride, void *out,
                      int64_t out_token_stride, int64_t out_head_stride, const int64_t *turns,
                      const int32_t *seq_lens, const int32_t *cu_seqlens, float amplitude, int layout,
                      int inverse, int N, int64_t T, int H, int d, int dtype, void *stream);

/*
 * kda_latent_append with the shared part rotated to the row's position on the
 * way (one rounding to bf16).  turns [d_pe / 2] int64; amplitude and layout as
 * for kda_latent_rotate; all else as for kda_latent_append.
 */
int kda_latent_append_rotated(const void *x, void *cache, const int32_t *block_table,
                              const int32_t *seq_lens, const int32_t *cu_seqlens, const float *norm_w,
                              float eps, const int64_t *turns, float amplitude, int layout, int N,
                              int64_t T, int64_t P, int page, int max_pages, int d_latent, int d_pe,
                              void *stream);

/* ---------------------------------------------------------------------------
 * The latent cache in 4 bits: 416 bytes a token instead of 1,152,
 *     row = [codes (256) | r (128, 64 bf16) | scales (32)].
 * The 512 latent channels are e2m1 codes, two a byte (the even channel in the
 * low half), in groups of 16 with an e4m3 scale each; a channel stands for
 * code * scale * 2^exponent, which bf16 holds exactly.  The exponent, -32 to 32,
 * is one number for a cache: group maxima below 6 * 2^-10 * 2^exponent are
 * stored as zeros and magnitudes above 2688 * 2^exponent saturate, so the
 * default 0 is right for latents of ordinary size.  The shared part keeps its
 * bits.  The cache is [P, page, 416] bytes, 32-byte aligned; pages, block tables,
 * offsets and errors are those of the bf16 cache.
 * ------------------------------------------------------------------------- */

/*
 * Write new tokens' rows: the row that kda_latent_append (turns NULL) or
 * kda_latent_append_rotated would store, in bf16, and then in 4 bits: a
 * group's scale is its largest magnitude over 6 rounded to e4m3, its codes are
 * the channels over that scale rounded to e2m1 (both to nearest even).  A group
 * with a NaN reads back as NaN; infinities saturate.
 */
int kda_latent4_append(const void *x, void *cache, const int32_t *block_table, const int32_t *seq_lens,
                       const int32_t *cu_seqlens, const float *norm_w, float eps, const int64_t *turns,
                       float amplitude, int layout, int exponent, int N, int64_t T, int64_t P, int page,
                       int max_pages, int d_latent, int d_pe, void *stream);

/* kda_latent_gather from a 4-bit cache: out [T, 576] bf16 holds what the rows
 * stand for. */
int kda_latent4_gather(const void *cache, const int32_t *block_table, const int32_t *cu_seqlens,
                       void *out, int exponent, int N, int64_t T, int64_t P, int page, int max_pages,
                       int d_latent, int d_pe, void *stream);

/*
 * kda_latent_decode over a 4-bit cache: the same arguments, outputs and rules,
 * with what the rows stand for in the rows' place.  The latent channels of a row
 * of q are held to 2^-38 of the row's largest magnitude (at exponents above 0 the
 * shared channels count 2^-exponent of theirs); shared channels of the cache are
 * below 2^75 in magnitude (2^107 at exponents of 0 and above).  workspace:
 * kda_latent4_decode_workspace_bytes(N, T, H, ...) bytes.
 */
int kda_latent4_decode(const void *q, const void *cache, const int32_t *block_table,
                       const int32_t *seq_lens, const int32_t *cu_seqlens, float scale, int exponent,
                       void *o, float *lse, int N, int64_t T, int H, int64_t P, int page, int max_pages,
                       int d_latent, int d_pe, void *workspace, size_t ws_bytes, void *stream);

/* Bytes of workspace of kda_latent4_decode (0 for invalid sizes). */
size_t kda_latent4_decode_workspace_bytes(int N, int64_t T, int H, int d_latent, int d_pe);

/*
 * Gives back the memory that the library's workspace pool on the current
 * device keeps between kda_prefill_chunked / _events / _gated /
 * kda_layer_prefill calls (one 60,416-byte record per (chunk, head) of the
 * largest call so far: about 6 GB after a 66,048-token, 96-head batch).
 * Memory still held by a call in flight is kept: synchronise the streams
 * those calls ran on first.  The next call grows the pool again (a driver
 * allocation).  Host-only bookkeeping plus cudaMemPoolTrimTo; returns KDA_OK
 * (also when the device has no pool yet) or KDA_ERR_CUDA.
 */
int kda_workspace_release(void);

/*
 * Device-side error word of the library.  The outputs of a call that raised
 * a bit are invalid.
 *   Bit 0: the tensor-core prefill kernels never wait without bound: if one
 *          of their waits on an asynchronous copy or on the tensor cores
 *          runs past its iteration limit they set this bit, release their
 *          tensor memory and exit.  Also set when cu_seqlens breaks its
 *          precondition (an entry below 0 or above T, or a decrease), by
 *          the prefill paths and the conv prologue, which then touch no
 *          memory outside their buffers; by the latent-attention calls
 *          also for a sequence length outside its block table.
 *   Bit 1: a kda_decode_step_pool or kda_decode_layer_step slot index was
 *          past the end of the pool, or a page index of a latent-attention
 *          call was outside the cache.
 *   Bit 2: the tensor-core prefill saw a gate g outside [-5, 0] or a NaN
 *          (its decay folding is sized for the model's gate bound).
 *   Bit 3: debug builds only (libkda_gb300_debug.so, built with
 *          python -m kda_linear_attention_gb300.build --debug and loaded by
 *          the Python binding when KDA_GB300_DEBUG=1): an index check on a
 *          kernel's global-memory addressing failed; the access was kept
 *          inside its buffer.
 *   Bit 4: the tensor-core prefill's intermediate u = beta (v - ...) (the
 *          delta-rule correction of each token, carried into its second
 *          state-pass product in fp16) reached 65504 in magnitude or NaN:
 *          v far outside a model's activation range.
 *
 *   code   host pointer, receives the word (0 = no error since the last reset)
 *   reset  nonzero: clear the word after reading it
 * Synchronous with respect to the device (a cudaMemcpyFromSymbol).  Returns
 * KDA_OK, KDA_ERR_NULL or KDA_ERR_CUDA.
 */
int kda_device_error(unsigned int *code, int reset);

#ifdef __cplusplus
}
#endif

#endif /* KDA_GB300_H */
