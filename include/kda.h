/*
 * kda.h -- C ABI of libkda, Kimi Delta Attention (KDA) on NVIDIA GB300 (sm_103a).
 *
 * KDA is the gated delta rule with a per-channel decay.  For one sequence and
 * one head the state S is a K x V fp32 matrix (K = d_k rows, V = d_v columns)
 * and each token t updates it and produces an output:
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(exp(g_t)) S_{t-1} + beta_t k_t v_t^T
 *     o_t = S_t^T (scale * q_t)
 *
 * with the gate g = -exp(A_log) * softplus(f + dt_bias) and beta = sigmoid(b).
 * The Kimi-K3 code audit (data/code-audit.json, finding
 * "dual-kda-execution-regimes") names the two regimes this library serves: a
 * chunked form for prefill and a fused recurrent form for one-token cached
 * decoding.  K3_ARTIFACT_AUDIT.md section 7.1 lists the interface facts of the
 * FlashKDA kernel library that this ABI also follows: K = V = 128, bf16 q/k/v,
 * fp32 A_log/dt_bias, fixed and variable length, initial and final recurrent
 * state.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every tensor argument is a DEVICE pointer to row-major contiguous memory
 *   owned by the caller.  libkda allocates nothing except where an entry
 *   point says otherwise; scratch memory is passed in as `workspace`.
 * - Token tensors are laid out [N, H, D] (token, head, channel); states are
 *   [B, H, K, V] with the d_k row index first; beta is [N, H].
 * - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *   stream).  Calls are asynchronous on it: the returned status covers host
 *   argument checks and launch errors only.
 * - Errors found on the device (an out-of-range cu_seqlens entry, a bounded
 *   wait that ran out) are recorded in a device error word and returned by
 *   kda_get_last_device_error().  No kernel traps or asserts.
 * - Pointers must be 16-byte aligned (KDA_ERR_MISALIGNED otherwise).
 * - No C++ exception crosses this ABI.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_VERSION 10200 /* 1.2.0 */

typedef enum kda_status {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1,        /* null pointer, negative size, bad enum, bad cu_seqlens */
    KDA_ERR_UNSUPPORTED_SHAPE = 2,  /* e.g. K or V != 128 for prefill/decode */
    KDA_ERR_UNSUPPORTED_DTYPE = 3,
    KDA_ERR_MISALIGNED = 4,         /* a pointer is not 16-byte aligned */
    KDA_ERR_WORKSPACE_TOO_SMALL = 5,
    KDA_ERR_CUDA = 6,               /* a CUDA runtime call or launch failed */
    KDA_ERR_DEVICE_TIMEOUT = 7,     /* a bounded device-side wait ran out */
    KDA_ERR_NONFINITE = 8,          /* reserved for debug checks */
    KDA_ERR_NOT_IMPLEMENTED = 9,
    KDA_ERR_NO_DEVICE = 10,         /* no usable sm_103 device / driver */
    KDA_ERR_DECAY_RANGE = 11        /* kda_chunk_backward: a (sequence, head) whose chunk
                                       decay exceeds one chunk's range (device-side) */
} kda_status;

typedef enum kda_dtype {
    KDA_BF16 = 0,
    KDA_FP32 = 1,
    KDA_FP8_E4M3 = 2                /* storage of a paged cache only (kda_paged_cache) */
} kda_dtype;

/*
 * Shape of A_log.  K3_ARTIFACT_AUDIT.md section 5.2 records that the public
 * configuration, the HF code and FlashKDA's check expect A_log of shape [H]
 * while the checkpoint header holds [128]; all three readings are accepted.
 */
typedef enum kda_alog_mode {
    KDA_ALOG_PER_HEAD = 0,          /* A_log [H] */
    KDA_ALOG_PER_CHANNEL = 1,       /* A_log [K] */
    KDA_ALOG_PER_HEAD_CHANNEL = 2   /* A_log [H, K] */
} kda_alog_mode;

/*
 * kda_gate_fused -- the KDA gate in one pass (parameters: K3_ARTIFACT_AUDIT.md
 * section 4.1 tensor table and section 5.1 statistics; beta as an fp32 sigmoid
 * of the raw gate: finding 1 of the "[OMNIML-6079] [20/21] Add the Kimi-K3
 * expert-parallel adapter" review).
 *
 *   g[n,h,c]  = -(exp(A_log[.]) * softplus(f[n,h,c] + dt_bias[h,c]))
 *   beta[n,h] = 1 / (1 + exp(-b[n,h]))
 *
 * with softplus(x) = max(x, 0) + log1p(exp(-|x|)).  The result is bit-exact
 * with respect to a fixed binary32 specification (libkda's own exp and log1p,
 * every operation rounded to nearest, no contraction).
 *
 *   f        [N, H, K] of f_dtype (bf16 or fp32)
 *   b        [N, H] of b_dtype (bf16 or fp32) beta logits; may be NULL, in
 *            which case beta_out must be NULL and no beta is written
 *   A_log    fp32, shape selected by alog_mode
 *   dt_bias  fp32 [H, K]
 *   g_out    fp32 [N, H, K] (written)
 *   beta_out fp32 [N, H] (written) or NULL
 *
 * Shape-generic in K.  N == 0 is a no-op.
 */
kda_status kda_gate_fused(const void *f, kda_dtype f_dtype,
                          const void *b, kda_dtype b_dtype,
                          const float *A_log, kda_alog_mode alog_mode,
                          const float *dt_bias,
                          float *g_out, float *beta_out,
                          int64_t N, int H, int K, void *stream);

/*
 * Bytes of device workspace kda_chunk_prefill needs for these sizes.
 * The value never exceeds a few kilobytes; it is 0 only when nothing runs.
 */
size_t kda_chunk_prefill_workspace_size(int64_t N, int B, int H, int K, int V);

/*
 * kda_chunk_prefill -- the chunked KDA regime for prefill (code-audit.json,
 * finding "dual-kda-execution-regimes"; varlen and initial/final state as in
 * K3_ARTIFACT_AUDIT.md section 7.1).  Computes o and the final state exactly
 * as the token recurrence above would, chunk by chunk.
 *
 *   q, k, v       bf16 [N, H, 128]; q and k are used as given (no normalisation)
 *   g             fp32 [N, H, 128] log-decay, g <= 0.  A positive or NaN entry
 *                 sets INVALID_ARG in the device error word (that sequence's
 *                 results are then unspecified).  Chunks whose decay in some
 *                 channel exceeds what one chunk represents (160) are split on
 *                 the device, and a token whose own g is below -160 is taken
 *                 as -160 (e^-160 underflows fp32 as any stronger decay does),
 *                 so every decay is computed.
 *   beta          fp32 [N, H], already passed through the sigmoid
 *   cu_seqlens    int32 [B+1] device offsets of B packed sequences
 *                 (cu_seqlens[0] = 0, non-decreasing, cu_seqlens[B] = N); NULL
 *                 means one sequence of N tokens (B must be 1).  Entries that
 *                 break these rules are caught on the device: the sequence is
 *                 skipped and the device error word is set to INVALID_ARG.
 *                 Zero-length sequences are allowed (final = initial).
 *   scale         multiplies q
 *   initial_state fp32 [B, H, 128, 128] or NULL (zero state)
 *   final_state   fp32 [B, H, 128, 128] (written) or NULL; may alias
 *                 initial_state (each state is read before it is written)
 *   o             [N, H, 128] of o_dtype (bf16 or fp32), written
 *   workspace     device scratch of at least
 *                 kda_chunk_prefill_workspace_size(N, B, H, 128, 128) bytes,
 *                 16-byte aligned; its contents need not be initialised and
 *                 it must not be used by another call running concurrently.
 *
 * K and V must be 128 (KDA_ERR_UNSUPPORTED_SHAPE otherwise).
 */
kda_status kda_chunk_prefill(const void *q, const void *k, const void *v,
                             const float *g, const float *beta,
                             const int32_t *cu_seqlens, int B,
                             int64_t N, int H, int K, int V, float scale,
                             const float *initial_state, float *final_state,
                             void *o, kda_dtype o_dtype,
                             void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_chunk_prefill_gated -- kda_chunk_prefill with the gate computed inside
 * the chunked kernel, the interface K3_ARTIFACT_AUDIT.md section 7.1 records for
 * FlashKDA (gate pre-activation in bf16, A_log/dt_bias in fp32, beta logits):
 *
 *   g[n,h,c]  = -exp(A_log[.]) * softplus(f[n,h,c] + dt_bias[h,c])
 *   beta[n,h] = sigmoid(b[n,h])
 *
 * evaluated with the special-function unit (relative error ~1e-6; it is not
 * the bit-exact specification of kda_gate_fused).  The fp32 g and beta never
 * reach global memory.
 *
 *   f        bf16 [N, H, 128] gate pre-activation (f_dtype must be KDA_BF16)
 *   b        [N, H] beta logits, bf16 or fp32 (b_dtype); the sigmoid is applied
 *            here, once (the EP-adapter review's finding 1: never pass raw
 *            logits where post-sigmoid beta is expected, or vice versa)
 *   A_log    fp32, shape by alog_mode;  dt_bias fp32 [H, 128]
 * All other arguments, layouts and results are those of kda_chunk_prefill
 * (same workspace size).
 */
kda_status kda_chunk_prefill_gated(const void *q, const void *k, const void *v,
                                   const void *f, kda_dtype f_dtype,
                                   const void *b, kda_dtype b_dtype,
                                   const float *A_log, kda_alog_mode alog_mode,
                                   const float *dt_bias,
                                   const int32_t *cu_seqlens, int B,
                                   int64_t N, int H, int K, int V, float scale,
                                   const float *initial_state, float *final_state,
                                   void *o, kda_dtype o_dtype,
                                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_chunk_prefill_noalloc -- kda_chunk_prefill without a workspace argument,
 * for callers that cannot allocate device memory: a host plugin interface that
 * hands the library only its input and output buffers and offers no way to ask
 * for scratch, or a serving process that reserved all device memory at start-up
 * and must not call cudaMalloc afterwards (it can fail, and it can synchronise
 * the device).  The pages this library follows have no counterpart to it.
 *
 * Arguments, layouts and results are those of kda_chunk_prefill.  The scratch
 * comes from a device array built into the library (4096 bytes; every GPU that
 * loads the library holds it until the process exits).  Sizes whose
 * kda_chunk_prefill_workspace_size() exceeds it are rejected with
 * KDA_ERR_WORKSPACE_TOO_SMALL.  The call allocates nothing: it never calls
 * cudaMalloc, cudaFree or any allocating library routine.  The first call on a
 * device looks up the array's device address (cudaGetSymbolAddress) with that
 * device current, so make that first call before any stream capture.  All
 * calls on a device share the array: calls whose kernels overlap on the GPU
 * (on different streams) race on it; calls in stream order do not.
 */
kda_status kda_chunk_prefill_noalloc(const void *q, const void *k, const void *v,
                                     const float *g, const float *beta,
                                     const int32_t *cu_seqlens, int B,
                                     int64_t N, int H, int K, int V, float scale,
                                     const float *initial_state, float *final_state,
                                     void *o, kda_dtype o_dtype, void *stream);

/*
 * kda_recurrent_decode -- the fused recurrent KDA regime for one-token cached
 * decoding (code-audit.json, finding "dual-kda-execution-regimes"): one new
 * token for each of B sequences, the state updated in place.
 *
 *   q, k, v   bf16 [B, H, 128]
 *   g         fp32 [B, H, 128];  beta fp32 [B, H] (post-sigmoid)
 *   state     fp32 [B, H, 128, 128], read and overwritten with S_t
 *   o         [B, H, 128] of o_dtype, written
 *
 * K and V must be 128.  B == 0 is a no-op.
 */
kda_status kda_recurrent_decode(const void *q, const void *k, const void *v,
                                const float *g, const float *beta,
                                float *state, int B, int H, int K, int V, float scale,
                                void *o, kda_dtype o_dtype, void *stream);

/*
 * kda_recurrent_decode_indexed -- kda_recurrent_decode over a pool of cached
 * states addressed by slot, with fp32 or bf16 state storage: the decode side
 * of continuous batching, where sequences come and go and their states live in
 * preallocated slots that are updated in place (indexed writes rather than
 * concatenation: the Kimi-K3 code audit's "repeated-mla-cache-concatenation"
 * recommendation; FlashKDA's bf16 / fp32 state modes, K3_ARTIFACT_AUDIT.md
 * section 7.4).
 *
 *   q, k, v        bf16 [B, H, 128];  g fp32 [B, H, 128];  beta fp32 [B, H]
 *   state_pool     [num_slots, H, 128, 128] of state_dtype (fp32 or bf16),
 *                  read and written in place; a bf16 state is computed in fp32
 *                  and rounded to nearest on the way back
 *   state_indices  int32 [B] device: the slot of each sequence.  A negative
 *                  index marks an inactive sequence (its state is untouched and
 *                  its output row is zero); an index >= num_slots is skipped the
 *                  same way and sets the device error word to INVALID_ARG.  Two
 *                  sequences must not share a slot.
 *   o              [B, H, 128] of o_dtype
 */
kda_status kda_recurrent_decode_indexed(const void *q, const void *k, const void *v,
                                        const float *g, const float *beta,
                                        void *state_pool, kda_dtype state_dtype,
                                        const int32_t *state_indices, int num_slots,
                                        int B, int H, int K, int V, float scale,
                                        void *o, kda_dtype o_dtype, void *stream);

/*
 * kda_recurrent_decode_gated -- the fused recurrent decode with the gate
 * computed in the same kernel, from the gate's own inputs (the interface
 * K3_ARTIFACT_AUDIT.md section 7.1 records for FlashKDA's prefill, applied to
 * the one-token regime of code-audit.json, finding "dual-kda-execution-
 * regimes").  g and beta are formed with exactly the binary32 operations of
 * kda_gate_fused, so the result equals kda_gate_fused followed by
 * kda_recurrent_decode_indexed bit for bit, with one launch and no fp32 g
 * buffer.  (Measured at B = 256, H = 96 on GB300 it is about 3 % slower than
 * the two launches: the exact gate arithmetic adds latency to every CTA of the
 * HBM-bound step.)
 *
 *   q, k, v        bf16 [B, H, 128]
 *   f              [B, H, 128] gate pre-activation, bf16 or fp32 (f_dtype)
 *   b              [B, H] beta logits, bf16 or fp32 (b_dtype); the sigmoid is
 *                  applied here, once
 *   A_log          fp32, shape by alog_mode;  dt_bias fp32 [H, 128]
 *   state_pool, state_dtype, state_indices, num_slots
 *                  as in kda_recurrent_decode_indexed; state_indices may be
 *                  NULL, meaning slot b for sequence b (then num_slots >= B)
 *   o              [B, H, 128] of o_dtype
 */
kda_status kda_recurrent_decode_gated(const void *q, const void *k, const void *v,
                                      const void *f, kda_dtype f_dtype,
                                      const void *b, kda_dtype b_dtype,
                                      const float *A_log, kda_alog_mode alog_mode,
                                      const float *dt_bias,
                                      void *state_pool, kda_dtype state_dtype,
                                      const int32_t *state_indices, int num_slots,
                                      int B, int H, int K, int V, float scale,
                                      void *o, kda_dtype o_dtype, void *stream);

/*
 * kda_recurrent_backward -- gradients of the KDA recurrence for training
 * ("chunked KDA for training", code-audit.json, finding
 * "dual-kda-execution-regimes"): given dL/do and dL/dS_final for the forward
 * pass that kda_chunk_prefill computes on the same inputs, the gradients with
 * respect to q, k, v, g, beta and the initial state.  With
 * S' = Diag(exp g_t) S_{t-1}, w = S'^T k_t, u = beta_t (v_t - w),
 * S_t = S' + k_t u^T, o_t = S_t^T (scale q_t), each reverse step from
 * G = dL/dS_t is
 *   G += (scale q_t) do_t^T;  du = G^T k_t;  dv_t = beta_t du;
 *   dbeta_t = du . (v_t - w);  dw = -beta_t du;  dk_t = G u + S' dw;
 *   dq_t = scale S_t do_t;  dg_t = rowsum((G + k_t dw^T) (.) S');
 *   G = Diag(exp g_t) (G + k_t dw^T)
 * (dL/dS_0 = G at the end).  Computed token by token in fp32 on CUDA cores:
 * a forward pass keeps the state every 16 tokens in the workspace, and each
 * 16-token segment is rerun from it in reverse order.
 *
 *   q, k, v        bf16 [N, H, 128];  g fp32 [N, H, 128];  beta fp32 [N, H]
 *   cu_seqlens, B, initial_state, scale   as in kda_chunk_prefill
 *   dO             [N, H, 128] of dO_dtype (bf16 or fp32)
 *   dS_final       fp32 [B, H, 128, 128] or NULL (zero)
 *   dq, dk, dv, dg fp32 [N, H, 128];  dbeta fp32 [N, H]   (all written)
 *   dS0            fp32 [B, H, 128, 128] or NULL (not computed)
 *   workspace      device, >= kda_recurrent_backward_workspace_size() bytes
 *                  (states every 16 tokens plus 1 MB per CTA; 1.7 GB for
 *                  N = 4096, H = 96); its contents are scratch
 *
 * The gate's own gradients (to f, A_log, dt_bias and the beta logits) are
 * the caller's: g and beta enter here as given tensors.  A bad cu_seqlens
 * entry sets the device error word to INVALID_ARG.
 */
size_t kda_recurrent_backward_workspace_size(int64_t N, int B, int H, int K, int V);

kda_status kda_recurrent_backward(const void *q, const void *k, const void *v,
                                  const float *g, const float *beta,
                                  const int32_t *cu_seqlens, int B,
                                  int64_t N, int H, int K, int V, float scale,
                                  const float *initial_state,
                                  const void *dO, kda_dtype dO_dtype, const float *dS_final,
                                  float *dq, float *dk, float *dv, float *dg, float *dbeta,
                                  float *dS0, void *workspace, size_t workspace_bytes,
                                  void *stream);

/*
 * kda_chunk_backward -- the same gradients as kda_recurrent_backward (same
 * arguments, layouts and results), in the chunked form the pages name for
 * training ("chunked KDA for training", code-audit.json, finding
 * "dual-kda-execution-regimes"), on the tensor cores.  A forward pass of the
 * chunked prefill keeps the state at the start of every 64-token chunk in the
 * workspace; then each (sequence, head) walks its chunks last to first, with
 * the state gradient in tensor memory, and per chunk forms the reverse mode
 * of the chunk-level (WY/UT) forward: dU = A_qk^T dO + Khat dS',
 * dS = Diag(e^{Gam_L}) dS' + Qbar^T dO - W^T dU, and the gradients of
 * A_qk, A_kk (through T = (I + A_kk)^-1), W, U-tilde and the decay factors,
 * down to dq, dk, dv, dg, dbeta.  Every product runs as tcgen05 bf16 MMAs on
 * operands split in a high and a low bf16 part (three products per pair,
 * a 16-bit significand) with fp32 accumulation; the chunk-start states come
 * from the tf32 forward, so the gradients agree with the exact reverse mode
 * to about 1e-3 relative L2 (the forward's state precision), not to fp32
 * rounding as kda_recurrent_backward does.  Every sum is added in a fixed
 * order, so two calls on the same inputs write the same bits.
 *
 * A (sequence, head) whose forward pass had to shorten a chunk (a chunk's
 * decay -sum(g) in some channel above 160) has no 64-token-aligned states:
 * its gradients are written as zeros and the device error word is set to
 * KDA_ERR_DECAY_RANGE; kda_recurrent_backward computes those.
 *
 *   workspace  device, >= kda_chunk_backward_workspace_size() bytes, 16-byte
 *              aligned: the chunk-start states ((N / 64 + B) H 64 KB, 400 MB
 *              for N = 4096, H = 96) plus 528 KB of operand scratch for each
 *              of up to min(B H, 160) CTAs; its contents are scratch.
 * The bounded waits use the product limit of kda_debug_set_wait_limit.
 */
size_t kda_chunk_backward_workspace_size(int64_t N, int B, int H, int K, int V);

kda_status kda_chunk_backward(const void *q, const void *k, const void *v,
                              const float *g, const float *beta,
                              const int32_t *cu_seqlens, int B,
                              int64_t N, int H, int K, int V, float scale,
                              const float *initial_state,
                              const void *dO, kda_dtype dO_dtype, const float *dS_final,
                              float *dq, float *dk, float *dv, float *dg, float *dbeta,
                              float *dS0, void *workspace, size_t workspace_bytes,
                              void *stream);

/*
 * kda_chunk_prefill_checkpointed / kda_chunk_backward_checkpointed -- the
 * training pair of the chunked form: the forward pass that a training step
 * runs anyway also keeps the chunk-start states, and the backward reads them
 * instead of running the forward a second time (kda_chunk_backward does both
 * in one call, about 0.5 ms of its time for N = 4096, H = 96).
 *
 * kda_chunk_prefill_checkpointed takes the arguments of kda_chunk_prefill and
 * writes the same o and final_state (the same kernel, bit for bit), and in
 * addition:
 *   checkpoints  device, >= kda_chunk_checkpoints_size() bytes, 16-byte
 *                aligned, written (caller-owned; nothing else is kept): first
 *                one int32 per (sequence, head), b H + h, set to 1 where a
 *                chunk had to be shortened (decay -sum(g) in some channel
 *                above 160 within 64 tokens), padded to 256 bytes; then the
 *                fp32 state S [K, V] at the start of every 64-token chunk,
 *                chunk c of sequence b (c = 0, 1, ..) in slot
 *                cu_seqlens[b] / 64 + b + c, [slot, H, K, V] row-major
 *                ((N / 64 + B) H 64 KB: 400 MB for N = 4096, H = 96).
 *   workspace    >= kda_chunk_prefill_workspace_size() bytes, as for
 *                kda_chunk_prefill.
 *
 * kda_chunk_backward_checkpointed takes the arguments of kda_chunk_backward
 * with the checkpoints of a kda_chunk_prefill_checkpointed call on the same
 * q, k, v, g, beta, cu_seqlens, scale and initial state in place of
 * initial_state, and writes the same gradients, bit for bit, with the same
 * KDA_ERR_DECAY_RANGE rule for a marked (sequence, head).  It only reads the
 * checkpoints (they may serve several backward calls).
 *   workspace    device, >= kda_chunk_backward_checkpointed_workspace_size()
 *                bytes (512 bytes plus 528 KB for each of up to
 *                min(B H, 160) CTAs), 16-byte aligned; scratch.
 * Both return KDA_ERR_WORKSPACE_TOO_SMALL when checkpoints_bytes is below the
 * size above, and otherwise fail as the calls they extend.  The sizes return
 * 0 for arguments those calls reject.
 */
size_t kda_chunk_checkpoints_size(int64_t N, int B, int H, int K, int V);

kda_status kda_chunk_prefill_checkpointed(const void *q, const void *k, const void *v,
                                          const float *g, const float *beta,
                                          const int32_t *cu_seqlens, int B,
                                          int64_t N, int H, int K, int V, float scale,
                                          const float *initial_state, float *final_state,
                                          void *o, kda_dtype o_dtype,
                                          void *checkpoints, size_t checkpoints_bytes,
                                          void *workspace, size_t workspace_bytes,
                                          void *stream);

size_t kda_chunk_backward_checkpointed_workspace_size(int64_t N, int B, int H, int K, int V);

kda_status kda_chunk_backward_checkpointed(const void *q, const void *k, const void *v,
                                           const float *g, const float *beta,
                                           const int32_t *cu_seqlens, int B,
                                           int64_t N, int H, int K, int V, float scale,
                                           const void *checkpoints, size_t checkpoints_bytes,
                                           const void *dO, kda_dtype dO_dtype,
                                           const float *dS_final,
                                           float *dq, float *dk, float *dv, float *dg,
                                           float *dbeta, float *dS0,
                                           void *workspace, size_t workspace_bytes,
                                           void *stream);

/*
 * kda_gate_backward -- gradients of the gate (the training regime, after
 * kda_recurrent_backward): from dL/dg and dL/dbeta to the gate's inputs.
 * With x = f + dt_bias, a = exp(A_log), g = -a softplus(x), beta = sigmoid(b)
 * (K3_ARTIFACT_AUDIT.md sections 4.1 and 5.1):
 *   df = dg (-a sigmoid(x));   d dt_bias = sum over tokens of df;
 *   d A_log = sum of dg g over the axes A_log is broadcast along;
 *   db = dbeta beta (1 - beta)
 * x, a, g and beta are formed with kda_gate_fused's binary32 specification.
 * The sums are added in a fixed order (the result does not depend on timing).
 *
 *   f            [N, H, K] of f_dtype (bf16 or fp32);  dg fp32 [N, H, K]
 *   b, dbeta     [N, H] (b_dtype) and fp32 [N, H], with db fp32 [N, H]
 *                written; all three NULL to skip beta
 *   A_log        fp32 by alog_mode;  dt_bias fp32 [H, K]
 *   df           fp32 [N, H, K] written
 *   dA_log       fp32, shape of A_log, written (or NULL)
 *   ddt_bias     fp32 [H, K] written (or NULL)
 *   workspace    >= kda_gate_backward_workspace_size(N, H, K) bytes (about
 *                (2 min(N, 256) + 1) H K 4 bytes), 16-byte aligned
 * K must be a multiple of 8; f, dg, df 16-byte aligned.
 */
size_t kda_gate_backward_workspace_size(int64_t N, int H, int K);

kda_status kda_gate_backward(const void *f, kda_dtype f_dtype,
                             const void *b, kda_dtype b_dtype,
                             const float *A_log, kda_alog_mode alog_mode,
                             const float *dt_bias,
                             const float *dg, const float *dbeta,
                             float *df, float *db, float *dA_log, float *ddt_bias,
                             int64_t N, int H, int K,
                             void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_short_conv_qkv -- the KDA input pre-step over a packed batch, on the three
 * projection streams at once: a depthwise causal convolution of kernel size 4
 * per channel (the checkpoint's q/k/v_conv1d.weight, fp32 [H*128, 1, 4];
 * K3_ARTIFACT_AUDIT.md section 4.1, KDA tensor table), then SiLU, then for q
 * and k an L2 norm over each head's 128 channels:
 *
 *   a[p, c] = sum_{j=0..3} w[c, j] x[p - 3 + j, c]     (tap 3 on the current token)
 *   y = a * sigmoid(a);   q, k: y / sqrt(sum_head y^2 + 1e-6);   v: y
 *
 * Positions before a sequence's first token read that sequence's carried
 * state (the last three raw inputs of its previous segment, oldest first), or
 * zeros when conv_state_in is NULL.  Sequences never see each other.
 *
 *   x_q, x_k, x_v     bf16 [N, C] each, C = H * 128 (the projection outputs)
 *   w_q, w_k, w_v     fp32 [C, 4] each
 *   cu_seqlens, B     as in kda_chunk_prefill (NULL: one sequence, B = 1)
 *   conv_state_in     bf16 [B, 3 (q, k, v), 3 (oldest first), C] or NULL
 *   conv_state_out    bf16 [B, 3, 3, C] or NULL: each sequence's last three
 *                     inputs (state rows fill in for sequences shorter than 3;
 *                     an empty sequence passes its state through).  Must not
 *                     overlap conv_state_in.
 *   q, k, v           bf16 [N, C] outputs, ready for kda_chunk_prefill as
 *                     [N, H, 128]; must not overlap any input
 *
 * C must be a positive multiple of 128 (KDA_ERR_UNSUPPORTED_SHAPE).  A bad
 * cu_seqlens array sets the device error word to INVALID_ARG.  N == 0 with
 * conv_state_out copies the states through.
 */
kda_status kda_short_conv_qkv(const void *x_q, const void *x_k, const void *x_v,
                              const float *w_q, const float *w_k, const float *w_v,
                              const int32_t *cu_seqlens, int B, int64_t N, int C,
                              const void *conv_state_in, void *conv_state_out,
                              void *q, void *k, void *v, void *stream);

/*
 * kda_short_conv_qkv_step -- the same pre-step for one new token per sequence,
 * the carried conv states kept in a pool addressed by slot and updated in
 * place (the decode side of kda_short_conv_qkv).
 *
 *   x_q, x_k, x_v     bf16 [B, C];  w_q, w_k, w_v fp32 [C, 4]
 *   conv_state_pool   bf16 [num_slots, 3, 3, C], read and shifted in place
 *   state_indices     int32 [B] device, or NULL for slot b = sequence b
 *                     (then num_slots >= B).  Negative: inactive sequence
 *                     (outputs zero, state untouched); >= num_slots: skipped
 *                     the same way and the device error word set to
 *                     INVALID_ARG.  Two sequences must not share a slot.
 *   q, k, v           bf16 [B, C] outputs (may be the inputs themselves)
 *
 * C must be a positive multiple of 128; B <= 65535.
 */
kda_status kda_short_conv_qkv_step(const void *x_q, const void *x_k, const void *x_v,
                                   const float *w_q, const float *w_k, const float *w_v,
                                   void *conv_state_pool, const int32_t *state_indices,
                                   int num_slots, int B, int C,
                                   void *q, void *k, void *v, void *stream);

/*
 * A paged key-value cache for softmax-attention layers that stand between KDA
 * layers and keep keys and values per head, of equal head_dim, in preallocated
 * pages that are written by index (what the Kimi-K3 code audit's finding
 * "repeated-mla-cache-concatenation" asks for, as for the state pool of
 * kda_recurrent_decode_indexed).  It does not hold that model's own attention
 * layers (K3_ARTIFACT_AUDIT.md section 3.1: 24 beside 69 KDA layers), whose cache
 * is one latent of 512 + 64 values a token for all heads.  Attention is for one
 * new token per sequence; a prompt's own attention over its keys is the caller's.
 * Three entry points serve one step of a batch:
 *
 *   kda_page_plan     block table, slot map and offsets of the step's tokens,
 *                     from the requests' lengths, on the device (once a step)
 *   kda_paged_append  the step's keys and values into the cache (each layer)
 *   kda_paged_decode  attention of one new token per sequence (each layer)
 *
 * A slot is page * page_size + offset: the place of one token.  A sequence's
 * position p lies in page block_table[b, p / page_size] at offset p % page_size.
 *
 * kda_paged_cache describes one layer's cache.  It is a host struct that the
 * calls read before they return; the memory it points to is the caller's.
 *
 *   k, v            device: the cache's keys and values (equal layouts)
 *   k_scale/v_scale fp32 [heads] device, or both NULL (1): an 8-bit cache holds
 *                   key / k_scale[h]; must be NULL for a bf16 cache
 *   page_stride, token_stride, head_stride
 *                   distances in elements from a page, a token of a page and a
 *                   head to the next; head_dim is contiguous.  Any order
 *                   of the three (pages stored token by token or head by head,
 *                   keys and values interleaved by page) whose rows do not
 *                   overlap; multiples of 16 bytes.
 *   dtype           KDA_BF16 or KDA_FP8_E4M3
 *   num_pages, page_size, heads
 *                   any positive numbers with num_pages * page_size < 2^31
 *   head_dim        64, 128 or 256
 */
typedef struct kda_paged_cache {
    void *k;
    void *v;
    const float *k_scale;
    const float *v_scale;
    int64_t page_stride;
    int64_t token_stride;
    int64_t head_stride;
    int32_t dtype;
    int32_t num_pages;
    int32_t page_size;
    int32_t heads;
    int32_t head_dim;
} kda_paged_cache;

/*
 * kda_page_plan -- places a step's new tokens: extends the block table by
 * pages from a free list and maps every new token to its slot.  With
 * c = cached_lens[b], n = new_lens[b] and ceil() the number of pages of a length,
 *
 *   need[b] = ceil(c + n) - ceil(c),   off[b] = sum of need[a] over a < b
 *   block_table[b, ceil(c) + i] = free_pages[off[b] + i],   i < need[b]
 *   seq_lens[b] = c + n,   cu_seqlens[b + 1] = cu_seqlens[b] + n
 *   slot_map[cu_seqlens[b] + j] = slot of position c + j of request b,  j < n
 *
 *   cached_lens  int32 [B] device: tokens already in the cache
 *   new_lens     int32 [B] device: tokens of this step (0: none)
 *   free_pages   int32 [num_free] device: pages to take, from the front (a list
 *                whose front was dropped: 4-byte aligned is enough)
 *   block_table  int32 [B, max_pages] device: the first ceil(c) entries of a
 *                row are read, the next need[b] written, the rest left alone
 *   seq_lens     int32 [B] written: what kda_paged_decode reads
 *   cu_seqlens   int32 [B+1] written: what kda_chunk_prefill reads
 *   slot_map     int32 [N] written: what kda_paged_append reads; entries past
 *                the step's tokens are -1 (N may exceed their number)
 *   pages_used   int32 [1] written: how many of free_pages were taken
 *
 * The lists are not advanced (the caller drops pages_used pages from the front),
 * so the call may be repeated.  A request is refused, with INVALID_ARG in the
 * device error word, if a length is negative, c + n exceeds
 * max_pages * page_size or 2^31 - 1, or its pages or tokens end past num_free or
 * N: its slots are -1, its row of the table is unchanged and seq_lens[b] = c (0
 * where c itself is out of range).  Its n > 0 tokens keep their rows (offsets
 * past N read N); its pages count for the requests after it, except where its
 * lengths are bad.  A page outside 0 .. num_pages-1 gives its tokens slot
 * -1 and sets INVALID_ARG too.  No output may overlap an input or another
 * output.  B == 0 and N == 0 are allowed.
 */
kda_status kda_page_plan(const int32_t *cached_lens, const int32_t *new_lens,
                         const int32_t *free_pages, int num_free, int32_t *block_table,
                         int max_pages, int B, int page_size, int num_pages, int32_t *seq_lens,
                         int32_t *cu_seqlens, int32_t *slot_map, int64_t N, int32_t *pages_used,
                         void *stream);

/*
 * kda_paged_append -- writes the keys and values of N tokens to their slots:
 *
 *   cache.k[slot_map[n], h, :] = k[n, h, :]                       (bf16 cache)
 *   cache.k[slot_map[n], h, :] = e4m3(k[n, h, :] / k_scale[h])    (8-bit cache)
 *
 * and v alike; e4m3 rounds the fp32 quotient to nearest, ties to even, and
 * limits its magnitude to 448 (NaN stays NaN).
 *
 *   k, v      bf16, token n's [heads, head_dim] values from k + n * k_row_stride
 *             (v_row_stride for v; in elements, multiples of 8, at least
 *             heads * head_dim: both may be slices of a fused projection)
 *   slot_map  int32 [N] device.  A negative slot leaves its token out; one past
 *             the cache is left out too and sets INVALID_ARG in the device error
 *             word.  Two tokens must not share a slot.
 * The sources must not overlap the cache.  N == 0 is a no-op.
 */
kda_status kda_paged_append(const void *k, const void *v, int64_t k_row_stride,
                            int64_t v_row_stride, const int32_t *slot_map, int64_t N,
                            const kda_paged_cache *cache, void *stream);

/* Bytes of device workspace kda_paged_decode needs (0 for sizes that it rejects). */
size_t kda_paged_decode_workspace_size(int B, int q_heads, int kv_heads, int head_dim);

/*
 * kda_paged_decode -- softmax attention of one new token per sequence over its
 * cached keys (its own among them, once appended).  With L = seq_lens[b] and
 * the key head of query head h being h / (q_heads / heads),
 *
 *   s[j] = scale * <q[b, h], key j>,  j < L
 *   o[b, h] = sum_j exp(s[j] - lse) value j,   lse[b, h] = log sum_j exp(s[j])
 *
 *   q           bf16, sequence b's [q_heads, head_dim] values from
 *               q + b * q_row_stride (elements, a multiple of 8)
 *   block_table int32 [B, max_pages] device;  seq_lens int32 [B] device
 *   q_heads     a positive multiple of cache->heads
 *   o           [B, q_heads, head_dim] of o_dtype (bf16 or fp32), written; a
 *               softmax weight is kept to 16 bits for bf16 outputs, 22 or more for
 *               fp32 ones; over an 8-bit cache, to that or to 2^-37 (fp32 outputs:
 *               2^-48) of the largest weight, whichever is coarser
 *   lse         fp32 [B, q_heads] written, or NULL: with fp32 outputs, what joins
 *               the results over two sets of keys
 *   workspace   device scratch, >= kda_paged_decode_workspace_size() bytes,
 *               16-byte aligned; not shared with a concurrent call
 *
 * An empty sequence gives o = 0 and lse = -inf.  A length below 0 or above
 * max_pages * page_size counts as empty, and keys on a page outside
 * 0 .. num_pages-1 are left out; both set INVALID_ARG in the device error word.
 * Memory past a sequence's last key is not read.  Infinities and NaN among q, the
 * keys and the values act as in fp32 arithmetic (an infinite value of a key with
 * weight gives an infinite output; a call that meets one takes longer).  Two calls
 * on the same inputs write the same bits.  B == 0 is a no-op.
 */
kda_status kda_paged_decode(const void *q, int64_t q_row_stride, const kda_paged_cache *cache,
                            const int32_t *block_table, int max_pages, const int32_t *seq_lens,
                            int B, int q_heads, float scale, void *o, kda_dtype o_dtype,
                            float *lse, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Drafted tokens.  A serving loop may run several drafted tokens of a request through the
 * layers at once, as a tree: each node is a token, its ancestors the tokens before it; then
 * one path is accepted and the rest is dropped.  A step of both kinds of layers:
 *
 *   kda_page_plan, kda_paged_append    place the nodes' keys and values, as for any new tokens
 *   kda_short_conv_qkv_tree            the KDA pre-step of every node
 *   kda_recurrent_tree_decode          the KDA recurrence to every node, the state unchanged
 *   kda_paged_tree_decode              attention of every node over the cache
 *   kda_recurrent_tree_commit, kda_short_conv_tree_commit, kda_paged_compact
 *                                      what the accepted path leaves in the three memories
 *
 * Arguments that these calls share:
 *
 *   cu_seqlens   int32 [B+1] device: request b's nodes are rows cu_seqlens[b] ..
 *                cu_seqlens[b+1] - 1 of the token tensors (what kda_page_plan writes); N rows
 *                in all.  Rows behind the last request's are neither read nor written.
 *   max_nodes    1 .. KDA_TREE_MAX_NODES: no request has more
 *   ancestors    uint64 [N] device: bit j of a node's word is set where it sees node j of its
 *                request.  The bits below its own number are its ancestors in the recurrence
 *                and the convolution, where the other bits are not looked at; attention takes
 *                the bits as they are, so a node's own bit belongs there.  (With parent[i] < i:
 *                word[i] = 1 << i | word[parent[i]].)
 *   last         int32 [B] device: the accepted path's last node; -1: nothing is accepted.
 *                The path is that node and its ancestors.
 *
 * A request whose offsets go back or leave the N rows is left out (its rows stay as they
 * were); one of more than max_nodes rows counts as inactive: outputs of its rows are zeros,
 * its memory stays as it is.  Both set INVALID_ARG in the device error word, and so does a
 * `last` past the request's nodes, which accepts nothing.  B is at most 65535.
 */
#define KDA_TREE_MAX_NODES 64

/*
 * kda_recurrent_tree_decode -- the KDA recurrence over trees of drafted tokens (the fused
 * recurrent regime for several tokens of a sequence that follow one another in more than one
 * order; code-audit.json, finding "dual-kda-execution-regimes").  Node i's state is its
 * parent's (the slot's, for a node without ancestors) after the update with i's k, v, g and
 * beta, as in kda_recurrent_decode; o is read from it.  No state is written: what the nodes
 * add to it is kept as one vector a node,
 *
 *   u_i = beta_i (v_i - S'^T k_i),  S' = Diag(exp g_i) S_parent
 *
 * from which kda_recurrent_tree_commit forms the state after any path.  Sums are fp32, and
 * operands are kept to 24 bits (a bf16 state is widened; unlike a chain of one-token decodes, it
 * is not rounded between the nodes of a path).  What a node does not see has no part in its output
 * and update, whatever it holds.  Infinities and NaN act as in fp32 arithmetic; a call that meets
 * them takes longer.  Two calls on the same inputs write the same bits.
 *
 *   q, k, v        bf16 [N, H, 128];  g fp32 [N, H, 128];  beta fp32 [N, H]
 *   state_pool     [num_slots, H, 128, 128] of state_dtype (fp32 or bf16), read
 *   state_indices  int32 [B] device: the slot of each request, or NULL for slot b (then
 *                  num_slots >= B).  Negative: inactive, its rows of o and u are zeros; one
 *                  >= num_slots is skipped the same way and sets INVALID_ARG.  Requests may
 *                  share a slot here.
 *   o              [N, H, 128] of o_dtype (bf16 or fp32), written
 *   u              fp32 [N, H, 128] written, or NULL
 * K and V must be 128.  No output may overlap an input or another output.  B == 0 is a no-op.
 */
kda_status kda_recurrent_tree_decode(const void *q, const void *k, const void *v, const float *g,
                                     const float *beta, const void *state_pool,
                                     kda_dtype state_dtype, const int32_t *state_indices,
                                     int num_slots, const int32_t *cu_seqlens,
                                     const uint64_t *ancestors, int B, int64_t N, int max_nodes,
                                     int H, int K, int V, float scale, void *o, kda_dtype o_dtype,
                                     float *u, void *stream);

/*
 * kda_recurrent_tree_commit -- the state after the accepted path, in place: with E_j the decays
 * of the path's nodes behind j multiplied up,
 *
 *   S <- Diag(prod exp g_j) S + sum_j (E_j k_j) u_j^T,   j over the path of node last[b]
 *
 *   k, g, u        of the kda_recurrent_tree_decode call (u as it was written there)
 *   state_pool, state_indices, num_slots
 *                  as there, but written; two requests must not share a slot
 * A bf16 state is rounded once, after the whole path.
 */
kda_status kda_recurrent_tree_commit(const void *k, const float *g, const float *u,
                                     void *state_pool, kda_dtype state_dtype,
                                     const int32_t *state_indices, int num_slots,
                                     const int32_t *cu_seqlens, const uint64_t *ancestors,
                                     const int32_t *last, int B, int64_t N, int max_nodes, int H,
                                     int K, int V, void *stream);

/*
 * kda_short_conv_qkv_tree -- kda_short_conv_qkv for trees of drafted tokens: the three inputs
 * before a node's own are those of its nearest ancestors, and the carried ones of its request
 * where it has fewer than three.  The pool is read, not changed.
 *
 *   x_q, x_k, x_v     bf16 [N, C];  w_q, w_k, w_v fp32 [C, 4]
 *   conv_state_pool   bf16 [num_slots, 3, 3, C];  state_indices, num_slots as in
 *                     kda_recurrent_tree_decode
 *   q, k, v           bf16 [N, C] written (zeros for an inactive request); must not overlap
 *                     an input or one another
 *
 * kda_short_conv_tree_commit -- the carried inputs after the path of node last[b], in place: the
 * last three of the carried ones and the path's.  Two requests must not share a slot.
 * C must be a positive multiple of 128.
 */
kda_status kda_short_conv_qkv_tree(const void *x_q, const void *x_k, const void *x_v,
                                   const float *w_q, const float *w_k, const float *w_v,
                                   const void *conv_state_pool, const int32_t *state_indices,
                                   int num_slots, const int32_t *cu_seqlens,
                                   const uint64_t *ancestors, int B, int64_t N, int max_nodes,
                                   int C, void *q, void *k, void *v, void *stream);

kda_status kda_short_conv_tree_commit(const void *x_q, const void *x_k, const void *x_v,
                                      void *conv_state_pool, const int32_t *state_indices,
                                      int num_slots, const int32_t *cu_seqlens,
                                      const uint64_t *ancestors, const int32_t *last, int B,
                                      int64_t N, int max_nodes, int C, void *stream);

/* Bytes of device workspace kda_paged_tree_decode needs (0 for sizes that it rejects). */
size_t kda_paged_tree_decode_workspace_size(int B, int max_nodes, int q_heads, int kv_heads,
                                            int head_dim);

/*
 * kda_paged_tree_decode -- softmax attention of a tree of drafted tokens per sequence over its
 * cached keys, the drafted tokens' own among them (appended before).  With L = seq_lens[b], n
 * nodes and C = L - n, node i sees the keys j < C and the keys C + j, j < n, whose bit j is set
 * in ancestors[cu_seqlens[b] + i]; over those keys it is kda_paged_decode's attention.
 *
 *   q           bf16, node's [q_heads, head_dim] values from q + row * q_row_stride (elements, a
 *               multiple of 8)
 *   cache, block_table, max_pages, seq_lens (drafted tokens included), q_heads, scale
 *               as in kda_paged_decode
 *   o           bf16 [N, q_heads, head_dim] written; a softmax weight is kept to 16 bits (over
 *               an 8-bit cache to 2^-37 of the largest, if that is coarser)
 *   lse         fp32 [N, q_heads] written, or NULL
 *   workspace   device scratch, >= kda_paged_tree_decode_workspace_size() bytes, 16-byte
 *               aligned; not shared with a concurrent call
 * o, lse and the workspace must not overlap an input or one another.
 *
 * A node that sees no key gives o = 0 and lse = -inf; what it does not see has no part in its
 * output, whatever it holds.  A length below n or above max_pages * page_size counts as no keys
 * for all the request's nodes, and keys on a page outside 0 .. num_pages-1 are left out; both
 * set INVALID_ARG in the device error word.  A request with more than max_nodes rows gives zeros
 * and -inf.  Infinities and NaN act as in fp32 arithmetic; a call that meets infinite or NaN
 * values takes longer.  Two calls on the same inputs write the same bits.
 */
kda_status kda_paged_tree_decode(const void *q, int64_t q_row_stride, const kda_paged_cache *cache,
                                 const int32_t *block_table, int max_pages,
                                 const int32_t *seq_lens, const int32_t *cu_seqlens,
                                 const uint64_t *ancestors, int B, int64_t N, int max_nodes,
                                 int q_heads, float scale, void *o, float *lse, void *workspace,
                                 size_t workspace_bytes, void *stream);

/*
 * kda_paged_compact -- keeps the accepted path's keys and values: the r-th node of the path of
 * last[b], r = 0, 1, .., moves to position C + r, C = seq_lens[b] - n (each layer).
 *
 *   kept_lens   int32 [B] written, or NULL: C + the path's nodes (for a request that is left
 *               out C, or 0 where its length is below its rows or does not fit its table);
 *               must not overlap an input
 * What lies behind kept_lens[b] afterwards is not defined; kda_page_release gives its pages
 * back.  The pages that hold drafted tokens must be the request's own.  Rows on a page outside
 * 0 .. num_pages-1 stay where they are and set INVALID_ARG.
 */
kda_status kda_paged_compact(const kda_paged_cache *cache, const int32_t *block_table,
                             int max_pages, const int32_t *seq_lens, const int32_t *cu_seqlens,
                             const uint64_t *ancestors, const int32_t *last, int B, int64_t N,
                             int max_nodes, int32_t *kept_lens, void *stream);

/*
 * kda_page_fork -- requests that go on from others (several continuations of one prompt): fork
 * f makes request dst[f] hold what request src[f] holds.  The source's full pages are shared;
 * its last, partly filled one gets a copy of its own, since both will write there.  Once for
 * all layers; kda_paged_copy then copies the listed pages in each.
 *
 *   src, dst     int32 [num_forks] device.  dst[f] must hold no pages (its row of the table is
 *                written over), be no fork's source and no other fork's destination; sources
 *                may repeat.
 *   seq_lens     int32 [B] device: seq_lens[dst[f]] = seq_lens[src[f]] is written
 *   free_pages   int32 [num_free] device, taken from the front in the order of the forks (4-byte
 *                aligned is enough)
 *   block_table  int32 [B, max_pages] device: rows dst[f] are written
 *   shares       int32 [num_pages] device: holders of each page beyond the first, so zeros for
 *                a pool that no fork has touched; + 1 for every page that is shared
 *   copies       int32 [num_forks, 3] written: source page, destination page and number of
 *                tokens (-1, -1, 0: nothing to copy)
 *   pages_used   int32 [1] written: how many of free_pages were taken
 *
 * A fork is refused, with INVALID_ARG in the device error word, if src or dst is out of range,
 * the source's length is negative or does not fit its row, dst[f] is a source or an earlier
 * fork's destination, or no page is left: nothing is written for it but its entry of copies.
 * (Where src and its length are good, the page that it would take counts as taken.)  A page
 * outside 0 .. num_pages-1 is neither counted nor copied and sets INVALID_ARG.  A source's last,
 * partly filled page may be shared itself.  No array may overlap another.  num_forks == 0 writes
 * pages_used = 0.
 */
kda_status kda_page_fork(const int32_t *src, const int32_t *dst, int num_forks, int32_t *seq_lens,
                         const int32_t *free_pages, int num_free, int32_t *block_table,
                         int max_pages, int B, int page_size, int num_pages, int32_t *shares,
                         int32_t *copies, int32_t *pages_used, void *stream);

/*
 * kda_paged_copy -- copies pages within a cache: for each entry (source page, destination page,
 * tokens) of copies int32 [num_copies, 3] the first `tokens` keys and values of all heads.  For
 * what kda_page_fork lists, or a caller's own list (pages moved together).  A page that one
 * entry writes must not be in another.  An entry of 0 tokens is skipped; one with a page
 * outside 0 .. num_pages-1 or tokens outside 0 .. page_size is skipped and sets INVALID_ARG.
 */
kda_status kda_paged_copy(const int32_t *copies, int num_copies, const kda_paged_cache *cache,
                          void *stream);

/*
 * kda_page_release -- gives pages back: request b keeps its first kept_lens[b] tokens of
 * seq_lens[b] (0: it has ended) and leaves the pages that only the others need.  A page with
 * shares has one less; one without is free.
 *
 *   seq_lens, kept_lens  int32 [B] device
 *   block_table  int32 [B, max_pages] device, read
 *   shares       int32 [num_pages] device, as in kda_page_fork; updated
 *   freed        int32 [max_freed] written: the pages that are free now, ascending; entries
 *                past num_freed stay as they were (it may be the end of the free list: 4-byte
 *                aligned is enough)
 *   num_freed    int32 [1] written
 *
 * A kept length may end inside a page that another request holds too (shares > 0: a fork, or
 * its source, that goes back behind the point where they parted).  The page stays shared, so the
 * request may be read, shortened, forked and released, but nothing may be appended to it or
 * compacted in it: that would write into the other's keys.  To go on from it, kda_page_fork it into an
 * empty row, which gives the last page a copy of its own, kda_paged_copy, and release the old row.
 *
 * A request with kept_lens[b] < 0 or > seq_lens[b], or a length that does not fit its row, is
 * refused and keeps its pages.  A page that is given back more often than it is held is freed
 * once; a page outside 0 .. num_pages-1 is passed over; pages past max_freed are not listed
 * (their shares are 0: they are lost to the caller).  Each sets INVALID_ARG in the device error
 * word.  No array may overlap another.  1024 rows of the table (or B, if fewer) must have fewer than
 * 2^31 entries.  B == 0 writes num_freed = 0.
 */
kda_status kda_page_release(const int32_t *seq_lens, const int32_t *kept_lens,
                            const int32_t *block_table, int max_pages, int B, int page_size,
                            int num_pages, int32_t *shares, int32_t *freed, int max_freed,
                            int32_t *num_freed, void *stream);

/*
 * kda_debug_check_gate_division -- test hook: the gate kernel's common path
 * (|f + dt_bias| < 87) divides with an fma-based correctly rounded division
 * (Markstein's method) instead of IEEE division; this call runs it against
 * IEEE division on the device for every operand pair that path can form
 * (about 1.07e9) and writes the number of differing results to *mismatches
 * (host pointer; 0 is the gate's bit-exactness).  Synchronises `stream`.
 */
kda_status kda_debug_check_gate_division(uint64_t *mismatches, void *stream);

/*
 * kda_debug_set_wait_limit -- test hook for the bounded device waits.  Every
 * wait of the chunked prefill kernels on a copy (TMA) or a tensor-core product
 * gives up after a bounded number of polls and records KDA_ERR_DEVICE_TIMEOUT
 * in the device error word instead of hanging (a failure is reported, never
 * turned into silent wrong numbers: the EP-adapter review, finding IMPORTANT
 * 1, asks for loud failure).  This call sets the bound of the main-loop waits
 * of later kda_chunk_prefill* launches in this process: copy_polls for copies,
 * product_polls for products; 0 gives up at the first poll, a negative value
 * restores the default.  A kernel that gives up stops issuing work and, before
 * it exits, waits for everything it had in flight with the default bound (this
 * drain is never shortened).  For tests only: the outputs of an aborted launch
 * are incomplete.  Always returns KDA_OK.
 */
kda_status kda_debug_set_wait_limit(int64_t copy_polls, int64_t product_polls);

/*
 * Synchronises `stream`, then returns and clears the device error word of the
 * current device (KDA_OK when no kernel recorded an error).  Returns
 * KDA_ERR_CUDA if the synchronisation itself fails.
 */
kda_status kda_get_last_device_error(void *stream);

/* A static, human-readable name for a status code. */
const char *kda_status_string(kda_status status);

/* KDA_VERSION of the built library. */
int kda_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
