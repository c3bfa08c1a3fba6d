/*
 * kda.h -- C ABI of libkda.so, the B200 (sm_100a) Kimi Delta Attention operator.
 *
 * The operator (per sequence b, head h; state S is d_k x d_v, fp32):
 *   S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *   o_t = S_t^T q_t,            alpha_t = exp(log_alpha_t) in (0, 1]^{d_k}
 * Sources: "Kimi Linear's 75% KV cache cut comes from making three of every
 * four layers recurrent" (theclarity.today), third paragraph (per-channel
 * decay, removal of the old projection onto the key, write of the new pair)
 * and fourth paragraph (chunked kernels with the WY representation: a chunk's
 * rank-1 updates become triangular solves and tensor-core matrix products);
 * "Kimi Linear wlasnie pokonal pelna uwage na wlasnych warunkach" (remio.ai),
 * section "Jak Kimi Linear wykorzystuje inteligentniejsza pamiec
 * rekurencyjna" (delta rule, finer-grained gates than Gated DeltaNet,
 * blockwise algorithm with a diagonal-plus-low-rank transition, fixed-size
 * recurrent state).
 *
 * Padding: a position whose pad_mask entry is 0 neither decays nor writes the
 * state and its output is exactly 0, whatever its gate and input values
 * ("Transformers Community Reports Kimi Linear Cache Bug: Padding May Change
 * Subsequent Inference State", ainews, paragraphs on the reproduction and the
 * follow-up investigation).
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers, owned by the caller, on the
 *     current CUDA device.  The library allocates no device memory.
 *   - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL = the
 *     legacy default stream).  Nothing is synchronised.
 *   - Argument errors are detected on the host and returned before anything
 *     is launched; no output is touched in that case.
 *   - Errors found on the device (an invalid cu_seqlens, a bounded wait that
 *     ran out) are latched in a per-device library word and reported by
 *     kda_get_device_status().  Kernels that follow a failed check on the same
 *     stream return without writing.
 *   - No C++ exception crosses the ABI.
 *   - Every launch is stream-ordered, so the calls can be captured into a CUDA
 *     graph; the first call on each device looks up the library's device error
 *     word (cudaGetSymbolAddress), so make one call before capturing.  The
 *     library keeps those device addresses for the life of the process: after
 *     a cudaDeviceReset(), unload and reload the library before calling it.
 *   - Layouts are row-major and contiguous.  N = total packed tokens,
 *     B = sequences (prefill) or rows (decode), H = heads.
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KDA_OK = 0,
  KDA_ERR_INVALID_ARG = 1,    /* bad pointer, size, alignment, overlap, dtype */
  KDA_ERR_UNSUPPORTED = 2,    /* valid but not built: head dims, chunk size */
  KDA_ERR_CUDA = 3,           /* a CUDA runtime call failed (launch, attribute) */
  KDA_ERR_DEVICE_TIMEOUT = 4, /* a bounded device-side wait gave up */
  KDA_ERR_DEVICE_CHECK = 5    /* a device-side argument check failed */
} kda_status;

/* KDA_E4M3 and KDA_I8 are output types of kda_rms_norm() only. */
typedef enum { KDA_F32 = 0, KDA_BF16 = 1, KDA_E4M3 = 2, KDA_I8 = 3 } kda_dtype;

/*
 * Layout of log_alpha.  KDA_GATE_CHANNEL: one decay per key channel, [.., H, dk]
 * (Kimi Delta Attention).  KDA_GATE_HEAD: one decay per token and head, [.., H],
 * applied to every channel of the state: the head-wise gate of Gated DeltaNet,
 * the coarser special case KDA refines ("Kimi Linear's 75% KV cache cut ...",
 * theclarity.today, third paragraph; "Kimi Linear wlasnie pokonal ...",
 * remio.ai, section "Jak Kimi Linear wykorzystuje inteligentniejsza pamiec
 * rekurencyjna").  The result equals the per-channel operator with the gate
 * broadcast over d_k; the head-wise layout reads 4 bytes of gate per token and
 * head instead of 4 * dk.
 */
typedef enum { KDA_GATE_CHANNEL = 0, KDA_GATE_HEAD = 1 } kda_gate;

/*
 * Chunkwise prefill over a packed variable-length batch.
 *
 * Fields (all device pointers, caller-owned):
 *   dtype        type of q, k, v and o.  log_alpha, beta and the states are
 *                always fp32.
 *   num_seqs     B >= 0 sequences; total_tokens N >= 0; H >= 1 heads;
 *   dk, dv       head dimensions, each 64 or 128.
 *   q, k         [N, H, dk]; v [N, H, dv]; 16-byte aligned.
 *   log_alpha    [N, H, dk] fp32 (gate = KDA_GATE_CHANNEL, 16-byte aligned) or
 *                [N, H] fp32 (gate = KDA_GATE_HEAD, 4-byte aligned): natural
 *                log of the forget gate; finite and <= 0 (values outside that
 *                range are not checked and give unspecified results).
 *   beta         [N, H] fp32, finite.
 *   cu_seqlens   [B+1] int32: cu[0] = 0, non-decreasing, cu[B] = N; sequence b
 *                owns packed rows [cu[b], cu[b+1]).  Checked on the device
 *                (KDA_ERR_DEVICE_CHECK, nothing written).
 *   pad_mask     [N] uint8, 1 = valid, 0 = pad; NULL = all valid.  A pad is an
 *                identity step with o = 0.  Pads at the two ends of a sequence
 *                are skipped outright, so a run with edge pads is bit-identical
 *                to the unpadded run; pads between valid tokens are identity
 *                steps inside a chunk (equal to the unpadded run up to
 *                rounding).  Requires a workspace.
 *   init_state   [B, H, dk, dv] fp32 (dv contiguous), 16-byte aligned; NULL = 0.
 *   o            [N, H, dv] of dtype; must not overlap any input.
 *   final_state  [B, H, dk, dv] fp32 or NULL (not written).  It may be the same
 *                pointer as init_state (in-place update) but may not otherwise
 *                overlap an input.
 *   chunk        0 (default: 64 for bf16, 16 for fp32), 16, 32 or 64; 128 or
 *                256 for bf16 with d_k = d_v = 128 and the full workspace (the
 *                tensor-core path merges 64-row chunks into longer ones: the
 *                pages' chunk of 256, "Kimi Linear's 75% KV cache cut ...",
 *                theclarity.today, fourth paragraph), else KDA_ERR_UNSUPPORTED.
 *                The result is defined by the recurrence and does not depend on
 *                the chunk size beyond rounding.
 *   workspace    device scratch, 256-byte aligned.  kda_prefill_workspace_size()
 *                bytes select the fastest path (for bf16, d_k = d_v = 128,
 *                chunk 64: a two-kernel path that stores each chunk's
 *                intermediate tiles, about 73 KB per 64 tokens and head; chunk
 *                128 / 256 also store the merged chunk items, about 2.5 / 3 KB
 *                per token and head in all).  A
 *                smaller workspace selects a fused single-kernel path; a pad
 *                mask needs at least 16 bytes per sequence (rounded up to 256).
 *                May be NULL when pad_mask is NULL.
 *   gate         layout of log_alpha (kda_gate); 0 = per channel.  With
 *                KDA_GATE_HEAD the single-kernel tensor-core path is not used
 *                (a small workspace selects the CUDA-core path).
 * Numerics: bf16 inputs take the tensor-core path (bf16 operands, fp32
 * accumulation, fp32 state); fp32 inputs take an fp32 CUDA-core path.  o is
 * rounded once (round to nearest even) to its dtype.
 */
typedef struct {
  kda_dtype dtype;
  int num_seqs;
  int total_tokens;
  int H;
  int dk;
  int dv;
  const void *q;
  const void *k;
  const void *v;
  const float *log_alpha;
  const float *beta;
  const int32_t *cu_seqlens;
  const uint8_t *pad_mask;
  const float *init_state;
  void *o;
  float *final_state;
  int chunk;
  void *workspace;
  size_t workspace_bytes;
  kda_gate gate;
} kda_prefill_args;

/* Bytes of workspace for the fastest path of kda_prefill() with these
 * arguments (reads only dtype, sizes and chunk).  Returns 0 if args is NULL. */
size_t kda_prefill_workspace_size(const kda_prefill_args *args);

/* Enqueue one prefill.  Returns KDA_OK or an argument/launch error. */
kda_status kda_prefill(const kda_prefill_args *args, void *stream);

/*
 * kda_prefill without a workspace argument.  The pages have no counterpart to
 * this call: it serves callers that cannot call cudaMalloc where they run the
 * operator (an engine whose device memory is owned up front by a host
 * framework that passes operators only their tensors, or a serving loop in
 * which cudaMalloc/cudaFree are not allowed because they may synchronise the
 * device).  Same arguments as kda_prefill; args->workspace and
 * args->workspace_bytes are ignored.  Its 64 KiB of scratch holds the span
 * table of the pad pre-pass but not the per-chunk items of the two-kernel
 * tensor-core path, so it runs the single-kernel tensor-core path (bf16,
 * d_k = 128, d_v a multiple of 64, chunk 64, per-channel gate) or the
 * CUDA-core path (everything else): its results equal kda_prefill's up to
 * rounding (within the same tolerances against the exact recurrence), not bit
 * for bit, and it is slower than kda_prefill with a full workspace.  The
 * scratch comes from a fixed device
 * array inside the library, sized for KDA_NOALLOC_MAX_SEQS sequences (64 KiB,
 * held by every GPU that loads the library until exit); a batch with more
 * sequences returns KDA_ERR_INVALID_ARG and launches nothing.  All calls on a
 * device share that array: calls whose kernels may overlap on the GPU race and
 * must be ordered by the caller.  The first call on each device looks up the
 * array's device address; make it before any stream capture.  Allocates no
 * memory.
 */
#define KDA_NOALLOC_MAX_SEQS 4096
kda_status kda_prefill_noalloc(const kda_prefill_args *args, void *stream);

/*
 * One decode step: one new token for each of B independent rows, all heads.
 *   q, k [B, H, dk]; v [B, H, dv] of dtype; log_alpha [B, H, dk] fp32, or
 *   [B, H] fp32 with gate = KDA_GATE_HEAD; beta [B, H] fp32; mask [B] uint8 (1 = active, NULL = all active);
 *   state [B, H, dk, dv] fp32, updated in place, 16-byte aligned;
 *   o [B, H, dv] of dtype, must not overlap any other argument.
 * A masked row's state is neither read nor written and its o is written as 0.
 * The step is: S' = Diag(alpha) S; p = S'^T k; S = S' + k (beta (v - p))^T;
 * o = S^T q.
 */
typedef struct {
  kda_dtype dtype;
  int B;
  int H;
  int dk;
  int dv;
  const void *q;
  const void *k;
  const void *v;
  const float *log_alpha;
  const float *beta;
  const uint8_t *mask;
  float *state;
  void *o;
  kda_gate gate;
} kda_decode_args;

kda_status kda_decode(const kda_decode_args *args, void *stream);

/*
 * Short causal convolution of the layer's inputs, padding-correct, with a
 * carried convolution state (the convolution window a cached continuation
 * keeps besides the recurrent state: "Transformers Community Reports Kimi
 * Linear Cache Bug", ainews, paragraphs on the reproduction and the follow-up
 * investigation -- padded entries must neither enter the window nor advance the
 * convolution state).  Depthwise, per channel c of sequence b, over the
 * sequence's VALID positions only:
 *   y_t[c] = bias[c] + sum_{i<W} weight[c*W + i] * u_i[c]
 * where u_0 .. u_{W-2} are the W-1 valid inputs before t (oldest first) and
 * u_{W-1} = x_t; before the sequence's first valid inputs the window holds the
 * incoming state.  A pad position has y = 0 and changes nothing.  No activation
 * is applied.  Fields (device pointers, caller-owned):
 *   dtype        type of x and y (KDA_BF16 or KDA_F32); everything else fp32.
 *   num_seqs     B >= 0; total_tokens N >= 0; D >= 8 channels, a multiple of 8.
 *   width        W in 1..4.
 *   x, y         [N, D], 16-byte aligned; y must not overlap any input.
 *   weight       [D, W]; bias [D] or NULL (zeros).
 *   cu_seqlens   [B+1] int32, as for kda_prefill (checked on the device).
 *   pad_mask     [N] uint8 (1 = valid) or NULL.
 *   state_in     [B, W-1, D] (oldest row first), 16-byte aligned, or NULL (zeros).
 *   state_out    [B, W-1, D]: the last W-1 valid inputs of each sequence
 *                (completed from state_in when the sequence has fewer), or
 *                NULL.  May be the same pointer as state_in (in-place update),
 *                may not otherwise overlap an input.
 * A decode step is a call with one token per sequence.  Allocates nothing.
 */
typedef struct {
  kda_dtype dtype;
  int num_seqs;
  int total_tokens;
  int D;
  int width;
  const void *x;
  const float *weight;
  const float *bias;
  const int32_t *cu_seqlens;
  const uint8_t *pad_mask;
  const float *state_in;
  float *state_out;
  void *y;
} kda_conv_args;

kda_status kda_short_conv(const kda_conv_args *args, void *stream);

/*
 * Backward pass of kda_prefill (training): the gradients of <o, grad_o> +
 * <final_state, grad_final_state> with respect to q, k, v, log_alpha, beta and
 * init_state, by the blockwise algorithm ("Kimi Linear wlasnie pokonal ...",
 * remio.ai, section "Jak Kimi Linear wykorzystuje inteligentniejsza pamiec
 * rekurencyjna": the chunked form serves training as well as inference).  Chunks
 * of 64 rows: the chunk quantities (pairwise decay products, so exact for any
 * log_alpha <= 0) and every gradient of a chunk's rows are computed for all
 * chunks in parallel; only the state at each chunk start (forward) and its
 * gradient at each chunk end (backward) are chained over a sequence's chunks.
 * fp32 accuracy throughout: the gradient kernel's dense products run on the tensor
 * cores with each fp32 operand split into two tf32 parts (three products), the
 * rest on CUDA cores in fp32.
 * Fields (device pointers, caller-owned):
 *   dtype, num_seqs, total_tokens, H, dk, dv, q, k, v, log_alpha, beta,
 *   cu_seqlens, pad_mask, init_state, gate   as for kda_prefill (chunk is not
 *                used; the result does not depend on it).
 *   grad_o           [N, H, dv] fp32.
 *   grad_final_state [B, H, dk, dv] fp32 or NULL (zero).
 *   grad_q, grad_k   [N, H, dk] fp32; grad_v [N, H, dv] fp32;
 *   grad_log_alpha   fp32, the layout of log_alpha; grad_beta [N, H] fp32;
 *   grad_init_state  [B, H, dk, dv] fp32 or NULL (not written).
 *                All outputs 16-byte aligned and not overlapping any input or
 *                each other; pad positions get zero gradients; rows outside
 *                every sequence are not written.
 *   workspace    kda_prefill_backward_workspace_size() bytes, 256-byte aligned:
 *                per 64-row chunk and head the chunk quantities, the state at
 *                the chunk start and its gradient at the chunk end, about
 *                5 KB per token and head for d_k = d_v = 128.
 */
typedef struct {
  kda_dtype dtype;
  int num_seqs;
  int total_tokens;
  int H;
  int dk;
  int dv;
  const void *q;
  const void *k;
  const void *v;
  const float *log_alpha;
  const float *beta;
  const int32_t *cu_seqlens;
  const uint8_t *pad_mask;
  const float *init_state;
  kda_gate gate;
  const float *grad_o;
  const float *grad_final_state;
  float *grad_q;
  float *grad_k;
  float *grad_v;
  float *grad_log_alpha;
  float *grad_beta;
  float *grad_init_state;
  void *workspace;
  size_t workspace_bytes;
} kda_backward_args;

size_t kda_prefill_backward_workspace_size(const kda_backward_args *args);
kda_status kda_prefill_backward(const kda_backward_args *args, void *stream);

/*
 * Linear attention with a decay for each head (the additive recurrence, without
 * KDA's removal of the old projection onto the key):
 *   S_t = a_t S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t,   a_t = exp(log_alpha_t)
 * per sequence b and value head h, with the state S d_k x d_v in fp32.  The same
 * conventions as kda_prefill: packed variable-length batch, pads are identity
 * steps with o = 0 whatever they hold (their memory may be read, but nothing there
 * has an effect), optional initial and final state.  An infinity or NaN in q, k or v of
 * a token that is no pad may reach o and the gradients of any token of its chunk (128
 * rows in bf16, 64 in fp32), earlier ones too: their weights are 0 there, not left
 * out.  Any result is independent of how the
 * library cuts sequences beyond rounding, and the same call gives the same bits.
 *
 * Fields (device pointers, caller-owned):
 *   dtype        type of q, k, v and o (KDA_BF16 or KDA_F32); everything else fp32.
 *   num_seqs     B >= 0; total_tokens N >= 0; H >= 1 value heads; Hk >= 1 query/key
 *                heads, a divisor of H: value head h reads query/key head
 *                h / (H / Hk).  dk, dv: each 64 or 128.
 *   q, k         [N, Hk, dk]; v, o [N, H, dv]; 16-byte aligned.
 *   log_alpha    decay = KDA_DECAY_TOKEN: [N, H], one decay per token and head;
 *                decay = KDA_DECAY_HEAD: [H], a constant of the head.  Natural
 *                log, <= 0 (not checked; positive values give unspecified results).
 *                A step below 2^-400 counts as 2^-400.  A NaN reaches o from its token
 *                on, the states behind it and the gradients, as far as later decays of the
 *                same head are not 0 in fp32.
 *   cu_seqlens   [B+1] int32 as for kda_prefill (checked on the device).
 *   pad_mask     [N] uint8, 1 = valid; NULL = all valid.
 *   init_state   [B, H, dk, dv] fp32, 16-byte aligned; NULL = 0.
 *   final_state  [B, H, dk, dv] fp32, 16-byte aligned, or NULL (not written); may be
 *                the same pointer as init_state, may not otherwise overlap an input.
 *   o            must not overlap any input.
 *   workspace    kda_linear_prefill_workspace_size() bytes, 256-byte aligned: the
 *                state at the start of every segment of a sequence.  Calls that may
 *                overlap on the GPU need workspaces of their own.
 * Numerics: products of bf16 inputs are accumulated in fp32; for o the weights
 * q.k a..a and the state are rounded to bf16 once as operands; final_state keeps fp32
 * accuracy.  fp32 inputs keep fp32 accuracy throughout.  Decays below 2^-126 count as 0.
 * The batch's lengths decide how its sequences are cut into segments, and with that the
 * order of the sums; the same lengths give the same bits.
 */
typedef enum { KDA_DECAY_TOKEN = 0, KDA_DECAY_HEAD = 1 } kda_decay;

typedef struct {
  kda_dtype dtype;
  int num_seqs;
  int total_tokens;
  int H;
  int Hk;
  int dk;
  int dv;
  const void *q;
  const void *k;
  const void *v;
  const float *log_alpha;
  const int32_t *cu_seqlens;
  const uint8_t *pad_mask;
  const float *init_state;
  void *o;
  float *final_state;
  kda_decay decay;
  void *workspace;
  size_t workspace_bytes;
} kda_linear_args;

/* Bytes of workspace (reads dtype, sizes and decay).  0 if args is NULL or invalid. */
size_t kda_linear_prefill_workspace_size(const kda_linear_args *args);
kda_status kda_linear_prefill(const kda_linear_args *args, void *stream);

/*
 * One step of the same recurrence for each of B independent rows, all heads.
 *   q, k [B, Hk, dk]; v, o [B, H, dv] of dtype; log_alpha [B, H] or [H] fp32
 *   (decay); mask [B] uint8 (1 = active, NULL = all active); state [B, H, dk, dv]
 *   fp32, updated in place, 16-byte aligned; o must not overlap any other argument.
 * A masked row's state is neither read nor written and its o is written as 0.
 */
typedef struct {
  kda_dtype dtype;
  int B;
  int H;
  int Hk;
  int dk;
  int dv;
  const void *q;
  const void *k;
  const void *v;
  const float *log_alpha;
  const uint8_t *mask;
  float *state;
  void *o;
  kda_decay decay;
} kda_linear_decode_args;

kda_status kda_linear_decode(const kda_linear_decode_args *args, void *stream);

/*
 * Backward pass of kda_linear_prefill (training): the gradients of <o, grad_o> +
 * <final_state, grad_final_state> with respect to q, k, v, log_alpha and
 * init_state.  dtype .. init_state and decay as for kda_linear_prefill.
 *   grad_o           [N, H, dv] of dtype, 16-byte aligned.
 *   grad_final_state [B, H, dk, dv] fp32 or NULL (zero).
 *   grad_q, grad_k   [N, Hk, dk], grad_v [N, H, dv] of dtype (the types in which
 *                    training hands them on); of a shared query/key head the sum
 *                    over its value heads, taken in fp32.
 *   grad_log_alpha   fp32, the layout of log_alpha ([H]: the sum over the tokens).
 *   grad_init_state  [B, H, dk, dv] fp32 or NULL (not written).
 *                    Outputs 16-byte aligned (grad_log_alpha 4), not overlapping any
 *                    input or each other; pads get zero gradients.
 *   workspace        kda_linear_prefill_backward_workspace_size() bytes, 256-byte aligned.
 * Sums over shared heads and tokens are taken in a fixed order: the same call gives
 * the same bits.
 * Numerics with bf16 inputs: on the way to grad_q, grad_k and grad_v the weights, the
 * states and their gradients are rounded to bf16 once as operands; grad_log_alpha and
 * grad_init_state take them as two and three bf16 parts (2^-16, 2^-24).
 */
typedef struct {
  kda_dtype dtype;
  int num_seqs;
  int total_tokens;
  int H;
  int Hk;
  int dk;
  int dv;
  const void *q;
  const void *k;
  const void *v;
  const float *log_alpha;
  const int32_t *cu_seqlens;
  const uint8_t *pad_mask;
  const float *init_state;
  kda_decay decay;
  const void *grad_o;
  const float *grad_final_state;
  void *grad_q;
  void *grad_k;
  void *grad_v;
  float *grad_log_alpha;
  float *grad_init_state;
  void *workspace;
  size_t workspace_bytes;
} kda_linear_backward_args;

size_t kda_linear_prefill_backward_workspace_size(const kda_linear_backward_args *args);
kda_status kda_linear_prefill_backward(const kda_linear_backward_args *args, void *stream);

/*
 * Root-mean-square norm of rows, with the residual's addition and an optional
 * 8-bit output with scales:
 *   r = x + residual (rounded to dtype; r = x without a residual)
 *   y = r / sqrt(mean(r^2) + eps) * weight
 * Fields (device pointers, caller-owned):
 *   dtype        type of x, residual, residual_out (KDA_BF16 or KDA_F32).
 *   out_dtype    type of y: dtype, KDA_E4M3 or KDA_I8 (8 bits, with scale).
 *   rows >= 0; D columns: a multiple of 8, 8 .. 16384.
 *   x            [rows, D]; residual [rows, D] or NULL; y [rows, D]; 16-byte aligned
 *                (an 8-bit y: 8-byte).
 *   weight       [D] fp32, 16-byte aligned, or NULL (ones).  eps >= 0, finite.
 *   group        8-bit output: 0 = one scale per row, or 32, 64 or 128 = one scale per
 *                group of that many columns (the last may be short).
 *   scale        8-bit output: fp32 [rows, 1] or [rows, ceil(D / group)]:
 *                max(max|y|, 2^-100) / 448 (e4m3) or / 127 (int8), and the stored value is
 *                y / scale (as y times the reciprocal of scale, both in fp32) rounded to nearest
 *                even.  A NaN in a group makes its scale NaN.
 *   residual_out [rows, D] r, or NULL; needs residual; may be the same pointer as residual.
 * The mean is taken in fp32: a row whose squares sum to more than 3.4e38 gives y = 0, and
 * with eps = 0 one whose squares sum to less than 1.2e-38 loses digits, down to y infinite.
 * Outputs may not otherwise overlap an input or each other.  Allocates nothing.
 */
typedef struct {
  kda_dtype dtype;
  kda_dtype out_dtype;
  int64_t rows;
  int D;
  const void *x;
  const void *residual;
  const float *weight;
  float eps;
  int group;
  void *y;
  float *scale;
  void *residual_out;
} kda_rms_norm_args;

kda_status kda_rms_norm(const kda_rms_norm_args *args, void *stream);

/*
 * Backward pass of kda_rms_norm (the output before any 8-bit rounding).
 *   x             [rows, D] of dtype: the normalised input (residual_out, or x).
 *   grad_y        [rows, D] of dtype; grad_residual [rows, D] of dtype or NULL: the
 *                 gradient that reaches r along the residual stream, added to grad_x.
 *   grad_x        [rows, D] of dtype: the gradient of r, which is that of x and of the
 *                 residual; may be the same pointer as grad_residual.
 *   grad_weight   [D] fp32 or NULL (not computed); the sum over rows in fp32, in a fixed order.
 *   workspace     kda_rms_norm_backward_workspace_size() bytes, 256-byte aligned; NULL
 *                 without grad_weight.
 */
typedef struct {
  kda_dtype dtype;
  int64_t rows;
  int D;
  const void *x;
  const float *weight;
  float eps;
  const void *grad_y;
  const void *grad_residual;
  void *grad_x;
  float *grad_weight;
  void *workspace;
  size_t workspace_bytes;
} kda_rms_norm_backward_args;

/* Bytes of workspace (reads dtype, rows and D).  0 if args is NULL or these are invalid. */
size_t kda_rms_norm_backward_workspace_size(const kda_rms_norm_backward_args *args);
kda_status kda_rms_norm_backward(const kda_rms_norm_backward_args *args, void *stream);

/* Synchronise `stream`, then return and clear the error latched on the
 * current device by earlier kernels (KDA_OK if none).  The word is the
 * device's, so an error of a call on another stream is returned and cleared
 * too.  A linear-attention call that was refused on the device stays refused
 * then (it keeps a mark of its own in its workspace); for kda_prefill,
 * kda_prefill_noalloc and kda_prefill_backward ask only once the calls on
 * other streams have ended. */
kda_status kda_get_device_status(void *stream);

/*
 * Test hook for failure detection without a GPU fault (the pages have no
 * counterpart).  Every device-side wait of the prefill kernels is bounded;
 * when one runs out the kernel drains what it has in flight, releases its
 * tensor memory, latches KDA_ERR_DEVICE_TIMEOUT and returns, so the context
 * stays usable.  This hook lets a test make that happen on purpose:
 *   fault        0 (normal operation) or KDA_FAULT_STARVE_STATE_LOADS: the
 *                state pass of the workspace-backed tensor-core prefill issues
 *                none of its item loads, so its waits run out; nothing is read
 *                or written out of bounds and the call's outputs are left
 *                unspecified.
 *   wait_cycles  the limit, in SM clock cycles, of every bounded wait in later
 *                prefill and linear-attention calls; <= 0 restores the default (about 2 s).
 * Process-wide and read at each call; meant for tests only.
 * Returns KDA_ERR_INVALID_ARG for an unknown fault bit.
 */
#define KDA_FAULT_STARVE_STATE_LOADS 1
kda_status kda_debug_set_fault(int fault, long long wait_cycles);

/*
 * Which bounded wait ran out first on the current device since the last call
 * (0: none): a diagnostic beside KDA_ERR_DEVICE_TIMEOUT.  Synchronises
 * `stream`, then returns and clears the code; -1 if a CUDA call failed.
 * Codes: workspace-backed tensor-core prefill, intra-chunk kernel: 1 Gram
 * products, 2 V tile, 3 W and U_v products, 4 staged log_alpha rows; its state
 * pass: 11 item load,
 * 12 first product group of a chunk, 13 second product group, 14 buffer
 * release (loading side); single-kernel tensor-core prefill: 21-26 (its six
 * waits in program order); chunks of 128 / 256: the state pass uses 11-14 as
 * above (11 any item tile) and 16 for the U_v block, the merge kernels 31
 * (operand loads), 32 and 33 (their two product groups); linear attention in bf16:
 * 41-51 a segment's share of the state, 55-69 a segment's outputs, 71-80 the backward
 * pass's states, 91-117 its gradients.
 */
int kda_debug_timeout_site(void *stream);

/* Static string for a status code; never NULL. */
const char *kda_status_string(kda_status status);

/* ABI version: (major << 16) | minor. */
int kda_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
