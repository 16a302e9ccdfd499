/*
 * fp8z1_ops.h -- model operators next to the optimizer step: what consumes
 * the FP8 weights the step writes and produces the FP32 weight gradients the
 * next step reads.  Part of libfp8z1.so (sm_103a).
 *
 *   embedding   rows of an FP8 table, scaled; the table's gradient;
 *   gated FFN   (silu(x Wg) * (x Wu)) Wd of each expert on its own tokens,
 *               forward and backward;
 *   distillation  loss against a teacher's top logits, and its gradient.
 *
 * Conventions, beside those of fp8z1.h (status codes, streams, no work
 * enqueued by a rejected call, no exception across the ABI):
 *   - An FP8 weight is row-major E4M3 codes [E, R, C] (uint8) and its FP32
 *     block scales [E, ceil(R/128), ceil(C/128)]: the value of code c of
 *     element (e, r, col) is e4m3(c) * scale[e][r/128][col/128].  That is what
 *     fp8z1_step_fused writes (the scales of a param are a view of the scale
 *     buffer, fp8z1_param_blocks).
 *   - Activations are row-major with a row stride ("ld") in elements.
 *   - Every buffer is the caller's.  A workspace is scratch: its contents need
 *     not be set before a call nor kept after it, and calls that may overlap
 *     on the device must not share one.
 */
#ifndef FP8Z1_OPS_H
#define FP8Z1_OPS_H

#include "fp8z1.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types of activations, logits and their gradients */
#define FP8Z1_F32 0
#define FP8Z1_BF16 1

/* ---- embedding -------------------------------------------------------------- */

/* out[t, d] = alpha * (e4m3(codes[id_t, d]) * scales[id_t / 128, d / 128]) in
 * FP32, rounded once to `out_type` (FP8Z1_F32 or FP8Z1_BF16).  `ids`: device,
 * `tokens` integers of `id_bytes` (4 or 8) bytes, signed; an id outside
 * [0, vocab) is no token and gives a row of zeros.  `codes`: [vocab, dim].
 * `out`: rows of `dim` elements, ld_out >= dim apart.  Any dim >= 1 and any
 * alignment of the element types; rows of a multiple of 8 elements, codes on
 * 8-byte and `out` on 16-byte boundaries, are read 8 and written 16 bytes at a
 * time.
 * tokens == 0 enqueues nothing.
 * Errors: EINVAL (null, vocab < 1 or >= 2^31, dim < 1 or > 2^23, tokens < 0 or
 * > 2^30, id_bytes, out_type, ld_out < dim, alpha not finite), EALIGN, ECUDA. */
int fp8z1_embed(int64_t vocab, int64_t dim, const uint8_t* codes, const float* scales, const void* ids,
                int32_t id_bytes, int64_t tokens, float alpha, void* out, int32_t out_type, int64_t ld_out,
                void* stream);

/* Bytes of workspace fp8z1_embed_grad needs.  Host only. */
int fp8z1_embed_grad_workspace(int64_t vocab, int64_t dim, int64_t tokens, int64_t* bytes);

/* d_table[v, d] = alpha * sum over {t : id_t = v} of dy[t, d]: every row of the
 * FP32 [vocab, dim] gradient is written (rows without a token with zeros), as
 * the optimizer's next step reads it.  The sum is FP32 in a fixed order (the
 * tokens are sorted by id, equal ids in order of t), so results repeat bit for
 * bit.  Ids outside [0, vocab) are skipped.  dy: `dy_type`, ld_dy apart.
 * Errors: EINVAL (null, sizes, id_bytes, dy_type, ld_dy < dim, alpha not
 * finite), EALIGN (workspace: 256 bytes), ECUDA. */
int fp8z1_embed_grad(int64_t vocab, int64_t dim, const void* ids, int32_t id_bytes, int64_t tokens, float alpha,
                     const void* dy, int32_t dy_type, int64_t ld_dy, float* d_table, void* workspace,
                     void* stream);

/* ---- gated feed-forward block -------------------------------------------------- */

/* Experts e = 0 .. experts-1, each on its own run of token rows:
 *   g = x Wg,  u = x Wu,  h = silu(g) * u,  y = h Wd,   silu(a) = a / (1 + exp(-a)),
 * with [Wg | Wu] = gate_up[e], FP8 [hidden, 2 * inner], and Wd = down[e], FP8
 * [inner, hidden].  experts = 1 is a dense block. */
typedef struct {
    int64_t tokens;  /* rows of x, 0 .. 2^30 */
    int64_t hidden;  /* a multiple of 16, below 2^24 */
    int64_t inner;   /* a multiple of 128, below 2^23 */
    int64_t experts; /* 1 .. 1024 */
} fp8z1_ffn_dims;

/* Bytes of the buffer a forward pass keeps for its backward pass, and of the
 * workspaces of both.  Host only.  Errors: EINVAL. */
int fp8z1_ffn_sizes(const fp8z1_ffn_dims* dims, int64_t* saved_bytes, int64_t* forward_bytes,
                    int64_t* backward_bytes);

/* y = the block of x.  `d_offsets`: device int32 [experts + 1], expert e has
 * rows [d_offsets[e], d_offsets[e + 1]) (ascending from 0; an empty run is an
 * expert without tokens), or NULL when experts == 1 (every row).  Rows from
 * d_offsets[experts] on belong to no expert and get y = 0.  x, y: BF16,
 * 16-byte aligned, ld_x, ld_y multiples of 8.  gate_up, down: 16-byte aligned.
 * `saved`: NULL, or fp8z1_ffn_sizes' saved_bytes for fp8z1_ffn_backward
 * (256-byte aligned, as `workspace`).
 * Accumulation is FP32; h is rounded between the two products, to 9 significant
 * bits (BF16 has 8) or 2^-17 of the largest of its 128 neighbours, and y once at
 * the end.  (One token, and up to four of small blocks, keep h in FP32: a token's y
 * may change in its last place when others join.)  x is held exactly down to
 * 2^-13 of the largest of its 128 neighbours, to 2^-21 of that below.  An infinity
 * or NaN in a row of x leaves that row of y without finite numbers.
 * y does not depend on `saved`; results repeat bit for bit.
 * Errors: EINVAL, EALIGN, ECUDA. */
int fp8z1_ffn_forward(const fp8z1_ffn_dims* dims, const void* x, int64_t ld_x, const int32_t* d_offsets,
                      const uint8_t* gate_up, const float* gate_up_scale, const uint8_t* down,
                      const float* down_scale, void* y, int64_t ld_y, void* saved, void* workspace, void* stream);

/* The gradients of sum(dy * y), from the same x, offsets and weights and the
 * buffer that forward pass filled:
 *   dh = dy Wd^T,  dg = dh * u * s (1 + g (1 - s)),  du = dh * silu(g),  s = sigmoid(g),
 *   dx = [dg | du] gate_up^T (BF16; NULL leaves it out; dg and du rounded for
 *        it as h is for y),
 *   d_gate_up = x^T [dg | du],  d_down = h^T dy,  FP32 [E, R, C] row-major: the
 * optimizer's grads.  Every element is written (zeros for an expert without
 * tokens; dx = 0 in rows of no expert).  dy, dx as x above; d_gate_up and
 * d_down 16-byte aligned.  The weight gradients carry FP32 accuracy, every column
 * of d_gate_up and row of d_down relative to its own size; of x and dy, elements
 * below 2^-32 of the expert's largest lose bits there.
 * Errors: EINVAL, EALIGN, ECUDA. */
int fp8z1_ffn_backward(const fp8z1_ffn_dims* dims, const void* dy, int64_t ld_dy, const void* x, int64_t ld_x,
                       const int32_t* d_offsets, const uint8_t* gate_up, const float* gate_up_scale,
                       const uint8_t* down, const float* down_scale, const void* saved, void* dx, int64_t ld_dx,
                       float* d_gate_up, float* d_down, void* workspace, void* stream);

/* The feed-forward kernels' warps wait for one another on barriers in shared
 * memory, and every wait ends: one that has not been answered after four seconds
 * and 100000 tries (a paused process does not run out of tries) gives up, and what
 * its CTA could not finish is NaN, in y, dx, the weight gradients or `saved`; a
 * NaN gradient sets the step's found_inf.  Reads and clears the number of threads
 * that gave up on the current device since the last call (synchronous; 0 in all
 * normal use).  Errors: EINVAL (null), ECUDA. */
int fp8z1_ffn_timeouts(uint32_t* count);

/* Test hook of a checked build (whose waits give up after 0.2 seconds): from the
 * next call on, the first CTA of the kernels of `kernels` does not announce its
 * first sums, so that the waits for them run out.  Bits: 1 gate_up, 2 down, 4 dh,
 * 8 dx, 16 a product split along K, 32 d_down, 64 d_gate_up; 0 ends it.
 * Synchronous.  Errors: EINVAL (a release build), ECUDA. */
int fp8z1_checked_ffn_stall(uint32_t kernels);

/* ---- distillation ----------------------------------------------------------------- */

/* Row r's loss against the teacher's `top` listed logits, at temperature tau:
 *   p = softmax(teacher_logits / tau) over the listed entries,
 *   q = softmax(logits / tau) over the vocabulary,
 *   loss[r] = tau^2 sum_k p_k (log p_k - log q[id_k]).
 * and, when `dlogits` is not NULL, the gradient of sum_r row_weight[r] loss[r]:
 *   dlogits[r, j] = row_weight[r] * tau * (q_j - sum over {k : id_k = j} of p_k).
 * `logits`: [rows, vocab] of `type` (FP8Z1_F32 or FP8Z1_BF16), ld apart;
 * `dlogits` the same type, ld_d apart; it may be `logits` itself (ld_d == ld).
 * `teacher_ids`, `teacher_logits`: [rows, top], int32 and FP32, dense; an entry
 * whose id lies outside [0, vocab) or whose logit is -inf is absent.  An id may
 * be listed twice (its p add up).  `row_weight`: FP32 [rows], or NULL for 1.
 * A row of weight 0, or without any teacher entry, is not read: its loss and
 * gradient are 0.  A row whose logits are all -inf has q = 0 (loss +inf).
 * `loss`: FP32 [rows], not weighted.  rows == 0 enqueues nothing.
 * Errors: EINVAL (null, rows < 0, vocab < 1 or >= 2^31, top outside 1 .. 1024,
 * type, ld < vocab, tau not positive and finite), EALIGN, ECUDA. */
#define FP8Z1_DISTILL_MAX_TOP 1024
int fp8z1_distill(const void* logits, int32_t type, int64_t ld, int64_t rows, int64_t vocab,
                  const int32_t* teacher_ids, const float* teacher_logits, int64_t top, float temperature,
                  const float* row_weight, float* loss, void* dlogits, int64_t ld_d, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8Z1_OPS_H */
