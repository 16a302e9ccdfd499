/*
 * fp8z1_ops.h -- model operators next to the optimizer step: what consumes
 * the FP8 weights the step writes and produces the FP32 weight gradients the
 * next step reads.  Part of libfp8z1.so (sm_103a).
 *
 *   embedding   rows of an FP8 table, scaled; the table's gradient;
 *   gated FFN   (silu(x Wg) * (x Wu)) Wd of each expert on its own tokens,
 *               forward and backward;
 *   distillation  loss against a teacher's top logits, and its gradient;
 *   RMS norm    of rows, the residual added first, in 16, 32 or 8 bits; its gradient;
 *   product     act(x W + bias) + residual, its gradients;
 *   routing     tokens sorted by expert, their rows gathered and joined again,
 *               and the gradients of both.
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
#define FP8Z1_E4M3 2 /* rows of codes with a scale for every 128 columns (fp8z1_linear's x) */

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

/* ---- root-mean-square norm --------------------------------------------------------- */

/* Row by row, in FP32:
 *   s = x + residual, rounded to `type` and written to `total` (without a residual s = x),
 *   y = s * (mean_j s_j^2 + eps)^-1/2 * weight,
 * y rounded once: to `type` in `y`, and to E4M3 in `codes` ([rows, dim], dense) with a
 * scale for every 128 columns in `scales` ([rows, ceil(dim / 128)], dense): c = max |y| / 448 of
 * the 128, codes those of y times 1 / c in FP32; a value is its code times its scale.  128 numbers
 * below 2^-117 are 0, with a scale of 1.  `y` or `codes` may be NULL (codes and scales together),
 * not both.
 * x, residual, total, y: `type`, rows of `dim` elements, ld >= dim apart; total and y may be
 * x or residual themselves (of one stride); else a result shares no memory with another one or
 * with what the norm reads (EINVAL).  weight: FP32 [dim].  Any alignment of the element types;
 * dim and strides of whole 16 bytes on 16-byte boundaries are moved 8 elements at a time.
 * No row is too large: squares beyond FP32 are summed scaled down.  An infinity or NaN
 * leaves its row without finite numbers (but 0 where a finite element meets an infinity's norm).
 * rows == 0 enqueues nothing.
 * Errors: EINVAL (null, rows < 0 or > 2^30, dim outside 1 .. 16384, type, strides, eps outside
 * 1e-20 .. 1e20, residual without total or total without residual, y == total), EALIGN, ECUDA. */
int fp8z1_rms_norm(int64_t rows, int64_t dim, const void* x, int32_t type, int64_t ld_x, const void* residual,
                   int64_t ld_r, const float* weight, float eps, void* total, int64_t ld_total, void* y, int64_t ld_y,
                   uint8_t* codes, float* scales, void* stream);

/* Bytes of workspace fp8z1_rms_norm_grad needs.  Host only. */
int fp8z1_rms_norm_grad_workspace(int64_t rows, int64_t dim, int64_t* bytes);

/* The gradients of sum(dy * y) from the rows s that were normed (`total`, or x itself):
 *   g = dy * weight,  h = s * rstd,  dx = rstd * (g - h * mean_j(g_j h_j)) + d_total,
 *   d_weight = sum over the rows of dy * h   (FP32 [dim], every element written).
 * dx is the gradient of x and of the residual; d_total (NULL: none) is what reaches s past the
 * norm.  dy, total, d_total, dx: `type`; dx may be dy, total or d_total itself (of one stride); else
 * it shares no memory with them, weight or d_weight (EINVAL).  Sums are FP32 in a
 * fixed order: results repeat bit for bit.
 * Errors: as fp8z1_rms_norm; EALIGN (workspace: 256 bytes). */
int fp8z1_rms_norm_grad(int64_t rows, int64_t dim, const void* dy, int32_t type, int64_t ld_dy, const void* total,
                        int64_t ld_total, const float* weight, float eps, const void* d_total, int64_t ld_dt, void* dx,
                        int64_t ld_dx, float* d_weight, void* workspace, void* stream);

/* As fp8z1_ffn_timeouts, of the norm's gradient, whose rows of more than 1024 columns are copied ahead to its
 * warps: a copy that does not come leaves NaN in its rows of dx and in d_weight. */
int fp8z1_rms_norm_timeouts(uint32_t* count);

/* As fp8z1_checked_ffn_stall.  Bits: of the first CTA's first row, 1 it is never copied, 2 a warp does
 * not give its place back to the next one. */
int fp8z1_checked_rms_norm_stall(uint32_t kernels);

/* ---- routing ------------------------------------------------------------------------- */

/* Sorts the choices (t, j), 0 <= t < tokens, 0 <= j < top, by their expert ids[t, j]
 * (`id_bytes` 4 or 8, signed; an id outside [0, experts) is no choice):
 *   offsets [experts + 1]: expert e has rows [offsets[e], offsets[e + 1]) (as
 *     fp8z1_ffn_forward takes them, over tokens * top rows);
 *   place [tokens, top]: the row of choice (t, j), -1 where there is none.
 * An expert's rows are in the order of the choices; an expert may be chosen twice by a
 * token and has two rows then.  tokens == 0 writes the offsets alone.
 * Errors: EINVAL (null, a result over the other or over ids, tokens < 0, tokens * top > 2^30, top outside 1 .. 64, experts
 * outside 1 .. 1024, id_bytes), EALIGN, ECUDA. */
int fp8z1_route(const void* ids, int32_t id_bytes, int64_t tokens, int64_t top, int64_t experts, int32_t* offsets,
                int32_t* place, void* stream);

/* rows[place[t, j]] = x[t], bit for bit; rows from offsets[experts] to tokens * top are
 * cleared.  x: [tokens, dim], rows: [tokens * top, dim], both `type`.  tokens == 0 enqueues
 * nothing.  Errors: EINVAL (as fp8z1_route, dim outside 1 .. 2^23, type, strides, rows sharing
 * memory with what the call reads), EALIGN, ECUDA. */
int fp8z1_dispatch(int64_t tokens, int64_t top, int64_t experts, int64_t dim, const void* x, int32_t type, int64_t ld_x,
                   const int32_t* offsets, const int32_t* place, void* rows, int64_t ld_rows, void* stream);

/* y[t] = residual[t] + sum_j weight[t, j] * rows[place[t, j]] over the choices that have a
 * row, in FP32 in the order of j, the residual last, rounded once to `type`.  weight: FP32
 * [tokens, top], NULL for 1 (which is fp8z1_dispatch's gradient); residual NULL: none; y may
 * be residual itself (of one stride); else it shares no memory with what the call reads.  Errors: as
 * fp8z1_dispatch. */
int fp8z1_combine(int64_t tokens, int64_t top, int64_t dim, const void* rows, int32_t type, int64_t ld_rows,
                  const int32_t* place, const float* weight, const void* residual, int64_t ld_residual, void* y,
                  int64_t ld_y, void* stream);

/* The gradients of sum(dy * y) of fp8z1_combine:
 *   d_rows[place[t, j]] = weight[t, j] * dy[t]  (rows from offsets[experts] on are cleared),
 *   d_weight[t, j] = sum over the columns of dy[t] * rows[place[t, j]], FP32, 0 without a row.
 * The residual's is dy.  d_rows may be rows itself (of one stride) and d_weight weight; else a result
 * shares no memory with the other or with what the call reads.  Results repeat bit for bit.  Errors: as
 * fp8z1_dispatch. */
int fp8z1_combine_grad(int64_t tokens, int64_t top, int64_t experts, int64_t dim, const void* dy, int32_t type,
                       int64_t ld_dy, const void* rows, int64_t ld_rows, const int32_t* offsets, const int32_t* place,
                       const float* weight, void* d_rows, int64_t ld_d, float* d_weight, void* stream);

/* ---- matrix product ------------------------------------------------------------------- */

/* activations: z; z sigmoid(z); z sigmoid(sqrt(8 / pi) (z + 0.044715 z^3)), GELU's tanh form */
#define FP8Z1_ACT_NONE 0
#define FP8Z1_ACT_SILU 1
#define FP8Z1_ACT_GELU_TANH 2

typedef struct {
    int64_t tokens;     /* rows of x, 0 .. 2^30 */
    int64_t rows, cols; /* of the FP8 weight w; cols a multiple of 16; both at most 2^22 */
    int32_t transposed; /* 0: x w, x [tokens, rows], y [tokens, cols]; 1: x w^T, x [tokens, cols], y [tokens, rows] */
    int32_t activation; /* FP8Z1_ACT_* */
    int32_t x_type;     /* FP8Z1_BF16 or FP8Z1_E4M3 */
    int32_t y_type;     /* FP8Z1_BF16 or FP8Z1_F32; dy's too */
} fp8z1_linear_dims;

/* Bytes of the workspaces of both directions (forward: 0 for E4M3 rows).  Host only.
 * Errors: EINVAL. */
int fp8z1_linear_sizes(const fp8z1_linear_dims* dims, int64_t* forward_bytes, int64_t* backward_bytes);

/* z = x w + bias (or x w^T + bias),  y = act(z) + residual, rounded once to `y_type`.
 * x: BF16 of any alignment and stride >= its width; or E4M3 codes, 16-byte aligned rows
 * (ld_x a multiple of 16), with `x_scale`, FP32 [tokens, ceil(width / 128)] dense, as
 * fp8z1_rms_norm writes them (x_scale is not read for BF16).  codes: 16-byte aligned.
 * bias: FP32 [width of y] or NULL; residual: BF16 or NULL; pre: NULL, or FP32 [tokens, width of
 * y] dense for z, which fp8z1_linear_grad reads.  y may be residual itself where both are BF16
 * of one stride; else a result shares no memory with the other or with what the product reads (EINVAL;
 * BF16 x has been read before).  Sums are FP32 over exact products of the codes and x (BF16 x down to 2^-13
 * of the largest of its 128 neighbours, to 2^-21 of that below); they repeat bit for
 * bit, and may change in their last places when other rows join.  An infinity or NaN in a row
 * of x leaves that row of y without finite numbers.  tokens == 0 enqueues nothing.
 * Errors: EINVAL, EALIGN, ECUDA. */
int fp8z1_linear(const fp8z1_linear_dims* dims, const void* x, int64_t ld_x, const float* x_scale, const uint8_t* codes,
                 const float* scales, const float* bias, const void* residual, int64_t ld_residual, void* y, int64_t ld_y,
                 float* pre, void* workspace, void* stream);

/* The gradients of sum(dy * y) for BF16 x, dz = dy * act'(z):
 *   dx = dz w^T (or dz w), BF16;  d_weight = x^T dz (or dz^T x), FP32 [rows, cols];  d_bias =
 *   sum over the rows of dz, FP32.
 * Each may be NULL, not all.  `pre`: z of the forward pass (not read without activation).
 * The residual's gradient is dy.  dy of `y_type`, dx: any alignment and stride; d_weight 16-byte
 * aligned.  The results share no memory with one another, dx none with the weight nor, where d_weight is
 * wanted, with x and (BF16 dy without activation, which d_weight's products read too) dy (EINVAL).  dz is dy itself, exact, for BF16 dy without activation; else it is rounded for dx to 9
 * significant bits (BF16 has 8) or 2^-17 of the largest of its 128 neighbours.  d_weight
 * and d_bias are FP32 sums of dz as it is, d_weight of every column relative to its own size (x: what
 * lies above 2^-31 of the largest of 256 rows x 128 columns): each 256 rows' sum is within 7e-7 of its
 * norm, and these are added one after the other (3e-6 at 8 million rows).  Every element is written.
 * Errors: EINVAL (E4M3 x too), EALIGN (workspace: 256 bytes), ECUDA. */
int fp8z1_linear_grad(const fp8z1_linear_dims* dims, const void* dy, int64_t ld_dy, const void* x, int64_t ld_x,
                      const uint8_t* codes, const float* scales, const float* pre, void* dx, int64_t ld_dx,
                      float* d_weight, float* d_bias, void* workspace, void* stream);

/* As fp8z1_ffn_timeouts, of the product's kernels (whose waits end as the
 * feed-forward kernels' do, and leave NaN in y, dx or d_weight). */
int fp8z1_linear_timeouts(uint32_t* count);

/* As fp8z1_checked_ffn_stall.  Bits: 1 products of many rows, 2 of few, 4 d_weight, 8 d_weight of a
 * transposed weight; 16 stalls nothing, but lets the kernel of few rows make every product. */
int fp8z1_checked_linear_stall(uint32_t kernels);

#ifdef __cplusplus
}
#endif

#endif /* FP8Z1_OPS_H */
