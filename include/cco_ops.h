/*
 * cco_ops.h -- operators around the MoE path of cco_moe.h, one MI355X
 * (gfx950): the router, the products grouped by expert with their
 * gradients, and the norms around a block fused with its gate and residual.
 *
 * Conventions are those of cco_moe.h: every call returns a cco_status,
 * argument errors are reported before anything is launched, launches are
 * asynchronous on `stream`, nothing is allocated, row-major tensors.
 * Beyond that:
 *   - the calls keep no state: any number may run at once, on any streams,
 *     and all may be captured into a graph;
 *   - `stream` belongs to the device that holds the tensors, and that
 *     device is current;
 *   - ld is the distance between rows in elements (at least the row's
 *     length); rows of T == 0 or zero-sized tensors may be NULL;
 *   - outputs must not overlap inputs or each other unless stated;
 *   - sums, softmax statistics and norms are held in 32 bits or more and
 *     results are rounded once, to nearest even.  Results are the same on
 *     every call: no atomics, fixed orders.
 */
#ifndef CCO_OPS_H
#define CCO_OPS_H

#include <stdint.h>

#include "cco_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
typedef enum { CCO_BF16 = 0, CCO_F16 = 1, CCO_F32 = 2 } cco_dtype;

/* -------------------------------------------------------- the router --- */

typedef enum { CCO_SCORE_SOFTMAX = 0, CCO_SCORE_SIGMOID = 1 } cco_score;

/* Choice of K experts per token out of E logits.
 *   scores   s = softmax(l) over the E logits, or s_e = 1 / (1 + exp(-l_e))
 *   choice   by the logits themselves when there is neither a bias nor
 *            groups (the scores order alike, without their rounding);
 *            otherwise by c_e = s_e + bias_e, computed in 64 bits
 *   groups   > 1: the experts form `groups` contiguous groups of E / groups;
 *            a group counts as the sum of its two largest c, the `kept`
 *            largest groups stay, and the choice is made among their experts
 *   ids      the K largest in descending order; equal values go to the lower
 *            id (groups too)
 *   weights  w_j = scale * s_j, or with renorm scale * s_j / sum_i s_i over
 *            the chosen ones (with softmax scores: the softmax over the
 *            chosen logits)
 * A logit of -inf is a masked expert: its score is 0 and its choice value
 * -inf whatever its bias, so that it is chosen only after all others (of the
 * kept groups) and with weight 0; a row of such logits gets the lowest ids
 * and weights 0.  A group's masked experts do not count in its sum.  NaN
 * logits are ordered like -inf, so the ids are valid and distinct whatever
 * the row holds; the weights follow the formula and become NaN where a NaN
 * (or, with softmax, +inf) enters it.
 */
typedef struct {
  int32_t num_experts; /* E, 1..1024 */
  int32_t topk;        /* K, 1..32, at most kept * E / groups */
  int32_t score;       /* cco_score */
  int32_t renorm;      /* nonzero: the chosen scores are divided by their sum */
  float scale;
  int32_t groups;      /* 1..64, divides E; 1: no groups */
  int32_t kept;        /* 1..groups */
} cco_route_desc;

/* logits device [T][E] of `dtype`, row distance ld, aligned to an element;
 * bias device fp32 [E] or NULL; idx device int32 [T][K]; w device fp32
 * [T][K]: the inputs of cco_moe_plan and cco_moe_dispatch. */
int cco_route(const cco_route_desc *d, const void *logits, int32_t dtype, int64_t ld,
              const float *bias, int32_t T, int32_t *idx, float *w, void *stream);

/* Gradient of the weights to the logits, for the chosen ids (the choice
 * itself has none): dlogits[t][e] = sum_j dw[t][j] * d w_j / d l_e, of the
 * logits' type, row distance lddl.  Of `d` the num_experts, topk, score,
 * renorm and scale count.  The ids may be any: one outside [0, E) takes no
 * part, one that occurs twice counts twice (in the renormalising sum too).
 * dw device fp32 [T][K].  dlogits may be logits (in place, lddl = ld). */
int cco_route_grad(const cco_route_desc *d, const void *logits, int32_t dtype, int64_t ld,
                   const int32_t *idx, const float *dw, int32_t T, void *dlogits, int64_t lddl,
                   void *stream);

/* ------------------------------------------------ products by group ---- */

/* Groups of rows: group g is the rows [first[g], first[g] + count[g]) that
 * lie in [0, rows) (device int32, read when the kernel runs: the expert_off
 * and counts of cco_moe_routing fit, for one slot's experts and its rows).
 * Any count may be zero or negative (no rows).  Groups may leave rows out:
 * such rows are neither read nor written.  Groups that share rows are
 * allowed in the weight gradient; in the other two they race on the shared
 * output rows. */
typedef struct {
  int32_t groups;       /* 1..1024 */
  int32_t rows;         /* rows of the row operands, >= 0 */
  const int32_t *first; /* [groups] */
  const int32_t *count; /* [groups] */
} cco_groups;

/* Which product (for the workspace query). */
typedef enum { CCO_GROUP_PRODUCT = 0, CCO_GROUP_DX = 1, CCO_GROUP_DW = 2 } cco_group_op;

/* Bytes of workspace with which a product of these sizes splits its
 * reduction over workgroups; 0: it never does (or invalid sizes).  Products
 * with few output tiles and long reductions are split, so that they occupy
 * the GPU: the parts' fp32 sums go to the workspace and a second kernel adds
 * them in order.  Without workspace the same products run unsplit, slower
 * (and may differ from the split ones by the order of their sums). */
uint64_t cco_group_product_workspace(int32_t op, const cco_groups *g, int32_t n, int32_t k);

/* y[r][n] = sum_k x[r][k] * w[g][n][k] for the rows r of every group g.
 *   dtype  CCO_BF16 or CCO_F16, for x, w and y; sums in fp32
 *   x      [rows][k], row distance ldx;  w  [groups][n][k], dense
 *   y      [rows][n], row distance ldy
 * n, k and the row distances lie in [1, 2^21).
 * Rows of whole 16 bytes (n, k and the distances multiples of 8, pointers
 * 16-byte aligned) take the fast kernel, others a general one.
 *   workspace  NULL, or device memory of at least the size above, 16-byte
 *              aligned, in use until the call's kernels have run */
int cco_group_product(const cco_groups *g, int32_t dtype, const void *x, int64_t ldx,
                      const void *w, int32_t n, int32_t k, void *y, int64_t ldy, void *workspace,
                      uint64_t workspace_bytes, void *stream);

/* Gradient to the rows: dx[r][k] = sum_n dy[r][n] * w[g][n][k]. */
int cco_group_product_dx(const cco_groups *g, int32_t dtype, const void *dy, int64_t lddy,
                         const void *w, int32_t n, int32_t k, void *dx, int64_t lddx,
                         void *workspace, uint64_t workspace_bytes, void *stream);

/* Gradient to the weights: dw[g][n][k] = sum over the rows r of group g of
 * dy[r][n] * x[r][k], a group without rows giving zeros; with `accumulate`
 * it is added to what dw holds (in fp32, rounded once).
 *   out_dtype  type of dw [groups][n][k], dense: that of the operands, or
 *              CCO_F32 */
int cco_group_product_dw(const cco_groups *g, int32_t dtype, const void *dy, int64_t lddy,
                         const void *x, int64_t ldx, int32_t n, int32_t k, void *dw,
                         int32_t out_dtype, int32_t accumulate, void *workspace,
                         uint64_t workspace_bytes, void *stream);

/* --------------------------------------------- norms around a block ---- */

typedef enum { CCO_GATE_NONE = 0, CCO_GATE_CHANNEL = 1, CCO_GATE_TOKEN = 2 } cco_gate;

/* Residual update around a block with output y, and the norm in front of
 * the next block:
 *   z   = post ? y / rms(y) * post : y           rms(v) = sqrt(mean(v^2) + eps)
 *   out = x + scale * gate * z
 *   u   = out / rms(out) * pre   (of the unrounded out; with pre only)
 * post, pre, and a gate per channel are device [hidden] vectors of `wdtype`
 * (CCO_F32 or the rows' type); a gate per token is device fp32 [T].  post
 * and pre may be NULL.
 * Sums of squares are fp32: a normalised row whose sum passes 2^128 becomes
 * zeros, and one whose mean square lies below 2^-126 counts as eps alone. */
typedef struct {
  int32_t hidden;    /* 1..16384 */
  int32_t dtype;     /* rows: CCO_BF16, CCO_F16 or CCO_F32 */
  int32_t wdtype;    /* vectors: CCO_F32 or dtype */
  int32_t gate_kind; /* cco_gate */
  float scale;
  float eps;         /* >= 0 */
  const void *post;
  const void *gate;  /* NULL with CCO_GATE_NONE */
  const void *pre;
} cco_block_norm_desc;

/* x, y, out, u: [T][hidden] dense, aligned to an element.  y may be NULL
 * (the norm in front of a first block): then out must be NULL too, post and
 * gate NULL, and u is the norm of x.  out may be NULL if pre is given; u is
 * NULL exactly when pre is.  out may be x, u may be y (in place). */
int cco_block_norm(const cco_block_norm_desc *d, const void *x, const void *y, int32_t T,
                   void *out, void *u, void *stream);

/* Bytes of workspace cco_block_norm_grad needs for T tokens (0: none, or an
 * invalid descriptor). */
uint64_t cco_block_norm_grad_workspace(const cco_block_norm_desc *d, int32_t T);

/* Gradients from dout (to out; NULL: zero) and du (to u; NULL exactly when
 * pre is), at least one given; the forward is recomputed from x and y.
 *   dx, dy        [T][hidden] of the rows' type; dy NULL exactly when y is.
 *                 dx may be dout or x, dy may be du or y.
 *   dpost, dpre   fp32 [hidden], NULL exactly when post / pre are
 *   dgate         fp32 [hidden] or [T], NULL without a gate
 *   workspace     device, 16-byte aligned, of the size above; in use until
 *                 the call's kernels have run */
int cco_block_norm_grad(const cco_block_norm_desc *d, const void *x, const void *y,
                        const void *dout, const void *du, int32_t T, void *dx, void *dy,
                        float *dpost, float *dgate, float *dpre, void *workspace,
                        uint64_t workspace_bytes, void *stream);

/* cco_moe_combine of the staging views and cco_block_norm of its result in
 * one launch: y = the combined rows rounded to bf16 (never written), then
 * out and u as above, bit for bit what the two calls give.  d->hidden is
 * the layer's, d->dtype CCO_BF16; x, out, u bf16 [T][hidden], 16-byte
 * aligned; weights fp32 [T][K]; y_out NULL, or bf16 [T][hidden] for the
 * combined rows (a gradient's y).  After an 8-bit dispatch to identity
 * experts it is refused as cco_moe_combine is.
 * One launch, for decoding batches: with 7168 columns and top-8 it takes two
 * thirds of the two calls' time up to 256 tokens, but 1.2 times as long for
 * thousands, where the two calls are the better choice. */
int cco_moe_combine_norm(cco_moe *m, const float *weights, const cco_block_norm_desc *d,
                         const void *x, int32_t T, void *y_out, void *out, void *u,
                         void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CCO_OPS_H */
