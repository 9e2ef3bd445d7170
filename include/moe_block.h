/*
 * moe_block.h -- C ABI of libmoe_block: what stands around the expert
 * contractions in a block (token rows to expert order and back, the norms
 * with gate and residual scale), with the gradients of these and of the
 * router.
 *
 * Conventions are those of moe.h (device pointers owned by the caller, no
 * allocation, host checks before anything is enqueued, MOE_DEV_* bits in
 * *dev_status, which may be NULL here), with these additions:
 *  - Rows may be fp32 or bf16 (moe_row_type) and may be strided: row i of a
 *    matrix starts ld * i ELEMENTS after its pointer, its elements are
 *    adjacent, and ld >= the row's width.  Columns between rows are not
 *    written, and no result depends on them (a norm's rows on odd elements are
 *    read in aligned 16-byte pieces, which may begin before the row).
 *  - Any width 1 <= H <= 65536 (the norms: 16384) and any alignment that the
 *    element type has by itself.  Fastest are rows that start on 8-element
 *    boundaries (bf16: pointer % 16 == 0, fp32: pointer % 32 == 0, ld % 8 == 0),
 *    then rows that start on even elements.
 *  - Every sum, norm factor, product and gradient is computed in fp32 in a
 *    fixed order: the same bits on every call.  A bf16 output is rounded once.
 *  - Outputs must not overlap inputs or one another, except where a call
 *    says so.
 *  - T == 0 is accepted: outputs per token are empty, and outputs per column
 *    or expert (the sum of nothing) are written as zeros.
 *  - k <= 32, E <= 1024, T <= 2^30, T * k < 2^31; anything else is
 *    MOE_ENOTSUP.
 *  - Values are not checked: infinities and NaN go where the formulas take
 *    them.  Rows that no route names are never read.  Sums of squares are
 *    fp32: a norm's rows have one below 3e38 (elements below 1e17 at the widest)
 *    and, with eps 0, above 1e-37; outside that the factor is 0 or infinite.
 *  - A call may be captured into a CUDA graph; make one call of its kind on
 *    the device before, which loads the library's device code.  Captured calls
 *    that share a workspace must not be replayed at the same time.
 */
#ifndef MOE_BLOCK_H_
#define MOE_BLOCK_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_row_type { MOE_ROW_F32 = 0, MOE_ROW_BF16 = 1 } moe_row_type;

/* ABI version of this header (major * 100 + minor). */
MOE_API int moe_block_abi_version(void);

/* ---------------------------------------------------------------------------
 * moe_dispatch -- token rows into expert order, with weights applied.
 *
 *   x_perm[inv_perm[t,j], :] = w[t,j] * x[t, :]          (w NULL: factor 1)
 *
 *   x [T,H], x_perm [R,H] (out): row_type both
 *   inv_perm [T,k] int32: the slot of each route as moe_permute writes it;
 *            -1 is a route without a slot (its expert was full, or the token
 *            is padding).  Any other value outside [0,R) is treated like -1
 *            and sets MOE_DEV_BAD_EXPERT.  The slots of a call are distinct.
 *   w        [T,k] f32 or NULL
 * Rows of x_perm that no route names are left as they were.  R == 0 is
 * accepted.
 * Source: AFN-019 "Hide SSD misses before the router knows they exist",
 * section "Why overlap alone cannot defeat the byte roofline" (grouping token
 * rows by expert), generalised to weighted rows and dropped routes.
 * ------------------------------------------------------------------------- */
MOE_API moe_status moe_dispatch(const void *x, int64_t ldx, int row_type, const int32_t *inv_perm, const float *w,
                                int T, int k, int H, int R, void *x_perm, int64_t ld_perm, int32_t *dev_status,
                                void *stream);

/* ---------------------------------------------------------------------------
 * moe_dispatch_backward -- gradient of moe_dispatch.
 *
 *   dx[t,:] = add[t,:] + sum_j w[t,j] * dx_perm[inv_perm[t,j], :]   (rank order)
 *   dw[t,j] = < dx_perm[inv_perm[t,j], :], x[t, :] >, 0 for a route without
 *             a slot
 *
 *   dx_perm [R,H] row_type;  dx (out), add [T,H] dx_type
 *   w       [T,k] f32 or NULL (factor 1)
 *   add     or NULL (0): a gradient that is already there; may be dx itself
 *           (then ld_add == ldx_grad)
 *   dw      [T,k] f32 (out) or NULL; with dw, x [T,H] row_type is required
 * ------------------------------------------------------------------------- */
MOE_API moe_status moe_dispatch_backward(const void *dx_perm, int64_t ld_perm, int row_type, const int32_t *inv_perm,
                                         const float *w, const void *x, int64_t ldx, int T, int k, int H, int R,
                                         void *dx, int64_t ldx_grad, int dx_type, const void *add, int64_t ld_add,
                                         float *dw, int32_t *dev_status, void *stream);

/* ---------------------------------------------------------------------------
 * moe_collect -- rows in expert order back to token order, weighted.
 *
 *   out[t,:] = add[t,:] + sum_j w[t,j] * y_perm[inv_perm[t,j], :]   (rank order)
 *
 * moe_combine for rows of either type, any width and stride, and routes
 * without a slot (a token none of whose routes has one gets add, or zero).
 *   y_perm [R,H] row_type;  out (out), add [T,H] out_type;  w [T,k] f32 or
 *   NULL (factor 1: rows that carry their weight);  add or NULL; may be out
 *   itself (then ld_add == ld_out)
 * Source: AFN-019, section "Hypothesis H4" (the weighted sum follows
 * route-rank order whatever order the experts ran in).
 * ------------------------------------------------------------------------- */
MOE_API moe_status moe_collect(const void *y_perm, int64_t ld_perm, int row_type, const int32_t *inv_perm,
                               const float *w, int T, int k, int H, int R, void *out, int64_t ld_out, int out_type,
                               const void *add, int64_t ld_add, int32_t *dev_status, void *stream);

/* ---------------------------------------------------------------------------
 * moe_collect_backward -- gradient of moe_collect (and of moe_combine).
 *
 *   dy_perm[inv_perm[t,j], :] = w[t,j] * dout[t, :]
 *   dw[t,j] = < dout[t, :], y_perm[inv_perm[t,j], :] >, 0 for a route without
 *             a slot
 *
 *   dout [T,H] out_type;  y_perm, dy_perm (out) [R,H] row_type
 *   w [T,k] f32 or NULL;  dw [T,k] f32 (out) or NULL; with dw, y_perm is
 *   required.  Rows of dy_perm that no route names are left as they were.
 * ------------------------------------------------------------------------- */
MOE_API moe_status moe_collect_backward(const void *dout, int64_t ld_dout, int out_type, const void *y_perm,
                                        int64_t ld_perm, int row_type, const int32_t *inv_perm, const float *w, int T,
                                        int k, int H, int R, void *dy_perm, int64_t ld_dperm, float *dw,
                                        int32_t *dev_status, void *stream);

/* ---------------------------------------------------------------------------
 * moe_block_norm -- from one block's output to the next block's input.
 *
 *   z      = y * r1 * (1 + gamma_post),  r1 = 1 / sqrt(mean(y^2) + eps)
 *            (post_norm != 0; else z = y)
 *   x_out  = scale * x + gate * z
 *   n_out  = x_out * r2 * (1 + gamma_pre),  r2 = 1 / sqrt(mean(x_out^2) + eps)
 * per row.  n_out and r2 use x_out before it is rounded to x_type.
 *
 *   x, x_out (out) [T,H] x_type: the residual stream; x_out may be x itself
 *            (then ldx_out == ldx), or NULL when only n_out is wanted
 *   y, n_out (out) [T,H] y_type: the block's output and the next one's input.
 *            y NULL: no block yet (z = 0; gate, gamma_post, rstd_post NULL,
 *            post_norm 0); n_out NULL: no norm after it (gamma_pre, rstd_pre
 *            NULL).  x_out and n_out are not both NULL.
 *   gate     by gate_kind: MOE_GATE_NONE (NULL, factor 1), MOE_GATE_CHANNEL
 *            [H] f32, MOE_GATE_TOKEN [T] f32, MOE_GATE_FULL [T,H] y_type with
 *            row stride ld_gate (ignored for the others)
 *   gamma_post, gamma_pre [H] f32 or NULL (gain 1)
 *   scale    finite;  eps >= 0
 *   rstd_post, rstd_pre [T] f32 (out) or NULL: r1 and r2, for the gradient
 * Source: AFN-001 "Porting Qwen3.8-Flash-Next to Hebrus", section "Phase 1:
 * separate math from acceleration" (zero-centred RMS normalisation), applied
 * on both sides of a block.
 * ------------------------------------------------------------------------- */
typedef enum moe_gate_kind {
  MOE_GATE_NONE = 0,
  MOE_GATE_CHANNEL = 1,
  MOE_GATE_TOKEN = 2,
  MOE_GATE_FULL = 3
} moe_gate_kind;

MOE_API moe_status moe_block_norm(const void *x, int64_t ldx, int x_type, const void *y, int64_t ldy, int y_type,
                                  const void *gate, int gate_kind, int64_t ld_gate, const float *gamma_post,
                                  const float *gamma_pre, int post_norm, float scale, float eps, int T, int H,
                                  void *x_out, int64_t ldx_out, void *n_out, int64_t ldn, float *rstd_post,
                                  float *rstd_pre, void *stream);

/* ---------------------------------------------------------------------------
 * moe_block_norm_backward -- gradient of moe_block_norm.
 *
 * With u = dn * (1 + gamma_pre), D = dx_out + r2 * u - x_out * r2^3 * mean(u * x_out)
 * (the gradient of x_out) and v = D * gate * (1 + gamma_post):
 *   dx         = scale * D
 *   dy         = r1 * v - y * r1^3 * mean(v * y)         (post_norm 0: D * gate)
 *   dgate      = D * z, summed over tokens (MOE_GATE_CHANNEL, [H] f32) or over
 *                columns (MOE_GATE_TOKEN, [T] f32), or as it is (MOE_GATE_FULL,
 *                [T,H] y_type, row stride ld_dgate)
 *   dgamma_post = sum_t D * gate * y * r1                                [H] f32
 *   dgamma_pre  = sum_t dn * x_out * r2                                  [H] f32
 *
 *   dx_out [T,H] x_type or NULL (0);  dn [T,H] y_type or NULL (0); not both NULL
 *   x_out, y, gate, gammas, scale, post_norm as the forward call had or wrote
 *   them; x_out may be NULL when dn is; y NULL as there
 *   rstd_post (post_norm), rstd_pre (dn): required as the forward wrote them
 *   dx (out) [T,H] x_type; may be dx_out itself (then ldx_grad == ld_dxo)
 *   dy (out) [T,H] y_type; required with y, else NULL
 *   dgate, dgamma_post, dgamma_pre (out): each NULL when not wanted; NULL
 *            where there is no gate / post_norm / dn
 *   workspace: >= moe_block_norm_workspace_size(T, H) bytes, 16-byte aligned,
 *            contents do not matter; not to be shared by calls that overlap
 *            on the GPU
 * ------------------------------------------------------------------------- */
MOE_API size_t moe_block_norm_workspace_size(int T, int H);
MOE_API moe_status moe_block_norm_backward(const void *dx_out, int64_t ld_dxo, const void *dn, int64_t ld_dn,
                                           const void *x_out, int64_t ldx_out, int x_type, const void *y, int64_t ldy,
                                           int y_type, const void *gate, int gate_kind, int64_t ld_gate,
                                           const float *gamma_post, const float *gamma_pre, int post_norm,
                                           float scale, const float *rstd_post, const float *rstd_pre, int T, int H,
                                           void *dx, int64_t ldx_grad, void *dy, int64_t ldy_grad, void *dgate,
                                           int64_t ld_dgate, float *dgamma_post, float *dgamma_pre, void *workspace,
                                           size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * moe_route_backward -- gradient of moe_route's renormalised top-k weights.
 *
 *   dlogits[t,j] = w[t,j] * (dw[t,j] - sum_i w[t,i] * dw[t,i])
 *   dx[t,:]        = add[t,:] + sum_j dlogits[t,j] * w_router[ids[t,j], :]
 *   dw_router[e,:] = sum over the routes (t,j) of expert e of dlogits[t,j] * x[t,:]
 *   dbias[e]       = sum over the routes of expert e of dlogits[t,j]
 * The selection itself has no gradient: logits outside the top k get none.
 *
 *   dw, topk_w [T,k] f32, topk_ids [T,k] int32 (moe_route); x [T,H], w_router
 *   [E,H] bf16; offsets [E+1], perm [T*k] int32 (moe_permute of topk_ids)
 *   dlogits   [T,k] f32 (out)
 *   dx        (out), add (or NULL; may be dx itself, then ld_add == ldx_grad)
 *             [T,H] dx_type; dx may be NULL
 *   dw_router [E,H] f32 (out) or NULL;  dbias [E] f32 (out) or NULL
 *   workspace: >= moe_route_backward_workspace_size(T, k, E, H) bytes, 16-byte
 *             aligned, contents do not matter; not to be shared by calls that
 *             overlap on the GPU
 * An expert ID outside [0,E) or a perm entry outside [0,T*k) sets
 * MOE_DEV_BAD_EXPERT and leaves that route out of dx or of dw_router and
 * dbias; offsets that do not rise from 0 to T*k set it and leave dw_router
 * and dbias unwritten.
 * Source: AFN-001, section "Phase 1" (float32 router softmax over the
 * normalised top-10); the gradient is its derivative.
 * ------------------------------------------------------------------------- */
MOE_API size_t moe_route_backward_workspace_size(int T, int k, int E, int H);
MOE_API moe_status moe_route_backward(const float *dw, const float *topk_w, const int32_t *topk_ids, const uint16_t *x,
                                      int64_t ldx, const uint16_t *w_router, int64_t ld_router, const int32_t *offsets,
                                      const int32_t *perm, int T, int k, int E, int H, float *dlogits, void *dx,
                                      int64_t ldx_grad, int dx_type, const void *add, int64_t ld_add,
                                      float *dw_router, int64_t ld_dw, float *dbias, void *workspace,
                                      size_t workspace_bytes, int32_t *dev_status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H_ */
