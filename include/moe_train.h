/*
 * moe_train.h -- C ABI of libmoe's operators around the layer in a training
 * step: the softmax cross entropy over a vocabulary with its gradient, the
 * gradient of the router (with its balance and z losses), and the global
 * gradient norm with clipping.  Conventions (device pointers owned by the
 * caller, asynchronous calls on `stream`, host-side validation, workspace and
 * device status word) are those of moe.h, moe_workspace_init before a
 * workspace's first use included; outputs must not overlap inputs unless a
 * declaration says so.  One workspace serves calls of any shapes and operators in
 * turn.  Its first 256 bytes outlive a call: the status word, and counters that
 * are zero between calls.  A call that reported MOE_ERR_CUDA may have left them
 * otherwise: moe_workspace_init before the next one.
 */
#ifndef MOE_TRAIN_H_
#define MOE_TRAIN_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Cross entropy of a linear classifier over a vocabulary
 *
 *   z_tv = <x_t, w_v>,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,target
 *
 * computed in pieces of the vocabulary: the [tokens, vocab] logits are never
 * stored.  A token whose target is ignore_index does not count: its loss, lse
 * and dx row are 0 and its x row is not read (it may hold anything).  A target
 * outside [0, vocab) that is not ignore_index is treated the same and sets
 * MOE_ERR_TARGET on the device.
 *   MOE_CE_NONE: the losses of the tokens;  MOE_CE_SUM: their sum;
 *   MOE_CE_MEAN: the sum over the number of tokens that count (0 when none).
 * Precision: bf16 inputs on the tensor cores with fp32 sums; fp32 inputs as three
 * bf16 planes each (all 24 mantissa bits, any finite magnitude; an infinite element
 * may give NaN where fp32 arithmetic gives an infinity), fp32 sums; statistics in
 * fp32; the gradient of the logits is rounded to bf16 (up to 32 tokens to two planes,
 * fp32 to three) as the operand of the two gradient products (before the total's gradient and the mean's
 * divisor, which scale the products in fp32); dx and dw are rounded once.
 * ------------------------------------------------------------------------- */
typedef enum { MOE_CE_NONE = 0, MOE_CE_SUM = 1, MOE_CE_MEAN = 2 } moe_ce_reduction;

typedef struct {
  int64_t tokens;       /* T >= 0, at most 2^28 */
  int32_t hidden;       /* H, a positive multiple of 8 */
  int32_t vocab;        /* V >= 1, at most 2^30 */
  int32_t dtype;        /* moe_dtype of x, w, dx, dw */
  int32_t reduction;    /* moe_ce_reduction */
  int32_t ignore_index; /* target of tokens that do not count */
  int64_t x_stride;     /* elements from one row of x to the next: 0 = H, else
                           at least H and a multiple of 8 */
  int64_t w_stride;     /* the same for w */
} moe_ce_shape;

/* Workspace of the two calls below (0 for an invalid shape).  Nothing of a call's
 * results or inputs is kept in it for the next. */
size_t moe_linear_ce_workspace_bytes(const moe_ce_shape *shape);

/* x [T, H], w [V, H] (16-byte aligned), target [T] int32.  Outputs (fp32):
 * loss [T] (may be NULL), lse [T] (may be NULL), stats [T, 4] (may be NULL; the
 * backward reads it: M, the row's largest z, S = sum_v e^(z - M), R the same without
 * the target, 0; from lse, rounded at its magnitude, probabilities near 1 would lose
 * digits; 16-byte aligned),
 * total [1] (the reduced loss; NULL with MOE_CE_NONE, else may be NULL). */
moe_status moe_linear_ce_forward(const moe_ce_shape *shape, const void *x, const void *w,
                                 const int32_t *target, float *loss, float *lse, float *stats,
                                 float *total, void *ws, size_t ws_bytes, void *stream);

/* Gradients of the reduced loss, g_t = d objective / d loss_t:
 *   d_tv = g_t (exp(z_tv - lse_t) - [v = target_t]), at the target -g_t R / S;  dx = d w;  dw = d^T x
 * stats as the forward wrote it for the same x and w.  dloss: MOE_CE_NONE: [T]
 * (needed); otherwise [1], the gradient of the total, or NULL for 1.
 * dx [T, H], dw [V, H], contiguous; either may be NULL (not computed).  Both
 * are overwritten. */
moe_status moe_linear_ce_backward(const moe_ce_shape *shape, const void *x, const void *w,
                                  const int32_t *target, const float *stats, const float *dloss,
                                  void *dx, void *dw, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * Gradient of the router (what moe_layer_backward leaves to its caller)
 *
 *   z = x . w_router^T (fp32),  p_t = softmax of z_t over the E experts
 *   topk_w[t, s]: softmax over the k selected logits (norm_topk) or p at them
 *   gate_t = sigmoid(z_tE) (shared_gate)
 *   balance = balance_coef * E * sum_e (n_e / (T k)) * mean_t p_te,
 *             n_e = slots routed to e (a constant for the gradient)
 *   zloss   = z_coef * mean_t lse_t^2
 * Given d_topk_w and d_gate it computes the gradient of the logits (of the
 * routed op's objective plus both losses) and
 *   dx = dx_add + dz . w_router,   dw_router = dz^T . x
 * The shape's tokens, hidden, topk_shape, shared_gate, norm_topk and dtype
 * count.  A route outside [0, E) is dropped and sets MOE_ERR_DEVICE_ROUTE; a
 * repeated route counts in each of its slots.
 * ------------------------------------------------------------------------- */
size_t moe_router_backward_workspace_bytes(const moe_shape *shape);

/* x [T, H], w_router [E + shared_gate, H], topk_idx [T, k], d_topk_w [T, k]
 * fp32 or NULL (zeros), d_gate [T] fp32 (iff shared_gate), dx_add [T, H] or
 * NULL (the experts' dx); outputs dx [T, H], dw_router [E + shared_gate, H] in
 * the activation type, aux [2] fp32 = {balance, zloss} or NULL.  dx_add may be
 * dx itself.  Coefficients finite and >= 0. */
moe_status moe_router_backward(const moe_shape *shape, const void *x, const void *w_router,
                               const int32_t *topk_idx, const float *d_topk_w,
                               const float *d_gate, double balance_coef, double z_coef,
                               const void *dx_add, void *dx, void *dw_router, float *aux,
                               void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * Global norm of many gradients, and clipping
 *
 *   norm = sqrt(sum over all tensors and elements of g^2)
 *   coef = min(1, max_norm / (norm + 1e-6));  1 when norm is not finite
 *   dst = g * coef, rounded once to dst's type
 * A norm that is not finite (an infinity or NaN among the gradients) thus leaves
 * them as they are, and the caller, who has the norm, skips the step; one beyond
 * fp32 clips and reads as infinity.  No two destinations may overlap, nor a
 * destination another tensor's source.  Squares are added in fp32 in
 * groups and in fp64 across them, in an order that depends on the list alone; a
 * group whose fp32 sum leaves the safe range is added again, scaled.
 * ------------------------------------------------------------------------- */
typedef struct {
  const void *src;    /* device, aligned to its element */
  void *dst;          /* device; src for in-place, NULL: only the norm counts */
  int64_t numel;      /* >= 0 */
  int32_t src_dtype;  /* moe_dtype */
  int32_t dst_dtype;
} moe_grad_tensor;

/* What moe_grad_clip needs on the host (filled by moe_grad_clip_plan). */
typedef struct {
  int64_t tensors, chunks;
  int32_t chunk_elems, reserved;
} moe_grad_plan;

/* Bytes of the list's table and the partial sums; tensors is the array on the
 * host.  0 for an invalid list. */
size_t moe_grad_clip_workspace_bytes(const moe_grad_tensor *tensors, int64_t n);

/* Write the list's table into ws (asynchronous on stream; the array on the
 * host is not read after the call).  ws belongs to the list from then on. */
moe_status moe_grad_clip_plan(const moe_grad_tensor *tensors, int64_t n, moe_grad_plan *plan,
                              void *ws, size_t ws_bytes, void *stream);

/* One norm and clipping over the planned list.  norm [1] fp32.  max_norm > 0,
 * infinity for the norm alone.  Where coef is 1 and dst is src, nothing is
 * written. */
moe_status moe_grad_clip(const moe_grad_plan *plan, double max_norm, float *norm, void *ws,
                         size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_TRAIN_H_ */
