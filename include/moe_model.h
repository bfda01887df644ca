/*
 * moe_model.h -- C ABI of libmoe's operators between the layer and the rest of a
 * model: the token embedding with its gradient, the norms before and after a
 * block with its gate and residual, and the orthogonalised update of weight
 * matrices.  Conventions (device pointers owned by the caller, asynchronous calls
 * on `stream`, host-side validation, workspace and device status word) are those
 * of moe.h and moe_train.h, moe_workspace_init before a workspace's first use and
 * one workspace for calls of any shapes in turn included; outputs must not overlap
 * inputs unless a declaration says so.
 */
#ifndef MOE_MODEL_H_
#define MOE_MODEL_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Token embedding and its gradient
 *
 *   y_t = scale * w[id_t]
 *   dw_v = dw_add_v + scale * sum over {t : id_t = v} of dy_t
 *
 * A token id outside [0, vocab) gives a zero row, has no gradient and sets
 * MOE_ERR_TOKEN on the device.  The rows of padding_idx (-1: none) are looked up
 * like the others and get no gradient.  The sums are in fp32 in an order that
 * depends on the ids alone (the tokens are sorted by id, no atomics on the
 * sums), each output rounded once.
 * ------------------------------------------------------------------------- */
typedef struct {
  int64_t tokens;       /* T >= 0, at most 2^28; T H below 2^47 */
  int32_t hidden;       /* H, a positive multiple of 8, at most 2^28 */
  int32_t vocab;        /* V >= 1, at most 2^30 */
  int32_t dtype;        /* moe_dtype of w, y, dy, dw_add, dw */
  int32_t padding_idx;  /* -1 or in [0, vocab) */
  double scale;         /* finite */
  int64_t w_stride;     /* elements from one row of w to the next: 0 = H, else at
                           least H and a multiple of 8 */
} moe_embed_shape;

/* Workspace of the two calls below (0 for an invalid shape). */
size_t moe_embed_workspace_bytes(const moe_embed_shape *shape);

/* w [V, H] (16-byte aligned), ids [T] int32 -> y [T, H]. */
moe_status moe_embed_forward(const moe_embed_shape *shape, const void *w, const int32_t *ids,
                             void *y, void *ws, size_t ws_bytes, void *stream);

/* ids [T], dy [T, H], dw_add [V, H] or NULL (zeros) -> dw [V, H], contiguous.
 * dw_add may be dw itself: only the rows that have tokens are then touched. */
moe_status moe_embed_backward(const moe_embed_shape *shape, const int32_t *ids, const void *dy,
                              const void *dw_add, void *dw, void *ws, size_t ws_bytes,
                              void *stream);

/* ---------------------------------------------------------------------------
 * Norms before and after a block, its gate and the residual, in one pass
 *
 *   r1_t = 1 / sqrt(mean_h y_th^2 + eps)         yn = y r1
 *   u    = yn (w_post + o)                       (u = y without w_post)
 *   s    = residual_scale x + g u                (s = residual_scale x without y)
 *   r2_t = 1 / sqrt(mean_h s_th^2 + eps)         sn = s r2
 *   h    = sn (w_pre + o)
 *
 * o = unit_offset (0 or 1); g = 1, a value for each channel or one for each
 * token.  x is the residual stream, y the block's output (NULL: only the norm
 * before the next block), s the new residual stream, h the next block's input,
 * computed from s before its rounding.  All in fp32, each output rounded once.
 * (moe_residual_setup of moe.h is the norm before a block too, to 2^-44 before its
 * rounding: what decides near ties of a router as the exact norm would is that one; here an
 * h may be the type's neighbouring value, and the routes those of the h that is fed.)
 * Rows are copied ahead under a bounded wait: where one never comes, the rows its block
 * had left become NaN, and the backward sets MOE_ERR_TIMEOUT (the forward, which has no
 * workspace, has no other sign).
 * ------------------------------------------------------------------------- */
typedef enum { MOE_GATE_NONE = 0, MOE_GATE_CHANNEL = 1, MOE_GATE_TOKEN = 2 } moe_gate_kind;

typedef struct {
  int64_t tokens;         /* T >= 0, at most 2^28 */
  int32_t hidden;         /* H, a positive multiple of 8, at most 32768 */
  int32_t dtype;          /* moe_dtype of everything but a token gate and rstd */
  int32_t gate;           /* moe_gate_kind */
  int32_t unit_offset;    /* 0 or 1 */
  double residual_scale;  /* finite */
  double eps;             /* positive and finite */
} moe_block_norm_shape;

/* Workspace of the backward (0 for an invalid shape); the forward needs none. */
size_t moe_block_norm_workspace_bytes(const moe_block_norm_shape *shape);

/* x, y [T, H] (y may be NULL: then w_post and gate must be too), w_post [H] or
 * NULL, gate [H] in dtype (MOE_GATE_CHANNEL) or [T] fp32 (MOE_GATE_TOKEN), w_pre [H]
 * or NULL (then h must be NULL).  Outputs s [T, H] (may be NULL; may be x), h
 * [T, H] (may be NULL without w_pre only), rstd [T, 2] fp32 {r1, r2} (may be NULL;
 * the backward reads it; 0 where there is no such norm). */
moe_status moe_block_norm_forward(const moe_block_norm_shape *shape, const void *x, const void *y,
                                  const void *w_post, const void *gate, const void *w_pre, void *s,
                                  void *h, float *rstd, void *stream);

/* Gradients given ds [T, H] (of s, or NULL: zeros) and dh [T, H] (of h; NULL iff
 * w_pre is NULL), for the same x, y, w_post, gate, w_pre and the forward's rstd:
 *   D = ds + r2 (dh (w_pre + o) - sn mean_h(dh (w_pre + o) sn))
 *   dx = residual_scale D,  dgate = sum_t D u (channel) or sum_h D u (token)
 *   dy = r1 (b - yn mean_h(b yn)) with b = g D (w_post + o)   (g D without w_post)
 *   dw_post = sum_t g D yn,  dw_pre = sum_t dh sn
 * dx, dy [T, H], dw_post, dw_pre [H], dgate [H] in dtype or [T] fp32; each may be
 * NULL (not computed) and must be NULL where its input is.  dx may be ds, dy may be
 * y.  The sums over tokens are in fp32 in a fixed order, in two stages. */
moe_status moe_block_norm_backward(const moe_block_norm_shape *shape, const void *ds,
                                   const void *dh, const void *x, const void *y,
                                   const void *w_post, const void *gate, const void *w_pre,
                                   const float *rstd, void *dx, void *dy, void *dw_post,
                                   void *dgate, void *dw_pre, void *ws, size_t ws_bytes,
                                   void *stream);

/* ---------------------------------------------------------------------------
 * Orthogonalised update of weight matrices (Newton-Schulz products)
 *
 *   X_0 = u / (|u|_F + eps),  |.|_F over one matrix
 *   X_{i+1} = a_i X_i + (b_i A + c_i A A) X_i,  A = X_i X_i^T   (X_i^T X_i for a
 *             matrix with more rows than columns: the same X by the smaller side)
 * which maps every singular value s of X_i to a_i s + b_i s^3 + c_i s^5 and
 * leaves the singular vectors.  A matrix of zeros stays zero; one with an
 * infinity or NaN becomes NaN, others in the batch do not see it.
 *
 * Precision: X is held under a fixed power of two, which the bounds below keep in
 * range.  bf16 matrices: one tensor-core product of fp16 operands (11 bits), while
 * a_i X_i takes X's 19 bits (an error outside X's row and column space grows by a_i
 * in every step); an X keeps 11 where the steps after it, and after any later X, grow such
 * an error by 4 or less.
 * Where n >= 2 m the first two of three or more steps are taken as one polynomial in
 * A (its coefficients allowing).  fp32 matrices: X in two fp16 parts (22 bits), the
 * three products above 2^-22.  A smaller side of at most 128 (up to a length): X in
 * fp32 between the steps.  Sums in fp32.  So a returned bf16 direction is some 2.3e-3 of its
 * norm off (its own rounding 1.7e-3 of it), an fp32 one 1e-6 to 5e-6.  Under the fixed power of
 * two entries of X below 2^-27 (fp32 matrices: 2^-16) have fewer bits and below 2^-38 none:
 * those of matrices far smaller than eps, and after steps that shrink singular values so far.
 * Matrices with a smaller side of at most 128 take clusters of up to 16 CTAs; where a
 * device or a part of one cannot hold those, the call returns MOE_ERR_CUDA.
 * ------------------------------------------------------------------------- */
#define MOE_ORTH_MAX_STEPS 16

typedef struct {
  int32_t steps;      /* 1 .. MOE_ORTH_MAX_STEPS */
  int32_t reserved;   /* 0 */
  double eps;         /* >= 0, finite */
  double coef[MOE_ORTH_MAX_STEPS][3];   /* (a_i, b_i, c_i); no step may take
                         singular values from [0, 1] (on the first step) past 3.5, or its
                         |b s^2 + c s^4| past 100 */
} moe_orth_coefs;

/* ---- the matrices alone: x [batch, rows, cols] -> out, contiguous ---- */
typedef struct {
  int64_t batch;      /* >= 0, at most 2^24 */
  int32_t rows, cols; /* 1 .. 65536 */
  int32_t dtype;      /* moe_dtype of x and out */
  int32_t reserved;   /* 0 */
} moe_orth_shape;

size_t moe_orthogonalize_workspace_bytes(const moe_orth_shape *shape, const moe_orth_coefs *coefs);

/* out may be x. */
moe_status moe_orthogonalize(const moe_orth_shape *shape, const moe_orth_coefs *coefs,
                             const void *x, void *out, void *ws, size_t ws_bytes, void *stream);

/* ---- one optimiser step over a list of parameters ----
 *   v = momentum * v + (1 - momentum) * g
 *   u = nesterov ? momentum * v + (1 - momentum) * g : v
 *   param = (1 - lr * weight_decay) * param - lr * size * orthogonalised(u)
 * size: 1 (MOE_MUON_SCALE_NONE), sqrt(max(1, rows / cols)) (_SPECTRAL) or
 * 0.2 sqrt(max(rows, cols)) (_RMS).  Each [rows, cols] matrix of a batch is
 * orthogonalised by itself; tensors whose smaller and larger sides agree share
 * their launches, whichever way round they are.  The parameter's type decides the
 * precision of its direction, whatever its gradient's is. */
typedef enum { MOE_MUON_SCALE_NONE = 0, MOE_MUON_SCALE_SPECTRAL = 1, MOE_MUON_SCALE_RMS = 2 } moe_muon_scale;

typedef struct {
  void *param;        /* [batch, rows, cols], updated in place */
  const void *grad;   /* the same, in param's type or the other one */
  float *momentum;    /* the same in fp32, updated in place */
  int64_t batch;
  int32_t rows, cols;
  int32_t param_dtype, grad_dtype;   /* moe_dtype; the param's decides the precision */
} moe_muon_tensor;

typedef struct {
  double lr, momentum, weight_decay;   /* finite; momentum in [0, 1) */
  int32_t nesterov;                    /* 0 or 1 */
  int32_t scale;                       /* moe_muon_scale */
  moe_orth_coefs coefs;
} moe_muon_config;

/* The array is on the host and is not read after the calls.  0: invalid list. */
size_t moe_muon_workspace_bytes(const moe_muon_tensor *tensors, int64_t n, const moe_muon_config *config);

/* No two of the list's params and momenta may overlap, nor one of them a
 * gradient. */
moe_status moe_muon_step(const moe_muon_tensor *tensors, int64_t n, const moe_muon_config *config,
                         void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_MODEL_H_ */
