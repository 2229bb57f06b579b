/*
 * vc_step.h -- the operators of a data-parallel training step between the
 * linear layers of vc_train.h and around the buckets of vc.h: the embedding
 * lookup and its gradient, the norms before and after a block with its gate
 * and residual, and the global norm of the gradients with clipping.
 *
 *   embedding   y_t = s W[id_t - first], zeros where the table has no such row;
 *               dW_v (+)= s * sum of dy_t over the tokens with id_t - first = v
 *   block norm  u = post(h),  r = a x + act(gate) * u,  n = pre(r)
 *   clipping    N = |all gradients|,  c = min(1, max_norm / (N + eps)),  g <- c g
 *
 * The rules are those of vc_train.h: the caller owns every buffer, workspaces
 * included (aligned to 256 bytes here), and the library allocates no device
 * memory and keeps no pointer after a call returns; calls are asynchronous on
 * `stream`; arguments are checked on the host and a call that returns an error
 * launches nothing; entry points are thread-safe.  Outputs must not overlap
 * inputs, except where a comment says that they may be the same matrix.
 *
 * Arithmetic is in 32 bits and rounded once where a value is stored.  (Clipping adds
 * squares in 32 bits over at most 33 values, and those sums as pairs of 32-bit values,
 * which keep 48 bits.)  The same call on the same inputs gives the same bits: no sum
 * depends on the order in which blocks run.
 */
#ifndef VC_STEP_H
#define VC_STEP_H

#include "vc.h"
#include "vc_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- embedding ----------------------------------------------------------- */

/* out row t <- scale * weight row (ids[t] - first), for t < tokens, and zeros
 * where 0 <= ids[t] - first < weight->rows does not hold: `weight` may be one
 * rank's part of a vocabulary, and the AllReduce (sum) of the ranks' outputs is
 * then the whole table's lookup.  ids: `tokens` values of VC_INT32 or VC_INT64
 * in device memory; weight [V, D] and out [tokens, D] float32 or bfloat16, each
 * by itself. */
vc_status_t vc_embedding_forward(const void *ids, vc_dtype_t id_dtype, long long tokens,
                                 const vc_matrix_t *weight, long long first, float scale,
                                 const vc_matrix_t *out, vc_stream_t stream);

/* Bytes of workspace that vc_embedding_backward needs; 0 where a size is
 * invalid. */
size_t vc_embedding_backward_workspace(long long tokens, long long rows, long long cols);

/* The gradient of vc_embedding_forward: dweight [V, D] row v (+)= scale * the
 * sum, in 32 bits and an order that depends on the ids alone, of the rows t of dy
 * [tokens, D] with ids[t] - first = v.  Tokens whose id is `padding` are left out
 * (and those outside of the table); a negative `padding` leaves none out.  Every
 * row of dweight is written: with zeros where no token is, unless `accumulate` is
 * non-zero, which adds to the rows that tokens have and leaves the others as they
 * are.  dy and dweight float32 or bfloat16, each by itself.  The tokens are sorted by
 * row first, so that no block adds to another's sums, whatever the ids are.  At most 2^30
 * tokens and 2^22 columns.  (Where accumulate adds to float32 values, sums below 2^-126
 * become 0.) */
vc_status_t vc_embedding_backward(const vc_matrix_t *dy, const void *ids, vc_dtype_t id_dtype,
                                  long long first, long long padding, float scale,
                                  const vc_matrix_t *dweight, int accumulate, void *workspace,
                                  size_t workspace_bytes, vc_stream_t stream);

/* ---- norms around a block ------------------------------------------------ */

/* RMS: v / sqrt(mean(v^2) + eps) * w.  LAYER: the same of v - mean(v), (+ b). */
typedef enum { VC_NORM_RMS = 0, VC_NORM_LAYER = 1 } vc_norm_t;
typedef enum { VC_GATE_NONE = 0, VC_GATE_SIGMOID = 1 } vc_gate_t;

typedef struct {
    vc_norm_t norm;
    vc_gate_t gate_act;    /* of the gate's values */
    float residual_scale;  /* a */
    float eps;             /* >= 0; shared by both norms */
} vc_block_norm_t;

/* A norm's weight and bias (D values each, contiguous, of one type: float32 or
 * bfloat16).  weight NULL: there is no such norm (and bias is NULL too).  RMS norms
 * have no bias: calls with one are refused. */
typedef struct {
    void *weight, *bias;
    vc_dtype_t dtype;
} vc_affine_t;

/* u = post-norm(h), or h without a post-norm;  r = residual_scale * x +
 * act(gate) * u;  n = pre-norm(r), the input of the next block.  h, n [T, D]
 * bfloat16; x, r [T, D] float32 or bfloat16, both of one type; x NULL: r =
 * act(gate) * u.  gate NULL (1), or [G, D] float32 or bfloat16 where G divides T: row g
 * is that of the T / G rows from g T / G on (G = 1: one vector for all; G = T:
 * a value for every element).  r or n NULL: not stored; n needs pre->weight.  n is computed
 * from r in 32 bits, before its rounding.  r may be x itself and n may be h
 * itself.  post and pre may be NULL where there is no such norm.  The squares of a row's
 * values must have a sum that float32 holds. */
vc_status_t vc_block_norm_forward(const vc_matrix_t *h, const vc_matrix_t *x,
                                  const vc_matrix_t *gate, const vc_affine_t *post,
                                  const vc_affine_t *pre, const vc_block_norm_t *args,
                                  const vc_matrix_t *r, const vc_matrix_t *n, vc_stream_t stream);

/* What the gradient reads (NULL where there is none) ... */
typedef struct {
    const vc_matrix_t *dr;  /* gradient at r from behind, of r's type; NULL: 0 */
    const vc_matrix_t *dn;  /* gradient at n, bfloat16; NULL: 0 */
    const vc_matrix_t *r;   /* as the forward pass stored it; read where dn is there */
    const vc_matrix_t *h;   /* read with a post-norm or for dgate */
    const vc_matrix_t *gate;
} vc_block_norm_in_t;
/* ... and writes (NULL: not computed). */
typedef struct {
    const vc_matrix_t *dx;     /* [T, D] of r's type; may be dr itself */
    const vc_matrix_t *dh;     /* [T, D] bfloat16; may be dn itself */
    const vc_matrix_t *dgate;  /* [G, D] float32 or bfloat16 */
    vc_affine_t dpost, dpre;   /* column sums over all rows; dtype is the gradients' */
} vc_block_norm_out_t;

/* Bytes of workspace that vc_block_norm_backward needs for [rows, cols], with
 * a gate of `gates` rows (0: none). */
size_t vc_block_norm_backward_workspace(long long rows, long long cols, long long gates);

/* The gradient of vc_block_norm_forward.  With hats for normalised rows and norm'
 * for the norms' own gradients,
 *   dr_all = dr + norm'(pre.weight * dn),       dx = residual_scale * dr_all
 *   dpre = sum dn * r^ (bias: sum dn),          dgate = sum dr_all * u * act'(gate)
 *   du = act(gate) * dr_all,                    dh = norm'(post.weight * du), or du
 *   dpost = sum du * h^ (bias: sum du)
 * with the sums over all rows, and over its own T / G rows for a row of dgate.
 * Both norms' statistics are computed again from r and h.  accumulate adds to dgate,
 * dpost and dpre in 32 bits.  The shape [T, D] is that of dr, or of dn where dr is
 * NULL. */
vc_status_t vc_block_norm_backward(const vc_block_norm_in_t *in, const vc_affine_t *post,
                                   const vc_affine_t *pre, const vc_block_norm_t *args,
                                   const vc_block_norm_out_t *out, int accumulate,
                                   void *workspace, size_t workspace_bytes, vc_stream_t stream);

/* ---- the norm of all gradients, and clipping ------------------------------ */

/* One tile of a plan: `count` consecutive elements of a gradient at src, and
 * where they go (NULL: nowhere).  flags bit 0: float32 (else bfloat16); bit 1: all
 * tiles of the plan are in place. */
typedef struct {
    const void *src;
    void *dst;
    int count;
    int flags;
    long long index;  /* its place in the plan */
} vc_clip_tile_t;

/* The largest tile that vc_clip_plan makes. */
#define VC_CLIP_TILE_MAX_BYTES (1u << 14)

/* Plans the norm of many gradients (host only; launches nothing).
 * grads, outs: HOST arrays of ntensors DEVICE pointers, counts[k] elements of
 *   dtypes[k] (VC_FLOAT32 or VC_BFLOAT16) each; outs NULL: nothing is clipped; outs[k] may
 *   be grads[k] (in place).  counts of 0 are allowed.
 * tiles: HOST array of max_tiles entries that receives the plan, or NULL to
 *   ask for their number only, which *ntiles receives.
 * VC_ERR_ALIAS (where tiles is given, which then holds nothing of use): an output
 * overlaps another output, or an input other than its own in place. */
vc_status_t vc_clip_plan(const void *const *grads, void *const *outs, const size_t *counts,
                         const vc_dtype_t *dtypes, int ntensors, vc_clip_tile_t *tiles,
                         int max_tiles, int *ntiles);

/* L2: sqrt of the sum of squares, which no value of the gradients' types is too large or
 * too small for: a sum of up to 33 squares that leaves [2^-90, 2^90] is taken in 64 bits.
 * MAX: the largest magnitude. */
typedef enum { VC_GRAD_NORM_L2 = 0, VC_GRAD_NORM_MAX = 1 } vc_grad_norm_t;

/* Bytes of workspace for both of the following. */
size_t vc_clip_workspace(int ntiles);

/* *norm (device memory, outside of the gradients and outputs; not checked) <- the norm
 * of the planned gradients.  dev_tiles: DEVICE
 * array of the ntiles tiles (16-byte aligned), as planned: tables that differ from the
 * planned ones are undefined behaviour, as for any device copy.  No tiles: 0. */
vc_status_t vc_grad_norm(const vc_clip_tile_t *dev_tiles, int ntiles, vc_grad_norm_t kind,
                         float *norm, void *workspace, size_t workspace_bytes, vc_stream_t stream);

/* The norm, and every output <- c * gradient, rounded to its type, with
 * c = min(1, max_norm / (norm + eps)) in 32 bits.  Gradients in place are left
 * as they are where c = 1.  A norm that is not a number, or infinite beside an
 * infinite max_norm, makes c NaN, and an infinite one beside a finite max_norm 0. max_norm >= 0, eps >= 0. */
vc_status_t vc_clip_grad_norm(const vc_clip_tile_t *dev_tiles, int ntiles, vc_grad_norm_t kind,
                              float max_norm, float eps, float *norm, void *workspace,
                              size_t workspace_bytes, vc_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* VC_STEP_H */
