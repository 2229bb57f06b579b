/*
 * vc_train.h -- the operators of a data-parallel training step that stand
 * beside the collectives of vc.h: the linear layer whose gradients fill the
 * buckets, its gradient, and the orthogonalised (Muon) update of a reduced
 * gradient.
 *
 *   forward     z = x W^T + b,  y = act(z) + r
 *   backward    dz = dy * act'(z),  dx = dz W,  dW (+)= dz^T x,
 *               db (+)= sum over the rows of dz       (dr is dy itself)
 *   orthogonalize (Newton-Schulz, on the smaller side of each matrix)
 *               X_0 = G / (|G|_F + eps),  A = X X^T,
 *               X <- a X + (b A + c A^2) X,  `steps` times
 *   muon step   M <- beta M + G,  O = orthogonalize(G + beta M, or M),
 *               W <- (1 - lr wd) W - lr scale O
 *
 * Rules shared with vc.h: the caller owns every buffer, workspaces included,
 * and the library allocates no device memory and keeps no pointer after a
 * call returns; calls are asynchronous on `stream`; arguments are checked on
 * the host and a call that returns an error launches nothing; entry points
 * are thread-safe.  Outputs must not overlap inputs, except where a comment
 * says that they may be the same matrix.  (Column slices of one wider tensor
 * do not overlap.)
 *
 * Arithmetic.  Products run on the tensor cores with 16-bit operands and
 * 32-bit accumulators; biases, activations, residuals, norms, column sums and
 * the momentum are computed in 32 bits and rounded once where they are
 * stored.  The same call on the same inputs gives the same bits.
 */
#ifndef VC_TRAIN_H
#define VC_TRAIN_H

#include "vc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A row-major matrix, or `batch` of them: element (i, j) of matrix k is
 * data[k * batch_stride + i * ld + j].  ld >= cols (any value where rows <= 1);
 * batch_stride is not read where batch is 1 and covers a whole matrix
 * otherwise.  dtype is VC_FLOAT32 or VC_BFLOAT16; data is aligned to its
 * element.  No side is above 2^30, no matrix or batch above 2^38 elements, no ld
 * above 2^39 - 8.  Bases on 16 bytes with an ld of whole 16 bytes take the fastest
 * path; others are copied into the workspace first (tensor-core operands) or
 * accessed element by element (the rest). */
typedef struct {
    void *data;
    long long batch, rows, cols;
    long long ld, batch_stride;
    vc_dtype_t dtype;
} vc_matrix_t;

/* Activations.  RELU2 is max(z, 0)^2; GELU uses the error function,
 * GELU_TANH its tanh approximation with the constants sqrt(2/pi) and
 * 0.044715.  RELU's derivative at 0 is 0.  At infinities an activation and its
 * derivative take their limits (0 or z, 0 or 1, and RELU2 its square). */
typedef enum {
    VC_ACT_NONE = 0,
    VC_ACT_RELU = 1,
    VC_ACT_RELU2 = 2,
    VC_ACT_GELU = 3,
    VC_ACT_GELU_TANH = 4,
    VC_ACT_SILU = 5
} vc_act_t;

/* Bytes of workspace that vc_linear_forward needs for these operands (0 where
 * both lie on 16 bytes); 0 too where they are invalid.  The linear layer's
 * workspaces are aligned to 16 bytes. */
size_t vc_linear_forward_workspace(const vc_matrix_t *x, const vc_matrix_t *weight);

/* y = act(x W^T + bias) + residual.  x [M, K], weight [N, K], y [M, N], all
 * bfloat16; bias: N bfloat16 values, or NULL; residual: [M, N] or NULL, and it
 * may be y itself; preact: receives z = x W^T + bias rounded to bfloat16, or
 * NULL.  M, N and K may be 0 (K = 0: z is the bias). */
vc_status_t vc_linear_forward(const vc_matrix_t *x, const vc_matrix_t *weight, const void *bias,
                              const vc_matrix_t *residual, const vc_matrix_t *y,
                              const vc_matrix_t *preact, vc_act_t act, void *workspace,
                              size_t workspace_bytes, vc_stream_t stream);

/* Bytes of workspace that vc_linear_backward needs. */
size_t vc_linear_backward_workspace(const vc_matrix_t *dy, const vc_matrix_t *x,
                                    const vc_matrix_t *weight, vc_act_t act, int has_dbias);

/* The gradient of vc_linear_forward.  dy [M, N], x [M, K], weight [N, K] and
 * preact [M, N] (what the forward pass stored; NULL for VC_ACT_NONE) are
 * bfloat16.  dx [M, K] bfloat16 or NULL; dweight [N, K] bfloat16 or float32, or
 * NULL; dbias: N values of dbias_dtype (bfloat16 or float32), or NULL.  With
 * accumulate non-zero dweight and dbias are added to (in 32 bits, then
 * rounded), else overwritten.  dz is rounded to bfloat16 before the products
 * (a tensor-core operand), so that dx and dweight, of whatever type, are 1.7e-3
 * of their norm off; batches of up to 64 rows keep the remainder of the rounding
 * (2e-5); with VC_ACT_NONE dz is dy and nothing is rounded.  dbias sums dz in 32
 * bits. */
vc_status_t vc_linear_backward(const vc_matrix_t *dy, const vc_matrix_t *x,
                               const vc_matrix_t *weight, const vc_matrix_t *preact, vc_act_t act,
                               const vc_matrix_t *dx, const vc_matrix_t *dweight, void *dbias,
                               vc_dtype_t dbias_dtype, int accumulate, void *workspace,
                               size_t workspace_bytes, vc_stream_t stream);

/* The Newton-Schulz iteration: `steps` (1 to 100) passes of the polynomial with the
 * coefficients a, b, c, after a division by the Frobenius norm plus eps.  The
 * squares of the values must have a sum that float32 holds: a norm from 1e-19
 * to 1.8e19.  (Below, a matrix counts as zero.)  The norm may be far below
 * eps. */
typedef struct {
    int steps;
    float a, b, c;
    float eps;
} vc_newton_schulz_t;

/* Bytes of workspace for matrices of these sizes (orthogonalize and muon
 * step), which is aligned to 256 bytes; 0 where a size is invalid. */
size_t vc_orthogonalize_workspace(long long batch, long long rows, long long cols);

/* out <- the orthogonalised g, each matrix of the batch by itself.  g float32
 * or bfloat16, out bfloat16, of the same sizes; out may be g (bfloat16).  Before
 * out's rounding the five default passes are within 1e-3 of the norm of the
 * exact iteration for matrices of full rank, within 3.3e-3 for sums of few outer
 * products; the worst measured is 5e-3 (rank one of 96 rows; matrices of a few
 * values).  A zero matrix gives zeros; a matrix with a
 * value that is not finite gives NaN. */
vc_status_t vc_orthogonalize(const vc_matrix_t *g, const vc_matrix_t *out,
                             const vc_newton_schulz_t *ns, void *workspace, size_t workspace_bytes,
                             vc_stream_t stream);

typedef struct {
    float lr, beta, weight_decay, scale;
    int nesterov;
    vc_newton_schulz_t ns;
} vc_muon_t;

/* One Muon step in place on weight and momentum: weight float32 or bfloat16,
 * grad float32 or bfloat16 (read only), momentum float32 or bfloat16, three
 * disjoint buffers of the same sizes. */
vc_status_t vc_muon_step(const vc_matrix_t *weight, const vc_matrix_t *grad,
                         const vc_matrix_t *momentum, const vc_muon_t *args, void *workspace,
                         size_t workspace_bytes, vc_stream_t stream);

/* Device-side waits of the product kernels, and of the block norms' clusters of
 * vc_step.h, are bounded (about two seconds each).  *count receives how many blocks of the current device have given up
 * since the library was loaded: 0 unless something is broken, and any other
 * value means that results computed since are not valid.  Waits for all
 * streams of the device, then copies one word to the host; not to be called
 * while a stream is captured.  (For tests: with VC_TEST_WAIT_OUT set to a
 * non-zero value in the environment a block that gives up runs first.) */
vc_status_t vc_train_timeouts(unsigned *count);

#ifdef __cplusplus
}
#endif

#endif /* VC_TRAIN_H */
