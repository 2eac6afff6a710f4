/*
 * soma_ops.h -- C ABI of the training operators for GB300 (sm_103a) whose
 * gradients the optimizer step of soma_opt.h takes: layer norm, linear layer
 * and distillation loss, each forward and backward.
 *
 * Matrices are row-major with unit stride along a row; `*_stride` is the
 * distance between rows in elements (at least the row's length; ignored when
 * there is one row).  Buffers are device memory of `device`, aligned to their
 * element size only; rows that start on 16-byte boundaries run fastest.
 * Outputs must not overlap inputs or each other except where a call says so.
 *
 * Types are SOMA_DTYPE_F32, _BF16 or _F16.  Every sum, statistic and
 * exponential is held in fp32; an output is rounded to its type once, to
 * nearest even.  Results do not depend on the schedule: the same call on the
 * same device gives the same bits.
 *
 * Memory belongs to the caller.  A call that needs scratch memory says how
 * much through its *_workspace function; the buffer (256-byte aligned device
 * memory) is in use until the call's work on `stream` is done.  Nothing is
 * allocated and nothing waits: calls enqueue on `stream` (a cudaStream_t;
 * NULL = the legacy default stream) and return, and may be captured in a CUDA
 * graph (make a first call of the same kind before: it loads the kernels).
 *
 * Errors: every call returns a status of soma_opt.h; arguments are checked
 * before anything is enqueued, and soma_ops_last_error() has the detail of
 * the calling thread's last failure.  A call with no rows to compute
 * succeeds; it writes only the outputs that have elements (zero gradients).
 *
 * Threads: calls are independent and may be made from several threads.
 */
#ifndef SOMA_OPS_H
#define SOMA_OPS_H

#include <stdint.h>

#include "soma_opt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Detail of the calling thread's last failed call of this header ("" if
 * none).  Valid until the thread's next call. */
const char *soma_ops_last_error(void);

/* Kernels that wait for their own asynchronous copies and products bound that
 * wait: a second, where a step of their pipelines takes microseconds, and 20 us
 * more for each 64 values that a sum of products runs over.  This call waits
 * for all work on `device`, on every stream, and returns SOMA_ERR_STATE if such
 * a wait ran out since the last check, which leaves that call's outputs
 * invalid: a fault of the library, not of its arguments.  Not while a stream is
 * being captured. */
soma_status_t soma_ops_check(int32_t device);

/* ---- layer norm -------------------------------------------------------------
 * Over each row of x[rows][cols]:
 *   mean = sum_c x_c / cols,  rstd = 1 / sqrt(sum_c (x_c - mean)^2 / cols + eps)
 *   y_c  = (x_c - mean) * rstd * weight_c + bias_c
 * x and y are in `dtype`; weight and bias [cols] (NULL = 1 and 0) in
 * param_dtype, fp32 or `dtype`.  mean and rstd [rows] fp32 are what the
 * backward pass takes; either may be NULL.  cols >= 1, eps >= 0 and finite.
 * y may be x itself (same pointer and stride). */
soma_status_t soma_layer_norm_forward(int32_t device, const void *x, int64_t x_stride, const void *weight,
                                      const void *bias, void *y, int64_t y_stride, float *mean, float *rstd,
                                      int64_t rows, int64_t cols, int32_t dtype, int32_t param_dtype, double eps,
                                      void *stream);

/* Gradients of the above for dy = dL/dy, with xh = (x - mean) * rstd and
 * g = dy * weight:
 *   dx      = rstd * (g - sum_c g / cols - xh * sum_c (g * xh) / cols)
 *   dweight = sum_rows dy * xh,   dbias = sum_rows dy        (in param_dtype)
 * dx, dweight and dbias may each be NULL (not wanted).  dx may be dy or x
 * itself (same pointer and stride).  The workspace is only needed when
 * dweight or dbias is wanted. */
soma_status_t soma_layer_norm_backward_workspace(int32_t device, int64_t rows, int64_t cols, int64_t *bytes);
soma_status_t soma_layer_norm_backward(int32_t device, const void *dy, int64_t dy_stride, const void *x,
                                       int64_t x_stride, const void *weight, const float *mean, const float *rstd,
                                       void *dx, int64_t dx_stride, void *dweight, void *dbias, void *workspace,
                                       int64_t workspace_bytes, int64_t rows, int64_t cols, int32_t dtype,
                                       int32_t param_dtype, void *stream);

/* ---- linear layer ------------------------------------------------------------
 *   z = x * weight^T + bias,   y = act(z) + residual
 * x[m][k], weight[n][k], bias[n] (NULL = 0), residual[m][n] (NULL = 0),
 * y[m][n], all bf16 or all fp16 (products are exact, sums fp32).  z_out[m][n]
 * receives z rounded, for the backward pass (NULL = not wanted).  residual
 * may be y itself (same pointer and stride).  1 <= k <= 2^30, m, n <= 2^30. */
#define SOMA_ACT_NONE      0  /* z */
#define SOMA_ACT_RELU      1  /* max(z, 0) */
#define SOMA_ACT_GELU      2  /* z * (1 + erf(z / sqrt(2))) / 2 */
#define SOMA_ACT_GELU_TANH 3  /* z * (1 + tanh(sqrt(2/pi) * (z + 0.044715 z^3))) / 2 */
#define SOMA_ACT_SILU      4  /* z / (1 + exp(-z)) */
soma_status_t soma_linear_forward_workspace(int32_t device, const void *x, int64_t x_stride, const void *weight,
                                            int64_t weight_stride, int64_t m, int64_t n, int64_t k, int32_t dtype,
                                            int64_t *bytes);
soma_status_t soma_linear_forward(int32_t device, const void *x, int64_t x_stride, const void *weight,
                                  int64_t weight_stride, const void *bias, const void *residual,
                                  int64_t residual_stride, void *y, int64_t y_stride, void *z_out, int64_t z_stride,
                                  void *workspace, int64_t workspace_bytes, int64_t m, int64_t n, int64_t k,
                                  int32_t dtype, int32_t activation, void *stream);

/* Gradients of the above for dy = dL/dy (dL/dresidual is dy itself):
 *   dz = dy * act'(z)
 *   dx = dz * weight,   dweight = dz^T * x,   dbias = sum_rows dz
 * z is the forward pass's z_out (ignored, may be NULL, for SOMA_ACT_NONE).
 * With an activation, dz is rounded once to the operands' type before the two
 * matrix products, whose tensor-core operands are 16-bit; dbias sums it
 * unrounded.  act'(0) = 0 for ReLU.  dx, dweight and dbias may each be NULL.
 * dweight has rows of dweight_stride elements; dbias has n elements. */
soma_status_t soma_linear_backward_workspace(int32_t device, const void *dy, int64_t dy_stride, const void *x,
                                             int64_t x_stride, const void *weight, int64_t weight_stride, int64_t m,
                                             int64_t n, int64_t k, int32_t dtype, int32_t activation,
                                             int64_t *bytes);
soma_status_t soma_linear_backward(int32_t device, const void *dy, int64_t dy_stride, const void *x,
                                   int64_t x_stride, const void *weight, int64_t weight_stride, const void *z,
                                   int64_t z_stride, void *dx, int64_t dx_stride, void *dweight,
                                   int64_t dweight_stride, void *dbias, void *workspace, int64_t workspace_bytes,
                                   int64_t m, int64_t n, int64_t k, int32_t dtype, int32_t activation,
                                   void *stream);

/* ---- distillation from a teacher's top logits -------------------------------
 * A teacher answers each row with `top` of its logits and their places in
 * the vocabulary.  With temperature T, 1e-6 <= T <= 1e6,
 *   p_j    = exp(t_j / T) / sum_j exp(t_j / T)      over the row's valid entries
 *   q_v    = exp(z_v / T - lse),  lse = log sum_v exp(z_v / T)
 *   loss_r = row_weight_r * T^2 * sum_j p_j * (log p_j - log q_{index_j})
 *   dL/dz_v = scale_r * T * (q_v - sum_{j: index_j = v} p_j)
 * An entry whose index is outside [0, vocab) is not valid (mark a short
 * teacher row with -1); a row without valid entries, or whose valid teacher
 * logits are all -inf, has loss 0 and gradient 0.  Entries with p_j = 0 do
 * not count; an index may occur more than once.  A logit of -inf has q = 0;
 * where p > 0 there the loss is +inf.  A row whose logits are all -inf has lse
 * -inf and, if it has valid entries, loss and gradient NaN.  Every other value
 * is an ordinary logit, the type's lowest too: beside larger ones its q is 0
 * by its size, p > 0 there costs p |z| T, and a row wholly at it is uniform.
 * z / T is taken in fp32; where that overflows, the logit counts as infinite.
 * row_weight[rows] fp32 (NULL = 1): a row of weight 0 does not count, its
 * logits are not read, and its loss, lse and gradient are 0, whatever its
 * grad_loss is.
 *
 * logits[rows][vocab] in dtype, teacher[rows][top] in teacher_dtype,
 * index[rows][top] int32 or int64, 0 <= top <= SOMA_DISTILL_MAX_TOP,
 * 1 <= vocab <= 2^30; loss and lse [rows] fp32.
 *
 *   forward    loss and lse
 *   backward   dlogits for grad_loss[rows] = dL/dloss: scale = grad_loss * row_weight
 *   loss_grad  loss, lse (may be NULL) and dlogits for grad_loss = 1 in one
 *              kernel; the row's second reading, for the gradient, is from
 *              shared memory or L2 as far as those hold the rows in progress
 * dlogits[rows][vocab] in dtype may be the logits themselves (same pointer
 * and stride). */
#define SOMA_INDEX_I32 0
#define SOMA_INDEX_I64 1
#define SOMA_DISTILL_MAX_TOP 1024
soma_status_t soma_distill_forward(int32_t device, const void *logits, int64_t logits_stride, const void *teacher,
                                   int64_t teacher_stride, const void *index, int64_t index_stride,
                                   const float *row_weight, double temperature, float *loss, float *lse,
                                   int64_t rows, int64_t vocab, int64_t top, int32_t dtype, int32_t teacher_dtype,
                                   int32_t index_type, void *stream);
soma_status_t soma_distill_backward(int32_t device, const float *grad_loss, const void *logits,
                                    int64_t logits_stride, const float *lse, const void *teacher,
                                    int64_t teacher_stride, const void *index, int64_t index_stride,
                                    const float *row_weight, double temperature, void *dlogits,
                                    int64_t dlogits_stride, int64_t rows, int64_t vocab, int64_t top, int32_t dtype,
                                    int32_t teacher_dtype, int32_t index_type, void *stream);
soma_status_t soma_distill_loss_grad(int32_t device, const void *logits, int64_t logits_stride, const void *teacher,
                                     int64_t teacher_stride, const void *index, int64_t index_stride,
                                     const float *row_weight, double temperature, float *loss, float *lse,
                                     void *dlogits, int64_t dlogits_stride, int64_t rows, int64_t vocab,
                                     int64_t top, int32_t dtype, int32_t teacher_dtype, int32_t index_type,
                                     void *stream);

#ifdef __cplusplus
}
#endif
#endif /* SOMA_OPS_H */
