// Host side of a language model's ends (include/soma_ops.h): argument checks,
// workspace layout and launches of the embedding and of the linear layer with
// cross entropy.
#include "soma_ops.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "ops_host.h"
#include "ops_kernels.h"

namespace {

using namespace soma;

soma_status_t check_tokens(const char* name, const TokenArgs& t, int64_t batch) {
    if (batch < 0 || t.length < 0 || (t.length > 0 && batch > kMaxInt / t.length))
        return fail(SOMA_ERR_INVALID_ARG, "batch and length must be >= 0 and their product below 2^31");
    if (t.type != SOMA_INDEX_I32 && t.type != SOMA_INDEX_I64)
        return fail(SOMA_ERR_DTYPE, "index_type = %d", (int)t.type);
    return check_matrix(name, t.index, t.stride, batch, t.length, t.type == SOMA_INDEX_I64 ? 8 : 4);
}

soma_status_t check_embedding(const TokenArgs& t, int64_t batch, int64_t vocab, int64_t cols, int32_t dtype,
                              double scale) {
    if (vocab < 1 || vocab > kMaxExtent) return fail(SOMA_ERR_INVALID_ARG, "vocab must be in [1, 2^30]");
    if (cols < 1 || cols > kMaxExtent) return fail(SOMA_ERR_INVALID_ARG, "cols must be in [1, 2^30]");
    if (!is_dtype(dtype)) return fail(SOMA_ERR_DTYPE, "dtype = %d", (int)dtype);
    if (!std::isfinite((float)scale)) return fail(SOMA_ERR_INVALID_ARG, "scale must be finite in fp32 (got %g)", scale);
    return check_tokens("index", t, batch);
}

soma_status_t check_head(const HeadArgs& a, int64_t batch, int64_t vocab, int64_t k) {
    if (vocab < 1 || vocab > kMaxExtent) return fail(SOMA_ERR_INVALID_ARG, "vocab must be in [1, 2^30]");
    if (k < 1 || k > kMaxExtent) return fail(SOMA_ERR_INVALID_ARG, "k must be in [1, 2^30]");
    if (a.dtype != SOMA_DTYPE_BF16 && a.dtype != SOMA_DTYPE_F16)
        return fail(SOMA_ERR_DTYPE, "dtype = %d: the products take bf16 or fp16", (int)a.dtype);
    SOMA_TRY(check_tokens("target", a.tokens, batch));
    if (batch * a.tokens.length > kMaxExtent) return fail(SOMA_ERR_INVALID_ARG, "more than 2^30 rows");
    SOMA_TRY(check_matrix("x", a.x, a.x_stride, a.rows, k, 2));
    SOMA_TRY(check_matrix("weight", a.weight, a.weight_stride, vocab, k, 2));
    SOMA_TRY(check_vector("row_weight", a.row_weight, a.rows, 4, true));
    SOMA_TRY(check_vector("loss", a.loss, a.rows, 4, true));
    SOMA_TRY(check_vector("lse", a.lse, a.rows, 4, true));
    SOMA_TRY(check_matrix("dx", a.dx, a.dx_stride, a.rows, k, 2, true));
    return check_matrix("dweight", a.dweight, a.dweight_stride, vocab, k, 2, true);
}

HeadArgs head_args(const void* x, int64_t x_stride, const void* weight, int64_t weight_stride, const void* target,
                   int64_t target_stride, int64_t batch, int64_t length, const float* row_weight, int64_t vocab, int64_t k,
                   int32_t dtype, int32_t index_type) {
    HeadArgs a{};
    a.x = x;
    a.x_stride = x_stride;
    a.weight = weight;
    a.weight_stride = weight_stride;
    a.tokens = {target, target_stride, length, index_type};
    a.row_weight = row_weight;
    // (a product that does not fit is refused by check_tokens)
    a.rows = batch >= 0 && length > 0 && batch <= kMaxInt / length ? batch * length : 0;
    a.vocab = (int32_t)vocab;
    a.k = (int32_t)k;
    a.dtype = dtype;
    return a;
}

// After the checks: the launches, or zeros where no row is.
soma_status_t run_head(int32_t device, const HeadArgs& a, bool forward, void* workspace, int64_t workspace_bytes,
                       void* stream, const char* what) {
    if (a.rows == 0 && !a.dweight) return SOMA_OK;
    SOMA_ON_DEVICE(device);
    if (a.rows == 0) {
        const size_t pitch = (size_t)(a.vocab > 1 ? a.dweight_stride : a.k) * 2;
        return cuda_status(
            cudaMemset2DAsync(a.dweight, pitch, 0, (size_t)a.k * 2, (size_t)a.vocab, (cudaStream_t)stream), what);
    }
    SOMA_TRY(check_workspace(workspace, workspace_bytes, head_workspace(a, forward, sms)));
    return cuda_status(launch_head(a, forward, workspace, sms, stream), what);
}

}  // namespace

extern "C" {

soma_status_t soma_embedding_forward(int32_t device, const void* weight, int64_t weight_stride, const void* index,
                                     int64_t index_stride, int64_t batch, int64_t length, void* y, int64_t y_stride,
                                     int64_t vocab, int64_t cols, int32_t dtype, int32_t index_type, double scale,
                                     void* stream) {
    const TokenArgs t{index, index_stride, length, index_type};
    SOMA_TRY(check_embedding(t, batch, vocab, cols, dtype, scale));
    const int64_t rows = batch * length;
    const int e = size_of(dtype);
    SOMA_TRY(check_matrix("weight", weight, weight_stride, vocab, cols, e));
    SOMA_TRY(check_matrix("y", y, y_stride, rows, cols, e));
    if (rows == 0) return SOMA_OK;
    SOMA_ON_DEVICE(device);
    (void)sms;
    return cuda_status(launch_embedding_fwd({t, weight, weight_stride, y, y_stride, rows, (int32_t)vocab, (int32_t)cols,
                                             dtype, (float)scale},
                                            stream),
                       "embedding");
}

soma_status_t soma_embedding_backward_workspace(int32_t device, int64_t rows, int64_t vocab, int64_t cols,
                                                int64_t* bytes) {
    (void)device;
    if (!bytes) return fail(SOMA_ERR_INVALID_ARG, "bytes is NULL");
    if (rows < 0 || rows > kMaxInt) return fail(SOMA_ERR_INVALID_ARG, "rows must be in [0, 2^31)");
    if (vocab < 1 || vocab > kMaxExtent) return fail(SOMA_ERR_INVALID_ARG, "vocab must be in [1, 2^30]");
    if (cols < 1 || cols > kMaxExtent) return fail(SOMA_ERR_INVALID_ARG, "cols must be in [1, 2^30]");
    *bytes = rows == 0 ? 0 : embedding_bwd_workspace(rows, cols);
    return SOMA_OK;
}

soma_status_t soma_embedding_backward(int32_t device, const void* dy, int64_t dy_stride, const void* index,
                                      int64_t index_stride, int64_t batch, int64_t length, void* dweight,
                                      int64_t dweight_stride, int32_t accumulate, void* workspace,
                                      int64_t workspace_bytes, int64_t vocab, int64_t cols, int32_t dtype,
                                      int32_t index_type, double scale, void* stream) {
    const TokenArgs t{index, index_stride, length, index_type};
    SOMA_TRY(check_embedding(t, batch, vocab, cols, dtype, scale));
    if (accumulate != 0 && accumulate != 1) return fail(SOMA_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    const int64_t rows = batch * length;
    const int e = size_of(dtype);
    SOMA_TRY(check_matrix("dy", dy, dy_stride, rows, cols, e));
    SOMA_TRY(check_matrix("dweight", dweight, dweight_stride, vocab, cols, e));
    if (rows == 0 && accumulate) return SOMA_OK;
    if (rows > 0) SOMA_TRY(check_workspace(workspace, workspace_bytes, embedding_bwd_workspace(rows, cols)));
    SOMA_ON_DEVICE(device);
    if (rows == 0) {
        const size_t pitch = (size_t)(vocab > 1 ? dweight_stride : cols) * e;
        return cuda_status(cudaMemset2DAsync(dweight, pitch, 0, (size_t)cols * e, (size_t)vocab, (cudaStream_t)stream),
                           "embedding backward");
    }
    return cuda_status(launch_embedding_bwd({t, nullptr, 0, dweight, dweight_stride, rows, (int32_t)vocab,
                                             (int32_t)cols, dtype, (float)scale},
                                            dy, dy_stride, accumulate != 0, workspace, sms, stream),
                       "embedding backward");
}

// ---- cross entropy of a linear layer ----------------------------------------

soma_status_t soma_linear_cross_entropy_workspace(int32_t device, const void* weight, int64_t weight_stride, int64_t rows,
                                                  int64_t vocab, int64_t k, int32_t dtype, int32_t forward, int32_t dx,
                                                  int32_t dweight, int64_t* bytes) {
    if (!bytes) return fail(SOMA_ERR_INVALID_ARG, "bytes is NULL");
    if (rows < 0 || rows > kMaxExtent) return fail(SOMA_ERR_INVALID_ARG, "rows must be in [0, 2^30]");
    if (vocab < 1 || vocab > kMaxExtent) return fail(SOMA_ERR_INVALID_ARG, "vocab must be in [1, 2^30]");
    if (k < 1 || k > kMaxExtent) return fail(SOMA_ERR_INVALID_ARG, "k must be in [1, 2^30]");
    if (dtype != SOMA_DTYPE_BF16 && dtype != SOMA_DTYPE_F16) return fail(SOMA_ERR_DTYPE, "dtype = %d: the products take bf16 or fp16", (int)dtype);
    const int sms = sm_count(device);
    if (sms <= 0) return fail(SOMA_ERR_CUDA, "no SM count for device %d", (int)device);
    static char wanted;
    HeadArgs a = head_args(nullptr, 0, weight, weight_stride, nullptr, 0, 1, rows, nullptr, vocab, k, dtype, 0);
    a.dx = dx ? &wanted : nullptr;
    a.dweight = dweight ? &wanted : nullptr;
    *bytes = rows == 0 ? 0 : head_workspace(a, forward != 0, sms);
    return SOMA_OK;
}

soma_status_t soma_linear_cross_entropy_forward(int32_t device, const void* x, int64_t x_stride, const void* weight,
                                                int64_t weight_stride, const void* target, int64_t target_stride,
                                                int64_t batch, int64_t length, const float* row_weight, float* loss,
                                                float* lse, void* workspace, int64_t workspace_bytes, int64_t vocab,
                                                int64_t k, int32_t dtype, int32_t index_type, void* stream) {
    HeadArgs a = head_args(x, x_stride, weight, weight_stride, target, target_stride, batch, length, row_weight, vocab, k,
                           dtype, index_type);
    a.loss = loss;
    a.lse = lse;
    SOMA_TRY(check_head(a, batch, vocab, k));
    return run_head(device, a, true, workspace, workspace_bytes, stream, "linear cross entropy");
}

soma_status_t soma_linear_cross_entropy_backward(int32_t device, const float* grad_loss, const void* x, int64_t x_stride,
                                                 const void* weight, int64_t weight_stride, const void* target,
                                                 int64_t target_stride, int64_t batch, int64_t length, const float* lse,
                                                 const float* row_weight, void* dx, int64_t dx_stride, void* dweight,
                                                 int64_t dweight_stride, void* workspace, int64_t workspace_bytes,
                                                 int64_t vocab, int64_t k, int32_t dtype, int32_t index_type,
                                                 void* stream) {
    HeadArgs a = head_args(x, x_stride, weight, weight_stride, target, target_stride, batch, length, row_weight, vocab, k,
                           dtype, index_type);
    a.grad_loss = grad_loss;
    a.lse_in = lse;
    a.dx = dx;
    a.dx_stride = dx_stride;
    a.dweight = dweight;
    a.dweight_stride = dweight_stride;
    SOMA_TRY(check_head(a, batch, vocab, k));
    SOMA_TRY(check_vector("grad_loss", grad_loss, a.rows, 4, false));
    SOMA_TRY(check_vector("lse", lse, a.rows, 4, false));
    if (!dx && !dweight) return SOMA_OK;
    return run_head(device, a, false, workspace, workspace_bytes, stream, "linear cross entropy backward");
}

soma_status_t soma_linear_cross_entropy_loss_grad(int32_t device, const void* x, int64_t x_stride, const void* weight,
                                                  int64_t weight_stride, const void* target, int64_t target_stride,
                                                  int64_t batch, int64_t length, const float* row_weight, float* loss,
                                                  float* lse, void* dx, int64_t dx_stride, void* dweight,
                                                  int64_t dweight_stride, void* workspace, int64_t workspace_bytes,
                                                  int64_t vocab, int64_t k, int32_t dtype, int32_t index_type,
                                                  void* stream) {
    HeadArgs a = head_args(x, x_stride, weight, weight_stride, target, target_stride, batch, length, row_weight, vocab, k,
                           dtype, index_type);
    a.loss = loss;
    a.lse = lse;
    a.dx = dx;
    a.dx_stride = dx_stride;
    a.dweight = dweight;
    a.dweight_stride = dweight_stride;
    SOMA_TRY(check_head(a, batch, vocab, k));
    SOMA_TRY(check_vector("loss", loss, a.rows, 4, false));
    return run_head(device, a, true, workspace, workspace_bytes, stream, "linear cross entropy and gradients");
}

}  // extern "C"
