// Host side of a language model's ends (include/soma_ops.h): argument checks,
// workspace layout and launches of the embedding.
#include "soma_ops.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "ops_host.h"
#include "ops_kernels.h"

namespace {

using namespace soma;

soma_status_t check_tokens(const TokenArgs& t, int64_t batch) {
    if (batch < 0 || t.length < 0 || (t.length > 0 && batch > kMaxInt / t.length))
        return fail(SOMA_ERR_INVALID_ARG, "batch and length must be >= 0 and their product below 2^31");
    if (t.type != SOMA_INDEX_I32 && t.type != SOMA_INDEX_I64)
        return fail(SOMA_ERR_DTYPE, "index_type = %d", (int)t.type);
    return check_matrix("index", t.index, t.stride, batch, t.length, t.type == SOMA_INDEX_I64 ? 8 : 4);
}

soma_status_t check_embedding(const TokenArgs& t, int64_t batch, int64_t vocab, int64_t cols, int32_t dtype,
                              double scale) {
    if (vocab < 1 || vocab > kMaxExtent) return fail(SOMA_ERR_INVALID_ARG, "vocab must be in [1, 2^30]");
    if (cols < 1 || cols > kMaxExtent) return fail(SOMA_ERR_INVALID_ARG, "cols must be in [1, 2^30]");
    if (!is_dtype(dtype)) return fail(SOMA_ERR_DTYPE, "dtype = %d", (int)dtype);
    if (!std::isfinite((float)scale)) return fail(SOMA_ERR_INVALID_ARG, "scale must be finite in fp32 (got %g)", scale);
    return check_tokens(t, batch);
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

}  // extern "C"
