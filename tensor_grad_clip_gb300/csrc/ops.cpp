// Host side of the C ABI declared in include/soma_ops.h: argument checks,
// workspace layout and launches.
#include "soma_ops.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <array>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <map>
#include <mutex>
#include <string>
#include <tuple>
#include <utility>

#include "ops_kernels.h"
#include "soma_kernels.h"

namespace {

thread_local std::string g_error;

soma_status_t fail(soma_status_t st, const char* fmt, ...) {
    char buf[400];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    try {
        g_error = std::string(soma_status_string(st)) + ": " + buf;
    } catch (...) {  // no memory for the text: the status alone
        g_error.clear();
    }
    return st;
}

soma_status_t cuda_status(int e, const char* what) {
    if (e == cudaSuccess) return SOMA_OK;
    cudaGetLastError();
    return fail(SOMA_ERR_CUDA, "%s: %s (%d)", what, cudaGetErrorString((cudaError_t)e), e);
}

// Makes `dev` current for the scope and restores the caller's device.
struct DeviceGuard {
    int prev = -1, dev;
    cudaError_t status;
    explicit DeviceGuard(int d) : dev(d) {
        status = cudaGetDevice(&prev);
        if (status == cudaSuccess && prev != dev) status = cudaSetDevice(dev);
    }
    ~DeviceGuard() {
        if (prev >= 0 && prev != dev) cudaSetDevice(prev);
    }
};

// SM count of a device, looked up once.
int sm_count(int device) {
    static std::array<std::atomic<int>, 64> known{};
    if (device < 0) return 0;
    if (device < 64 && known[device].load(std::memory_order_relaxed) > 0) return known[device].load();
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (device < 64) known[device].store(n);
    return n;
}

constexpr int64_t kMaxInt = 0x7fffffff;
constexpr int64_t kMaxExtent = 1 << 30;  // of a dimension that kernels index with an int, sums of a few included

std::mutex g_facts_mu;
// (device, kernel, block or -1, shared memory) -> resident CTAs, or 1 where the shared memory is allowed
std::map<std::tuple<int, const void*, int, int>, int> g_facts;

// What the last check of a device found its kernels' counts of expired waits
// at: layer norm, linear, distillation.
using Counts = std::array<unsigned, 3>;
std::map<int, Counts> g_gave_up;

bool is_dtype(int32_t d) { return d == SOMA_DTYPE_F32 || d == SOMA_DTYPE_BF16 || d == SOMA_DTYPE_F16; }
int size_of(int32_t d) { return d == SOMA_DTYPE_F32 ? 4 : 2; }
int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// Checks a matrix argument.  A matrix without elements may be NULL.
soma_status_t check_matrix(const char* name, const void* p, int64_t stride, int64_t rows, int64_t cols, int esize,
                           bool optional = false) {
    if (rows == 0 || cols == 0) return SOMA_OK;
    if (!p) return optional ? SOMA_OK : fail(SOMA_ERR_INVALID_ARG, "%s is NULL", name);
    if (rows > 1 && stride < cols)
        return fail(SOMA_ERR_INVALID_ARG, "%s: stride %lld is below the row length %lld", name, (long long)stride,
                    (long long)cols);
    if (rows > 1 && stride > INT64_MAX / esize / rows)
        return fail(SOMA_ERR_LIMIT, "%s: stride %lld x %lld rows does not fit 64 bits", name, (long long)stride,
                    (long long)rows);
    if ((uintptr_t)p % esize) return fail(SOMA_ERR_ALIGNMENT, "%s is not aligned to its element size", name);
    return SOMA_OK;
}

soma_status_t check_vector(const char* name, const void* p, int64_t n, int esize, bool optional) {
    return check_matrix(name, p, n, 1, n, esize, optional);
}

soma_status_t check_workspace(const void* workspace, int64_t have, int64_t need) {
    if (need == 0) return SOMA_OK;
    if (!workspace) return fail(SOMA_ERR_INVALID_ARG, "workspace is NULL, %lld bytes are needed", (long long)need);
    if (have < need)
        return fail(SOMA_ERR_LIMIT, "workspace has %lld bytes, %lld are needed", (long long)have, (long long)need);
    if ((uintptr_t)workspace % 256) return fail(SOMA_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
    return SOMA_OK;
}

// A 16-bit operand of a matrix product: where it is, or the part of the
// workspace that a copy with aligned rows takes.
struct Operand {
    const void* p;
    int64_t stride, rows, cols;
    bool copy;
    Operand(const void* q, int64_t s, int64_t r, int64_t c)
        : p(q), stride(s), rows(r), cols(c), copy(soma::gemm_operand_needs_copy(q, s, r)) {}
    int64_t bytes() const { return copy ? align256(rows * ((cols + 7) / 8 * 8) * 2) : 0; }
    // Enqueues the copy, if any, and advances the workspace past it.
    int place(char*& workspace, int dtype, int sms, void* stream) {
        if (!copy) return cudaSuccess;
        const int64_t to = (cols + 7) / 8 * 8;
        const int e = soma::launch_repack(p, stride, workspace, to, rows, cols, dtype, sms, stream);
        p = workspace;
        stride = to;
        workspace += align256(rows * to * 2);
        copy = false;
        return e;
    }
};

#define SOMA_TRY(x)                              \
    do {                                         \
        const soma_status_t st_ = (x);           \
        if (st_ != SOMA_OK) return st_;          \
    } while (0)

// Start of a launching entry point, after its argument checks.
#define SOMA_ON_DEVICE(device)                                                             \
    DeviceGuard guard(device);                                                             \
    if (guard.status != cudaSuccess) return cuda_status((int)guard.status, "cudaSetDevice"); \
    const int sms = sm_count(device);                                                      \
    if (sms <= 0) return fail(SOMA_ERR_CUDA, "no SM count for device %d", (int)(device))

soma_status_t check_norm(int64_t rows, int64_t cols, int32_t dtype, int32_t param_dtype) {
    if (rows < 0) return fail(SOMA_ERR_INVALID_ARG, "rows < 0");
    if (cols < 1 || cols > kMaxInt) return fail(SOMA_ERR_INVALID_ARG, "cols must be in [1, 2^31)");
    if (!is_dtype(dtype)) return fail(SOMA_ERR_DTYPE, "dtype = %d", (int)dtype);
    if (param_dtype != SOMA_DTYPE_F32 && param_dtype != dtype)
        return fail(SOMA_ERR_DTYPE, "param_dtype = %d must be fp32 or dtype (%d)", (int)param_dtype, (int)dtype);
    return SOMA_OK;
}

soma_status_t check_linear(int64_t m, int64_t n, int64_t k, int32_t dtype, int32_t act) {
    if (m < 0 || n < 0 || m > kMaxExtent || n > kMaxExtent)
        return fail(SOMA_ERR_INVALID_ARG, "m and n must be in [0, 2^30]");
    if (k < 1 || k > kMaxExtent) return fail(SOMA_ERR_INVALID_ARG, "k must be in [1, 2^30]");
    if (dtype != SOMA_DTYPE_BF16 && dtype != SOMA_DTYPE_F16)
        return fail(SOMA_ERR_DTYPE, "dtype = %d: the linear layer takes bf16 or fp16", (int)dtype);
    if (act < SOMA_ACT_NONE || act > SOMA_ACT_SILU) return fail(SOMA_ERR_INVALID_ARG, "activation = %d", (int)act);
    return SOMA_OK;
}

// Workspace of the backward pass: the bias gradient's partial sums, dz (with
// an activation, or where dy's rows are not aligned), and copies of x and
// weight where theirs are not.
int64_t backward_bytes(const Operand& dy, const Operand& x, const Operand& weight, int32_t act, int sms) {
    const bool dz = act != SOMA_ACT_NONE || dy.copy;
    return align256(soma::act_bwd_workspace(dy.rows, dy.cols, sms)) +
           (dz ? align256(dy.rows * ((dy.cols + 7) / 8 * 8) * 2) : 0) + x.bytes() + weight.bytes();
}

soma_status_t check_distill(const soma::DistillArgs& a, int64_t vocab, int64_t top, double temperature) {
    if (a.rows < 0) return fail(SOMA_ERR_INVALID_ARG, "rows < 0");
    if (vocab < 1 || vocab > kMaxExtent) return fail(SOMA_ERR_INVALID_ARG, "vocab must be in [1, 2^30]");
    if (top < 0) return fail(SOMA_ERR_INVALID_ARG, "top < 0");
    if (top > SOMA_DISTILL_MAX_TOP)
        return fail(SOMA_ERR_LIMIT, "top = %lld, at most %d entries per row", (long long)top, SOMA_DISTILL_MAX_TOP);
    if (!is_dtype(a.dtype)) return fail(SOMA_ERR_DTYPE, "dtype = %d", (int)a.dtype);
    if (!is_dtype(a.teacher_dtype)) return fail(SOMA_ERR_DTYPE, "teacher_dtype = %d", (int)a.teacher_dtype);
    if (a.index_type != SOMA_INDEX_I32 && a.index_type != SOMA_INDEX_I64)
        return fail(SOMA_ERR_DTYPE, "index_type = %d", (int)a.index_type);
    if (!std::isfinite(temperature) || !(temperature >= 1e-6) || temperature > 1e6)
        return fail(SOMA_ERR_INVALID_ARG, "temperature must be in [1e-6, 1e6] (got %g)", temperature);
    SOMA_TRY(check_matrix("logits", a.logits, a.logits_stride, a.rows, vocab, size_of(a.dtype)));
    SOMA_TRY(check_matrix("teacher", a.teacher, a.teacher_stride, a.rows, top, size_of(a.teacher_dtype)));
    SOMA_TRY(check_matrix("index", a.index, a.index_stride, a.rows, top, a.index_type == SOMA_INDEX_I64 ? 8 : 4));
    return check_vector("row_weight", a.row_weight, a.rows, 4, true);
}

soma::DistillArgs distill_args(const void* logits, int64_t logits_stride, const void* teacher, int64_t teacher_stride,
                               const void* index, int64_t index_stride, const float* row_weight, double temperature,
                               int64_t rows, int64_t vocab, int64_t top, int32_t dtype, int32_t teacher_dtype,
                               int32_t index_type) {
    soma::DistillArgs a{};
    a.logits = logits;
    a.logits_stride = logits_stride;
    a.teacher = teacher;
    a.teacher_stride = teacher_stride;
    a.index = index;
    a.index_stride = index_stride;
    a.row_weight = row_weight;
    a.temperature = (float)temperature;
    a.inv_temperature = (float)(1.0 / temperature);
    a.rows = rows;
    a.vocab = (int32_t)vocab;
    a.top = (int32_t)top;
    a.dtype = dtype;
    a.teacher_dtype = teacher_dtype;
    a.index_type = index_type;
    return a;
}

}  // namespace

namespace soma {

int allow_smem(const void* kernel, int bytes) {
    int device = 0;
    if (const cudaError_t e = cudaGetDevice(&device)) return e;
    try {
        std::lock_guard<std::mutex> lk(g_facts_mu);
        int& most = g_facts[{device, kernel, -1, 0}];
        if (most >= bytes) return cudaSuccess;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) most = bytes;
        return e;
    } catch (...) {
        return cudaErrorMemoryAllocation;
    }
}

int resident_ctas(const void* kernel, int block, int smem, int* ctas) {
    int device = 0;
    if (const cudaError_t e = cudaGetDevice(&device)) return e;
    try {
        std::lock_guard<std::mutex> lk(g_facts_mu);
        int& n = g_facts[{device, kernel, block, smem}];
        cudaError_t e = cudaSuccess;
        if (n == 0) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, block, smem);
        *ctas = n;
        return e;
    } catch (...) {
        return cudaErrorMemoryAllocation;
    }
}

}  // namespace soma

extern "C" {

const char* soma_ops_last_error(void) { return g_error.c_str(); }

soma_status_t soma_ops_check(int32_t device) {
    SOMA_ON_DEVICE(device);
    (void)sms;
    SOMA_TRY(cuda_status(cudaDeviceSynchronize(), "check"));
    Counts now{};
    SOMA_TRY(cuda_status(soma::read_norm_gave_up(&now[0]), "check"));
    SOMA_TRY(cuda_status(soma::read_linear_gave_up(&now[1]), "check"));
    SOMA_TRY(cuda_status(soma::read_distill_gave_up(&now[2]), "check"));
    Counts before{};
    try {
        std::lock_guard<std::mutex> lk(g_facts_mu);
        before = std::exchange(g_gave_up[device], now);
    } catch (...) {
        return fail(SOMA_ERR_OOM, "no host memory");
    }
    if (now == before) return SOMA_OK;
    return fail(SOMA_ERR_STATE, "a %s kernel gave up waiting for its own copies: its results are not valid",
                now[0] != before[0] ? "layer norm" : now[1] != before[1] ? "linear" : "distillation");
}

// ---- layer norm -----------------------------------------------------------

soma_status_t soma_layer_norm_forward(int32_t device, const void* x, int64_t x_stride, const void* weight,
                                      const void* bias, void* y, int64_t y_stride, float* mean, float* rstd,
                                      int64_t rows, int64_t cols, int32_t dtype, int32_t param_dtype, double eps,
                                      void* stream) {
    SOMA_TRY(check_norm(rows, cols, dtype, param_dtype));
    if (!std::isfinite(eps) || eps < 0) return fail(SOMA_ERR_INVALID_ARG, "eps must be finite and >= 0 (got %g)", eps);
    const int e = size_of(dtype), pe = size_of(param_dtype);
    SOMA_TRY(check_matrix("x", x, x_stride, rows, cols, e));
    SOMA_TRY(check_matrix("y", y, y_stride, rows, cols, e));
    SOMA_TRY(check_vector("weight", weight, cols, pe, true));
    SOMA_TRY(check_vector("bias", bias, cols, pe, true));
    SOMA_TRY(check_vector("mean", mean, rows, 4, true));
    SOMA_TRY(check_vector("rstd", rstd, rows, 4, true));
    if (rows == 0) return SOMA_OK;
    SOMA_ON_DEVICE(device);
    soma::NormFwdArgs a{x, x_stride, weight, bias, y, y_stride, mean, rstd, rows, (int32_t)cols, dtype, param_dtype,
                        (float)eps};
    return cuda_status(soma::launch_norm_fwd(a, sms, stream), "layer norm");
}

soma_status_t soma_layer_norm_backward_workspace(int32_t device, int64_t rows, int64_t cols, int64_t* bytes) {
    if (!bytes) return fail(SOMA_ERR_INVALID_ARG, "bytes is NULL");
    SOMA_TRY(check_norm(rows, cols, SOMA_DTYPE_F32, SOMA_DTYPE_F32));
    const int sms = sm_count(device);
    if (sms <= 0) return fail(SOMA_ERR_CUDA, "no SM count for device %d", (int)device);
    *bytes = soma::norm_bwd_workspace(rows, cols, sms);
    return SOMA_OK;
}

soma_status_t soma_layer_norm_backward(int32_t device, const void* dy, int64_t dy_stride, const void* x,
                                       int64_t x_stride, const void* weight, const float* mean, const float* rstd,
                                       void* dx, int64_t dx_stride, void* dweight, void* dbias, void* workspace,
                                       int64_t workspace_bytes, int64_t rows, int64_t cols, int32_t dtype,
                                       int32_t param_dtype, void* stream) {
    SOMA_TRY(check_norm(rows, cols, dtype, param_dtype));
    const int e = size_of(dtype), pe = size_of(param_dtype);
    SOMA_TRY(check_matrix("dy", dy, dy_stride, rows, cols, e));
    SOMA_TRY(check_matrix("x", x, x_stride, rows, cols, e));
    SOMA_TRY(check_vector("weight", weight, cols, pe, true));
    SOMA_TRY(check_vector("mean", mean, rows, 4, false));
    SOMA_TRY(check_vector("rstd", rstd, rows, 4, false));
    SOMA_TRY(check_matrix("dx", dx, dx_stride, rows, cols, e, true));
    SOMA_TRY(check_vector("dweight", dweight, cols, pe, true));
    SOMA_TRY(check_vector("dbias", dbias, cols, pe, true));
    const bool params = dweight || dbias;
    if (!params && (!dx || rows == 0)) return SOMA_OK;
    SOMA_ON_DEVICE(device);
    if (params) SOMA_TRY(check_workspace(workspace, workspace_bytes, soma::norm_bwd_workspace(rows, cols, sms)));
    soma::NormBwdArgs a{dy, dy_stride, x,     x_stride, weight, mean, rstd, dx, dx_stride, dweight, dbias,
                        static_cast<float*>(workspace), rows, (int32_t)cols, dtype, param_dtype};
    return cuda_status(soma::launch_norm_bwd(a, sms, stream), "layer norm backward");
}

// ---- linear layer ---------------------------------------------------------

soma_status_t soma_linear_forward_workspace(int32_t device, const void* x, int64_t x_stride, const void* weight,
                                            int64_t weight_stride, int64_t m, int64_t n, int64_t k, int32_t dtype,
                                            int64_t* bytes) {
    (void)device;
    if (!bytes) return fail(SOMA_ERR_INVALID_ARG, "bytes is NULL");
    SOMA_TRY(check_linear(m, n, k, dtype, SOMA_ACT_NONE));
    *bytes = m == 0 || n == 0 ? 0 : Operand(x, x_stride, m, k).bytes() + Operand(weight, weight_stride, n, k).bytes();
    return SOMA_OK;
}

soma_status_t soma_linear_forward(int32_t device, const void* x, int64_t x_stride, const void* weight,
                                  int64_t weight_stride, const void* bias, const void* residual,
                                  int64_t residual_stride, void* y, int64_t y_stride, void* z_out, int64_t z_stride,
                                  void* workspace, int64_t workspace_bytes, int64_t m, int64_t n, int64_t k,
                                  int32_t dtype, int32_t activation, void* stream) {
    SOMA_TRY(check_linear(m, n, k, dtype, activation));
    SOMA_TRY(check_matrix("x", x, x_stride, m, k, 2));
    SOMA_TRY(check_matrix("weight", weight, weight_stride, n, k, 2));
    SOMA_TRY(check_vector("bias", bias, n, 2, true));
    SOMA_TRY(check_matrix("residual", residual, residual_stride, m, n, 2, true));
    SOMA_TRY(check_matrix("y", y, y_stride, m, n, 2));
    SOMA_TRY(check_matrix("z_out", z_out, z_stride, m, n, 2, true));
    if (m == 0 || n == 0) return SOMA_OK;
    Operand a(x, x_stride, m, k), b(weight, weight_stride, n, k);
    SOMA_TRY(check_workspace(workspace, workspace_bytes, a.bytes() + b.bytes()));
    SOMA_ON_DEVICE(device);
    char* ws = static_cast<char*>(workspace);
    int e = a.place(ws, dtype, sms, stream);
    if (e == cudaSuccess) e = b.place(ws, dtype, sms, stream);
    if (e == cudaSuccess)
        e = soma::launch_gemm({a.p, a.stride, true, b.p, b.stride, true, bias, residual, residual_stride, y, y_stride,
                               z_out, z_stride, (int32_t)m, (int32_t)n, (int32_t)k, dtype, activation},
                              sms, stream);
    return cuda_status(e, "linear");
}

soma_status_t soma_linear_backward_workspace(int32_t device, const void* dy, int64_t dy_stride, const void* x,
                                             int64_t x_stride, const void* weight, int64_t weight_stride, int64_t m,
                                             int64_t n, int64_t k, int32_t dtype, int32_t activation,
                                             int64_t* bytes) {
    if (!bytes) return fail(SOMA_ERR_INVALID_ARG, "bytes is NULL");
    SOMA_TRY(check_linear(m, n, k, dtype, activation));
    const int sms = sm_count(device);
    if (sms <= 0) return fail(SOMA_ERR_CUDA, "no SM count for device %d", (int)device);
    *bytes = m == 0 || n == 0 ? 0 : backward_bytes(Operand(dy, dy_stride, m, n), Operand(x, x_stride, m, k),
                                                   Operand(weight, weight_stride, n, k), activation, sms);
    return SOMA_OK;
}

soma_status_t soma_linear_backward(int32_t device, const void* dy, int64_t dy_stride, const void* x,
                                   int64_t x_stride, const void* weight, int64_t weight_stride, const void* z,
                                   int64_t z_stride, void* dx, int64_t dx_stride, void* dweight,
                                   int64_t dweight_stride, void* dbias, void* workspace, int64_t workspace_bytes,
                                   int64_t m, int64_t n, int64_t k, int32_t dtype, int32_t activation,
                                   void* stream) {
    SOMA_TRY(check_linear(m, n, k, dtype, activation));
    SOMA_TRY(check_matrix("dy", dy, dy_stride, m, n, 2));
    SOMA_TRY(check_matrix("x", x, x_stride, m, k, 2, !dweight));
    SOMA_TRY(check_matrix("weight", weight, weight_stride, n, k, 2, !dx));
    if (activation != SOMA_ACT_NONE) SOMA_TRY(check_matrix("z", z, z_stride, m, n, 2));
    SOMA_TRY(check_matrix("dx", dx, dx_stride, m, k, 2, true));
    SOMA_TRY(check_matrix("dweight", dweight, dweight_stride, n, k, 2, true));
    SOMA_TRY(check_vector("dbias", dbias, n, 2, true));
    SOMA_ON_DEVICE(device);
    cudaStream_t st = (cudaStream_t)stream;
    int e = cudaSuccess;
    if (n == 0) {  // nothing flows back
        if (dx && m > 0) e = cudaMemset2DAsync(dx, (size_t)std::max(dx_stride, k) * 2, 0, (size_t)k * 2, (size_t)m, st);
        return cuda_status(e, "linear backward");
    }
    if (m == 0) {
        if (dweight)
            e = cudaMemset2DAsync(dweight, (size_t)std::max(dweight_stride, k) * 2, 0, (size_t)k * 2, (size_t)n, st);
        if (dbias && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, (size_t)n * 2, st);
        return cuda_status(e, "linear backward");
    }
    Operand g(dy, dy_stride, m, n), a(x, x_stride, m, k), b(weight, weight_stride, n, k);
    SOMA_TRY(check_workspace(workspace, workspace_bytes, backward_bytes(g, a, b, activation, sms)));
    char* ws = static_cast<char*>(workspace);
    const bool products = dx || dweight;
    const bool store = products && (activation != SOMA_ACT_NONE || g.copy);
    if (store || dbias) {
        const int64_t dz_stride = (n + 7) / 8 * 8;
        char* dz = ws + align256(soma::act_bwd_workspace(m, n, sms));
        e = soma::launch_act_bwd({dy, dy_stride, z, z_stride, store ? dz : nullptr, dz_stride, dbias,
                                  reinterpret_cast<float*>(ws), m, (int32_t)n, dtype, activation},
                                 sms, stream);
        if (store) {
            g = Operand(dz, dz_stride, m, n);
            ws = dz + align256(m * dz_stride * 2);
        }
    }
    if (dx && e == cudaSuccess) e = b.place(ws, dtype, sms, stream);
    if (dx && e == cudaSuccess)
        e = soma::launch_gemm({g.p, g.stride, true, b.p, b.stride, false, nullptr, nullptr, 0, dx, dx_stride, nullptr, 0,
                               (int32_t)m, (int32_t)k, (int32_t)n, dtype, SOMA_ACT_NONE},
                              sms, stream);
    if (dweight && e == cudaSuccess) e = a.place(ws, dtype, sms, stream);
    if (dweight && e == cudaSuccess)
        e = soma::launch_gemm({g.p, g.stride, false, a.p, a.stride, false, nullptr, nullptr, 0, dweight, dweight_stride,
                               nullptr, 0, (int32_t)n, (int32_t)k, (int32_t)m, dtype, SOMA_ACT_NONE},
                              sms, stream);
    return cuda_status(e, "linear backward");
}

// ---- distillation loss ----------------------------------------------------

soma_status_t soma_distill_forward(int32_t device, const void* logits, int64_t logits_stride, const void* teacher,
                                   int64_t teacher_stride, const void* index, int64_t index_stride,
                                   const float* row_weight, double temperature, float* loss, float* lse,
                                   int64_t rows, int64_t vocab, int64_t top, int32_t dtype, int32_t teacher_dtype,
                                   int32_t index_type, void* stream) {
    soma::DistillArgs a = distill_args(logits, logits_stride, teacher, teacher_stride, index, index_stride, row_weight,
                                       temperature, rows, vocab, top, dtype, teacher_dtype, index_type);
    SOMA_TRY(check_distill(a, vocab, top, temperature));
    SOMA_TRY(check_vector("loss", loss, rows, 4, false));
    SOMA_TRY(check_vector("lse", lse, rows, 4, false));
    if (rows == 0) return SOMA_OK;
    SOMA_ON_DEVICE(device);
    a.loss = loss;
    a.lse = lse;
    return cuda_status(soma::launch_distill(a, soma::kDistillForward, sms, stream), "distillation loss");
}

soma_status_t soma_distill_backward(int32_t device, const float* grad_loss, const void* logits,
                                    int64_t logits_stride, const float* lse, const void* teacher,
                                    int64_t teacher_stride, const void* index, int64_t index_stride,
                                    const float* row_weight, double temperature, void* dlogits,
                                    int64_t dlogits_stride, int64_t rows, int64_t vocab, int64_t top, int32_t dtype,
                                    int32_t teacher_dtype, int32_t index_type, void* stream) {
    soma::DistillArgs a = distill_args(logits, logits_stride, teacher, teacher_stride, index, index_stride, row_weight,
                                       temperature, rows, vocab, top, dtype, teacher_dtype, index_type);
    SOMA_TRY(check_distill(a, vocab, top, temperature));
    SOMA_TRY(check_vector("grad_loss", grad_loss, rows, 4, false));
    SOMA_TRY(check_vector("lse", lse, rows, 4, false));
    SOMA_TRY(check_matrix("dlogits", dlogits, dlogits_stride, rows, vocab, size_of(dtype)));
    if (rows == 0) return SOMA_OK;
    SOMA_ON_DEVICE(device);
    a.grad_loss = grad_loss;
    a.lse_in = lse;
    a.dlogits = dlogits;
    a.dlogits_stride = dlogits_stride;
    return cuda_status(soma::launch_distill(a, soma::kDistillBackward, sms, stream), "distillation backward");
}

soma_status_t soma_distill_loss_grad(int32_t device, const void* logits, int64_t logits_stride, const void* teacher,
                                     int64_t teacher_stride, const void* index, int64_t index_stride,
                                     const float* row_weight, double temperature, float* loss, float* lse,
                                     void* dlogits, int64_t dlogits_stride, int64_t rows, int64_t vocab,
                                     int64_t top, int32_t dtype, int32_t teacher_dtype, int32_t index_type,
                                     void* stream) {
    soma::DistillArgs a = distill_args(logits, logits_stride, teacher, teacher_stride, index, index_stride, row_weight,
                                       temperature, rows, vocab, top, dtype, teacher_dtype, index_type);
    SOMA_TRY(check_distill(a, vocab, top, temperature));
    SOMA_TRY(check_vector("loss", loss, rows, 4, false));
    SOMA_TRY(check_vector("lse", lse, rows, 4, true));
    SOMA_TRY(check_matrix("dlogits", dlogits, dlogits_stride, rows, vocab, size_of(dtype)));
    if (rows == 0) return SOMA_OK;
    SOMA_ON_DEVICE(device);
    a.loss = loss;
    a.lse = lse;
    a.dlogits = dlogits;
    a.dlogits_stride = dlogits_stride;
    return cuda_status(soma::launch_distill(a, soma::kDistillLossGrad, sms, stream), "distillation loss and gradient");
}

}  // extern "C"
