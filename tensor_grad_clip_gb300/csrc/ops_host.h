// What the host sides of the training operators share: errors, the current
// device, argument checks.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "soma_ops.h"

namespace soma {

// Notes the calling thread's error text and returns the status.
soma_status_t fail(soma_status_t st, const char* fmt, ...);
soma_status_t cuda_status(int e, const char* what);

// SM count of a device, looked up once.
int sm_count(int device);

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

constexpr int64_t kMaxInt = 0x7fffffff;
constexpr int64_t kMaxExtent = 1 << 30;  // of a dimension that kernels index with an int, sums of a few included

inline bool is_dtype(int32_t d) { return d == SOMA_DTYPE_F32 || d == SOMA_DTYPE_BF16 || d == SOMA_DTYPE_F16; }
inline int size_of(int32_t d) { return d == SOMA_DTYPE_F32 ? 4 : 2; }
inline int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// Checks a matrix argument.  A matrix without elements may be NULL.
inline soma_status_t check_matrix(const char* name, const void* p, int64_t stride, int64_t rows, int64_t cols, int esize,
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

inline soma_status_t check_vector(const char* name, const void* p, int64_t n, int esize, bool optional) {
    return check_matrix(name, p, n, 1, n, esize, optional);
}

inline soma_status_t check_workspace(const void* workspace, int64_t have, int64_t need) {
    if (need == 0) return SOMA_OK;
    if (!workspace) return fail(SOMA_ERR_INVALID_ARG, "workspace is NULL, %lld bytes are needed", (long long)need);
    if (have < need)
        return fail(SOMA_ERR_LIMIT, "workspace has %lld bytes, %lld are needed", (long long)have, (long long)need);
    if ((uintptr_t)workspace % 256) return fail(SOMA_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
    return SOMA_OK;
}

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

}  // namespace soma
