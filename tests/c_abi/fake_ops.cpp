// Fakes of what csrc/ops.cpp calls, so that its host side runs without a GPU:
// the CUDA runtime's functions and the kernels' launchers.  A test sets what
// they return and reads in which order they were called.
#include <cuda_runtime.h>

#include <cstring>

#include "ops_kernels.h"
#include "soma_opt.h"

extern "C" {
unsigned fake_counts[3];  // expired waits: layer norm, linear, distillation
int fake_sync_error, fake_read_error;
char fake_calls[256];

static int called(const char* what, int result) {
    strncat(fake_calls, what, sizeof fake_calls - strlen(fake_calls) - 1);
    return result;
}

const char* soma_status_string(soma_status_t) { return "status"; }

cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "error"; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { return *v = 152, cudaSuccess; }
cudaError_t cudaDeviceSynchronize(void) { return (cudaError_t)called("sync ", fake_sync_error); }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*, int, size_t) { return *n = 1, cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemset2DAsync(void*, size_t, int, size_t, size_t, cudaStream_t) { return cudaSuccess; }
}

namespace soma {
static int read(int which, unsigned* count) {
    *count = fake_counts[which];
    return called("read ", fake_read_error);
}
int read_norm_gave_up(unsigned* count) { return read(0, count); }
int read_linear_gave_up(unsigned* count) { return read(1, count); }
int read_distill_gave_up(unsigned* count) { return read(2, count); }

int launch_norm_fwd(const NormFwdArgs&, int, void*) { return called("norm ", 0); }
int64_t norm_bwd_workspace(int64_t, int64_t, int) { return 0; }
int launch_norm_bwd(const NormBwdArgs&, int, void*) { return called("norm ", 0); }
int launch_gemm(const GemmArgs&, int, void*) { return called("gemm ", 0); }
bool gemm_operand_needs_copy(const void*, int64_t, int64_t) { return false; }
int launch_repack(const void*, int64_t, void*, int64_t, int64_t, int64_t, int, int, void*) { return called("repack ", 0); }
int64_t act_bwd_workspace(int64_t, int64_t, int) { return 0; }
int launch_act_bwd(const ActBwdArgs&, int, void*) { return called("act ", 0); }
int launch_distill(const DistillArgs&, DistillPass, int, void*) { return called("distill ", 0); }
}  // namespace soma
