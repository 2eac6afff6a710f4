// Argument blocks and launchers of the training operators (layer norm,
// linear layer, distillation loss), shared by the host checks (ops.cpp) and
// the kernels.  Every launcher returns the cudaError_t of its launches as int.
#pragma once

#include <cstdint>

namespace soma {

struct NormFwdArgs {
    const void* x;
    int64_t x_stride;
    const void* weight;  // or nullptr
    const void* bias;    // or nullptr
    void* y;
    int64_t y_stride;
    float* mean;         // or nullptr
    float* rstd;         // or nullptr
    int64_t rows;
    int32_t cols;
    int32_t dtype, param_dtype;
    float eps;
};

struct NormBwdArgs {
    const void* dy;
    int64_t dy_stride;
    const void* x;
    int64_t x_stride;
    const void* weight;  // or nullptr
    const float* mean;
    const float* rstd;
    void* dx;            // or nullptr
    int64_t dx_stride;
    void* dweight;       // or nullptr
    void* dbias;         // or nullptr
    float* partials;     // workspace, see norm_bwd_workspace
    int64_t rows;
    int32_t cols;
    int32_t dtype, param_dtype;
};

// What a kernel needs to know of the current device, looked up once per
// kernel (and block and shared-memory size) and device: the driver's own
// answers take microseconds per call.
int allow_smem(const void* kernel, int bytes);
int resident_ctas(const void* kernel, int block, int smem, int* ctas);

int launch_norm_fwd(const NormFwdArgs& a, int sm_count, void* stream);
int64_t norm_bwd_workspace(int64_t rows, int64_t cols, int sm_count);
int launch_norm_bwd(const NormBwdArgs& a, int sm_count, void* stream);

// out[m][n] = act(sum_k A(m, k) B(n, k) + bias[n]) + residual[m][n], all
// operands of one 16-bit type.  A(m, k) is a[m * a_stride + k] when a_kmajor,
// else a[k * a_stride + m]; B likewise.
struct GemmArgs {
    const void* a;
    int64_t a_stride;
    bool a_kmajor;
    const void* b;
    int64_t b_stride;
    bool b_kmajor;
    const void* bias;      // or nullptr
    const void* residual;  // or nullptr
    int64_t residual_stride;
    void* out;
    int64_t out_stride;
    void* z_out;           // or nullptr: the sum with bias, before act
    int64_t z_stride;
    int32_t m, n, k;
    int32_t dtype;
    int32_t act;
};

int launch_gemm(const GemmArgs& a, int sm_count, void* stream);

// launch_gemm reads operands by TMA: rows that do not start on 16-byte
// boundaries (needs_copy) are first copied into rows that do.
bool gemm_operand_needs_copy(const void* p, int64_t stride, int64_t rows);
int launch_repack(const void* src, int64_t src_stride, void* dst, int64_t dst_stride, int64_t rows, int64_t cols,
                  int dtype, int sm_count, void* stream);

// dz = dy * act'(z) (dz == nullptr: not stored), and dbias = column sums of
// the unrounded dz (dbias == nullptr: not wanted).
struct ActBwdArgs {
    const void* dy;
    int64_t dy_stride;
    const void* z;
    int64_t z_stride;
    void* dz;
    int64_t dz_stride;
    void* dbias;
    float* partials;  // workspace, see act_bwd_workspace; only with dbias
    int64_t rows;
    int32_t cols;
    int32_t dtype;
    int32_t act;
};

int64_t act_bwd_workspace(int64_t rows, int64_t cols, int sm_count);
int launch_act_bwd(const ActBwdArgs& a, int sm_count, void* stream);

struct DistillArgs {
    const void* logits;
    int64_t logits_stride;
    const void* teacher;
    int64_t teacher_stride;
    const void* index;
    int64_t index_stride;
    const float* row_weight;  // or nullptr
    const float* grad_loss;   // backward only
    const float* lse_in;      // backward only
    float* loss;              // forward, loss_grad
    float* lse;               // forward, loss_grad (or nullptr)
    void* dlogits;            // backward, loss_grad
    int64_t dlogits_stride;
    float temperature, inv_temperature;
    int64_t rows;
    int32_t vocab, top;
    int32_t dtype, teacher_dtype, index_type;
};

enum DistillPass : int32_t { kDistillForward, kDistillBackward, kDistillLossGrad };

int launch_distill(const DistillArgs& a, DistillPass pass, int sm_count, void* stream);

// How often a bounded wait inside a kernel of the current device has run out:
// a count that only grows (modulo 2^32).  The copy waits for the legacy default
// stream alone; kernels on others may still be running.
int read_norm_gave_up(unsigned* count);
int read_linear_gave_up(unsigned* count);
int read_distill_gave_up(unsigned* count);

}  // namespace soma
