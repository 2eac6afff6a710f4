// Distillation loss from a teacher's top logits (formulas in soma_ops.h).
#include <math.h>

#include "ops_device.cuh"
#include "ops_kernels.h"
#include "soma_ops.h"

namespace soma {
namespace {

constexpr int kBlock = 256;

__device__ __forceinline__ float block_sum(float x, float* scratch) {
    __syncthreads();
    scratch[threadIdx.x] = x;
    __syncthreads();
    float r = 0.f;
    for (int i = 0; i < kBlock; ++i) r += scratch[i];
    return r;
}
__device__ __forceinline__ float block_max(float x, float* scratch) {
    __syncthreads();
    scratch[threadIdx.x] = x;
    __syncthreads();
    float r = -INFINITY;
    for (int i = 0; i < kBlock; ++i) r = fmaxf(r, scratch[i]);
    return r;
}

template <typename T, typename U, int PASS>
__global__ void __launch_bounds__(kBlock) distill_kernel(const __grid_constant__ DistillArgs a) {
    __shared__ float scratch[kBlock];
    __shared__ float p[SOMA_DISTILL_MAX_TOP], zt[SOMA_DISTILL_MAX_TOP];
    __shared__ int at[SOMA_DISTILL_MAX_TOP];
    const int t = threadIdx.x;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* z = static_cast<const T*>(a.logits) + r * a.logits_stride;
        T* dz = static_cast<T*>(a.dlogits) + r * a.dlogits_stride;
        const float w = a.row_weight ? a.row_weight[r] : 1.f;
        const float scale = PASS == kDistillBackward ? a.grad_loss[r] * w : w;
        if (scale == 0.f) {
            if (t == 0 && PASS != kDistillBackward) a.loss[r] = 0.f;
            if (t == 0 && PASS != kDistillBackward && a.lse) a.lse[r] = 0.f;
            if (PASS != kDistillForward)
                for (int v = t; v < a.vocab; v += kBlock) dz[v] = from_f32<T>(0.f);
            continue;
        }
        __syncthreads();
        float top = -INFINITY;
        for (int j = t; j < a.top; j += kBlock) {
            const int64_t i = a.index_type == SOMA_INDEX_I64
                                  ? static_cast<const int64_t*>(a.index)[r * a.index_stride + j]
                                  : static_cast<const int32_t*>(a.index)[r * a.index_stride + j];
            const bool ok = i >= 0 && i < a.vocab;
            at[j] = ok ? (int)i : -1;
            p[j] = ok ? to_f32(static_cast<const U*>(a.teacher)[r * a.teacher_stride + j]) : -INFINITY;
            zt[j] = ok ? to_f32(z[i]) : 0.f;
            top = isnan(p[j]) ? p[j] : fmaxf(top, p[j]);
        }
        top = block_max(top, scratch);
        float total = 0.f;
        for (int j = t; j < a.top; j += kBlock)
            if (p[j] != -INFINITY) total += expf((p[j] - top) * a.inv_temperature);
        total = block_sum(total, scratch);
        const bool any = !(top == -INFINITY && total == 0.f);
        float lse, m = 0.f;
        if (PASS == kDistillBackward) {
            lse = a.lse_in[r];
        } else {
            m = -INFINITY;
            for (int v = t; v < a.vocab; v += kBlock) m = fmaxf(m, to_f32(z[v]));
            m = block_max(m, scratch);
            float s = 0.f;
            for (int v = t; v < a.vocab; v += kBlock) {
                const float x = to_f32(z[v]);
                if (x != -INFINITY) s += expf((x - m) * a.inv_temperature);
            }
            s = block_sum(s, scratch);
            lse = m * a.inv_temperature + logf(s);
        }
        float loss = 0.f;
        for (int j = t; j < a.top; j += kBlock) {
            const float logp = (p[j] - top) * a.inv_temperature - logf(total);
            const float pj = any && at[j] >= 0 ? expf(logp) : 0.f;
            if (pj != 0.f) loss += pj * (logp - zt[j] * a.inv_temperature + lse);
            p[j] = pj;
        }
        if (PASS != kDistillBackward) {
            loss = block_sum(loss, scratch);
            if (t == 0) {
                a.loss[r] = w * a.temperature * a.temperature * loss;
                if (a.lse) a.lse[r] = lse;
            }
        }
        if (PASS != kDistillForward) {
            __syncthreads();
            const float g = scale * a.temperature;
            for (int v = t; v < a.vocab; v += kBlock)
                dz[v] = from_f32<T>(any ? g * expf(fmaf(to_f32(z[v]), a.inv_temperature, -lse)) : 0.f);
            __syncthreads();
            for (int j = t; j < a.top; j += kBlock) {
                if (at[j] < 0) continue;
                float sum = 0.f;
                bool first = true;
                for (int i = 0; i < a.top; ++i) {
                    if (at[i] != at[j]) continue;
                    if (i < j) first = false;
                    sum += p[i];
                }
                if (first && any)
                    dz[at[j]] = from_f32<T>(g * (expf(fmaf(zt[j], a.inv_temperature, -lse)) - sum));
            }
        }
    }
}

}  // namespace

int launch_distill(const DistillArgs& a, DistillPass pass, int sm_count, void* stream) {
    return with_type(a.dtype, [&](auto t) {
        return with_type(a.teacher_dtype, [&](auto u) {
            using T = decltype(t);
            using U = decltype(u);
            const int grid = (int)(a.rows < 8 * sm_count ? a.rows : 8 * sm_count);
            cudaStream_t st = (cudaStream_t)stream;
            if (pass == kDistillForward) distill_kernel<T, U, kDistillForward><<<grid, kBlock, 0, st>>>(a);
            else if (pass == kDistillBackward) distill_kernel<T, U, kDistillBackward><<<grid, kBlock, 0, st>>>(a);
            else distill_kernel<T, U, kDistillLossGrad><<<grid, kBlock, 0, st>>>(a);
            return (int)cudaGetLastError();
        });
    });
}

}  // namespace soma
