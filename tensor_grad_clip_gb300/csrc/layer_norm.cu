// Layer norm, forward and backward (formulas in soma_ops.h).
#include "ops_device.cuh"
#include "ops_kernels.h"

namespace soma {
namespace {

constexpr int kBlock = 256;

// Sum over the block, valid in every thread.
__device__ __forceinline__ float block_total(float x, float* scratch) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();  // the previous total has been read
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
    __syncthreads();
    float r = 0.f;
#pragma unroll
    for (int w = 0; w < kBlock / 32; ++w) r += scratch[w];
    return r;
}

template <typename T, typename W>
__global__ void __launch_bounds__(kBlock) norm_fwd_kernel(const __grid_constant__ NormFwdArgs a) {
    __shared__ float scratch[kBlock / 32];
    const W* w = static_cast<const W*>(a.weight);
    const W* b = static_cast<const W*>(a.bias);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
        T* y = static_cast<T*>(a.y) + r * a.y_stride;
        float s = 0.f;
        for (int c = threadIdx.x; c < a.cols; c += kBlock) s += to_f32(x[c]);
        const float mean = block_total(s, scratch) / (float)a.cols;
        s = 0.f;
        for (int c = threadIdx.x; c < a.cols; c += kBlock) {
            const float d = to_f32(x[c]) - mean;
            s = fmaf(d, d, s);
        }
        const float rstd = 1.f / sqrtf(block_total(s, scratch) / (float)a.cols + a.eps);
        for (int c = threadIdx.x; c < a.cols; c += kBlock) {
            const float v = (to_f32(x[c]) - mean) * rstd;
            y[c] = from_f32<T>(v * (w ? to_f32(w[c]) : 1.f) + (b ? to_f32(b[c]) : 0.f));
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

template <typename T, typename W>
__global__ void __launch_bounds__(kBlock) norm_dx_kernel(const __grid_constant__ NormBwdArgs a) {
    __shared__ float scratch[kBlock / 32];
    const W* w = static_cast<const W*>(a.weight);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
        const T* dy = static_cast<const T*>(a.dy) + r * a.dy_stride;
        T* dx = static_cast<T*>(a.dx) + r * a.dx_stride;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s0 = 0.f, s1 = 0.f;
        for (int c = threadIdx.x; c < a.cols; c += kBlock) {
            const float g = to_f32(dy[c]) * (w ? to_f32(w[c]) : 1.f);
            s0 += g;
            s1 = fmaf(g, (to_f32(x[c]) - mean) * rstd, s1);
        }
        s0 = block_total(s0, scratch) / (float)a.cols;
        s1 = block_total(s1, scratch) / (float)a.cols;
        for (int c = threadIdx.x; c < a.cols; c += kBlock) {
            const float g = to_f32(dy[c]) * (w ? to_f32(w[c]) : 1.f);
            const float xh = (to_f32(x[c]) - mean) * rstd;
            dx[c] = from_f32<T>(rstd * (g - s0 - xh * s1));
        }
    }
}

// Sums of dy * xh and dy over the rows of one part, a thread per column.
template <typename T>
__global__ void __launch_bounds__(kBlock) norm_dw_partial_kernel(const __grid_constant__ NormBwdArgs a, int parts) {
    const int c = blockIdx.x * kBlock + threadIdx.x;
    if (c >= a.cols) return;
    float dw = 0.f, db = 0.f;
    for (int64_t r = blockIdx.y; r < a.rows; r += parts) {
        const float g = to_f32(static_cast<const T*>(a.dy)[r * a.dy_stride + c]);
        const float xh = (to_f32(static_cast<const T*>(a.x)[r * a.x_stride + c]) - a.mean[r]) * a.rstd[r];
        dw = fmaf(g, xh, dw);
        db += g;
    }
    a.partials[(int64_t)blockIdx.y * a.cols + c] = dw;
    a.partials[(int64_t)(parts + blockIdx.y) * a.cols + c] = db;
}

template <typename W>
__global__ void __launch_bounds__(kBlock) norm_dw_kernel(const __grid_constant__ NormBwdArgs a, int parts) {
    const int c = blockIdx.x * kBlock + threadIdx.x;
    if (c >= a.cols) return;
    float dw = 0.f, db = 0.f;
    for (int p = 0; p < parts; ++p) {
        dw += a.partials[(int64_t)p * a.cols + c];
        db += a.partials[(int64_t)(parts + p) * a.cols + c];
    }
    if (a.dweight) static_cast<W*>(a.dweight)[c] = from_f32<W>(dw);
    if (a.dbias) static_cast<W*>(a.dbias)[c] = from_f32<W>(db);
}

int row_parts(int64_t rows) { return (int)(rows < 64 ? (rows > 0 ? rows : 1) : 64); }

template <typename F>
int with_types(int dtype, int param_dtype, F&& f) {
    return with_type(dtype, [&](auto t) {
        using T = decltype(t);
        return param_dtype == kF32 ? f(t, float{}) : f(t, T{});
    });
}

}  // namespace

int launch_norm_fwd(const NormFwdArgs& a, int sm_count, void* stream) {
    return with_types(a.dtype, a.param_dtype, [&](auto t, auto w) {
        const int grid = (int)(a.rows < 16 * sm_count ? a.rows : 16 * sm_count);
        norm_fwd_kernel<decltype(t), decltype(w)><<<grid, kBlock, 0, (cudaStream_t)stream>>>(a);
        return (int)cudaGetLastError();
    });
}

int64_t norm_bwd_workspace(int64_t rows, int64_t cols, int) { return 2 * (int64_t)row_parts(rows) * cols * 4; }

int launch_norm_bwd(const NormBwdArgs& a, int sm_count, void* stream) {
    return with_types(a.dtype, a.param_dtype, [&](auto t, auto w) {
        using T = decltype(t);
        using W = decltype(w);
        cudaStream_t st = (cudaStream_t)stream;
        const int cblocks = (a.cols + kBlock - 1) / kBlock;
        if (a.dweight || a.dbias) {
            const int parts = row_parts(a.rows);
            norm_dw_partial_kernel<T><<<dim3(cblocks, parts), kBlock, 0, st>>>(a, parts);
            norm_dw_kernel<W><<<cblocks, kBlock, 0, st>>>(a, parts);
        }
        if (a.dx && a.rows > 0) {
            const int grid = (int)(a.rows < 16 * sm_count ? a.rows : 16 * sm_count);
            norm_dx_kernel<T, W><<<grid, kBlock, 0, st>>>(a);
        }
        return (int)cudaGetLastError();
    });
}

}  // namespace soma
