// Linear layer: matrix products with their epilogue, and the activation's
// backward pass (formulas in soma_ops.h).
#include <math.h>

#include "ops_device.cuh"
#include "ops_kernels.h"
#include "soma_ops.h"

namespace soma {
namespace {

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f;
constexpr float kCubic = 0.044715f;

// 1 / (1 + exp(-x)); exp overflows to inf far left, where the result is 0.
__device__ __forceinline__ float logistic(float x) { return 1.f / (1.f + expf(-x)); }

__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case SOMA_ACT_RELU: return z < 0.f ? 0.f : z;  // NaN stays NaN
        case SOMA_ACT_GELU: return 0.5f * z * (1.f + erff(z * kSqrtHalf));
        // (1 + tanh u) / 2 is the logistic function of 2u
        case SOMA_ACT_GELU_TANH: return z * logistic(2.f * kSqrt2OverPi * z * fmaf(kCubic * z, z, 1.f));
        case SOMA_ACT_SILU: return z * logistic(z);
        default: return z;
    }
}

__device__ __forceinline__ float act_slope(float z, int act) {
    switch (act) {
        case SOMA_ACT_RELU: return z > 0.f ? 1.f : 0.f;
        case SOMA_ACT_GELU: return fmaf(z * kInvSqrt2Pi, expf(-0.5f * z * z), 0.5f * (1.f + erff(z * kSqrtHalf)));
        case SOMA_ACT_GELU_TANH: {
            const float s = logistic(2.f * kSqrt2OverPi * z * fmaf(kCubic * z, z, 1.f));
            const float du = 2.f * kSqrt2OverPi * fmaf(3.f * kCubic * z, z, 1.f);
            return fmaf(z * s * (1.f - s), du, s);
        }
        case SOMA_ACT_SILU: {
            const float s = logistic(z);
            return s * fmaf(z, 1.f - s, 1.f);
        }
        default: return 1.f;
    }
}

constexpr int kTile = 16;

template <typename T>
__global__ void __launch_bounds__(kTile* kTile) gemm_kernel(const __grid_constant__ GemmArgs a) {
    __shared__ float sa[kTile][kTile + 1], sb[kTile][kTile + 1];
    const T* A = static_cast<const T*>(a.a);
    const T* B = static_cast<const T*>(a.b);
    const int tx = threadIdx.x % kTile, ty = threadIdx.x / kTile;
    const int64_t m0 = (int64_t)blockIdx.y * kTile, n0 = (int64_t)blockIdx.x * kTile;
    float acc = 0.f;
    for (int64_t k0 = 0; k0 < a.k; k0 += kTile) {
        const int64_t k = k0 + (a.a_kmajor ? tx : ty), m = m0 + (a.a_kmajor ? ty : tx);
        const float va = m < a.m && k < a.k ? to_f32(A[a.a_kmajor ? m * a.a_stride + k : k * a.a_stride + m]) : 0.f;
        sa[a.a_kmajor ? ty : tx][a.a_kmajor ? tx : ty] = va;
        const int64_t kb = k0 + (a.b_kmajor ? tx : ty), n = n0 + (a.b_kmajor ? ty : tx);
        const float vb = n < a.n && kb < a.k ? to_f32(B[a.b_kmajor ? n * a.b_stride + kb : kb * a.b_stride + n]) : 0.f;
        sb[a.b_kmajor ? ty : tx][a.b_kmajor ? tx : ty] = vb;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTile; ++i) acc = fmaf(sa[ty][i], sb[tx][i], acc);
        __syncthreads();
    }
    const int64_t m = m0 + ty, n = n0 + tx;
    if (m >= a.m || n >= a.n) return;
    if (a.bias) acc += to_f32(static_cast<const T*>(a.bias)[n]);
    if (a.z_out) static_cast<T*>(a.z_out)[m * a.z_stride + n] = from_f32<T>(acc);
    float y = activate(acc, a.act);
    if (a.residual) y += to_f32(static_cast<const T*>(a.residual)[m * a.residual_stride + n]);
    static_cast<T*>(a.out)[m * a.out_stride + n] = from_f32<T>(y);
}

constexpr int kBlock = 256;

template <typename T>
__global__ void __launch_bounds__(kBlock) act_bwd_kernel(const __grid_constant__ ActBwdArgs a, int parts) {
    const int c = blockIdx.x * kBlock + threadIdx.x;
    if (c >= a.cols) return;
    float db = 0.f;
    for (int64_t r = blockIdx.y; r < a.rows; r += parts) {
        float g = to_f32(static_cast<const T*>(a.dy)[r * a.dy_stride + c]);
        if (a.act != SOMA_ACT_NONE) g *= act_slope(to_f32(static_cast<const T*>(a.z)[r * a.z_stride + c]), a.act);
        if (a.dz) static_cast<T*>(a.dz)[r * a.dz_stride + c] = from_f32<T>(g);
        db += g;
    }
    if (a.dbias) a.partials[(int64_t)blockIdx.y * a.cols + c] = db;
}

template <typename T>
__global__ void __launch_bounds__(kBlock) bias_grad_kernel(const __grid_constant__ ActBwdArgs a, int parts) {
    const int c = blockIdx.x * kBlock + threadIdx.x;
    if (c >= a.cols) return;
    float db = 0.f;
    for (int p = 0; p < parts; ++p) db += a.partials[(int64_t)p * a.cols + c];
    static_cast<T*>(a.dbias)[c] = from_f32<T>(db);
}

int row_parts(int64_t rows) { return (int)(rows < 64 ? (rows > 0 ? rows : 1) : 64); }

template <typename F>
int with_type16(int dtype, F&& f) {
    return dtype == kBF16 ? f(__nv_bfloat16{}) : f(__half{});
}

}  // namespace

int launch_gemm(const GemmArgs& a, int, void* stream) {
    return with_type16(a.dtype, [&](auto t) {
        const dim3 grid((a.n + kTile - 1) / kTile, (a.m + kTile - 1) / kTile);
        gemm_kernel<decltype(t)><<<grid, kTile * kTile, 0, (cudaStream_t)stream>>>(a);
        return (int)cudaGetLastError();
    });
}

int64_t act_bwd_workspace(int64_t rows, int64_t cols, int) { return (int64_t)row_parts(rows) * cols * 4; }

int launch_act_bwd(const ActBwdArgs& a, int, void* stream) {
    return with_type16(a.dtype, [&](auto t) {
        using T = decltype(t);
        const int cblocks = (a.cols + kBlock - 1) / kBlock, parts = row_parts(a.rows);
        act_bwd_kernel<T><<<dim3(cblocks, parts), kBlock, 0, (cudaStream_t)stream>>>(a, parts);
        if (a.dbias) bias_grad_kernel<T><<<cblocks, kBlock, 0, (cudaStream_t)stream>>>(a, parts);
        return (int)cudaGetLastError();
    });
}

}  // namespace soma
