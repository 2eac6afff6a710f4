// Element types of the training operators' kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <cstdint>

#include "soma_kernels.h"

namespace soma {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// Two fp32 values per instruction (each lane rounded like the scalar form).
__device__ __forceinline__ uint64_t bits2(float2 a) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ float2 float2_of(uint64_t r) {
    float2 a;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
    return a;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return float2_of(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return float2_of(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return float2_of(r);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A 16-byte vector as fp32 values, and back with one rounding.
__device__ __forceinline__ void widen16(const uint4& v, float* x, float) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void widen16(const uint4& v, float* x, __nv_bfloat16) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // bf16 is the upper half of a binary32
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void widen16(const uint4& v, float* x, __half) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __half2 h;
        memcpy(&h, &w[i], 4);
        const float2 f = __half22float2(h);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ uint4 narrow16(const float* x, float) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}
__device__ __forceinline__ uint4 narrow16(const float* x, __nv_bfloat16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        memcpy(&w[i], &h, 4);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 narrow16(const float* x, __half) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        memcpy(&w[i], &h, 4);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The 16 bytes from byte `phase` (< 16, a multiple of the element size) of
// two consecutive words on.  phase is the same for all lanes of a warp.
template <typename T>
__device__ __forceinline__ uint4 shifted(const uint4& u, const uint4& v, int phase) {
    uint32_t x0, x1, x2, x3, x4;
    switch (phase >> 2) {
        case 0: x0 = u.x; x1 = u.y; x2 = u.z; x3 = u.w; x4 = v.x; break;
        case 1: x0 = u.y; x1 = u.z; x2 = u.w; x3 = v.x; x4 = v.y; break;
        case 2: x0 = u.z; x1 = u.w; x2 = v.x; x3 = v.y; x4 = v.z; break;
        default: x0 = u.w; x1 = v.x; x2 = v.y; x3 = v.z; x4 = v.w; break;
    }
    if (sizeof(T) == 4) return make_uint4(x0, x1, x2, x3);
    const int bits = (phase & 3) * 8;
    return make_uint4(__funnelshift_r(x0, x1, bits), __funnelshift_r(x1, x2, bits), __funnelshift_r(x2, x3, bits),
                      __funnelshift_r(x3, x4, bits));
}

// Stores a vector x of elements c .. of `row`.  Not kAligned: the row starts
// `phase` bytes after a 16-byte boundary; each lane joins the end of its
// vector and the start of the next lane's into one aligned word, and the
// elements at a warp's two ends go one by one.  All lanes of a warp call this
// together, with consecutive vectors.
template <typename T, bool kAligned>
__device__ __forceinline__ void store_vector(T* row, int c, int cols, int phase, const float* x) {
    constexpr int kVec = 16 / sizeof(T);
    const uint4 own = narrow16(x, T{});
    if (kAligned || phase == 0) {
        if (c + kVec <= cols) {
            *reinterpret_cast<uint4*>(row + c) = own;
        } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (c + i < cols) row[c + i] = from_f32<T>(x[i]);
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    uint4 next;
    next.x = __shfl_down_sync(0xffffffffu, own.x, 1);
    next.y = __shfl_down_sync(0xffffffffu, own.y, 1);
    next.z = __shfl_down_sync(0xffffffffu, own.z, 1);
    next.w = __shfl_down_sync(0xffffffffu, own.w, 1);
    const int head = (16 - phase) / (int)sizeof(T);  // elements before the first aligned word after the vector's start
    const bool joins = lane < 31 && c + kVec + head <= cols, joined = lane > 0 && c + head <= cols;
    if (joins) *reinterpret_cast<uint4*>(row + c + head) = shifted<T>(own, next, 16 - phase);
    if (!joins || !joined) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (c + i < cols && (i < head ? !joined : !joins)) row[c + i] = from_f32<T>(x[i]);
    }
}

// A row as vectors of kVec elements, vector i from element kVec i
// on, wherever the row starts: where that is inside a 16-byte word, a vector
// is shifted out of two words.
template <typename T, bool kKeep>
struct RowReader {
    static constexpr int kVec = 16 / sizeof(T);
    const T* row;
    const uint4* words;  // the word that holds the row's first element
    int phase, cols;
    // Vectors [inner_begin, inner_end) are whole and lie in words inside the
    // matrix, whose first and last rows may end inside a word.
    int inner_begin, inner_end;

    __device__ __forceinline__ RowReader(const T* base, int64_t stride, int64_t rows, int64_t r, int n)
        : row(base + r * stride), phase((int)((uintptr_t)row & 15)), cols(n) {
        words = reinterpret_cast<const uint4*>((uintptr_t)row & ~(uintptr_t)15);
        inner_begin = (uintptr_t)words < (uintptr_t)base ? 1 : 0;
        const uintptr_t end = (uintptr_t)(base + (rows - 1) * stride + cols) & ~(uintptr_t)15;
        // vector i takes bytes up to 16 (i + 1), or 16 (i + 2) when shifted
        const int64_t fit = ((int64_t)(end - (uintptr_t)words) >> 4) - (phase ? 1 : 0);
        inner_end = (int)min(fit < 0 ? (int64_t)0 : fit, (int64_t)(cols / kVec));
    }
    // One vector anywhere in the row; elements past the row's end are `missing`.
    __device__ __forceinline__ void gather(int i, float (&x)[kVec], float missing = -INFINITY) const {
#pragma unroll
        for (int q = 0; q < kVec; ++q) x[q] = kVec * i + q < cols ? to_f32(row[kVec * i + q]) : missing;
    }
    // Vectors [i, i + n step) of whole words, step apart.
    template <bool kShift, int kN>
    __device__ __forceinline__ void load(int i, int step, uint4 (&u)[kN], uint4 (&v)[kShift ? kN : 1]) const {
#pragma unroll
        for (int q = 0; q < kN; ++q) {
            const uint4* w = words + i + q * step;
            if (kShift) {  // the neighbouring vector's word comes out of L1
                u[q] = w[0];
                v[kShift ? q : 0] = w[1];
            } else if (kKeep) {  // read again, from L2
                asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(u[q].x), "=r"(u[q].y), "=r"(u[q].z), "=r"(u[q].w)
                             : "l"(w)
                             : "memory");
            } else {
                u[q] = __ldcs(w);
            }
        }
    }
    template <bool kShift>
    __device__ __forceinline__ void widen(const uint4& u, const uint4& v, float (&x)[kVec]) const {
        widen16(kShift ? shifted<T>(u, v, phase) : u, x, T{});
    }
};

// Calls f with a value of the C++ type that a dtype code stands for.
template <typename F>
inline int with_type(int dtype, F&& f) {
    if (dtype == kF32) return f(float{});
    if (dtype == kBF16) return f(__nv_bfloat16{});
    return f(__half{});
}

}  // namespace soma
