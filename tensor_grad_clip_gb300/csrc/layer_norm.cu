// Layer norm, forward and backward (formulas in soma_ops.h).
//
// Both passes stream rows from HBM (forward: read x, write y; backward: read
// dy and x, write dx) at 8 to 14 flops per element, so the bound is HBM
// bandwidth.  The CTAs are persistent.  A ring of row slots in shared memory
// keeps the next rows' bulk copies in flight while a row is reduced, and a
// thread keeps its columns for all rows, so that weight, bias and the
// backward pass's sums over rows stay in registers.
//
//   rows of               a row belongs to
//   up to 512 elements    a warp (8 or 16 elements per thread, no barriers)
//   up to 1024            two warps (16 elements per thread)
//   up to 16384           a CTA (16 or 32 elements per thread)
//   more                  a CTA of 256 threads that re-reads it through L2
//
// Measured (GB300, 6682 GB/s copy): 16384 x 4096 bf16 forward 49.2 us, 5460
// GB/s; backward 82.1 us, 4905 GB/s.  fp32: 8192 x 4096 forward 50.6 us, 5305
// GB/s; 16384 x 4096 backward 126 us, 6402 GB/s.  16381 x 4099 fp16 (padded
// rows) backward 125 us, 3226 GB/s.  2000 x 40000 bf16, which takes the last
// path, 206 us forward and 436 us backward (1553 and 1102 GB/s).  The 16-bit
// passes are bound by the latency of a row's chain (copy, statistics over the
// CTA, output) at the two or three rows an SM's registers hold, not by DRAM:
// ncu has DRAM at 57 to 60 % and the issue slots at 48 to 65 %.  Tried and
// slower: more rows per SM with the parameters read again for every row from
// L1 (74 us forward), a warp of its own to fill the ring (57 us; warps are
// allocated in fours), 24 or 32 elements per thread for rows of 4099 (206 us
// backward).
//
// A row may start at any element: its slot holds the whole 16-byte words that
// cover it, and threads shift their vectors into place.  Which thread sums
// which columns does not depend on the alignment, so neither do the results.
#include <algorithm>
#include <type_traits>

#include "mbarrier.cuh"
#include "ops_device.cuh"
#include "ops_kernels.h"

namespace soma {
namespace {

__device__ unsigned g_gave_up;  // threads that saw a bounded wait run out, on this device

// Rows first, first + step, ... of a group of threads, counted by an int.
struct Walk {
    int64_t first, step;
    int count;
    __device__ __forceinline__ Walk(int64_t f, int64_t s, int64_t rows)
        : first(f), step(s), count(f < rows ? (int)((rows - 1 - f) / s) + 1 : 0) {}
    __device__ __forceinline__ int64_t row(int i) const { return first + i * step; }
    // How many of its rows are below `row`.
    __device__ __forceinline__ int below(int64_t row) const {
        return row <= first ? 0 : (int)min((int64_t)count, (row - 1 - first) / step + 1);
    }
};

constexpr int kCtaWarps = 4;    // warps of a CTA whose rows take one or two of them
constexpr int kMaxDepth = 8;    // rows in flight per warp or CTA

// A matrix operand as the kernels see it.  Row r's window is the run of whole
// 16-byte words that covers it; slots hold windows, so a row's first element
// sits `phase` bytes into its slot.
template <typename T>
struct Rows {
    const T* base;
    int64_t stride, rows;
    int cols;

    __device__ __forceinline__ int phase(int64_t r) const { return (int)((uintptr_t)(base + r * stride) & 15); }
    // The window of the row at address s, clipped to the matrix's own span
    // where it may stick out of it; patch() fills in those few elements.
    template <bool kAligned>
    __device__ __forceinline__ void window(uintptr_t s, bool edge, uintptr_t& lo, uint32_t& skip, uint32_t& bytes) const {
        const uintptr_t e = s + (uint32_t)cols * (uint32_t)sizeof(T);
        lo = kAligned ? s : s & ~(uintptr_t)15;
        uintptr_t hi = (e + 15) & ~(uintptr_t)15;
        skip = 0;
        if (edge) {
            if (lo < (uintptr_t)base) {
                lo += 16;
                skip = 16;
            }
            if (hi > (uintptr_t)(base + (rows - 1) * stride + cols)) hi -= 16;
        }
        bytes = hi > lo ? (uint32_t)(hi - lo) : 0;
    }
    // Rows outside [inner_begin, inner_end) may have a window that sticks out.
    __device__ __forceinline__ int64_t edge_rows() const {
        return rows <= 1 ? rows : min(rows, 1 + 16 / (stride * (int64_t)sizeof(T)));
    }
    __device__ __forceinline__ int64_t inner_begin() const { return (uintptr_t)base % 16 ? edge_rows() : 0; }
    __device__ __forceinline__ int64_t inner_end() const {
        return (uintptr_t)(base + (rows - 1) * stride + cols) % 16 ? rows - edge_rows() : rows;
    }
    // The elements of row r in its first and last word, copied one by one.
    __device__ __forceinline__ void patch(int64_t r, char* slot, int t) const {
        constexpr int kVec = 16 / sizeof(T);
        const T* row = base + r * stride;
        T* to = reinterpret_cast<T*>(slot + phase(r));
        if (t >= 2 * kVec) return;
        const int c = t < kVec ? t : cols - 1 - (t - kVec);
        if (c >= 0 && c < cols) to[c] = row[c];
        fence_to_async();  // (before a later copy into the slot)
    }
};

// Elements c .. c + 16 / sizeof(T) - 1 of a row in a slot, c a multiple of
// their number.  kAligned: phase is 0.
template <typename T, bool kAligned>
__device__ __forceinline__ uint4 slot_vector(const char* slot, int c, int phase) {
    const uint4 u = *reinterpret_cast<const uint4*>(slot + c * sizeof(T));
    if (kAligned) return u;
    return shifted<T>(u, *reinterpret_cast<const uint4*>(slot + c * sizeof(T) + 16), phase);
}

// kN elements of a parameter vector from c on, `missing` where there is none.
template <typename T, int kN>
__device__ __forceinline__ void parameter(const void* v, bool f32, int c, int cols, float missing, float* w) {
    if (v && ((uintptr_t)v & 15) == 0 && c + kN <= cols) {  // (c is a multiple of kN)
        if (f32) {
#pragma unroll
            for (int i = 0; i < kN; i += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(v) + c + i));
                w[i] = f.x; w[i + 1] = f.y; w[i + 2] = f.z; w[i + 3] = f.w;
            }
        } else {
            widen16(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(v) + c)), w, T{});
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        w[i] = missing;
        if (v && c + i < cols) w[i] = f32 ? static_cast<const float*>(v)[c + i] : to_f32(static_cast<const T*>(v)[c + i]);
    }
}

__device__ __forceinline__ float warp_total(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <int kWarps>
__device__ __forceinline__ void group_sync(int group, int warps);

// Totals of x and y over the threads of a row, in every thread.  Within a
// warp the lower half sums x and the upper half y; across warps every thread
// adds the warps' sums in a fixed order.  Consecutive calls alternate between
// two scratch rows, so that one barrier per call is enough.
template <int kWarps>
__device__ __forceinline__ float2 row_totals(float x, float y, float2 (*scratch)[16], int group, int warps, int& turn) {
    const unsigned all = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    float v = lane < 16 ? x : y;
    v += __shfl_xor_sync(all, lane < 16 ? y : x, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(all, v, o);
    if (kWarps == 1) return make_float2(__shfl_sync(all, v, 0), __shfl_sync(all, v, 16));
    float* mine = reinterpret_cast<float*>(&scratch[turn][threadIdx.x >> 5]);
    if ((lane & 15) == 0) mine[lane >> 4] = v;
    group_sync<kWarps>(group, warps);
    const float4* from = reinterpret_cast<const float4*>(scratch[turn] + (kWarps == 2 ? 2 * group : 0));
    turn ^= 1;
    const float4 v0 = from[0];
    float2 s = make_float2(v0.x, v0.y), u = make_float2(v0.z, v0.w);
    if (kWarps == 0) {
        auto more = [&](int w) {  // (entries past the last warp are 0)
            const float4 v4 = from[w];
            s = add2(s, make_float2(v4.x, v4.y));
            u = add2(u, make_float2(v4.z, v4.w));
        };
        more(1);
        if (warps > 4) {
            more(2);
            more(3);
        }
        if (warps > 8) {
#pragma unroll
            for (int w = 4; w < 8; ++w) more(w);
        }
    }
    return add2(s, u);
}

// The ring of row slots of one group of threads: slots of kOperands windows,
// an mbarrier each that counts the slot's copies.
template <int kOperands>
struct Ring {
    char* slots;
    uint32_t full;
    int depth, slot_bytes;  // bytes of one window's room
    __device__ __forceinline__ char* window(int slot, int operand) const {
        return slots + (slot * kOperands + operand) * slot_bytes;
    }
};

// Starts the copies of one row.  Every instruction here delays a row's
// threads at their next barrier.
template <bool kAligned, int kOperands, typename T>
__device__ __forceinline__ void fill_row(const Ring<kOperands>& ring, const Rows<T> (&m)[kOperands], int64_t row,
                                         bool edge, int slot) {
    const uint32_t bar = ring.full + 8 * slot, to = smem_addr(ring.slots) + slot * kOperands * ring.slot_bytes;
    uintptr_t lo[kOperands];
    uint32_t skip[kOperands], bytes[kOperands], total = 0;
#pragma unroll
    for (int o = 0; o < kOperands; ++o) {
        m[o].template window<kAligned>((uintptr_t)(m[o].base + row * m[o].stride), edge, lo[o], skip[o], bytes[o]);
        total += bytes[o];
    }
    mbar_expect(bar, total);
#pragma unroll
    for (int o = 0; o < kOperands; ++o)
        if (bytes[o]) bulk_load(to + o * ring.slot_bytes + skip[o], reinterpret_cast<const void*>(lo[o]), bytes[o], bar);
}

// Threads of one row: kWarps warps where that is 1 or 2 (the CTA then has
// kCtaWarps / kWarps rows at a time), else all warps of the CTA (kWarps = 0).
template <int kWarps>
__device__ __forceinline__ void group_sync(int group, int warps) {
    if (kWarps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(warps * 32) : "memory");
}

// kPer elements per thread; a row belongs to a warp, to two (kWarps) or to all
// warps of the CTA (kWarps = 0).
//
// The statistics take one pass over the thread's elements and one reduction:
// mean = sum x / n and var = sum x^2 / n - mean^2.  That loses up to two bits
// of the variance while mean^2 <= 4 var; beyond, the thread's elements, which
// it holds, become x - k with k the mean just found, and both sums are taken
// again of those (16384 x 4096 bf16: 49.2 us, and 62.6 us where every row's
// mean is that far from 0).  A shift by some element of the row instead would
// round all others at that one's size, and the mean with them.
template <typename T, int kPer, bool kAligned, int kWarps>
__global__ void __maxnreg__(kPer == 32 ? 128 : kWarps ? 96 : 80)
    norm_fwd_kernel(const __grid_constant__ NormFwdArgs a, int depth, int slot_bytes) {
    constexpr int kVec = 16 / sizeof(T), kPieces = kPer / kVec;
    extern __shared__ __align__(16) char dynamic[];
    __shared__ __align__(8) uint64_t bars[kWarps ? kCtaWarps / kWarps : 1][kMaxDepth];
    __shared__ __align__(16) float2 scratch[2][16];
    __shared__ int gave_up;
    constexpr int kGroups = kWarps ? kCtaWarps / kWarps : 1;
    const int warps = kWarps ? kWarps : blockDim.x / 32, threads = warps * 32;
    const int group = kWarps ? threadIdx.x / (32 * kWarps) : 0, t = threadIdx.x - group * threads;
    const Ring<1> ring{dynamic + group * depth * slot_bytes, smem_addr(bars[group]), depth, slot_bytes};
    const Rows<T> x[1] = {{static_cast<const T*>(a.x), a.x_stride, a.rows, a.cols}};
    const Walk walk((int64_t)blockIdx.x * kGroups + group, (int64_t)gridDim.x * kGroups, a.rows);
    const int inner_begin = walk.below(x[0].inner_begin()), inner_end = walk.below(x[0].inner_end());
    if (threadIdx.x == 0) gave_up = 0;
    if (threadIdx.x < 32) scratch[threadIdx.x >> 4][threadIdx.x & 15] = both(0.f);
    if (t == 0) {
        for (int i = 0; i < depth; ++i) mbar_init(ring.full + 8 * i, 1);
        mbar_init_fence();
        for (int i = 0; i < min(depth, walk.count); ++i) fill_row<kAligned>(ring, x, walk.row(i), i < inner_begin || i >= inner_end, i);
    }
    __syncthreads();
    const bool f32 = a.param_dtype == kF32;
    float w[kPer], b[kPer];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        parameter<T, kVec>(a.weight, f32, (p * threads + t) * kVec, a.cols, 1.f, w + p * kVec);
        parameter<T, kVec>(a.bias, f32, (p * threads + t) * kVec, a.cols, 0.f, b + p * kVec);
    }
    const float inv = 1.f / (float)a.cols;
    T* y = static_cast<T*>(a.y) + walk.first * a.y_stride;
    int turn = 0, slot = 0;
    uint32_t parity = 0;
    for (int it = 0; it < walk.count; ++it, y += walk.step * a.y_stride) {
        mbar_wait(ring.full + 8 * slot, parity, &gave_up);  // (after giving up, garbage follows)
        char* window = ring.window(slot, 0);
        if (it < inner_begin || it >= inner_end) {
            x[0].patch(walk.row(it), window, t);
            group_sync<kWarps>(group, warps);
        }
        const int phase = kAligned ? 0 : x[0].phase(walk.row(it));
        float2 e[kPer / 2], sum = both(0.f), square = both(0.f);  // x, 0 past the row's end
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int c = (p * threads + t) * kVec;
            float v[kVec];
            if (c < a.cols) widen16(slot_vector<T, kAligned>(window, c, phase), v, T{});
#pragma unroll
            for (int i = 0; i < kVec / 2; ++i) e[p * kVec / 2 + i] = make_float2(v[2 * i], v[2 * i + 1]);
            if (c + kVec > a.cols) {
#pragma unroll
                for (int i = 0; i < kVec / 2; ++i) {
                    if (c + 2 * i >= a.cols) e[p * kVec / 2 + i].x = 0.f;
                    if (c + 2 * i + 1 >= a.cols) e[p * kVec / 2 + i].y = 0.f;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kPer / 2; ++i) {
            sum = add2(sum, e[i]);
            square = fma2(e[i], e[i], square);
        }
        float2 s = row_totals<kWarps>(sum.x + sum.y, square.x + square.y, scratch, group, warps, turn);
        // (every thread has its part of the row in registers now)
        if (t == 0 && it + depth < walk.count) fill_row<kAligned>(ring, x, walk.row(it + depth), it + depth >= inner_end || it + depth < inner_begin, slot);
        float k = 0.f, shift = s.x * inv, var = fmaf(-shift, shift, s.y * inv);
        if (shift * shift > 4.f * var) {  // the same for all threads of the row
            k = shift;
            sum = square = both(0.f);
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                const int c = (p * threads + t) * kVec;
#pragma unroll
                for (int i = 0; i < kVec / 2; ++i) e[p * kVec / 2 + i] = add2(e[p * kVec / 2 + i], both(-k));
                if (c + kVec > a.cols) {
#pragma unroll
                    for (int i = 0; i < kVec / 2; ++i) {
                        if (c + 2 * i >= a.cols) e[p * kVec / 2 + i].x = 0.f;
                        if (c + 2 * i + 1 >= a.cols) e[p * kVec / 2 + i].y = 0.f;
                    }
                }
#pragma unroll
                for (int i = 0; i < kVec / 2; ++i) {
                    sum = add2(sum, e[p * kVec / 2 + i]);
                    square = fma2(e[p * kVec / 2 + i], e[p * kVec / 2 + i], square);
                }
            }
            s = row_totals<kWarps>(sum.x + sum.y, square.x + square.y, scratch, group, warps, turn);
            shift = s.x * inv;
            var = fmaf(-shift, shift, s.y * inv);
            if (var < 0.f) var = 0.f;  // (the rounding of a constant row)
        }
        const float rstd = rsqrtf(var + a.eps);
        const int out_phase = kAligned ? 0 : (int)((uintptr_t)y & 15);
        const float2 scale = both(rstd), offset = both(-shift * rstd);
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            float out[kVec];
#pragma unroll
            for (int i = 0; i < kVec / 2; ++i) {
                const int j = p * kVec + 2 * i;
                const float2 xh = fma2(e[p * kVec / 2 + i], scale, offset);
                const float2 v = fma2(xh, make_float2(w[j], w[j + 1]), make_float2(b[j], b[j + 1]));
                out[2 * i] = v.x;
                out[2 * i + 1] = v.y;
            }
            store_vector<T, kAligned>(y, (p * threads + t) * kVec, a.cols, out_phase, out);
        }
        if (t == 0) {
            if (a.mean) a.mean[walk.row(it)] = k + shift;
            if (a.rstd) a.rstd[walk.row(it)] = rstd;
        }
        if (++slot == depth) {
            slot = 0;
            parity ^= 1;
        }
    }
    if (gave_up) {
        atomicAdd(&g_gave_up, 1u);
        outlast_copies();
    }
}

// dx of every row, and this CTA's sums of dy * xh and dy over its rows into
// partials[blockIdx.x][0 / 1][cols] (when wanted).
template <typename T, int kPer, bool kAligned, int kWarps>
__global__ void __maxnreg__(128)
    norm_bwd_kernel(const __grid_constant__ NormBwdArgs a, int depth, int slot_bytes) {
    constexpr int kVec = 16 / sizeof(T), kPieces = kPer / kVec;
    // weight, xh and g stay in registers; else they are formed again from the slot for dx
    constexpr bool kHold = kPer <= 16;
    extern __shared__ __align__(16) char dynamic[];
    __shared__ __align__(8) uint64_t bars[kWarps ? kCtaWarps / kWarps : 1][kMaxDepth];
    __shared__ __align__(16) float2 scratch[2][16];
    __shared__ int gave_up;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kGroups = kWarps ? kCtaWarps / kWarps : 1;
    const int warps = kWarps ? kWarps : blockDim.x / 32, threads = warps * 32;
    const int group = kWarps ? threadIdx.x / (32 * kWarps) : 0, t = threadIdx.x - group * threads;
    const Ring<2> ring{dynamic + group * depth * 2 * slot_bytes, smem_addr(bars[group]), depth, slot_bytes};
    const Rows<T> m[2] = {{static_cast<const T*>(a.x), a.x_stride, a.rows, a.cols},
                          {static_cast<const T*>(a.dy), a.dy_stride, a.rows, a.cols}};
    const Walk walk((int64_t)blockIdx.x * kGroups + group, (int64_t)gridDim.x * kGroups, a.rows);
    const int inner_begin = walk.below(max(m[0].inner_begin(), m[1].inner_begin()));
    const int inner_end = walk.below(min(m[0].inner_end(), m[1].inner_end()));
    if (threadIdx.x == 0) gave_up = 0;
    if (threadIdx.x < 32) scratch[threadIdx.x >> 4][threadIdx.x & 15] = both(0.f);
    if (t == 0) {
        for (int i = 0; i < depth; ++i) mbar_init(ring.full + 8 * i, 1);
        mbar_init_fence();
        for (int i = 0; i < min(depth, walk.count); ++i) fill_row<kAligned>(ring, m, walk.row(i), i < inner_begin || i >= inner_end, i);
    }
    __syncthreads();
    float next_mean = 0.f, next_rstd = 0.f;
    if (walk.count > 0) {
        next_mean = a.mean[walk.first];
        next_rstd = a.rstd[walk.first];
    }
    const bool f32 = a.param_dtype == kF32;
    float w[kHold ? kPer : kVec];
    float2 dw[kPer / 2], db[kPer / 2];
#pragma unroll
    for (int p = 0; p < kPieces; ++p)
        if (kHold) parameter<T, kVec>(a.weight, f32, (p * threads + t) * kVec, a.cols, 1.f, w + (kHold ? p * kVec : 0));
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) dw[i] = db[i] = both(0.f);
    const float inv = 1.f / (float)a.cols;
    T* dx = static_cast<T*>(a.dx) + walk.first * a.dx_stride;
    int turn = 0, slot = 0, last_slot = 0;
    uint32_t parity = 0;
    for (int it = 0; it < walk.count; ++it, dx += walk.step * a.dx_stride) {
        const float rstd = next_rstd, mean = next_mean;
        if (it + 1 < walk.count) {
            next_mean = a.mean[walk.row(it + 1)];
            next_rstd = a.rstd[walk.row(it + 1)];
        }
        mbar_wait(ring.full + 8 * slot, parity, &gave_up);  // (after giving up, garbage follows)
        char *window_x = ring.window(slot, 0), *window_dy = ring.window(slot, 1);
        if (it < inner_begin || it >= inner_end) {
            m[0].patch(walk.row(it), window_x, t);
            m[1].patch(walk.row(it), window_dy, t);
            group_sync<kWarps>(group, warps);
        }
        const int phase_x = kAligned ? 0 : m[0].phase(walk.row(it)), phase_dy = kAligned ? 0 : m[1].phase(walk.row(it));
        float2 xh[kHold ? kPer / 2 : kVec / 2], g[kHold ? kPer / 2 : kVec / 2];
        // xh and dy of piece p (0 past the row's end), and its weights.  x - mean
        // before the product: x rstd - mean rstd would cancel where the mean is
        // many standard deviations from 0.
        auto take = [&](int p, float2* to_xh, float2* to_dy) {
            const int c = (p * threads + t) * kVec;
            float ex[kVec], ed[kVec];
            if (c < a.cols) {
                widen16(slot_vector<T, kAligned>(window_x, c, phase_x), ex, T{});
                widen16(slot_vector<T, kAligned>(window_dy, c, phase_dy), ed, T{});
            }
#pragma unroll
            for (int i = 0; i < kVec / 2; ++i) {
                to_xh[i] = mul2(add2(make_float2(ex[2 * i], ex[2 * i + 1]), both(-mean)), both(rstd));
                to_dy[i] = make_float2(ed[2 * i], ed[2 * i + 1]);
            }
            if (c + kVec > a.cols) {
#pragma unroll
                for (int i = 0; i < kVec / 2; ++i) {
                    if (c + 2 * i >= a.cols) to_xh[i].x = to_dy[i].x = 0.f;
                    if (c + 2 * i + 1 >= a.cols) to_xh[i].y = to_dy[i].y = 0.f;
                }
            }
            if (!kHold) parameter<T, kVec>(a.weight, f32, c, a.cols, 1.f, w);
        };
        float2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int j0 = kHold ? p * kVec / 2 : 0;
            take(p, xh + j0, g + j0);
#pragma unroll
            for (int i = 0; i < kVec / 2; ++i) {
                const int j = j0 + i, q = p * kVec / 2 + i;
                dw[q] = fma2(g[j], xh[j], dw[q]);
                db[q] = add2(db[q], g[j]);
                g[j] = mul2(g[j], make_float2(w[2 * j], w[2 * j + 1]));
                s0 = add2(s0, g[j]);
                s1 = fma2(g[j], xh[j], s1);
            }
        }
        const float2 s = row_totals<kWarps>(s0.x + s0.y, s1.x + s1.y, scratch, group, warps, turn);
        if (t == 0) {
            // every warp is done with this row's slot (kHold), or with that of the row before it
            const int next = it + depth - (kHold ? 0 : 1);
            if (next < walk.count && (kHold || (depth > 1 && it > 0)))
                fill_row<kAligned>(ring, m, walk.row(next), next < inner_begin || next >= inner_end, kHold ? slot : last_slot);
        }
        last_slot = slot;
        if (a.dx) {
            // dx = rstd g - rstd mean(g) - xh rstd mean(g xh)
            const float2 scale = both(rstd), m0 = both(-s.x * inv * rstd), m1 = both(-s.y * inv * rstd);
            const int out_phase = kAligned ? 0 : (int)((uintptr_t)dx & 15);
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                const int j0 = kHold ? p * kVec / 2 : 0;
                if (!kHold) take(p, xh, g);
                float e[kVec];
#pragma unroll
                for (int i = 0; i < kVec / 2; ++i) {
                    const int j = j0 + i;
                    if (!kHold) g[j] = mul2(g[j], make_float2(w[2 * j], w[2 * j + 1]));
                    const float2 v = fma2(xh[j], m1, fma2(g[j], scale, m0));
                    e[2 * i] = v.x;
                    e[2 * i + 1] = v.y;
                }
                store_vector<T, kAligned>(dx, (p * threads + t) * kVec, a.cols, out_phase, e);
            }
        }
        if (!kHold && depth == 1) {  // the only slot: its next row can start now
            __syncthreads();
            if (t == 0 && it + 1 < walk.count) fill_row<kAligned>(ring, m, walk.row(it + 1), it + 1 < inner_begin || it + 1 >= inner_end, 0);
        }
        if (++slot == depth) {
            slot = 0;
            parity ^= 1;
        }
    }
    if (gave_up) {
        atomicAdd(&g_gave_up, 1u);
        outlast_copies();
    }
    if (!a.dweight && !a.dbias) return;
    float* out = a.partials + 2 * (int64_t)blockIdx.x * a.cols;
    auto sums_of = [&](auto&& f) {  // f(column, dw, db) for the thread's columns
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = (i / kVec * threads + t) * kVec + i % kVec;
            if (c < a.cols) f(c, i % 2 ? dw[i / 2].y : dw[i / 2].x, i % 2 ? db[i / 2].y : db[i / 2].x);
        }
    };
    if (kWarps == 0) {
        sums_of([&](int c, float u, float v) {
            out[c] = u;
            out[a.cols + c] = v;
        });
        return;
    }
    // the CTA's groups join their sums, in order, in the first slots' place
    float* sums = reinterpret_cast<float*>(dynamic);
    __syncthreads();
    for (int q = 0; q < kGroups; ++q) {
        if (group == q)
            sums_of([&](int c, float u, float v) {
                float* to = q == kGroups - 1 ? out : sums;
                to[c] = q ? sums[c] + u : u;
                to[a.cols + c] = q ? sums[a.cols + c] + v : v;
            });
        __syncthreads();
    }
}

// dweight and dbias: the partial sums added in a fixed order.  A CTA takes 32
// columns; its 32 warps take the parts in turn.
constexpr int kJoinWarps = 32;
template <typename W>
__global__ void __launch_bounds__(32 * kJoinWarps) norm_join_kernel(const __grid_constant__ NormBwdArgs a, int parts) {
    __shared__ float scratch[2][kJoinWarps][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float dw = 0.f, db = 0.f;
    if (c < a.cols) {
#pragma unroll 4
        for (int p = warp; p < parts; p += kJoinWarps) {
            dw += a.partials[2 * (int64_t)p * a.cols + c];
            db += a.partials[(2 * (int64_t)p + 1) * a.cols + c];
        }
    }
    scratch[0][warp][lane] = dw;
    scratch[1][warp][lane] = db;
    __syncthreads();
    if (warp >= 2 || c >= a.cols) return;
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < kJoinWarps; ++q) s += scratch[warp][q][lane];
    W* out = static_cast<W*>(warp == 0 ? a.dweight : a.dbias);
    if (out) out[c] = from_f32<W>(s);
}

// ---- rows too long for the registers of a CTA ------------------------------------

constexpr int kLoopBlock = 256;

__device__ __forceinline__ float block_total(float x, float* scratch) {
    x = warp_total(x);
    __syncthreads();  // the previous total has been read
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
    __syncthreads();
    float r = 0.f;
#pragma unroll
    for (int w = 0; w < kLoopBlock / 32; ++w) r += scratch[w];
    return r;
}

template <typename T, typename W>
__global__ void __launch_bounds__(kLoopBlock) norm_fwd_loop_kernel(const __grid_constant__ NormFwdArgs a) {
    __shared__ float scratch[kLoopBlock / 32];
    const W* w = static_cast<const W*>(a.weight);
    const W* b = static_cast<const W*>(a.bias);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
        T* y = static_cast<T*>(a.y) + r * a.y_stride;
        float s = 0.f;
        for (int64_t c = threadIdx.x; c < a.cols; c += kLoopBlock) s += to_f32(x[c]);
        const float mean = block_total(s, scratch) / (float)a.cols;
        s = 0.f;
        for (int64_t c = threadIdx.x; c < a.cols; c += kLoopBlock) {
            const float d = to_f32(x[c]) - mean;
            s = fmaf(d, d, s);
        }
        const float rstd = 1.f / sqrtf(block_total(s, scratch) / (float)a.cols + a.eps);
        for (int64_t c = threadIdx.x; c < a.cols; c += kLoopBlock) {
            const float v = (to_f32(x[c]) - mean) * rstd;
            y[c] = from_f32<T>(fmaf(v, w ? to_f32(w[c]) : 1.f, b ? to_f32(b[c]) : 0.f));
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

template <typename T, typename W>
__global__ void __launch_bounds__(kLoopBlock) norm_dx_loop_kernel(const __grid_constant__ NormBwdArgs a) {
    __shared__ float scratch[kLoopBlock / 32];
    const W* w = static_cast<const W*>(a.weight);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
        const T* dy = static_cast<const T*>(a.dy) + r * a.dy_stride;
        T* dx = static_cast<T*>(a.dx) + r * a.dx_stride;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s0 = 0.f, s1 = 0.f;
        for (int64_t c = threadIdx.x; c < a.cols; c += kLoopBlock) {
            const float g = to_f32(dy[c]) * (w ? to_f32(w[c]) : 1.f);
            s0 += g;
            s1 = fmaf(g, (to_f32(x[c]) - mean) * rstd, s1);
        }
        s0 = block_total(s0, scratch) / (float)a.cols;
        s1 = block_total(s1, scratch) / (float)a.cols;
        for (int64_t c = threadIdx.x; c < a.cols; c += kLoopBlock) {
            const float g = to_f32(dy[c]) * (w ? to_f32(w[c]) : 1.f);
            const float xh = (to_f32(x[c]) - mean) * rstd;
            dx[c] = from_f32<T>(rstd * (g - fmaf(xh, s1, s0)));
        }
    }
}

// Sums over the rows of one part, a thread per column.
template <typename T>
__global__ void __launch_bounds__(kLoopBlock) norm_dw_loop_kernel(const __grid_constant__ NormBwdArgs a, int parts) {
    const int64_t c = (int64_t)blockIdx.x * kLoopBlock + threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (c >= a.cols) return;
    float dw = 0.f, db = 0.f;
    for (int64_t r = blockIdx.y; r < a.rows; r += parts) {
        const float g = to_f32(static_cast<const T*>(a.dy)[r * a.dy_stride + c]);
        const float xh = (to_f32(static_cast<const T*>(a.x)[r * a.x_stride + c]) - a.mean[r]) * a.rstd[r];
        dw = fmaf(g, xh, dw);
        db += g;
    }
    a.partials[2 * (int64_t)blockIdx.y * a.cols + c] = dw;
    a.partials[(2 * (int64_t)blockIdx.y + 1) * a.cols + c] = db;
}

// ---- launch shapes ------------------------------------------------------------

constexpr int kCtasMost = 8;   // persistent CTAs per SM; bounds the partial sums
constexpr int kLoopParts = 64;
constexpr int kLongest = 512 * 32;  // elements of a row that a CTA takes
constexpr int kRingBytes = 200 * 1024;  // of an SM's shared memory, for all its CTAs
// The forward pass is faster with fewer rows in flight, two at least: 100 KB
// instead of 200 take 16384 x 4096 bf16 from 52.3 to 49.2 us and 8192 x 5000
// fp32 from 61.3 to 56.7.
constexpr int kForwardRing = 100 * 1024;

template <typename F>
int with_types(int dtype, int param_dtype, F&& f) {
    return with_type(dtype, [&](auto t) {
        using T = decltype(t);
        return param_dtype == kF32 ? f(t, float{}) : f(t, T{});
    });
}

bool vector_rows(const void* p, int64_t stride, int64_t rows, int esize) {
    return !p || ((uintptr_t)p % 16 == 0 && (rows <= 1 || stride * esize % 16 == 0));
}

// Calls f(elements per thread, warps per row or 0, warps of a CTA).
template <typename F>
int with_shape(int cols, F&& f) {
    using std::integral_constant;
    using OneWarp = integral_constant<int, 1>;
    using TwoWarps = integral_constant<int, 2>;
    using AllWarps = integral_constant<int, 0>;
    using Eight = integral_constant<int, 8>;
    using Sixteen = integral_constant<int, 16>;
    using ThirtyTwo = integral_constant<int, 32>;
    if (cols <= 32 * 8) return f(Eight{}, OneWarp{}, kCtaWarps);
    if (cols <= 32 * 16) return f(Sixteen{}, OneWarp{}, kCtaWarps);
    if (cols <= 64 * 16) return f(Sixteen{}, TwoWarps{}, kCtaWarps);
    if (cols <= 512 * 16) return f(Sixteen{}, AllWarps{}, (cols + 511) / 512);
    return f(ThirtyTwo{}, AllWarps{}, (cols + 1023) / 1024);
}

// Enqueues a persistent kernel on as many CTAs as the device holds, at most
// one per row (or group of rows), and says how many.
template <typename Args>
int launch_rows(void (*kernel)(Args, int, int), const Args& a, int operands, int esize, int row_warps, int warps,
                int sm_count, cudaStream_t st, int* ctas) {
    const int groups = row_warps ? kCtaWarps / row_warps : 1, block = 32 * warps;
    // a window is up to 15 bytes longer than its row at either end; a vector read may run 16 bytes past it
    const int slot = (a.cols * esize + 15) / 16 * 16 + 32, bytes = groups * operands * slot;
    int per_sm = 0;
    int e = resident_ctas((const void*)kernel, block, 0, &per_sm);
    if (e != cudaSuccess) return e;
    per_sm = std::min(kCtasMost, std::max(1, per_sm));
    while (per_sm > 1 && kRingBytes / per_sm / bytes < 2) --per_sm;
    const int ring = operands == 1 ? kForwardRing : kRingBytes;
    const int depth = std::max(operands == 1 ? 2 : 1, std::min(kMaxDepth, ring / per_sm / bytes));
    const size_t smem = (size_t)bytes * depth;
    if (smem > 40 * 1024) e = allow_smem((const void*)kernel, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t work = (a.rows + groups - 1) / groups;
    *ctas = (int)std::max<int64_t>(1, std::min<int64_t>(work, (int64_t)sm_count * per_sm));
    kernel<<<*ctas, block, smem, st>>>(a, depth, slot);
    return (int)cudaGetLastError();
}

// Enqueues norm_join_kernel so that it may be set up while the kernel before
// it runs.
template <typename W>
int launch_join(NormBwdArgs a, int parts, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(((int64_t)a.cols + 31) / 32));
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, norm_join_kernel<W>, a, parts);
}

}  // namespace

int launch_norm_fwd(const NormFwdArgs& a, int sm_count, void* stream) {
    cudaStream_t st = (cudaStream_t)stream;
    if (a.cols > kLongest)
        return with_types(a.dtype, a.param_dtype, [&](auto t, auto w) {
            const int grid = (int)std::min<int64_t>(a.rows, kCtasMost * sm_count);
            norm_fwd_loop_kernel<decltype(t), decltype(w)><<<grid, kLoopBlock, 0, st>>>(a);
            return (int)cudaGetLastError();
        });
    return with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        const bool vec = vector_rows(a.x, a.x_stride, a.rows, sizeof(T)) && vector_rows(a.y, a.y_stride, a.rows, sizeof(T));
        return with_shape(a.cols, [&](auto per, auto row_warps, int warps) {
            constexpr int kPer = decltype(per)::value;
            constexpr int kWarps = decltype(row_warps)::value;
            int ctas;
            return launch_rows(vec ? norm_fwd_kernel<T, kPer, true, kWarps> : norm_fwd_kernel<T, kPer, false, kWarps>, a,
                               1, sizeof(T), kWarps, warps, sm_count, st, &ctas);
        });
    });
}

int64_t norm_bwd_workspace(int64_t rows, int64_t cols, int sm_count) {
    const int64_t parts = cols > kLongest ? kLoopParts : (int64_t)kCtasMost * sm_count;
    return 2 * std::max<int64_t>(1, std::min(rows, parts)) * cols * 4;
}

int launch_norm_bwd(const NormBwdArgs& a, int sm_count, void* stream) {
    cudaStream_t st = (cudaStream_t)stream;
    const bool params = a.dweight || a.dbias;
    int parts = 1, e = cudaSuccess;
    if (a.cols > kLongest) {
        e = with_type(a.dtype, [&](auto t) {
            using T = decltype(t);
            if (params) {
                parts = (int)std::max<int64_t>(1, std::min<int64_t>(a.rows, kLoopParts));
                const dim3 grid((unsigned)(((int64_t)a.cols + kLoopBlock - 1) / kLoopBlock), parts);
                norm_dw_loop_kernel<T><<<grid, kLoopBlock, 0, st>>>(a, parts);
            }
            return (int)cudaGetLastError();
        });
    } else {
        e = with_type(a.dtype, [&](auto t) {
            using T = decltype(t);
            const bool vec = vector_rows(a.x, a.x_stride, a.rows, sizeof(T)) &&
                             vector_rows(a.dy, a.dy_stride, a.rows, sizeof(T)) &&
                             vector_rows(a.dx, a.dx_stride, a.rows, sizeof(T));
            return with_shape(a.cols, [&](auto per, auto row_warps, int warps) {
                constexpr int kPer = decltype(per)::value;
                constexpr int kWarps = decltype(row_warps)::value;
                return launch_rows(vec ? norm_bwd_kernel<T, kPer, true, kWarps> : norm_bwd_kernel<T, kPer, false, kWarps>,
                                   a, 2, sizeof(T), kWarps, warps, sm_count, st, &parts);
            });
        });
    }
    if (e == cudaSuccess && params)
        e = a.param_dtype == kF32    ? launch_join<float>(a, parts, st)
            : a.param_dtype == kBF16 ? launch_join<__nv_bfloat16>(a, parts, st)
                                     : launch_join<__half>(a, parts, st);
    // (dweight and dbias first: dx may take the place of dy or x)
    if (e == cudaSuccess && a.cols > kLongest && a.dx && a.rows > 0)
        e = with_types(a.dtype, a.param_dtype, [&](auto t, auto w) {
            const int grid = (int)std::min<int64_t>(a.rows, kCtasMost * sm_count);
            norm_dx_loop_kernel<decltype(t), decltype(w)><<<grid, kLoopBlock, 0, st>>>(a);
            return (int)cudaGetLastError();
        });
    return e;
}

int read_norm_gave_up(unsigned* count) { return (int)cudaMemcpyFromSymbol(count, g_gave_up, sizeof(*count)); }

}  // namespace soma
