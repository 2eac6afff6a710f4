// Linear layer: matrix products with their epilogue, and the activation's
// backward pass (formulas in soma_ops.h).
//
// Many rows are bound by the tensor cores: 256 x 256 tiles on CTA pairs, 64
// k-values per pipeline stage, operands by TMA, two accumulators in TMEM so
// that a tile's epilogue (bias, activation, residual, rounding) runs under the
// next tile's products.  Few rows are bound by reading the weight: there its
// rows are the tile's, and k is split over a cluster so that every SM reads.
// Operands may run along k or across it, so no product needs a transpose.
//
// Measured (GB300, cuBLAS bf16 1924 TFLOP/s in a burst): 16384 x 4096 x 11008
// bf16 with residual 818 us in a burst, 1807 TFLOP/s, and 944 us in a steady
// loop, which power limits; 4096 x 4096 x 1024 with gelu and saved
// pre-activation 32.8 us, 1048 TFLOP/s (3.4 waves of tiles whose epilogue is as
// long as their products); its three gradients in fp16 71.5 us, 961 TFLOP/s;
// through 11008 x 4096, one row 18.2 us, 4960 GB/s, 16 rows 20.3, 64 rows 28.2
// and 128 rows 47.8 us.
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "ops_device.cuh"
#include "ops_kernels.h"
#include "soma_ops.h"
#include "tcgen05.cuh"

namespace soma {
namespace {

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f;
constexpr float kCubic = 0.044715f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float reciprocal_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + exp(-x)); the exponential overflows to inf far left, where the result is 0.
__device__ __forceinline__ float logistic(float x) { return reciprocal_fast(1.f + exp2_fast(-kLog2e * x)); }

// The normal distribution's cdf and exp(-z^2 / 2), by Abramowitz and Stegun's
// formula 7.1.26 for erf (absolute error below 1.5e-7): one exponential, one
// reciprocal and a polynomial of degree 5, where the outputs have 8 or 11 bits.
// z cdf(z) errs by at most 2.2e-7.  Relative to itself that is 5e-5 for z > -3,
// 5e-4 to -4 (an eighth of a bf16 unit, one of fp16), 0.0016 to -5 and 0.0065
// to -7, where the value is 1e-11; fp32's 1 + erf(z / sqrt 2) loses it all by -5.
__device__ __forceinline__ float normal_cdf(float z, float& bell) {
    const float x = fabsf(z) * kSqrtHalf;
    const float t = reciprocal_fast(fmaf(0.3275911f, x, 1.f));
    bell = exp2_fast(-kLog2e * x * x);
    float q = fmaf(1.061405429f, t, -1.453152027f);
    q = fmaf(q, t, 1.421413741f);
    q = fmaf(q, t, -0.284496736f);
    q = fmaf(q, t, 0.254829592f);
    const float tail = 0.5f * q * t * bell;
    return z > 0.f ? 1.f - tail : tail;
}

template <int kAct>
__device__ __forceinline__ float activate(float z) {
    if (kAct == SOMA_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN stays NaN
    if (kAct == SOMA_ACT_GELU) {
        float bell;
        return z * normal_cdf(z, bell);
    }
    // (1 + tanh u) / 2 is the logistic function of 2u
    if (kAct == SOMA_ACT_GELU_TANH) return z * logistic(2.f * kSqrt2OverPi * z * fmaf(kCubic * z, z, 1.f));
    if (kAct == SOMA_ACT_SILU) return z * logistic(z);
    return z;
}

template <int kAct>
__device__ __forceinline__ float act_slope(float z) {
    if (kAct == SOMA_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if (kAct == SOMA_ACT_GELU) {
        float bell;
        const float cdf = normal_cdf(z, bell);
        return fmaf(z * kInvSqrt2Pi, bell, cdf);
    }
    if (kAct == SOMA_ACT_GELU_TANH) {
        const float s = logistic(2.f * kSqrt2OverPi * z * fmaf(kCubic * z, z, 1.f));
        const float near = fminf(fabsf(z), 64.f);  // s (1 - s) is 0 beyond; z^2 may leave fp32's range
        const float du = 2.f * kSqrt2OverPi * fmaf(3.f * kCubic * near, near, 1.f);
        return fmaf(z * s * (1.f - s), du, s);
    }
    if (kAct == SOMA_ACT_SILU) {
        const float s = logistic(z);
        return s * fmaf(z, 1.f - s, 1.f);
    }
    return 1.f;
}

// Calls f with the activation as a compile-time constant (f is a function of
// the host or of the device, as the caller is).
#pragma nv_exec_check_disable
template <typename F>
__host__ __device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case SOMA_ACT_RELU: f(std::integral_constant<int, SOMA_ACT_RELU>{}); break;
        case SOMA_ACT_GELU: f(std::integral_constant<int, SOMA_ACT_GELU>{}); break;
        case SOMA_ACT_GELU_TANH: f(std::integral_constant<int, SOMA_ACT_GELU_TANH>{}); break;
        case SOMA_ACT_SILU: f(std::integral_constant<int, SOMA_ACT_SILU>{}); break;
        default: f(std::integral_constant<int, SOMA_ACT_NONE>{}); break;
    }
}

constexpr int kBM = 128;                    // rows of one CTA's tile: the TMEM lanes
constexpr int kBK = 64;                     // k-values of a pipeline stage: one 128-byte swizzle row
constexpr int kOperandRows = 64;            // m- or n-values of an mn-major box
constexpr uint32_t kMaxSmem = 232448;       // 227 KB

__device__ unsigned g_gave_up;  // threads that saw a bounded wait run out, on this device

template <typename T>
constexpr bool kIsBf16 = std::is_same<T, __nv_bfloat16>::value;

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    __half2 h;
    memcpy(&h, &w, 4);
    return __half22float2(h);
}

// x += eight packed values.
template <typename T>
__device__ __forceinline__ void add8(float* x, const uint4& w) {
    float2 t;
    t = unpack2<T>(w.x); x[0] += t.x; x[1] += t.y;
    t = unpack2<T>(w.y); x[2] += t.x; x[3] += t.y;
    t = unpack2<T>(w.z); x[4] += t.x; x[5] += t.y;
    t = unpack2<T>(w.w); x[6] += t.x; x[7] += t.y;
}

// Lets the next kernel of the stream be set up, and waits until the one
// before it is done and its results are visible.
__device__ __forceinline__ void follow_stream() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Copies an operand into rows that start on 16-byte boundaries, as TMA needs.
// A thread shifts whole vectors into place, four rows in flight; the new
// rows' padding is 0.  (T: either 16-bit type, for its size.)
constexpr int kRepackRows = 4;
template <typename T>
__global__ void __launch_bounds__(256) repack_kernel(const T* src, int64_t src_stride, T* dst, int64_t dst_stride,
                                                     int64_t rows, int32_t cols) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i * 8 >= cols) return;
    const int64_t step = gridDim.y;
    for (int64_t r0 = blockIdx.y; r0 < rows; r0 += kRepackRows * step) {
        uint4 u[kRepackRows], v[kRepackRows];
        int phase[kRepackRows];
#pragma unroll
        for (int k = 0; k < kRepackRows; ++k) {
            const int64_t r = r0 + k * step;
            if (r >= rows) break;
            const RowReader<T, false> row(src, src_stride, rows, r, cols);
            phase[k] = -1;
            if (i >= row.inner_begin && i < row.inner_end) {
                phase[k] = row.phase;
                u[k] = row.words[i];
                if (row.phase) v[k] = row.words[i + 1];
            } else {
                float x[8];
                row.gather(i, x, 0.f);
                u[k] = narrow16(x, T{});
            }
        }
#pragma unroll
        for (int k = 0; k < kRepackRows; ++k) {
            const int64_t r = r0 + k * step;
            if (r >= rows) break;
            reinterpret_cast<uint4*>(dst + r * dst_stride)[i] = phase[k] > 0 ? shifted<T>(u[k], v[k], phase[k]) : u[k];
        }
    }
}

struct TileArgs {
    CUtensorMap a, b, out, z;
    GemmArgs g;
    int32_t tiles_m, tiles_n;
    int32_t strip;         // columns of tiles that are walked through together
    int32_t whole;         // tiles from this one on are done in two halves of their columns
    bool tma_out, tma_z;   // rows of out / z start on 16-byte boundaries
};

// The boxes of one operand stage: `rows` m- (or n-) values from row0, k-values from k0.
template <int CG>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, bool kmajor, int rows, int row0,
                                             int k0, uint32_t bar) {
    if (kmajor) {
        tma_load<CG>(dst, map, k0, row0, bar);
    } else {
        for (int i = 0; i < rows / kOperandRows; ++i)
            tma_load<CG>(dst + i * kOperandRows * kBK * 2, map, row0 + i * kOperandRows, k0, bar);
    }
}

// The MMAs of one stage.
template <int CG>
__device__ __forceinline__ void stage_mma(uint32_t acc, uint32_t a, uint32_t b, bool a_kmajor, bool b_kmajor,
                                          uint32_t idesc, bool first) {
    const uint64_t da = operand_desc(a, a_kmajor), db = operand_desc(b, b_kmajor);
    const uint32_t sa = a_kmajor ? kStepKMajor : kStepMnMajor, sb = b_kmajor ? kStepKMajor : kStepMnMajor;
#pragma unroll
    for (int i = 0; i < kBK / 16; ++i) mma_f16<CG>(acc, da + i * sa, db + i * sb, idesc, !(first && i == 0));
}

// ---- many rows: a tile of 128 x BN (CG = 1) or 256 x BN (CG = 2) ------------

// Sixteen warps for the epilogue: with eight, 4096 x 4096 x 1024 with gelu and
// a saved pre-activation took 38.4 us instead of 34.6 (1.0 to 2 % the other way
// for products with a long k and a short epilogue).
constexpr int kEpilogueWarps = 16;
constexpr uint32_t kStagerBytes = 32 * 64;  // a warp's output buffer: 32 rows of 32 values
constexpr int kTileThreads = 32 * (kEpilogueWarps + 2);

template <int CG, int BN>
struct TileShape {
    static constexpr int kRowsB = BN / CG;  // rows of B that one CTA stages
    static constexpr uint32_t kBytesA = kBM * kBK * 2, kBytesB = kRowsB * kBK * 2, kStage = kBytesA + kBytesB;
    static constexpr uint32_t kStaging = kEpilogueWarps * (kStagerBytes + 32 * 2);  // output block and bias of each warp
    static constexpr int kStages = (int)((kMaxSmem - 1024 - 512 - kStaging) / kStage) > 8
                                       ? 8 : (int)((kMaxSmem - 1024 - 512 - kStaging) / kStage);
    static constexpr uint32_t kSmem = 1024 + kStages * kStage + kStaging + 512;
    static constexpr uint32_t kTmemCols = 2 * BN;
};

// Staging of a warp's output: 32 rows x 32 columns, 64-byte rows whose 16-byte
// pieces are swizzled like the output's tensor map.
template <typename T>
struct Stager {
    char* block;
    int row0, m, n;
    // Packs this lane's row of 32 values and stores the block at (row0, col0).
    __device__ __forceinline__ void store(const float (&x)[32], int col0, const CUtensorMap* map, bool tma, T* out,
                                          int64_t stride) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) tma_store_wait_read();  // the block before has been read
        __syncwarp();
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            uint4 w;
            w.x = pack2<T>(x[8 * v], x[8 * v + 1]);
            w.y = pack2<T>(x[8 * v + 2], x[8 * v + 3]);
            w.z = pack2<T>(x[8 * v + 4], x[8 * v + 5]);
            w.w = pack2<T>(x[8 * v + 6], x[8 * v + 7]);
            *reinterpret_cast<uint4*>(block + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4)) = w;
        }
        if (tma) {
            fence_to_async();
            __syncwarp();
            if (lane == 0) tma_store(map, smem_addr(block), col0, row0);
        } else {
            __syncwarp();
            if (col0 + lane < n) {
#pragma unroll 4
                for (int r = 0; r < 32 && row0 + r < m; ++r)
                    out[(row0 + r) * stride + col0 + lane] = *reinterpret_cast<const T*>(
                        block + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2);
            }
        }
    }
};

// One warp's 32 rows x `cols` columns (a multiple of 32) at (row0, col0):
// out of TMEM at `acc`, through the epilogue, into out (and z_out).
template <typename T>
__device__ __forceinline__ void epilogue(const TileArgs& p, uint32_t acc, int row0, int col0, int cols, Stager<T>& stager,
                                         T* bias) {
    const int lane = threadIdx.x & 31;
    const GemmArgs& g = p.g;
    const bool has_row = row0 + lane < g.m;
    const T* res =
        g.residual && has_row ? static_cast<const T*>(g.residual) + (int64_t)(row0 + lane) * g.residual_stride : nullptr;
    const bool res_vec = ((uintptr_t)g.residual % 16 == 0) && g.residual_stride % 8 == 0;
    stager.row0 = row0;
    for (int c0 = 0; c0 < cols && col0 + c0 < g.n; c0 += 32) {
        const int col = col0 + c0;
        uint32_t raw[32];
        tmem_ld32(acc + c0, raw);
        uint4 r4[4] = {};
        const bool whole = res && res_vec && col + 32 <= g.n;
        if (whole) {
#pragma unroll
            for (int v = 0; v < 4; ++v) r4[v] = *reinterpret_cast<const uint4*>(res + col + 8 * v);
        }
        if (g.bias) {
            __syncwarp();
            bias[lane] = col + lane < g.n ? static_cast<const T*>(g.bias)[col + lane] : from_f32<T>(0.f);
            __syncwarp();
        }
        tmem_ld_wait(raw);
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(raw[i]);
        if (g.bias) {
#pragma unroll
            for (int v = 0; v < 4; ++v) add8<T>(x + 8 * v, *reinterpret_cast<const uint4*>(bias + 8 * v));
        }
        if (g.z_out) stager.store(x, col, &p.z, p.tma_z, static_cast<T*>(g.z_out), g.z_stride);
        if (g.act != SOMA_ACT_NONE)
            with_act(g.act, [&](auto act) {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = activate<decltype(act)::value>(x[i]);
            });
        if (whole) {
#pragma unroll
            for (int v = 0; v < 4; ++v) add8<T>(x + 8 * v, r4[v]);
        } else if (res) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (col + i < g.n) x[i] += to_f32(res[col + i]);
        }
        stager.store(x, col, &p.out, p.tma_out, static_cast<T*>(g.out), g.out_stride);
    }
}

// Persistent: cluster i takes units i, i + clusters, ...  Warps 0-15 drain
// accumulators, the next loads operands, the last issues the MMAs; two
// accumulators in TMEM let a tile's epilogue run under the next tile's MMAs.
// CG = 2: a pair of CTAs shares one 256-row tile, each staging half of both
// operands; the leader (rank 0) issues the MMAs for both.
template <int CG, int BN, typename T>
__global__ void __launch_bounds__(kTileThreads, 1) tile_kernel(const __grid_constant__ TileArgs p) {
    using S = TileShape<CG, BN>;
    extern __shared__ char dynamic[];
    __shared__ int gave_up;
    __shared__ uint32_t tmem_slot;
    char* base = reinterpret_cast<char*>(((uintptr_t)dynamic + 1023) & ~(uintptr_t)1023);
    char* staging = base + S::kStages * S::kStage;
    const uint32_t stages = smem_addr(base);
    const uint32_t bars = smem_addr(staging + S::kStaging);
    auto full = [&](int s) { return bars + 8 * s; };
    auto empty = [&](int s) { return bars + 8 * (S::kStages + s); };
    auto acc_full = [&](int i) { return bars + 8 * (2 * S::kStages + i); };
    auto acc_empty = [&](int i) { return bars + 8 * (2 * S::kStages + 2 + i); };

    const GemmArgs& g = p.g;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full(i), 1);
            mbar_init(acc_empty(i), kEpilogueWarps * CG);
        }
        mbar_init_fence();
    }
    if (warp == kEpilogueWarps + 1) tmem_alloc<CG>(smem_addr(&tmem_slot), S::kTmemCols);
    if (threadIdx.x == kEpilogueWarps * 32) {
        prefetch_map(&p.a);
        prefetch_map(&p.b);
    }
    tcgen05_before_sync();
    if (CG == 2) cluster_sync_all();
    else __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = tmem_slot;
    follow_stream();

    // units of work: whole tiles, then halves
    const int tiles = p.tiles_m * p.tiles_n, units = 2 * tiles - p.whole;
    const int first = blockIdx.x / CG, step = gridDim.x / CG;
    const int kts = (g.k + kBK - 1) / kBK;
    auto tile_at = [&](int u, int& row0, int& col0) {  // returns the unit's columns
        const bool half = u >= p.whole;
        const int t = half ? p.whole + (u - p.whole) / 2 : u;
        const int strip = t / (p.tiles_m * p.strip) * p.strip, width = min(p.strip, p.tiles_n - strip);
        const int in_strip = t - strip * p.tiles_m;
        col0 = (strip + in_strip % width) * BN + (half && (u - p.whole) % 2 ? BN / 2 : 0);
        row0 = in_strip / width * (kBM * CG) + (int)rank * kBM;
        return half ? BN / 2 : BN;
    };

    if (warp == kEpilogueWarps && lane == 0) {
        int s = 0;
        uint32_t parity = 1;  // a fresh barrier's previous phase counts as done
        bool ok = true;
        for (int u = first; u < units && ok; u += step) {
            int row0, col0;
            // (of a half, the second half of B's rows is loaded and not used)
            const int b0 = tile_at(u, row0, col0) / CG * (int)rank + col0;
            for (int kt = 0; kt < kts; ++kt) {
                if (!(ok = mbar_wait(empty(s), parity, &gave_up))) break;
                const uint32_t bar = CG == 2 ? cluster_map(full(s), 0) : full(s);
                if (rank == 0) mbar_expect(full(s), CG * S::kStage);
                const uint32_t dst = stages + s * S::kStage;
                load_operand<CG>(dst, &p.a, g.a_kmajor, kBM, row0, kt * kBK, bar);
                load_operand<CG>(dst + S::kBytesA, &p.b, g.b_kmajor, S::kRowsB, b0, kt * kBK, bar);
                if (++s == S::kStages) {
                    s = 0;
                    parity ^= 1;
                }
            }
        }
        // The MMAs' last arrivals (of a pair, from the other CTA) land before the
        // CTA's memory is given back: other commits' arrivals do not promise it.
        for (int i = 0; i < S::kStages && ok; ++i) {
            ok = mbar_wait(empty(s), parity, &gave_up);
            if (++s == S::kStages) {
                s = 0;
                parity ^= 1;
            }
        }
    } else if (warp == kEpilogueWarps + 1 && lane == 0 && rank == 0) {
        int s = 0, i = 0;
        uint32_t parity = 0, acc_parity = 1;
        bool ok = true;
        for (int u = first; u < units && ok; u += step) {
            const uint32_t idesc =
                instruction_desc(kIsBf16<T>, g.a_kmajor, g.b_kmajor, kBM * CG, u >= p.whole ? BN / 2 : BN);
            if (!(ok = mbar_wait(acc_empty(i), acc_parity, &gave_up))) break;
            tcgen05_after_sync();
            for (int kt = 0; kt < kts; ++kt) {
                if (!(ok = mbar_wait(full(s), parity, &gave_up))) break;
                tcgen05_after_sync();
                const uint32_t src = stages + s * S::kStage;
                stage_mma<CG>(tmem + i * BN, src, src + S::kBytesA, g.a_kmajor, g.b_kmajor, idesc, kt == 0);
                mma_commit<CG>(empty(s));
                if (++s == S::kStages) {
                    s = 0;
                    parity ^= 1;
                }
            }
            mma_commit<CG>(acc_full(i));
            i ^= 1;
            if (i == 0) acc_parity ^= 1;
        }
    } else if (warp < kEpilogueWarps) {
        Stager<T> stager{staging + warp * kStagerBytes, 0, g.m, g.n};
        T* bias = reinterpret_cast<T*>(staging + kEpilogueWarps * kStagerBytes) + warp * 32;
        const int quarter = warp & 3;
        int i = 0;
        uint32_t parity = 0;
        for (int u = first; u < units; u += step) {
            int row0, col0;
            const int cols = tile_at(u, row0, col0) / (kEpilogueWarps / 4), at = (warp >> 2) * cols;  // the warp's
            if (!mbar_wait(acc_full(i), parity, &gave_up, product_limit(kts))) break;
            __syncwarp();
            tcgen05_after_sync();
            if (row0 + quarter * 32 < g.m)
                epilogue<T>(p, tmem + i * BN + at + ((uint32_t)(quarter * 32) << 16), row0 + quarter * 32, col0 + at, cols,
                            stager, bias);
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(CG == 2 ? cluster_map(acc_empty(i), 0) : acc_empty(i));
            i ^= 1;
            if (i == 0) parity ^= 1;
        }
        if (lane == 0) tma_store_wait();
    }
    __syncwarp();
    if (gave_up) outlast_copies();  // what is still in flight lands before the CTA's memory is given back
    tcgen05_before_sync();
    if (CG == 2) cluster_sync_all();
    else __syncthreads();
    tcgen05_after_sync();
    if (threadIdx.x == 0 && gave_up) atomicAdd(&g_gave_up, 1u);
    if (warp == kEpilogueWarps + 1) tmem_free<CG>(tmem, S::kTmemCols);
}

// ---- few tiles: k split over a cluster ------------------------------------------
//
// For products that have too few 128 x 128 tiles for the SMs, those with few
// rows above all.  The roles are swapped, out^T = B A^T: the rows of `b` (the
// weight, in the forward pass) are the tile's 128 TMEM lanes and up to BN rows
// of `a` its columns, so that one row of x costs no more than it must.  A
// cluster of CTAs splits k; each leaves a partial 128 x BN sum in TMEM, sends
// every CTA its share of the columns through distributed shared memory, and
// finishes its own share, adding the partial sums in rank order.

constexpr int kFewThreads = 32 * 6;

template <int BN>
struct FewShape {
    static constexpr uint32_t kBytesW = kBM * kBK * 2, kBytesX = BN * kBK * 2, kStage = kBytesW + kBytesX;
    static constexpr uint32_t kExchange = kBM * BN * 4;
    // two CTAs per SM where the columns are few
    static constexpr int kCtasPerSm = BN <= 64 ? 2 : 1;
    static constexpr uint32_t kBudget = (kCtasPerSm == 2 ? 113 * 1024 : kMaxSmem) - 1024 - 512 - kExchange;
    static constexpr int kStages = (int)(kBudget / kStage) > 8 ? 8 : (int)(kBudget / kStage);
    static constexpr uint32_t kSmem = 1024 + kStages * kStage + kExchange + 512;
    static constexpr uint32_t kTmemCols = BN < 32 ? 32 : BN;
};

template <int BN, typename T>
__global__ void __launch_bounds__(kFewThreads) few_kernel(const __grid_constant__ TileArgs p, int splits) {
    using S = FewShape<BN>;
    extern __shared__ char dynamic[];
    __shared__ int gave_up;
    __shared__ uint32_t tmem_slot;
    char* base = reinterpret_cast<char*>(((uintptr_t)dynamic + 1023) & ~(uintptr_t)1023);
    float* exchange = reinterpret_cast<float*>(base + S::kStages * S::kStage);
    const uint32_t stages = smem_addr(base);
    const uint32_t bars = smem_addr(base) + S::kStages * S::kStage + S::kExchange;
    auto full = [&](int s) { return bars + 8 * s; };
    auto empty = [&](int s) { return bars + 8 * (S::kStages + s); };
    const uint32_t done = bars + 8 * (2 * S::kStages);

    const GemmArgs& g = p.g;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)blockIdx.x % splits;
    const int64_t tile = blockIdx.x / splits;
    const int n0 = (int)(tile % p.tiles_n) * kBM, m0 = (int)(tile / p.tiles_n) * BN;
    const int kts = (g.k + kBK - 1) / kBK;
    const int kt0 = (int)((int64_t)rank * kts / splits), kt1 = (int)((int64_t)(rank + 1) * kts / splits);
    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(done, 1);
        mbar_init_fence();
    }
    if (warp == 5) tmem_alloc<1>(smem_addr(&tmem_slot), S::kTmemCols);
    if (threadIdx.x == 4 * 32) {
        prefetch_map(&p.a);
        prefetch_map(&p.b);
    }
    tcgen05_before_sync();
    if (splits > 1) cluster_sync_all();  // (no CTA writes into another that has not started)
    else __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = tmem_slot;
    follow_stream();

    if (warp == 4 && lane == 0) {
        int s = 0;
        uint32_t parity = 1;
        bool ok = true;
        for (int kt = kt0; kt < kt1; ++kt) {
            if (!(ok = mbar_wait(empty(s), parity, &gave_up))) break;
            mbar_expect(full(s), S::kStage);
            const uint32_t dst = stages + s * S::kStage;
            load_operand<1>(dst, &p.b, g.b_kmajor, kBM, n0, kt * kBK, full(s));
            load_operand<1>(dst + S::kBytesW, &p.a, g.a_kmajor, BN, m0, kt * kBK, full(s));
            if (++s == S::kStages) {
                s = 0;
                parity ^= 1;
            }
        }
        // (as in the tile kernel)
        for (int i = 0; i < S::kStages && ok; ++i) {
            ok = mbar_wait(empty(s), parity, &gave_up);
            if (++s == S::kStages) {
                s = 0;
                parity ^= 1;
            }
        }
    } else if (warp == 5 && lane == 0) {
        const uint32_t idesc = instruction_desc(kIsBf16<T>, g.b_kmajor, g.a_kmajor, kBM, BN);
        int s = 0;
        uint32_t parity = 0;
        for (int kt = kt0; kt < kt1; ++kt) {
            if (!mbar_wait(full(s), parity, &gave_up)) break;
            tcgen05_after_sync();
            const uint32_t src = stages + s * S::kStage;
            stage_mma<1>(tmem, src, src + S::kBytesW, g.b_kmajor, g.a_kmajor, idesc, kt == kt0);
            mma_commit<1>(empty(s));
            if (++s == S::kStages) {
                s = 0;
                parity ^= 1;
            }
        }
        mma_commit<1>(done);
    }
    __syncwarp();
    // columns that each CTA finishes (splits is a power of two)
    const int log_share = __ffs(BN) - __ffs(splits), share = 1 << log_share;
    if (warp < 4) {
        if (mbar_wait(done, 0, &gave_up, product_limit(kt1 - kt0))) {
            __syncwarp();
            tcgen05_after_sync();
            const uint32_t mine = smem_addr(exchange) + (rank * share * kBM + warp * 32 + lane) * 4;
#pragma unroll
            for (int c0 = 0; c0 < BN; c0 += 16) {
                uint32_t raw[16];
                tmem_ld16(tmem + ((uint32_t)(warp * 32) << 16) + c0, raw);
                tmem_ld_wait(raw);
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const int col = c0 + c;
                    const uint32_t at = mine + (col & (share - 1)) * (kBM * 4);
                    st_cluster_f32(splits == 1 ? at : cluster_map(at, col >> log_share), __uint_as_float(raw[c]));
                }
            }
        }
        tcgen05_before_sync();
    }
    __syncwarp();
    if (gave_up) outlast_copies();
    if (splits > 1) cluster_sync_all();  // every partial sum has arrived; no CTA's memory is written after this
    else __syncthreads();
    if (threadIdx.x == 0 && gave_up) atomicAdd(&g_gave_up, 1u);
    if (warp < 4) {
        const int n = n0 + warp * 32 + lane;
        const int count = min(share, g.m - m0 - rank * share);
        if (n < g.n && count > 0) {
            const float bias = g.bias ? to_f32(static_cast<const T*>(g.bias)[n]) : 0.f;
            const float* from = exchange + warp * 32 + lane;
            const int64_t m = m0 + rank * share;
            const T* res = g.residual ? static_cast<const T*>(g.residual) + m * g.residual_stride + n : nullptr;
            T* out = static_cast<T*>(g.out) + m * g.out_stride + n;
            T* z_out = g.z_out ? static_cast<T*>(g.z_out) + m * g.z_stride + n : nullptr;
            with_act(g.act, [&](auto act) {
#pragma unroll 4
                for (int c = 0; c < count; ++c) {
                    float z = 0.f;
                    for (int r = 0; r < splits; ++r) z += from[(r * share + c) * kBM];
                    z += bias;
                    if (z_out) z_out[c * g.z_stride] = from_f32<T>(z);
                    float y = activate<decltype(act)::value>(z);
                    if (res) y += to_f32(res[c * g.residual_stride]);
                    out[c * g.out_stride] = from_f32<T>(y);
                }
            });
        }
    }
    if (warp == 5) {
        tcgen05_after_sync();
        tmem_free<1>(tmem, S::kTmemCols);
    }
}

// ---- host side ----------------------------------------------------------------

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess || found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

bool aligned_rows(const void* p, int64_t stride, int64_t rows) {
    return (uintptr_t)p % 16 == 0 && (rows <= 1 || stride % 8 == 0);
}

// Tensor map of a 16-bit matrix with boxes of box_rows rows x 64 or 32
// columns, swizzled over the box's 128- or 64-byte rows.
int make_map(CUtensorMap* map, int dtype, const void* p, int64_t stride, int64_t rows, int64_t cols, int box_rows,
             int box_cols = 64) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return cudaErrorNotSupported;
    if (rows <= 1) stride = (cols + 7) / 8 * 8;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, steps[2] = {1, 1};
    const CUresult r = fn(map, dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                          const_cast<void*>(p), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int operand_map(CUtensorMap* map, const GemmArgs& g, const void* p, int64_t stride, bool kmajor, int64_t rows,
                int box_rows) {
    return kmajor ? make_map(map, g.dtype, p, stride, rows, g.k, box_rows)
                  : make_map(map, g.dtype, p, stride, g.k, rows, kBK);
}

int launch(const void* kernel, void** args, int grid, int threads, uint32_t smem, int cluster, void* stream) {
    const int e = allow_smem(kernel, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    // may be set up while the kernel before it ends (it waits before it reads or writes)
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

template <int CG, int BN, typename T>
int launch_tile(TileArgs& p, int sm_count, void* stream) {
    using S = TileShape<CG, BN>;
    const GemmArgs& g = p.g;
    int e;
    if ((e = operand_map(&p.a, g, g.a, g.a_stride, g.a_kmajor, g.m, kBM)) ||
        (e = operand_map(&p.b, g, g.b, g.b_stride, g.b_kmajor, g.n, S::kRowsB)))
        return e;
    p.tma_out = aligned_rows(g.out, g.out_stride, g.m);
    p.tma_z = g.z_out && aligned_rows(g.z_out, g.z_stride, g.m);
    if (p.tma_out && (e = make_map(&p.out, g.dtype, g.out, g.out_stride, g.m, g.n, 32, 32))) return e;
    if (p.tma_z && (e = make_map(&p.z, g.dtype, g.z_out, g.z_stride, g.m, g.n, 32, 32))) return e;
    p.tiles_m = (g.m + kBM * CG - 1) / (kBM * CG);
    p.tiles_n = (g.n + BN - 1) / BN;
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n, workers = std::max(1, sm_count / CG);
    if (tiles > (1 << 29)) return cudaErrorInvalidValue;
    // Strips of columns of B of at most 48 MB, which stay in L2 while A passes,
    // are done one after another: 8192^3 605 us instead of 643 in one strip,
    // 16384 x 4096 x 11008 822 instead of 830 (ncu had 1.9 GB read there for
    // 0.6 GB of operands).
    const int64_t fit = std::max<int64_t>(1, (48ll << 20) / ((int64_t)BN * g.k * 2));
    const int64_t strips = (p.tiles_n + fit - 1) / fit;
    p.strip = (int32_t)((p.tiles_n + strips - 1) / strips);
    // a last wave that at most half of the workers have is done in half tiles by all
    const int64_t rest = tiles % workers;
    p.whole = (int32_t)(CG == 2 && 2 * rest <= workers ? tiles - rest : tiles);
    const int64_t units = 2 * tiles - p.whole;
    void* args[] = {&p};
    return launch((const void*)tile_kernel<CG, BN, T>, args, CG * (int)std::min(units, workers), kTileThreads,
                  S::kSmem, CG, stream);
}

template <int BN, typename T>
int launch_few(TileArgs& p, int sm_count, void* stream) {
    using S = FewShape<BN>;
    const GemmArgs& g = p.g;
    int e;
    if ((e = operand_map(&p.a, g, g.a, g.a_stride, g.a_kmajor, g.m, BN)) ||
        (e = operand_map(&p.b, g, g.b, g.b_stride, g.b_kmajor, g.n, kBM)))
        return e;
    p.tiles_n = (g.n + kBM - 1) / kBM;
    p.tiles_m = (g.m + BN - 1) / BN;
    const int tiles = p.tiles_n * p.tiles_m, kts = (g.k + kBK - 1) / kBK;
    int splits = 1;
    while (splits < 8 && 4 * splits <= kts && tiles * splits * 2 <= S::kCtasPerSm * sm_count) splits *= 2;
    void* args[] = {&p, &splits};
    return launch((const void*)few_kernel<BN, T>, args, tiles * splits, kFewThreads, S::kSmem, splits, stream);
}

// ---- the activation's backward pass -------------------------------------------

// A warp takes 256 columns, a vector of 8 per lane; the CTA's warps, and the
// CTAs of a column block, take rows in turn.  dz is rounded and stored, the
// column sums of the unrounded dz stay in registers and end as one partial
// row per CTA.  Reads dy and z, writes dz: HBM (or L2) bound.
constexpr int kActWarps = 8, kActCols = 256;

// kWhole: the rows of dy and z start on 16-byte boundaries and hold whole
// vectors; four rows' loads are then in flight per thread.
template <typename T, int kAct, bool kWhole>
__global__ void __launch_bounds__(32 * kActWarps) act_bwd_kernel(const __grid_constant__ ActBwdArgs a) {
    __shared__ float sums[kActWarps][kActCols];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane, c0 = i * 8;  // this lane's vector
    const int64_t step = (int64_t)gridDim.y * kActWarps;
    float db[8] = {};
    struct Raw {
        uint4 u, v;
        int phase;  // -1: u is the vector itself
    };
    auto fetch = [&](const void* base, int64_t stride, int64_t r) {
        const RowReader<T, false> row(static_cast<const T*>(base), stride, a.rows, r, a.cols);
        Raw raw;
        raw.phase = -1;
        if (i >= row.inner_begin && i < row.inner_end) {
            raw.phase = row.phase;
            raw.u = row.words[i];
            if (row.phase) raw.v = row.words[i + 1];
        } else {
            float x[8];
            row.gather(i, x, 0.f);
            raw.u = narrow16(x, T{});
        }
        return raw;
    };
    auto expand = [](const Raw& raw, float (&x)[8]) {
        widen16(raw.phase > 0 ? shifted<T>(raw.u, raw.v, raw.phase) : raw.u, x, T{});
    };
    int64_t r = (int64_t)blockIdx.y * kActWarps + warp;
    auto finish = [&](int64_t row, float (&g)[8], const float (&z)[8]) {
        if (kAct != SOMA_ACT_NONE) {
#pragma unroll
            for (int q = 0; q < 8; ++q) g[q] *= act_slope<kAct>(z[q]);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (kWhole || c0 + q < a.cols) db[q] += g[q];
        // (dz's rows are padded to whole vectors)
        if (a.dz && c0 < a.cols) *reinterpret_cast<uint4*>(static_cast<T*>(a.dz) + row * a.dz_stride + c0) = narrow16(g, T{});
    };
    if (kWhole && c0 < a.cols) {
        constexpr int kAhead = 4;
        const T *dy = static_cast<const T*>(a.dy) + c0, *z0 = static_cast<const T*>(a.z) + c0;
        for (; r + (kAhead - 1) * step < a.rows; r += kAhead * step) {
            uint4 u[kAhead], v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                u[k] = *reinterpret_cast<const uint4*>(dy + (r + k * step) * a.dy_stride);
                if (kAct != SOMA_ACT_NONE) v[k] = *reinterpret_cast<const uint4*>(z0 + (r + k * step) * a.z_stride);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                float g[8], z[8];
                widen16(u[k], g, T{});
                if (kAct != SOMA_ACT_NONE) widen16(v[k], z, T{});
                finish(r + k * step, g, z);
            }
        }
    }
    for (; r < a.rows; r += 2 * step) {
        const bool second = r + step < a.rows;
        Raw dy[2], zr[2];
        dy[0] = fetch(a.dy, a.dy_stride, r);
        if (kAct != SOMA_ACT_NONE) zr[0] = fetch(a.z, a.z_stride, r);
        if (second) {
            dy[1] = fetch(a.dy, a.dy_stride, r + step);
            if (kAct != SOMA_ACT_NONE) zr[1] = fetch(a.z, a.z_stride, r + step);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k && !second) break;
            float g[8], z[8];
            expand(dy[k], g);
            if (kAct != SOMA_ACT_NONE) expand(zr[k], z);
            finish(r + k * step, g, z);
        }
    }
    if (!a.dbias) return;
#pragma unroll
    for (int q = 0; q < 8; ++q) sums[warp][lane * 8 + q] = db[q];
    __syncthreads();
    const int c = blockIdx.x * kActCols + threadIdx.x;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kActWarps; ++w) s += sums[w][threadIdx.x];
    if (c < a.cols) a.partials[(int64_t)blockIdx.y * a.cols + c] = s;
}

// dbias: the partial rows added in a fixed order, 32 columns per CTA.
template <typename T>
__global__ void __launch_bounds__(32 * kActWarps) bias_grad_kernel(const __grid_constant__ ActBwdArgs a, int parts) {
    __shared__ float scratch[kActWarps][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float db = 0.f;
    if (c < a.cols) {
#pragma unroll 4
        for (int p = warp; p < parts; p += kActWarps) db += a.partials[(int64_t)p * a.cols + c];
    }
    scratch[warp][lane] = db;
    __syncthreads();
    if (warp || c >= a.cols) return;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kActWarps; ++w) s += scratch[w][lane];
    static_cast<T*>(a.dbias)[c] = from_f32<T>(s);
}

// CTAs of a column block: about six CTAs per SM in all, eight rows each at least.
int row_parts(int64_t rows, int64_t cols, int sm_count) {
    const int64_t blocks = (cols + kActCols - 1) / kActCols, by_rows = (rows + kActWarps - 1) / kActWarps;
    return (int)std::max<int64_t>(1, std::min<int64_t>(by_rows, 6 * (int64_t)sm_count / blocks));
}

template <typename F>
int with_type16(int dtype, F&& f) {
    return dtype == kBF16 ? f(__nv_bfloat16{}) : f(__half{});
}

}  // namespace

bool gemm_operand_needs_copy(const void* p, int64_t stride, int64_t rows) { return !aligned_rows(p, stride, rows); }

int launch_repack(const void* src, int64_t src_stride, void* dst, int64_t dst_stride, int64_t rows, int64_t cols,
                  int dtype, int sm_count, void* stream) {
    const unsigned blocks = (unsigned)((cols + 2047) / 2048);
    const int64_t by_rows = (rows + kRepackRows - 1) / kRepackRows;
    const dim3 grid(blocks, (unsigned)std::max<int64_t>(1, std::min<int64_t>(by_rows, 8 * (int64_t)sm_count / blocks)));
    auto kernel = dtype == kBF16 ? (const void*)repack_kernel<__nv_bfloat16> : (const void*)repack_kernel<__half>;
    int32_t n = (int32_t)cols;
    void* args[] = {&src, &src_stride, &dst, &dst_stride, &rows, &n};
    return (int)cudaLaunchKernel(kernel, grid, dim3(256), args, 0, (cudaStream_t)stream);
}

int launch_gemm(const GemmArgs& a, int sm_count, void* stream) {
    return with_type16(a.dtype, [&](auto t) {
        using T = decltype(t);
        TileArgs p{};
        p.g = a;
        // Few rows, or a long k over too few tiles for the SMs: k is split.
        // (Joining costs about as much as 26 pipeline stages: 1021 x 1111 x 1003
        // took 26.8 us split in two and 18.6 us whole, 300 x 300 x 10000 15.5 us
        // split in eight and 50 us whole.)
        const int64_t small = (int64_t)((a.m + 127) / 128) * ((a.n + 127) / 128), kts = (a.k + kBK - 1) / kBK;
        const int64_t splits = small * 8 <= sm_count ? 8 : small * 4 <= sm_count ? 4 : small * 2 <= sm_count ? 2 : 1;
        if (a.m <= 128 || kts - kts / splits > 26) {
            if (a.a_kmajor && a.m <= 16) return launch_few<16, T>(p, sm_count, stream);
            if (a.a_kmajor && a.m <= 32) return launch_few<32, T>(p, sm_count, stream);
            if (a.m <= 64) return launch_few<64, T>(p, sm_count, stream);
            return launch_few<128, T>(p, sm_count, stream);
        }
        // A 256 x 256 tile on two SMs takes as long as a 128 x 128 tile on one
        // (0.36 and 0.34 us per 64 k-values: the small one moves twice the
        // operand bytes per product), so the fewer waves win.
        const int64_t big = (int64_t)((a.m + 255) / 256) * ((a.n + 255) / 256), pairs = std::max(1, sm_count / 2);
        const int64_t waves_big = (big + pairs - 1) / pairs, waves_small = (small + sm_count - 1) / sm_count;
        if (waves_big < waves_small) return launch_tile<2, 256, T>(p, sm_count, stream);
        return launch_tile<1, 128, T>(p, sm_count, stream);
    });
}

int read_linear_gave_up(unsigned* count) { return (int)cudaMemcpyFromSymbol(count, g_gave_up, sizeof(*count)); }

int64_t act_bwd_workspace(int64_t rows, int64_t cols, int sm_count) {
    return (int64_t)row_parts(rows, cols, sm_count) * cols * 4;
}

int launch_act_bwd(const ActBwdArgs& a, int sm_count, void* stream) {
    return with_type16(a.dtype, [&](auto t) {
        using T = decltype(t);
        const int blocks = (a.cols + kActCols - 1) / kActCols, parts = row_parts(a.rows, a.cols, sm_count);
        cudaStream_t st = (cudaStream_t)stream;
        const bool whole = a.cols % 8 == 0 && aligned_rows(a.dy, a.dy_stride, a.rows) &&
                           (a.act == SOMA_ACT_NONE || aligned_rows(a.z, a.z_stride, a.rows));
        with_act(a.act, [&](auto act) {
            constexpr int kAct = decltype(act)::value;
            auto kernel = whole ? act_bwd_kernel<T, kAct, true> : act_bwd_kernel<T, kAct, false>;
            kernel<<<dim3(blocks, parts), 32 * kActWarps, 0, st>>>(a);
        });
        int e = (int)cudaGetLastError();
        if (e != cudaSuccess || !a.dbias) return e;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((a.cols + 31) / 32);
        cfg.blockDim = dim3(32 * kActWarps);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return (int)cudaLaunchKernelEx(&cfg, bias_grad_kernel<T>, a, parts);
    });
}

}  // namespace soma
