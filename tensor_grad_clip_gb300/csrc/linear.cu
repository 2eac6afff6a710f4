// Linear layer: matrix products with their epilogue, and the activation's
// backward pass (formulas in soma_ops.h).
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

constexpr int kBM = 128;                    // rows of one CTA's tile: the TMEM lanes
constexpr int kBK = 64;                     // k-values of a pipeline stage: one 128-byte swizzle row
constexpr int kOperandRows = 64;            // m- or n-values of an mn-major box
constexpr uint32_t kMaxSmem = 232448;       // 227 KB

__device__ int g_gave_up;                   // a kernel's bounded wait ran out on this device

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
__device__ __forceinline__ void add8(float (&x)[8], const uint4& w) {
    float2 t;
    t = unpack2<T>(w.x); x[0] += t.x; x[1] += t.y;
    t = unpack2<T>(w.y); x[2] += t.x; x[3] += t.y;
    t = unpack2<T>(w.z); x[4] += t.x; x[5] += t.y;
    t = unpack2<T>(w.w); x[6] += t.x; x[7] += t.y;
}

// Copies an operand into rows that start on 16-byte boundaries, as TMA needs.
template <typename T>
__global__ void __launch_bounds__(256) repack_kernel(const T* src, int64_t src_stride, T* dst, int64_t dst_stride,
                                                     int64_t rows, int32_t cols) {
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y)
        for (int c = blockIdx.x * 256 + threadIdx.x; c < cols; c += gridDim.x * 256)
            dst[r * dst_stride + c] = src[r * src_stride + c];
}

struct TileArgs {
    CUtensorMap a, b, out, z;
    GemmArgs g;
    int32_t tiles_m, tiles_n;
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

constexpr int kEpilogueWarps = 8;
constexpr int kTileThreads = 32 * (kEpilogueWarps + 2);

template <int CG, int BN>
struct TileShape {
    static constexpr int kRowsB = BN / CG;  // rows of B that one CTA stages
    static constexpr uint32_t kBytesA = kBM * kBK * 2, kBytesB = kRowsB * kBK * 2, kStage = kBytesA + kBytesB;
    static constexpr uint32_t kStaging = kEpilogueWarps * (32 * 128 + 64 * 2);  // output block and bias of each warp
    static constexpr int kStages = (int)((kMaxSmem - 1024 - 512 - kStaging) / kStage) > 8
                                       ? 8 : (int)((kMaxSmem - 1024 - 512 - kStaging) / kStage);
    static constexpr uint32_t kSmem = 1024 + kStages * kStage + kStaging + 512;
    static constexpr uint32_t kTmemCols = 2 * BN;
};

// One warp's 32 x 64 block: rows row0.., columns col0... `acc` is the block's
// TMEM address; block is 4 KB of staging (128-byte rows, 16-byte pieces
// swizzled by the row like the output's tensor map), bias 64 values.
template <typename T>
__device__ __forceinline__ void epilogue_block(const TileArgs& p, uint32_t acc, int row0, int col0, char* block,
                                               T* bias) {
    const int lane = threadIdx.x & 31;
    const GemmArgs& g = p.g;
    const int row = row0 + lane;
    const bool has_row = row < g.m;
    if (g.bias) {
        const T* b = static_cast<const T*>(g.bias) + col0;
        bias[lane] = col0 + lane < g.n ? b[lane] : from_f32<T>(0.f);
        bias[lane + 32] = col0 + lane + 32 < g.n ? b[lane + 32] : from_f32<T>(0.f);
    }
    __syncwarp();
    char* mine = block + lane * 128;
    const int sw = lane & 7;
    const T* res = g.residual ? static_cast<const T*>(g.residual) + (int64_t)row * g.residual_stride + col0 : nullptr;
    const bool res_vec = g.residual && ((uintptr_t)g.residual % 16 == 0) && g.residual_stride % 8 == 0;
    // pass 0 writes z, pass 1 writes out
    for (int pass = g.z_out ? 0 : 1; pass < 2; ++pass) {
        // the previous block's store has read the staging rows
        if (lane == 0) tma_store_wait_read();
        __syncwarp();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t raw[32];
            tmem_ld32(acc + half * 32, raw);
            tmem_ld_wait(raw);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(raw[v * 8 + i]);
                const int c = half * 32 + v * 8;
                if (g.bias) {
                    add8<T>(x, *reinterpret_cast<const uint4*>(bias + c));
                }
                if (pass == 1) {
                    if (g.act != SOMA_ACT_NONE) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = activate(x[i], g.act);
                    }
                    if (res && has_row) {
                        if (res_vec && col0 + c + 8 <= g.n) {
                            add8<T>(x, *reinterpret_cast<const uint4*>(res + c));
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (col0 + c + i < g.n) x[i] += to_f32(res[c + i]);
                        }
                    }
                }
                uint4 w;
                w.x = pack2<T>(x[0], x[1]);
                w.y = pack2<T>(x[2], x[3]);
                w.z = pack2<T>(x[4], x[5]);
                w.w = pack2<T>(x[6], x[7]);
                *reinterpret_cast<uint4*>(mine + (((half * 4 + v) ^ sw) << 4)) = w;
            }
        }
        if (pass == 0 ? p.tma_z : p.tma_out) {
            fence_to_async();
            __syncwarp();
            if (lane == 0) tma_store(pass == 0 ? &p.z : &p.out, smem_addr(block), col0, row0);
        } else {
            __syncwarp();
            T* out = static_cast<T*>(pass == 0 ? g.z_out : g.out);
            const int64_t stride = pass == 0 ? g.z_stride : g.out_stride;
            for (int r = 0; r < 32 && row0 + r < g.m; ++r) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = h * 32 + lane;
                    const T v = *reinterpret_cast<const T*>(block + r * 128 + (((c >> 3) ^ (r & 7)) << 4) + (c & 7) * 2);
                    if (col0 + c < g.n) out[(row0 + r) * stride + col0 + c] = v;
                }
            }
            __syncwarp();
        }
    }
}

// Persistent: cluster i takes tiles i, i + clusters, ...  Warps 0-7 drain
// accumulators, warp 8 loads operands, warp 9 issues the MMAs; two
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
    tcgen05_before_sync();
    if (CG == 2) cluster_sync_all();
    else __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = tmem_slot;

    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    const int64_t first = blockIdx.x / CG, step = gridDim.x / CG;
    const int kts = (g.k + kBK - 1) / kBK;
    auto tile_at = [&](int64_t t, int& row0, int& col0) {
        col0 = (int)(t % p.tiles_n) * BN;
        row0 = (int)(t / p.tiles_n) * (kBM * CG) + (int)rank * kBM;
    };

    if (warp == kEpilogueWarps && lane == 0) {
        prefetch_map(&p.a);
        prefetch_map(&p.b);
        int s = 0;
        uint32_t parity = 1;  // a fresh barrier's previous phase counts as done
        bool ok = true;
        for (int64_t t = first; t < tiles && ok; t += step) {
            int row0, col0;
            tile_at(t, row0, col0);
            const int b0 = col0 + (int)rank * S::kRowsB;
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
    } else if (warp == kEpilogueWarps + 1 && lane == 0 && rank == 0) {
        const uint32_t idesc = instruction_desc(kIsBf16<T>, g.a_kmajor, g.b_kmajor, kBM * CG, BN);
        int s = 0, i = 0;
        uint32_t parity = 0, acc_parity = 1;
        bool ok = true;
        for (int64_t t = first; t < tiles && ok; t += step) {
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
        char* block = staging + warp * (32 * 128);
        T* bias = reinterpret_cast<T*>(staging + kEpilogueWarps * (32 * 128)) + warp * 64;
        const int quarter = warp & 3, half = warp >> 2;
        int i = 0;
        uint32_t parity = 0;
        for (int64_t t = first; t < tiles; t += step) {
            int row0, col0;
            tile_at(t, row0, col0);
            if (!mbar_wait(acc_full(i), parity, &gave_up)) break;
            __syncwarp();
            tcgen05_after_sync();
            for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 64)
                if (row0 + quarter * 32 < g.m && col0 + c < g.n)
                    epilogue_block<T>(p, tmem + i * BN + c + ((uint32_t)(quarter * 32) << 16), row0 + quarter * 32,
                                      col0 + c, block, bias);
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(CG == 2 ? cluster_map(acc_empty(i), 0) : acc_empty(i));
            i ^= 1;
            if (i == 0) parity ^= 1;
        }
        if (lane == 0) tma_store_wait();
    }
    __syncwarp();
    if (gave_up) {  // what is still in flight lands before the CTA's memory is given back
        if (threadIdx.x == 0) g_gave_up = 1;
        outlast_copies();
    }
    tcgen05_before_sync();
    if (CG == 2) cluster_sync_all();
    else __syncthreads();
    tcgen05_after_sync();
    if (warp == kEpilogueWarps + 1) tmem_free<CG>(tmem, S::kTmemCols);
}

// ---- few rows: the weight's rows are the tile's 128 TMEM lanes ---------------
//
// out^T = B' A'^T with the roles swapped: `a` of the arguments is the operand
// with few rows (k-major, at most BN), `b` the weight.  A cluster of S CTAs
// splits k; each CTA leaves a partial 128 x BN sum in TMEM, sends every CTA
// its share of the columns through distributed shared memory, and finishes
// its own share, adding the partial sums in rank order.

constexpr int kFewThreads = 32 * 6;

template <int BN>
struct FewShape {
    static constexpr uint32_t kBytesW = kBM * kBK * 2, kBytesX = BN * kBK * 2, kStage = kBytesW + kBytesX;
    static constexpr uint32_t kExchange = kBM * BN * 4;
    // two CTAs per SM where the columns are few
    static constexpr uint32_t kBudget = (BN <= 64 ? 113 * 1024 : kMaxSmem) - 1024 - 512 - kExchange;
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
    const int n0 = (int)(blockIdx.x / splits) * kBM;
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
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = tmem_slot;

    if (warp == 4 && lane == 0) {
        prefetch_map(&p.a);
        prefetch_map(&p.b);
        int s = 0;
        uint32_t parity = 1;
        for (int kt = kt0; kt < kt1; ++kt) {
            if (!mbar_wait(empty(s), parity, &gave_up)) break;
            mbar_expect(full(s), S::kStage);
            const uint32_t dst = stages + s * S::kStage;
            load_operand<1>(dst, &p.b, g.b_kmajor, kBM, n0, kt * kBK, full(s));
            load_operand<1>(dst + S::kBytesW, &p.a, true, BN, 0, kt * kBK, full(s));
            if (++s == S::kStages) {
                s = 0;
                parity ^= 1;
            }
        }
    } else if (warp == 5 && lane == 0) {
        const uint32_t idesc = instruction_desc(kIsBf16<T>, g.b_kmajor, true, kBM, BN);
        int s = 0;
        uint32_t parity = 0;
        for (int kt = kt0; kt < kt1; ++kt) {
            if (!mbar_wait(full(s), parity, &gave_up)) break;
            tcgen05_after_sync();
            const uint32_t src = stages + s * S::kStage;
            stage_mma<1>(tmem, src, src + S::kBytesW, g.b_kmajor, true, idesc, kt == kt0);
            mma_commit<1>(empty(s));
            if (++s == S::kStages) {
                s = 0;
                parity ^= 1;
            }
        }
        mma_commit<1>(done);
    }
    __syncwarp();
    const int share = BN / splits;  // columns that each CTA finishes
    if (warp < 4) {
        if (mbar_wait(done, 0, &gave_up)) {
            __syncwarp();
            tcgen05_after_sync();
            const int lane_n = warp * 32 + lane;
#pragma unroll
            for (int c0 = 0; c0 < BN; c0 += 16) {
                uint32_t raw[16];
                tmem_ld16(tmem + ((uint32_t)(warp * 32) << 16) + c0, raw);
                tmem_ld_wait(raw);
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const int col = c0 + c, to = col / share;
                    const uint32_t at = smem_addr(exchange + ((rank * share + col % share) * kBM + lane_n));
                    if (splits == 1) exchange[col * kBM + lane_n] = __uint_as_float(raw[c]);
                    else st_cluster_f32(cluster_map(at, to), __uint_as_float(raw[c]));
                }
            }
        }
        tcgen05_before_sync();
    }
    __syncwarp();
    if (gave_up) {
        if (threadIdx.x == 0) g_gave_up = 1;
        outlast_copies();
    }
    if (splits > 1) cluster_sync_all();  // every partial sum has arrived; no CTA's memory is written after this
    else __syncthreads();
    if (warp < 4) {
        const int n = n0 + warp * 32 + lane;
        const float bias = g.bias && n < g.n ? to_f32(static_cast<const T*>(g.bias)[n]) : 0.f;
        for (int c = 0; c < share; ++c) {
            const int m = rank * share + c;
            if (m >= g.m || n >= g.n) break;
            float z = 0.f;
            for (int r = 0; r < splits; ++r) z += exchange[(r * share + c) * kBM + warp * 32 + lane];
            z += bias;
            if (g.z_out) static_cast<T*>(g.z_out)[m * g.z_stride + n] = from_f32<T>(z);
            float y = activate(z, g.act);
            if (g.residual) y += to_f32(static_cast<const T*>(g.residual)[m * g.residual_stride + n]);
            static_cast<T*>(g.out)[m * g.out_stride + n] = from_f32<T>(y);
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

// Tensor map of a 16-bit matrix with boxes of box_rows x 64 columns.
int make_map(CUtensorMap* map, int dtype, const void* p, int64_t stride, int64_t rows, int64_t cols, int box_rows) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return cudaErrorNotSupported;
    if (rows <= 1) stride = (cols + 7) / 8 * 8;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, steps[2] = {1, 1};
    const CUresult r = fn(map, dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                          const_cast<void*>(p), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int operand_map(CUtensorMap* map, const GemmArgs& g, const void* p, int64_t stride, bool kmajor, int64_t rows,
                int box_rows) {
    return kmajor ? make_map(map, g.dtype, p, stride, rows, g.k, box_rows)
                  : make_map(map, g.dtype, p, stride, g.k, rows, kBK);
}

int launch(const void* kernel, void** args, int grid, int threads, uint32_t smem, int cluster, void* stream) {
    int e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
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
    if (p.tma_out && (e = make_map(&p.out, g.dtype, g.out, g.out_stride, g.m, g.n, 32))) return e;
    if (p.tma_z && (e = make_map(&p.z, g.dtype, g.z_out, g.z_stride, g.m, g.n, 32))) return e;
    p.tiles_m = (g.m + kBM * CG - 1) / (kBM * CG);
    p.tiles_n = (g.n + BN - 1) / BN;
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    const int64_t workers = std::max(1, sm_count / CG);
    void* args[] = {&p};
    return launch((const void*)tile_kernel<CG, BN, T>, args, CG * (int)std::min(tiles, workers), kTileThreads,
                  S::kSmem, CG, stream);
}

template <int BN, typename T>
int launch_few(TileArgs& p, int sm_count, void* stream) {
    using S = FewShape<BN>;
    const GemmArgs& g = p.g;
    int e;
    if ((e = operand_map(&p.a, g, g.a, g.a_stride, true, g.m, BN)) ||
        (e = operand_map(&p.b, g, g.b, g.b_stride, g.b_kmajor, g.n, kBM)))
        return e;
    const int tiles = (g.n + kBM - 1) / kBM, kts = (g.k + kBK - 1) / kBK;
    int splits = 1;
    while (splits < 8 && 2 * splits <= kts && tiles * splits * 2 <= 2 * sm_count) splits *= 2;
    void* args[] = {&p, &splits};
    return launch((const void*)few_kernel<BN, T>, args, tiles * splits, kFewThreads, S::kSmem, splits, stream);
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

bool gemm_operand_needs_copy(const void* p, int64_t stride, int64_t rows) { return !aligned_rows(p, stride, rows); }

int launch_repack(const void* src, int64_t src_stride, void* dst, int64_t dst_stride, int64_t rows, int64_t cols,
                  void* stream) {
    const dim3 grid((unsigned)std::min<int64_t>((cols + 255) / 256, 64), (unsigned)std::min<int64_t>(rows, 2048));
    repack_kernel<uint16_t><<<grid, 256, 0, (cudaStream_t)stream>>>(static_cast<const uint16_t*>(src), src_stride,
                                                                   static_cast<uint16_t*>(dst), dst_stride, rows,
                                                                   (int32_t)cols);
    return (int)cudaGetLastError();
}

int launch_gemm(const GemmArgs& a, int sm_count, void* stream) {
    return with_type16(a.dtype, [&](auto t) {
        using T = decltype(t);
        TileArgs p{};
        p.g = a;
        if (a.a_kmajor && a.m <= 128) {
            if (a.m <= 16) return launch_few<16, T>(p, sm_count, stream);
            if (a.m <= 32) return launch_few<32, T>(p, sm_count, stream);
            if (a.m <= 64) return launch_few<64, T>(p, sm_count, stream);
            return launch_few<128, T>(p, sm_count, stream);
        }
        const int64_t big = (int64_t)((a.m + 255) / 256) * ((a.n + 255) / 256);
        if (big * 2 >= sm_count) return launch_tile<2, 256, T>(p, sm_count, stream);
        return launch_tile<1, 128, T>(p, sm_count, stream);
    });
}

int take_linear_gave_up(int* value) {
    int e = cudaMemcpyFromSymbol(value, g_gave_up, sizeof(int));
    if (e == cudaSuccess && *value) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_gave_up, &zero, sizeof(int));
    }
    return e;
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
