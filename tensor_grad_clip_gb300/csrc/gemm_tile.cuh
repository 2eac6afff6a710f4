// Matrix products of 16-bit operands on the tensor cores: tiles, their
// pipeline, and the host's side of TMA.  What becomes of a tile's sums is the
// caller's.
#pragma once

#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "ops_device.cuh"
#include "ops_kernels.h"
#include "tcgen05.cuh"

namespace soma {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
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

// Lets the next kernel of the stream be set up, and waits until the one
// before it is done and its results are visible.
__device__ __forceinline__ void follow_stream() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

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

// What a product has to do: m rows (those of 32 that begin below it are
// drained), k values a sum, tiles, of which those from `whole` on are done in
// two halves of their columns, walked through in strips of `strip` columns of
// tiles; or, with splits > 1 (then whole = all tiles), every tile once for each
// part of k.  The sum of a unit is handed over every `chunk` stages, anew each
// time.
struct TilePlan {
    int m, k, tiles_m, tiles_n, strip, whole, splits, chunk;
};
constexpr int kOneChunk = 1 << 26;  // stages: more than any sum has

// ---- a tile of 128 x BN (CG = 1) or 256 x BN (CG = 2) ------------

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

// Persistent: cluster i takes units i, i + clusters, ...  Warps 0-15 drain
// accumulators, the next loads operands, the last issues the MMAs; two
// accumulators in TMEM let a tile's epilogue run under the next tile's MMAs.
// CG = 2: a pair of CTAs shares one 256-row tile, each staging half of both
// operands; the leader (rank 0) issues the MMAs for both.
//
// plan() says what there is to do, once the kernels before this one are done
// (a row count may come from one of them).  Each warp of the first sixteen
// calls drain(accumulator's address, part, staging, done) for its 32 rows of a
// unit (or of a chunk of it), which calls done() when it has read the
// accumulator.  `columns` (0 = BN) is the width of tiles narrower than BN, a
// multiple of 32; CG = 1 and no halves then.
struct Part {
    int row0, col0, cols, split;
    bool first, last;  // of the unit's chunks
};
template <int CG, int BN, typename T, typename Plan, typename Drain>
__device__ __forceinline__ void tile_products(const CUtensorMap* map_a, const CUtensorMap* map_b, bool a_kmajor,
                                              bool b_kmajor, Plan&& make_plan, Drain&& drain, int columns = 0) {
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
        prefetch_map(map_a);
        prefetch_map(map_b);
    }
    tcgen05_before_sync();
    if (CG == 2) cluster_sync_all();
    else __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = tmem_slot;
    follow_stream();

    // units of work: whole tiles, then halves; or every part of k of every tile
    const TilePlan p = make_plan();
    const int tiles = p.tiles_m * p.tiles_n, units = (2 * tiles - p.whole) * p.splits;
    const int first = blockIdx.x / CG, step = gridDim.x / CG;
    const int all_kts = (p.k + kBK - 1) / kBK;
    auto kt_begin = [&](int u) { return p.splits == 1 ? 0 : (int)((int64_t)(u / tiles) * all_kts / p.splits); };
    auto kt_end = [&](int u) { return p.splits == 1 ? all_kts : (int)((int64_t)(u / tiles + 1) * all_kts / p.splits); };
    const int bn = columns ? columns : BN;
    const uint32_t stage_bytes = columns ? S::kBytesA + columns * kBK * 2 : S::kStage;
    auto tile_at = [&](int u, int& row0, int& col0) {  // returns the unit's columns
        if (p.splits > 1) u %= tiles;
        const bool half = u >= p.whole;
        const int t = half ? p.whole + (u - p.whole) / 2 : u;
        const int strip = t / (p.tiles_m * p.strip) * p.strip, width = min(p.strip, p.tiles_n - strip);
        const int in_strip = t - strip * p.tiles_m;
        col0 = (strip + in_strip % width) * bn + (half && (u - p.whole) % 2 ? BN / 2 : 0);
        row0 = in_strip / width * (kBM * CG) + (int)rank * kBM;
        return half ? BN / 2 : bn;
    };

    if (warp == kEpilogueWarps && lane == 0) {
        int s = 0;
        uint32_t parity = 1;  // a fresh barrier's previous phase counts as done
        bool ok = true;
        for (int u = first; u < units && ok; u += step) {
            int row0, col0;
            // (of a half, the second half of B's rows is loaded and not used)
            const int b0 = tile_at(u, row0, col0) / CG * (int)rank + col0;
            const int kt1 = kt_end(u);
            for (int kt = kt_begin(u); kt < kt1; ++kt) {
                if (!(ok = mbar_wait(empty(s), parity, &gave_up))) break;
                const uint32_t bar = CG == 2 ? cluster_map(full(s), 0) : full(s);
                if (rank == 0) mbar_expect(full(s), CG * stage_bytes);
                const uint32_t dst = stages + s * S::kStage;
                load_operand<CG>(dst, map_a, a_kmajor, kBM, row0, kt * kBK, bar);
                load_operand<CG>(dst + S::kBytesA, map_b, b_kmajor, S::kRowsB, b0, kt * kBK, bar);
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
                instruction_desc(kIsBf16<T>, a_kmajor, b_kmajor, kBM * CG, p.splits == 1 && u >= p.whole ? BN / 2 : bn);
            const int kt0 = kt_begin(u), kt1 = kt_end(u);
            for (int c0 = kt0; c0 < kt1 && ok; c0 += p.chunk) {
                if (!(ok = mbar_wait(acc_empty(i), acc_parity, &gave_up))) break;
                tcgen05_after_sync();
                const int c1 = min(kt1, c0 + p.chunk);
                for (int kt = c0; kt < c1; ++kt) {
                    if (!(ok = mbar_wait(full(s), parity, &gave_up))) break;
                    tcgen05_after_sync();
                    const uint32_t src = stages + s * S::kStage;
                    stage_mma<CG>(tmem + i * BN, src, src + S::kBytesA, a_kmajor, b_kmajor, idesc, kt == c0);
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
        }
    } else if (warp < kEpilogueWarps) {
        const int quarter = warp & 3;
        int i = 0;
        uint32_t parity = 0;
        bool ok = true;
        for (int u = first; u < units && ok; u += step) {
            Part part;
            int row0, col0;
            // the warp's columns: a quarter of the tile's (of narrow tiles, of BN's)
            const int width = tile_at(u, row0, col0), quarter_cols = (columns ? BN : width) / (kEpilogueWarps / 4);
            const int at = (warp >> 2) * quarter_cols;
            part.row0 = row0 + quarter * 32;
            part.col0 = col0 + at;
            part.cols = min(quarter_cols, width - at);
            part.split = p.splits == 1 ? 0 : u / tiles;
            const int kt0 = kt_begin(u), kt1 = kt_end(u);
            for (int c0 = kt0; c0 < kt1; c0 += p.chunk) {
                if (!(ok = mbar_wait(acc_full(i), parity, &gave_up, product_limit(all_kts)))) break;
                __syncwarp();
                tcgen05_after_sync();
                part.first = c0 == kt0;
                part.last = kt1 - c0 <= p.chunk;
                auto done = [&] {
                    tcgen05_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(CG == 2 ? cluster_map(acc_empty(i), 0) : acc_empty(i));
                };
                if (part.row0 < p.m && part.cols > 0)
                    drain(tmem + i * BN + at + ((uint32_t)(quarter * 32) << 16), part, staging, done);
                else
                    done();
                i ^= 1;
                if (i == 0) parity ^= 1;
            }
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

int launch_cluster(const void* kernel, void** args, int grid, int threads, uint32_t smem, int cluster, void* stream) {
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

}  // namespace
}  // namespace soma
