// Softmax cross entropy of a linear layer over a large vocabulary (formulas in
// soma_ops.h): logits are made on the tensor cores, a tile at a time, and used
// where they are, in registers.
//
//   select   rows that count are numbered, in order; what the others get is written
//   gather   those rows of x, one after the other on 16-byte boundaries: rows
//            that do not count cost nothing in the products, and what they
//            hold (NaN, say) reaches no gradient
//   stats    z = x W^T; maximum and sum of exponentials of every 32 logits
//   join     log-sum-exp and loss
// and for the gradients, for one piece of the vocabulary after the other,
//   dz       z again; dz = g (exp(z - lse) - [its token]), rounded to the
//            operands' 16 bits into a buffer of the piece's size; where one
//            piece is the whole vocabulary and the loss is wanted too, `stats`
//            leaves exp(z - the 32 logits' maximum) there, and a pass over the
//            buffer makes dz of it, instead of a fourth product
//   dweight  dz^T x, the piece's rows, complete
//   dx       dz W added to fp32 sums, which a last kernel rounds
// The number of rows that count is only known on the device: the products read
// it there.
#include <math.h>

#include <algorithm>

#include "gemm_tile.cuh"
#include "soma_ops.h"

namespace soma {
namespace {

constexpr float kLowest = -3.402823466e38f;

// What `select` finds out.
struct Counted {
    int32_t rows;           // that count
    int32_t padded;         // the next multiple of 64, 64 at least: what the products run over
    float scale, unscale;   // a power of two that brings the largest |g| to about 2^14, and its inverse
};

// Row pointers are numbered by counted rows, up to Counted::padded.
struct HeadRows {
    Counted* counted;
    int32_t* row;           // its number among all rows, -1 in the padding
    int32_t* place;         // [all rows] the counted row's number, or -1
    int32_t* token;         // -1 in the padding
    float* weight;          // row_weight
    float* g;               // row_weight * grad_loss
    float* lse;
    float* z_token;         // its token's logit
};

constexpr int kSelectThreads = 1024, kSelectEach = 4;

__device__ __forceinline__ int64_t token_of(const TokenArgs& t, int64_t r) {
    const int64_t at = t.length == t.stride ? r : r / t.length * t.stride + r % t.length;
    return t.type == SOMA_INDEX_I64 ? (int64_t)__ldg(static_cast<const long long*>(t.index) + at)
                                    : (int64_t)__ldg(static_cast<const int*>(t.index) + at);
}

// One CTA: it has a few microseconds' work where the products have hundreds.
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ HeadArgs a, HeadRows h) {
    __shared__ int sums[32];
    __shared__ float tops[32];
    follow_stream();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int done = 0;  // rows counted so far
    float top = 0.f;
    for (int64_t base = 0; base < a.rows; base += kSelectThreads * kSelectEach) {
        const int64_t r0 = base + threadIdx.x * kSelectEach;
        int token[kSelectEach], mine = 0;
        float weight[kSelectEach], g[kSelectEach];
#pragma unroll
        for (int q = 0; q < kSelectEach; ++q) {
            token[q] = -1;
            weight[q] = g[q] = 0.f;
            if (r0 + q >= a.rows) continue;
            const int64_t t = token_of(a.tokens, r0 + q);
            weight[q] = a.row_weight ? a.row_weight[r0 + q] : 1.f;
            g[q] = a.grad_loss ? a.grad_loss[r0 + q] : 1.f;
            const bool counts = t >= 0 && t < a.vocab && weight[q] != 0.f && g[q] != 0.f;
            if (counts) {
                token[q] = (int)t;
                g[q] *= weight[q];
                if (isfinite(g[q])) top = fmaxf(top, fabsf(g[q]));
                ++mine;
            } else {
                h.place[r0 + q] = -1;
                if (a.loss) a.loss[r0 + q] = 0.f;
                if (a.lse) a.lse[r0 + q] = 0.f;
            }
        }
        int before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += t;
        }
        if (lane == 31) sums[warp] = before;
        __syncthreads();
        int total = 0, earlier = 0;
        for (int w = 0; w < kSelectThreads / 32; ++w) {
            if (w == warp) earlier = total;
            total += sums[w];
        }
        int at = done + earlier + before - mine;
#pragma unroll
        for (int q = 0; q < kSelectEach; ++q) {
            if (token[q] < 0) continue;
            h.row[at] = (int)(r0 + q);
            h.place[r0 + q] = at;
            h.token[at] = token[q];
            h.weight[at] = weight[q];
            h.g[at] = g[q];
            if (a.lse_in) h.lse[at] = a.lse_in[r0 + q];
            ++at;
        }
        done += total;
        __syncthreads();
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    const int padded = max(64, (done + 63) / 64 * 64);
    for (int i = done + threadIdx.x; i < padded; i += kSelectThreads) {
        h.row[i] = h.token[i] = -1;
        h.weight[i] = h.g[i] = h.lse[i] = 0.f;
    }
    if (threadIdx.x == 0) {
        for (int w = 1; w < kSelectThreads / 32; ++w) top = fmaxf(top, tops[w]);
        int e = 0;
        if (top > 0.f) frexpf(top, &e);
        e = min(max(14 - e, -100), 100);
        *h.counted = {done, padded, ldexpf(1.f, e), ldexpf(1.f, -e)};
    }
}

// The counted rows of x, and zeros in the padding: a warp copies 32 vectors.
template <typename T>
__global__ void __launch_bounds__(256) gather_kernel(const T* x, int64_t stride, int64_t rows, int32_t cols, T* out,
                                                     int64_t out_stride, HeadRows h, int pieces) {
    follow_stream();
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int to = (int)(item / pieces), i = (int)(item - (int64_t)to * pieces) * 32 + (threadIdx.x & 31);
    if (to >= h.counted->padded || i * 8 >= cols) return;
    const int from = h.row[to];
    uint4 v = make_uint4(0, 0, 0, 0);
    if (from >= 0) {
        const RowReader<T, false> row(x, stride, rows, from, cols);
        if (i >= row.inner_begin && i < row.inner_end) {
            v = row.words[i];
            if (row.phase) v = shifted<T>(v, row.words[i + 1], row.phase);
        } else {
            float e[8];
            row.gather(i, e, 0.f);
            v = narrow16(e, T{});
        }
    }
    reinterpret_cast<uint4*>(out + to * out_stride)[i] = v;
}

// ---- logits -------------------------------------------------------------------

struct LogitArgs {
    CUtensorMap a, b, out;
    HeadRows h;
    float2* parts;          // [rows][slices of 32 columns] maximum and sum of exponentials
    int64_t slices;
    bool keep;              // stats: store the exponentials too
    int32_t n, k;           // columns (of the piece), their first in the vocabulary, sum length
    int32_t first;
    int32_t tiles_n, strip;
};

// Rows of tiles, and where halves begin so that a last wave that at most half
// of the workers have is done by all.
template <int CG>
__device__ __forceinline__ TilePlan plan_rows(int rows, int k, int tiles_n, int strip, bool halves, int splits) {
    TilePlan p{rows, k, (rows + kBM * CG - 1) / (kBM * CG), tiles_n, strip, 0, splits};
    const int tiles = p.tiles_m * tiles_n, workers = (int)gridDim.x / CG, rest = tiles % workers;
    p.whole = halves && CG == 2 && splits == 1 && 2 * rest <= workers ? tiles - rest : tiles;
    return p;
}

// A row's 32 logits from column col on, out of TMEM; those past the end are -inf.
__device__ __forceinline__ void load_logits(uint32_t acc, int col, int n, float (&z)[32]) {
    uint32_t raw[32];
    tmem_ld32(acc, raw);
    tmem_ld_wait(raw);
#pragma unroll
    for (int i = 0; i < 32; ++i) z[i] = __uint_as_float(raw[i]);
    if (col + 32 > n) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (col + i >= n) z[i] = -INFINITY;
    }
}

// What the kept exponentials, at most 1, are multiplied by: fp16 has no
// small enough numbers for what a vocabulary's tail weighs.
template <typename T>
constexpr float kKeepScale = kIsBf16<T> ? 1.f : 16384.f;

template <int CG, int BN, typename T>
__global__ void __launch_bounds__(kTileThreads, 1) stats_kernel(const __grid_constant__ LogitArgs p) {
    tile_products<CG, BN, T>(
        &p.a, &p.b, true, true,
        [&] { return plan_rows<CG>(p.h.counted->padded, p.k, p.tiles_n, p.strip, true, 1); },
        [&](uint32_t acc, int row0, int col0, int cols, int, const TilePlan&, char* staging) {
            const int row = row0 + (threadIdx.x & 31);
            const int at = p.h.token[row] - col0;  // the token's column here
            Stager<T> stager{staging + (threadIdx.x >> 5) * kStagerBytes, row0, 0, p.n};
            for (int c = 0; c < cols && col0 + c < p.n; c += 32) {
                float z[32];
                load_logits(acc + c, col0 + c, p.n, z);
                float m = kLowest;
#pragma unroll
                for (int i = 0; i < 32; ++i) m = fmaxf(m, z[i]);
                const int d = at - c;
                if (__any_sync(0xffffffffu, d >= 0 && d < 32) && d >= 0 && d < 32) {
                    float t = z[0];
#pragma unroll
                    for (int i = 1; i < 32; ++i) t = d == i ? z[i] : t;
                    p.h.z_token[row] = t;
                }
                float even = 0.f, odd = 0.f;
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    z[i] = exp2_fast((z[i] - m) * kLog2e);
                    z[i + 1] = exp2_fast((z[i + 1] - m) * kLog2e);
                    even += z[i];
                    odd += z[i + 1];
                }
                p.parts[row * p.slices + (col0 + c) / 32] = make_float2(m, even + odd);
                if (p.keep) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) z[i] *= kKeepScale<T>;
                    stager.store(z, col0 + c, &p.out, true, nullptr, 0);
                }
            }
        });
}

__device__ __forceinline__ float2 join_stats(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x);
    return make_float2(m, a.y * exp2_fast((a.x - m) * kLog2e) + b.y * exp2_fast((b.x - m) * kLog2e));
}

// Log-sum-exp and loss of a counted row per CTA.
constexpr int kJoinWarps = 4;
__global__ void __launch_bounds__(32 * kJoinWarps) stats_join_kernel(const float2* parts, int64_t slices, HeadRows h,
                                                                     float* loss, float* lse) {
    __shared__ float2 sums[kJoinWarps];
    follow_stream();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.x;
    if (i >= h.counted->rows) return;
    float2 own = make_float2(kLowest, 0.f);
#pragma unroll 8
    for (int64_t q = threadIdx.x; q < slices; q += 32 * kJoinWarps) own = join_stats(own, __ldcg(parts + i * slices + q));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        own = join_stats(own, make_float2(__shfl_xor_sync(0xffffffffu, own.x, o), __shfl_xor_sync(0xffffffffu, own.y, o)));
    if (lane == 0) sums[warp] = own;
    __syncthreads();
    if (threadIdx.x) return;
    for (int w = 1; w < kJoinWarps; ++w) own = join_stats(own, sums[w]);
    const float log_s = logf(own.y), total = own.x + log_s;
    const int r = h.row[i];
    h.lse[i] = total;
    if (lse) lse[r] = total;
    // (m - z) + log s: near 0 it keeps its digits where lse - z would not
    if (loss) loss[r] = h.weight[i] * ((own.x - h.z_token[i]) + log_s);
}

// dz of the kept exponentials, in place: a thread 8 of them.  What rounding
// them once more costs is at most another half step of 16 bits; the token's
// own element, a difference from 1, is made of its logit.
template <typename T>
__global__ void __launch_bounds__(256) keep_kernel(T* dz, int64_t stride, const float2* parts, int64_t slices, HeadRows h,
                                                   int32_t n) {
    follow_stream();
    const int row = blockIdx.y;
    if (row >= h.counted->padded) return;
    const int c = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 8;
    if (c >= n) return;
    const float lse = h.lse[row], g = h.g[row] * h.counted->scale;
    const float f = g * (1.f / kKeepScale<T>) * exp2_fast((__ldg(&parts[row * slices + c / 32].x) - lse) * kLog2e);
    uint4* at = reinterpret_cast<uint4*>(dz + row * stride + c);
    float x[8];
    widen16(*at, x, T{});
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= f;
    const int d = h.token[row] - c;
    if (d >= 0 && d < 8) {
        const float own = g * (exp2_fast((h.z_token[row] - lse) * kLog2e) - 1.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = d == i ? own : x[i];
    }
    *at = narrow16(x, T{});
}

// dz of a piece, scaled.
template <int CG, int BN, typename T>
__global__ void __launch_bounds__(kTileThreads, 1) dz_kernel(const __grid_constant__ LogitArgs p) {
    tile_products<CG, BN, T>(
        &p.a, &p.b, true, true,
        [&] { return plan_rows<CG>(p.h.counted->padded, p.k, p.tiles_n, p.strip, true, 1); },
        [&](uint32_t acc, int row0, int col0, int cols, int, const TilePlan&, char* staging) {
            const int row = row0 + (threadIdx.x & 31);
            const int at = p.h.token[row] - p.first - col0;
            const float lse = p.h.lse[row], g = p.h.g[row] * p.h.counted->scale;
            Stager<T> stager{staging + (threadIdx.x >> 5) * kStagerBytes, row0, 0, p.n};
            for (int c = 0; c < cols && col0 + c < p.n; c += 32) {
                float z[32];
                load_logits(acc + c, col0 + c, p.n, z);
                const int d = at - c;
                const bool here = __any_sync(0xffffffffu, d >= 0 && d < 32);
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] = g * exp2_fast((z[i] - lse) * kLog2e);
                if (here) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (d == i) z[i] -= g;
                }
                stager.store(z, col0 + c, &p.out, true, nullptr, 0);
            }
        });
}

// ---- gradients ------------------------------------------------------------------

struct GradArgs {
    CUtensorMap a, b, out;
    HeadRows h;
    float* sums;            // dx: [splits][pitch rows][sums_stride]
    int64_t pitch, sums_stride;
    bool add;               // dx: to what is there
    void* dweight;          // its piece
    int64_t dweight_stride;
    bool tma_out;
    int32_t m, n, k;        // dweight: m; dx: k (the others are the device's)
    int32_t tiles_m, tiles_n, strip, splits;
};

template <int CG, int BN, typename T>
__global__ void __launch_bounds__(kTileThreads, 1) dweight_kernel(const __grid_constant__ GradArgs p) {
    tile_products<CG, BN, T>(
        &p.a, &p.b, false, false,
        [&] { return plan_rows<CG>(p.m, p.h.counted->padded, p.tiles_n, p.strip, true, 1); },
        [&](uint32_t acc, int row0, int col0, int cols, int, const TilePlan&, char* staging) {
            const float unscale = p.h.counted->unscale;
            Stager<T> stager{staging + (threadIdx.x >> 5) * kStagerBytes, row0, p.m, p.n};
            for (int c = 0; c < cols && col0 + c < p.n; c += 32) {
                uint32_t raw[32];
                tmem_ld32(acc + c, raw);
                tmem_ld_wait(raw);
                float x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(raw[i]) * unscale;
                stager.store(x, col0 + c, &p.out, p.tma_out, static_cast<T*>(p.dweight), p.dweight_stride);
            }
        });
}

// A lane's row of 32 sums, 32 bytes at a time (rows of sums start on 32-byte boundaries).
__device__ __forceinline__ void add_or_store(float* to, const uint32_t (&raw)[32], bool add) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(raw[8 * v + i]);
        if (add) {
            float y[8];
            asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=f"(y[0]), "=f"(y[1]), "=f"(y[2]), "=f"(y[3]), "=f"(y[4]), "=f"(y[5]), "=f"(y[6]), "=f"(y[7])
                         : "l"(to + 8 * v)
                         : "memory");
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] += y[i];
        }
        asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to + 8 * v), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                     "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                     : "memory");
    }
}

template <int CG, int BN, typename T>
__global__ void __launch_bounds__(kTileThreads, 1) dx_kernel(const __grid_constant__ GradArgs p) {
    tile_products<CG, BN, T>(
        &p.a, &p.b, true, false,
        [&] { return plan_rows<CG>(p.h.counted->padded, p.k, p.tiles_n, p.strip, true, p.splits); },
        [&](uint32_t acc, int row0, int col0, int cols, int split, const TilePlan&, char*) {
            float* to = p.sums + (split * p.pitch + row0 + (threadIdx.x & 31)) * p.sums_stride;
            // (the sums' rows are as long as whole tiles)
            for (int c = 0; c < cols && col0 + c < p.n; c += 32) {
                uint32_t raw[32];
                tmem_ld32(acc + c, raw);
                tmem_ld_wait(raw);
                add_or_store(to + col0 + c, raw, p.add);
            }
        });
}

// dx of all rows: the sums of the parts, unscaled and rounded; 0 for rows that
// do not count.
template <typename T>
__global__ void __launch_bounds__(256) dx_round_kernel(const float* sums, int64_t pitch, int64_t sums_stride, int splits,
                                                       HeadRows h, T* dx, int64_t dx_stride, int64_t rows, int32_t cols,
                                                       int pieces) {
    follow_stream();
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t r = item / pieces;
    const int c = ((int)(item - r * pieces) * 32 + (threadIdx.x & 31)) * 8;
    if (r >= rows || c >= cols) return;
    const int at = h.place[r];
    float x[8] = {};
    if (at >= 0) {
        for (int s = 0; s < splits; ++s) {
            const float4* from = reinterpret_cast<const float4*>(sums + (s * pitch + at) * sums_stride + c);
            const float4 u = __ldcs(from), v = __ldcs(from + 1);
            x[0] += u.x; x[1] += u.y; x[2] += u.z; x[3] += u.w;
            x[4] += v.x; x[5] += v.y; x[6] += v.z; x[7] += v.w;
        }
        const float unscale = h.counted->unscale;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= unscale;
    }
    T* to = dx + r * dx_stride + c;
    if ((uintptr_t)to % 16 == 0 && c + 8 <= cols) {
        *reinterpret_cast<uint4*>(to) = narrow16(x, T{});
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) to[i] = from_f32<T>(x[i]);
    }
}

// ---- host side ----------------------------------------------------------------------

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// The buffer for a piece's dz: half a gigabyte or as much as the weight has,
// or what one column of tiles needs.
constexpr int64_t kPieceBytes = 512ll << 20;

struct HeadLayout {
    int64_t counted, row, place, token, weight, g, lse, z_token, x, w, parts, dz, sums, bytes;
    int64_t pitch;                   // rows, rounded up to whole tiles
    int64_t x_stride, w_stride, sums_stride;
    int64_t piece, pieces;           // columns of the vocabulary
    int32_t splits;                  // parts of the vocabulary in which dx is summed side by side
    bool big;                        // tiles on pairs of SMs
    HeadLayout(int64_t rows, int64_t vocab, int64_t k, bool copy_weight, bool forward, bool dx, bool dweight, int sms) {
        pitch = (rows + 255) / 256 * 256;
        // As for a linear layer: a 256 x 256 tile on two SMs takes as long as a
        // 128 x 128 tile on one, so the fewer waves win.
        const int64_t pairs = std::max(1, sms / 2);
        const int64_t t256 = (rows + 255) / 256 * ((vocab + 255) / 256), t128 = (rows + 127) / 128 * ((vocab + 127) / 128);
        big = rows > 128 && (t256 + pairs - 1) / pairs < (t128 + sms - 1) / sms;
        const int64_t buffer = std::max(kPieceBytes, vocab * k * 2);
        const int64_t most = std::max<int64_t>(256, buffer / (2 * pitch) / 256 * 256);
        pieces = (vocab + most - 1) / most;
        piece = ((vocab + pieces - 1) / pieces + 255) / 256 * 256;
        pieces = (vocab + piece - 1) / piece;
        // dx has few tiles and long sums: parts of the sums make the last wave
        // full, or the only one.  (A part more costs its share of writing and
        // reading the sums, about as much as four of its pipeline stages.)
        const int64_t edge = big ? 256 : 128, workers = big ? pairs : sms, kts = std::min(piece, vocab) / kBK + 1;
        const int64_t tiles = (rows + edge - 1) / edge * ((k + edge - 1) / edge);
        splits = 1;
        double least = 0;
        for (int s = 1; s <= 16 && kts >= 16 * s && tiles <= 4 * workers; ++s) {
            const double time = (double)((tiles * s + workers - 1) / workers) * ((double)kts / s + 4) + 0.05 * kts * (s > 1);
            if (s == 1 || time < least) {
                least = time;
                splits = s;
            }
        }
        x_stride = (k + 7) / 8 * 8;
        w_stride = x_stride;
        sums_stride = (k + 255) / 256 * 256;
        int64_t at = 0;
        auto take = [&](int64_t n) { const int64_t here = at; at += align256(n); return here; };
        counted = take(sizeof(Counted));
        row = take(pitch * 4);
        place = take(rows * 4);
        token = take(pitch * 4);
        weight = take(pitch * 4);
        g = take(pitch * 4);
        lse = take(pitch * 4);
        z_token = take(pitch * 4);
        x = take(pitch * x_stride * 2);
        w = take(copy_weight ? vocab * w_stride * 2 : 0);
        parts = take(forward ? pitch * slices(vocab) * 8 : 0);
        dz = take(dx || dweight ? pitch * piece * 2 : 0);
        sums = take(dx ? splits * pitch * sums_stride * 4 : 0);
        bytes = at;
    }
    static int64_t slices(int64_t vocab) { return (vocab + 31) / 32; }
};

int launch_after(const void* kernel, dim3 grid, int threads, void** args, void* stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelExC(&cfg, kernel, args);
}

// Strips of columns of B of at most 48 MB, as for a linear layer.
int32_t strip_of(int64_t tiles_n, int bn, int64_t k) {
    const int64_t fit = std::max<int64_t>(1, (48ll << 20) / (bn * k * 2)), strips = (tiles_n + fit - 1) / fit;
    return (int32_t)((tiles_n + strips - 1) / strips);
}

template <int CG, int BN, typename T>
struct Head {
    using S = TileShape<CG, BN>;
    const HeadArgs& a;
    const HeadLayout& at;
    HeadRows h;
    char* ws;
    const void* w;
    int64_t w_stride;
    int sms;
    void* stream;

    int grid(int64_t units) const { return (int)std::max<int64_t>(1, std::min<int64_t>(units, sms / CG)) * CG; }
    int64_t rows_of_tiles(int64_t m) const { return (m + kBM * CG - 1) / (kBM * CG); }
    int tiles(const void* kernel, int64_t units, void** args) const {
        if (units > (1 << 29)) return cudaErrorInvalidValue;
        return launch_cluster(kernel, args, grid(units), kTileThreads, S::kSmem, CG, stream);
    }
    // z = x W^T over columns [first, first + n) of the vocabulary.
    int logits(LogitArgs& p, int64_t first, int64_t n, const void* kernel) const {
        p.h = h;
        p.slices = HeadLayout::slices(a.vocab);
        p.n = (int32_t)n;
        p.k = a.k;
        p.first = (int32_t)first;
        p.tiles_n = (int32_t)((n + BN - 1) / BN);
        p.strip = strip_of(p.tiles_n, BN, a.k);
        const char* b = static_cast<const char*>(w) + first * w_stride * 2;
        if (const int e = make_map(&p.a, a.dtype, ws + at.x, at.x_stride, at.pitch, a.k, kBM)) return e;
        if (const int e = make_map(&p.b, a.dtype, b, w_stride, n, a.k, S::kRowsB)) return e;
        void* args[] = {&p};
        // (half tiles make at most twice as many units)
        return tiles(kernel, rows_of_tiles(a.rows) * p.tiles_n * 2, args);
    }
    int forward(bool keep) const {
        LogitArgs p{};
        p.parts = reinterpret_cast<float2*>(ws + at.parts);
        p.keep = keep;
        int e = keep ? make_map(&p.out, a.dtype, ws + at.dz, at.piece, at.pitch, a.vocab, 32, 32) : cudaSuccess;
        if (!e) e = logits(p, 0, a.vocab, (const void*)stats_kernel<CG, BN, T>);
        if (e) return e;
        const float2* parts = p.parts;
        int64_t slices = p.slices, stride = at.piece;
        HeadRows rows = h;
        float *loss = a.loss, *lse = a.lse;
        void* args[] = {&parts, &slices, &rows, &loss, &lse};
        e = launch_after((const void*)stats_join_kernel, dim3((unsigned)a.rows), 32 * kJoinWarps, args, stream);
        if (e || !keep) return e;
        T* dz = reinterpret_cast<T*>(ws + at.dz);
        int32_t n = a.vocab;
        void* keep_args[] = {&dz, &stride, &parts, &slices, &rows, &n};
        return launch_after((const void*)keep_kernel<T>, dim3((a.vocab + 2047) / 2048, (unsigned)std::max<int64_t>(64, (a.rows + 63) / 64 * 64)),
                            256, keep_args, stream);
    }
    int gradients(bool kept) const {
        for (int64_t first = 0; first < a.vocab; first += at.piece) {
            const int64_t n = std::min<int64_t>(at.piece, a.vocab - first);
            int e = cudaSuccess;
            if (!kept) {
                LogitArgs p{};
                e = make_map(&p.out, a.dtype, ws + at.dz, at.piece, at.pitch, n, 32, 32);
                if (!e) e = logits(p, first, n, (const void*)dz_kernel<CG, BN, T>);
            }
            if (!e && a.dweight) e = dweight(first, n);
            if (!e && a.dx) e = dx(first, n);
            if (e) return e;
        }
        if (!a.dx) return cudaSuccess;
        const float* sums = reinterpret_cast<const float*>(ws + at.sums);
        int64_t pitch = at.pitch, sums_stride = at.sums_stride, stride = a.dx_stride, rows = a.rows;
        int splits = at.splits, pieces = (a.k + 255) / 256;
        int32_t cols = a.k;
        HeadRows hr = h;
        T* out = static_cast<T*>(a.dx);
        void* args[] = {&sums, &pitch, &sums_stride, &splits, &hr, &out, &stride, &rows, &cols, &pieces};
        const int64_t grid = (rows * pieces + 7) / 8;
        if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
        return launch_after((const void*)dx_round_kernel<T>, dim3((unsigned)grid), 256, args, stream);
    }
    int dweight(int64_t first, int64_t n) const {
        GradArgs p{};
        p.h = h;
        p.m = (int32_t)n;
        p.n = a.k;
        p.dweight = static_cast<T*>(a.dweight) + first * a.dweight_stride;
        p.dweight_stride = a.dweight_stride;
        p.tma_out = aligned_rows(p.dweight, a.dweight_stride, n);
        p.tiles_m = (int32_t)rows_of_tiles(n);
        p.tiles_n = (a.k + BN - 1) / BN;
        p.strip = strip_of(p.tiles_n, BN, a.rows);
        // both operands run along their rows' other dimension
        if (const int e = make_map(&p.a, a.dtype, ws + at.dz, at.piece, at.pitch, n, kBK)) return e;
        if (const int e = make_map(&p.b, a.dtype, ws + at.x, at.x_stride, at.pitch, a.k, kBK)) return e;
        if (p.tma_out)
            if (const int e = make_map(&p.out, a.dtype, p.dweight, a.dweight_stride, n, a.k, 32, 32)) return e;
        void* args[] = {&p};
        return tiles((const void*)dweight_kernel<CG, BN, T>, (int64_t)p.tiles_m * p.tiles_n * 2, args);
    }
    int dx(int64_t first, int64_t n) const {
        GradArgs p{};
        p.h = h;
        p.sums = reinterpret_cast<float*>(ws + at.sums);
        p.pitch = at.pitch;
        p.sums_stride = at.sums_stride;
        p.add = first > 0;
        p.n = a.k;
        p.k = (int32_t)n;
        // (a last piece that has less than a stage for each part is added to the first part's sums)
        p.splits = (n + kBK - 1) / kBK >= at.splits ? at.splits : 1;
        p.tiles_n = (a.k + BN - 1) / BN;
        p.strip = strip_of(p.tiles_n, BN, n);
        const char* b = static_cast<const char*>(w) + first * w_stride * 2;
        if (const int e = make_map(&p.a, a.dtype, ws + at.dz, at.piece, at.pitch, n, kBM)) return e;
        if (const int e = make_map(&p.b, a.dtype, b, w_stride, n, a.k, kBK)) return e;
        void* args[] = {&p};
        return tiles((const void*)dx_kernel<CG, BN, T>, rows_of_tiles(a.rows) * p.tiles_n * p.splits * 2, args);
    }
};

}  // namespace

int64_t head_workspace(const HeadArgs& a, bool forward, int sm_count) {
    return HeadLayout(a.rows, a.vocab, a.k, !aligned_rows(a.weight, a.weight_stride, a.vocab), forward, a.dx != nullptr,
                      a.dweight != nullptr, sm_count)
        .bytes;
}

int launch_head(const HeadArgs& a, bool forward, void* workspace, int sm_count, void* stream) {
    const bool copy = !aligned_rows(a.weight, a.weight_stride, a.vocab);
    const HeadLayout at(a.rows, a.vocab, a.k, copy, forward, a.dx != nullptr, a.dweight != nullptr, sm_count);
    char* ws = static_cast<char*>(workspace);
    auto i32 = [&](int64_t o) { return reinterpret_cast<int32_t*>(ws + o); };
    auto f32 = [&](int64_t o) { return reinterpret_cast<float*>(ws + o); };
    HeadRows h{reinterpret_cast<Counted*>(ws + at.counted), i32(at.row), i32(at.place), i32(at.token), f32(at.weight),
               f32(at.g), f32(at.lse), f32(at.z_token)};
    const void* w = a.weight;
    int64_t w_stride = a.weight_stride;
    int e;
    if (copy) {
        if ((e = launch_repack(a.weight, a.weight_stride, ws + at.w, at.w_stride, a.vocab, a.k, a.dtype, sm_count, stream)))
            return e;
        w = ws + at.w;
        w_stride = at.w_stride;
    }
    {
        HeadArgs copy_of = a;
        void* args[] = {&copy_of, &h};
        if ((e = launch_after((const void*)select_kernel, dim3(1), kSelectThreads, args, stream))) return e;
    }
    auto run = [&](auto t) -> int {
        using T = decltype(t);
        const T* x = static_cast<const T*>(a.x);
        T* out = reinterpret_cast<T*>(ws + at.x);
        int64_t stride = a.x_stride, rows = a.rows, out_stride = at.x_stride;
        int32_t cols = a.k;
        int pieces = (a.k + 255) / 256;
        void* args[] = {&x, &stride, &rows, &cols, &out, &out_stride, &h, &pieces};
        const int64_t padded = std::max<int64_t>(64, (a.rows + 63) / 64 * 64);
        const int64_t grid = (padded * pieces + 7) / 8;
        if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
        if (const int e = launch_after((const void*)gather_kernel<T>, dim3((unsigned)grid), 256, args, stream)) return e;
        auto products = [&](const auto& head) {
            const bool gradients = a.dx || a.dweight;
            // (a row of the pass over the kept exponentials is a row of its grid)
            const bool keep = forward && gradients && at.pieces == 1 && a.rows <= 65472;
            int e = forward ? head.forward(keep) : cudaSuccess;
            if (!e && gradients) e = head.gradients(keep);
            return e;
        };
        if (at.big) return products(Head<2, 256, T>{a, at, h, ws, w, w_stride, sm_count, stream});
        return products(Head<1, 128, T>{a, at, h, ws, w, w_stride, sm_count, stream});
    };
    return a.dtype == kBF16 ? run(__nv_bfloat16{}) : run(__half{});
}

int read_head_gave_up(unsigned* count) { return (int)cudaMemcpyFromSymbol(count, g_gave_up, sizeof(*count)); }

}  // namespace soma
