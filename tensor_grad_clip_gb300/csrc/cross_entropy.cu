// Softmax cross entropy of a linear layer over a large vocabulary (formulas in
// soma_ops.h): logits are made on the tensor cores, a tile at a time, and used
// where they are, in registers.
//
//   select   rows that count are numbered, in order; what the others get is written
//   gather   those rows of x, one after the other on 16-byte boundaries: rows
//            that do not count cost nothing in the products, and what they
//            hold (NaN, say) reaches no gradient
//   stats    z = x W^T; maximum and sum of exponentials of every 32 logits
//   join     log-sum-exp and loss; where the statistics of all logits would
//            take more than 512 MB, the two run over one piece of the vocabulary
//            after the other, and the rows' running statistics are carried on
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
//
// Bound by the tensor cores, for few rows by reading the weight.  Measured
// (GB300, cuBLAS bf16 1916 TFLOP/s in a burst, 1723 in a loop; 85 % of the rows
// count; calls in a row, and graph replays after the slash): loss of 8192 rows,
// 32000 x 4096, 1.13 to 1.22 / 1.07 to 1.13 ms, 1500 to 1700 TFLOP/s; loss and
// gradients of 4096 rows, 131072 x 4096, 7.2 to 7.5 / 7.2 ms, 1500 to 1560
// TFLOP/s counted as three products; of 2500 rows, 32000 x 1024 fp16, 370 to 382
// / 360 us; loss of 16 rows, 32000 x 1024, 25 to 28 / 22 us, 3 TB/s.  Where
// the rows are two pieces, the logits are made twice: loss and gradients of 8192
// rows (all count), 131072 x 4096, 22.0 ms, 1600 TFLOP/s counted as four products.
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
    // What brings the largest |g| to 2^14, in fp16's range, and its inverse.  It
    // also spares the rows of that g, often all, the rounding of -g: of p - 1
    // times 2^14, near which most tokens' elements lie, little is lost.
    float scale, unscale;
    int32_t parts;          // in which the sums of dx were made
    uint32_t ticket;        // CTAs of the few rows' statistics that are done
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

constexpr int kSelectEach = 4;

__device__ __forceinline__ int64_t token_of(const TokenArgs& t, int64_t r) {
    const int64_t at = t.length == t.stride ? r : r / t.length * t.stride + r % t.length;
    return t.type == SOMA_INDEX_I64 ? (int64_t)__ldg(static_cast<const long long*>(t.index) + at)
                                    : (int64_t)__ldg(static_cast<const int*>(t.index) + at);
}

// Numbers the rows that count, by one CTA of kThreads; returns how many there
// are.  kWrite: it writes what the other kernels read, and what the other
// rows get.  here(number, row), if any, is told of each.
template <int kThreads, bool kWrite, typename Here>
__device__ __forceinline__ int select_rows(const HeadArgs& a, const HeadRows& h, Here&& here) {
    constexpr int kWarps = kThreads / 32;
    __shared__ int sums[kWarps];
    __shared__ float tops[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int done = 0;  // rows counted so far
    float top = 0.f;
    for (int64_t base = 0; base < a.rows; base += kThreads * kSelectEach) {
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
            } else if (kWrite) {
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
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) earlier = total;
            total += sums[w];
        }
        int at = done + earlier + before - mine;
#pragma unroll
        for (int q = 0; q < kSelectEach; ++q) {
            if (token[q] < 0) continue;
            here(at, (int)(r0 + q));
            if (kWrite) {
                h.row[at] = (int)(r0 + q);
                h.place[r0 + q] = at;
                h.token[at] = token[q];
                h.weight[at] = weight[q];
                h.g[at] = g[q];
                if (a.lse_in) h.lse[at] = a.lse_in[r0 + q];
            }
            ++at;
        }
        done += total;
        __syncthreads();
    }
    if constexpr (kWrite) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) tops[warp] = top;
        __syncthreads();
        const int padded = max(64, (done + 63) / 64 * 64);
        for (int i = done + threadIdx.x; i < padded; i += kThreads) {
            h.row[i] = h.token[i] = -1;
            h.weight[i] = h.g[i] = h.lse[i] = 0.f;
        }
        if (threadIdx.x == 0) {
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, tops[w]);
            const float largest = top > 0.f ? fminf(fmaxf(top, 0x1p-100f), 0x1p100f) : 1.f;
            *h.counted = {done, padded, 16384.f / largest, largest * (1.f / 16384.f), 1, 0};
        }
    }
    return done;
}

// One CTA: it has a few microseconds' work where the products have hundreds.
constexpr int kSelectThreads = 1024;
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ HeadArgs a, HeadRows h) {
    follow_stream();
    select_rows<kSelectThreads, true>(a, h, [](int, int) {});
}

// Vector i of a counted row of x (from < 0: of the padding), to its place.
template <typename T>
__device__ __forceinline__ void gather_vector(const T* x, int64_t stride, int64_t rows, int32_t cols, T* out,
                                              int64_t out_stride, int from, int to, int i) {
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

// Both in one launch, for rows that one pass of a CTA counts: every CTA counts
// them and copies its share.
constexpr int kFewThreads = 256, kFewRows = kFewThreads * kSelectEach;
template <typename T>
__global__ void __launch_bounds__(kFewThreads) select_few_kernel(const __grid_constant__ HeadArgs a, HeadRows h, T* out,
                                                                 int64_t out_stride, int pieces) {
    __shared__ int row[kFewRows];
    follow_stream();
    auto here = [&](int number, int r) { row[number] = r; };
    const int count = blockIdx.x == 0 ? select_rows<kFewThreads, true>(a, h, here) : select_rows<kFewThreads, false>(a, h, here);
    __syncthreads();
    const int padded = max(64, (count + 63) / 64 * 64), warps = gridDim.x * (kFewThreads / 32);
    for (int item = blockIdx.x * (kFewThreads / 32) + (threadIdx.x >> 5); item < padded * pieces; item += warps) {
        const int to = item / pieces, i = (item - to * pieces) * 32 + (threadIdx.x & 31);
        if (i * 8 < a.k)
            gather_vector<T>(static_cast<const T*>(a.x), a.x_stride, a.rows, a.k, out, out_stride, to < count ? row[to] : -1,
                             to, i);
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
    gather_vector<T>(x, stride, rows, cols, out, out_stride, h.row[to], to, i);
}

// ---- logits -------------------------------------------------------------------

struct LogitArgs {
    CUtensorMap a, b, out;
    HeadRows h;
    float2* parts;          // [slices of 32 columns][pitch rows] maximum and sum of exponentials
    int64_t pitch;
    float2* joined;         // few rows: [rows][CTAs]
    bool keep;              // stats: store the exponentials too
    int32_t columns;        // stats: of narrow tiles, or 0
    float *loss, *lse;      // stats of few rows: what the last CTA writes (either may be nullptr)
    bool join;
    int32_t n, k;           // columns (of the piece), their first in the vocabulary, sum length
    int32_t first;
    int32_t tiles_n, strip;
};

// Rows of tiles, and where halves begin so that a last wave that at most half
// of the workers have is done by all.
template <int CG>
__device__ __forceinline__ TilePlan plan_rows(int rows, int k, int tiles_n, int strip, bool halves, int splits = 1,
                                              int chunk = kOneChunk) {
    TilePlan p{rows, k, (rows + kBM * CG - 1) / (kBM * CG), tiles_n, strip, 0, splits, chunk};
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

// The kept exponentials, at most 1, are fp16 whatever the operands are: its 11
// bits lose little beside the 8 that bf16's dz is rounded to (in bf16 they
// would cost as much again as that).  Times 2^14, so that fp16 has numbers for
// what a vocabulary's tail weighs: down to 2^-38.
constexpr float kKeepScale = 16384.f;

__device__ __forceinline__ float2 join_stats(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x);
    return make_float2(m, a.y * exp2_fast((a.x - m) * kLog2e) + b.y * exp2_fast((b.x - m) * kLog2e));
}

// Joins parts q, q + step, ... of what `at` points to, eight reads at a time.
__device__ __forceinline__ float2 join_parts(const float2* at, int64_t pitch, int q, int step, int count) {
    float2 own = make_float2(kLowest, 0.f);
    for (; q < count; q += 8 * step) {
        float2 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = q + k * step < count ? __ldcg(at + (q + k * step) * pitch) : make_float2(kLowest, 0.f);
        float m = own.x;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = fmaxf(m, v[k].x);
        float s = own.y * exp2_fast((own.x - m) * kLog2e);
#pragma unroll
        for (int k = 0; k < 8; ++k) s += v[k].y * exp2_fast((v[k].x - m) * kLog2e);
        own = make_float2(m, s);
    }
    return own;
}

// A counted row's loss and log-sum-exp.
__device__ __forceinline__ void write_loss(const HeadRows& h, int i, float2 sum, float* loss, float* lse) {
    const float log_s = logf(sum.y), total = sum.x + log_s;
    const int r = h.row[i];
    h.lse[i] = total;
    if (lse) lse[r] = total;
    // (m - z) + log s: near 0 it keeps its digits where lse - z would not
    if (loss) loss[r] = h.weight[i] * ((sum.x - __ldcg(h.z_token + i)) + log_s);
}

// A tensor core drops the last bits of a long sum's every step.  The loss is
// an fp32 number, so its logits are summed in chunks of 1024 products that are
// added in registers: at k = 4096 the loss errs by 3.6e-7 (fp32 products: 4.5e-7)
// instead of 1.6e-6, for 4 % of 8192 x 32000 x 4096's time; chunks of 512 err by
// 1.7e-7 for 7 %, of 2048 by 7.8e-7.
constexpr int kLogitChunk = 1024 / kBK;

// "Few rows": about one for each warp of the last CTA.  16 rows, 32000 x 1024
// 22.0 us (22.1 with a kernel of its own), 131072 x 4096 175 us (189); 32 rows,
// whose warps take two each, 22.7 and 176 us (22.0 and 188).
constexpr int kJoinedRows = 16;

template <int CG, int BN, typename T>
__global__ void __launch_bounds__(kTileThreads, 1) stats_kernel(const __grid_constant__ LogitArgs p) {
    constexpr int kCols = BN / (kEpilogueWarps / 4);  // of a warp, at most
    float z[kCols];
    float2 run = make_float2(kLowest, 0.f);  // few rows: of this thread's row, over all its tiles
    tile_products<CG, BN, T>(
        &p.a, &p.b, true, true,
        [&] { return plan_rows<CG>(p.h.counted->padded, p.k, p.tiles_n, p.strip, p.columns == 0, 1, kLogitChunk); },
        [&](uint32_t acc, const Part& part, char* staging, auto&& done) {
#pragma unroll
            for (int c = 0; c < kCols; c += 16) {
                if (c >= part.cols) break;
                uint32_t raw[16];
                tmem_ld16(acc + c, raw);
                tmem_ld_wait(raw);
#pragma unroll
                for (int i = 0; i < 16; ++i) z[c + i] = part.first ? __uint_as_float(raw[i]) : z[c + i] + __uint_as_float(raw[i]);
            }
            done();
            if (!part.last) return;
            const int row = part.row0 + (threadIdx.x & 31);
            const int at = p.h.token[row] - p.first - part.col0;  // the token's column here
            Stager<__half> stager{staging + (threadIdx.x >> 5) * kStagerBytes, part.row0, 0, p.n};
#pragma unroll
            for (int c = 0; c < kCols; c += 32) {
                const int col = part.col0 + c;
                if (c >= part.cols || col >= p.n) break;
                float (&x)[32] = *reinterpret_cast<float (*)[32]>(z + c);
                if (col + 32 > p.n) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (col + i >= p.n) x[i] = -INFINITY;
                }
                float m = kLowest;
#pragma unroll
                for (int i = 0; i < 32; ++i) m = fmaxf(m, x[i]);
                const int d = at - c;
                if (__any_sync(0xffffffffu, d >= 0 && d < 32) && d >= 0 && d < 32) {
                    float t = x[0];
#pragma unroll
                    for (int i = 1; i < 32; ++i) t = d == i ? x[i] : t;
                    p.h.z_token[row] = t;
                }
                float even = 0.f, odd = 0.f;
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    x[i] = exp2_fast((x[i] - m) * kLog2e);
                    x[i + 1] = exp2_fast((x[i + 1] - m) * kLog2e);
                    even += x[i];
                    odd += x[i + 1];
                }
                if (p.join) run = join_stats(run, make_float2(m, even + odd));
                if (!p.join || p.keep) p.parts[col / 32 * p.pitch + row] = make_float2(m, even + odd);
                if (p.keep) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] *= kKeepScale;
                    stager.store(x, col, &p.out, true, nullptr, 0);
                }
            }
        },
        p.columns);
    if (!p.join) return;
    // Few rows, all in the first 32 of the tile: a CTA joins what its warps have,
    // and the last CTA to finish what the CTAs have, a warp a row; that saves a
    // launch.
    __shared__ bool last;
    extern __shared__ char dynamic[];  // (nothing is on its way there any more)
    float2 (*sums)[32] = reinterpret_cast<float2 (*)[32]>(dynamic);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp < kEpilogueWarps && warp % 4 == 0) sums[warp / 4][lane] = run;
    __syncthreads();
    if (warp == 0) {
        for (int w = 1; w < kEpilogueWarps / 4; ++w) run = join_stats(run, sums[w][lane]);
        if (lane < kJoinedRows) p.joined[lane * gridDim.x + blockIdx.x] = run;
        __threadfence();
    }
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(&p.h.counted->ticket, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    for (int i = warp; i < p.h.counted->rows; i += kTileThreads / 32) {
        float2 own = join_parts(p.joined + i * gridDim.x, 1, lane, 32, gridDim.x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            own = join_stats(own, make_float2(__shfl_xor_sync(0xffffffffu, own.x, o), __shfl_xor_sync(0xffffffffu, own.y, o)));
        if (lane == 0) write_loss(p.h, i, own, p.loss, p.lse);
    }
}

// Log-sum-exp and loss of 8 counted rows per CTA, or of 4 where rows are few:
// kRows lanes take neighbouring rows, the others slices in turn.  Of a piece
// of the vocabulary: joined with those before it; the last one writes the loss.
constexpr int kJoinThreads = 512;
template <int kRows>
__global__ void __launch_bounds__(kJoinThreads) stats_join_kernel(const float2* parts, int64_t pitch, int slices, HeadRows h,
                                                                  float* loss, float* lse, float2* run, bool first, bool last) {
    constexpr int kTurns = kJoinThreads / kRows;
    __shared__ float2 sums[kTurns][kRows];
    follow_stream();
    const int at = threadIdx.x % kRows, turn = threadIdx.x / kRows, i = blockIdx.x * kRows + at;
    if ((int)blockIdx.x * kRows >= h.counted->rows) return;
    float2 own = join_parts(parts + i, pitch, turn, kTurns, slices);
    sums[turn][at] = own;
    __syncthreads();
    for (int o = kTurns / 2; o > 0; o /= 2) {
        if (turn < o) sums[turn][at] = own = join_stats(own, sums[turn + o][at]);
        __syncthreads();
    }
    if (turn || i >= h.counted->rows) return;
    if (!first) own = join_stats(run[i], own);
    if (last) write_loss(h, i, own, loss, lse);
    else run[i] = own;
}

// dz of the kept exponentials, in place: a CTA 32 rows of 256 columns.  The
// token's own element, a difference from 1, is made of its logit.
constexpr int kKeepRows = 32, kKeepCols = 256;
template <typename T>
__global__ void __launch_bounds__(256) keep_kernel(T* dz, int64_t stride, const float2* parts, int64_t pitch, HeadRows h,
                                                   int32_t n) {
    __shared__ float factor[kKeepCols / 32][kKeepRows];
    follow_stream();
    const int row0 = blockIdx.y * kKeepRows, col0 = blockIdx.x * kKeepCols;
    if (row0 >= h.counted->padded) return;
    {
        const int r = threadIdx.x % kKeepRows, q = threadIdx.x / kKeepRows;
        if (col0 + 32 * q < n)
            factor[q][r] = h.g[row0 + r] * h.counted->scale * (1.f / kKeepScale) *
                           exp2_fast((__ldcs(&parts[(col0 / 32 + q) * pitch + row0 + r].x) - h.lse[row0 + r]) * kLog2e);
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = col0 + lane * 8;
    if (c >= n) return;
    uint4 v[kKeepRows / 8];
    T* at = dz + (int64_t)(row0 + warp) * stride + c;
#pragma unroll
    for (int k = 0; k < kKeepRows / 8; ++k) v[k] = *reinterpret_cast<const uint4*>(at + 8 * k * stride);
#pragma unroll
    for (int k = 0; k < kKeepRows / 8; ++k) {
        const int r = warp + 8 * k, row = row0 + r;
        const float f = factor[lane / 4][r];
        float x[8];
        widen16(v[k], x, __half{});
        const int token = h.token[row], d = token - c;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = token < 0 ? 0.f : x[i] * f;  // (the padding: NaN where weight is not finite)
        if (d >= 0 && d < 8) {
            const float own =
                h.g[row] * h.counted->scale * (exp2_fast((h.z_token[row] - h.lse[row]) * kLog2e) - 1.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = d == i ? own : x[i];
        }
        *reinterpret_cast<uint4*>(at + 8 * k * stride) = narrow16(x, T{});
    }
}

// dz of a piece, scaled.
template <int CG, int BN, typename T>
__global__ void __launch_bounds__(kTileThreads, 1) dz_kernel(const __grid_constant__ LogitArgs p) {
    tile_products<CG, BN, T>(
        &p.a, &p.b, true, true,
        [&] { return plan_rows<CG>(p.h.counted->padded, p.k, p.tiles_n, p.strip, true); },
        [&](uint32_t acc, const Part& part, char* staging, auto&& done) {
            const int row0 = part.row0, col0 = part.col0, cols = part.cols, row = row0 + (threadIdx.x & 31);
            const int at = p.h.token[row] - p.first - col0;
            const float lse = p.h.lse[row], g = p.h.g[row] * p.h.counted->scale;
            // (the padding's g is 0, but where weight is not finite its logits are not either)
            const bool padding = row0 + 32 > p.h.counted->rows;
            Stager<T> stager{staging + (threadIdx.x >> 5) * kStagerBytes, row0, 0, p.n};
            for (int c = 0; c < cols && col0 + c < p.n; c += 32) {
                float z[32];
                load_logits(acc + c, col0 + c, p.n, z);
                const int d = at - c;
                const bool here = __any_sync(0xffffffffu, d >= 0 && d < 32);
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] = g * exp2_fast((z[i] - lse) * kLog2e);
                if (padding && p.h.token[row] < 0) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) z[i] = 0.f;
                }
                if (here) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (d == i) z[i] -= g;
                }
                stager.store(z, col0 + c, &p.out, true, nullptr, 0);
            }
            done();
        });
}

// ---- gradients ------------------------------------------------------------------

struct GradArgs {
    CUtensorMap a, b, out;
    HeadRows h;
    float* sums;            // dx: [parts][pitch rows][sums_stride]
    int64_t pitch, sums_stride;
    bool add;               // dx: to what is there
    void* dweight;          // its piece
    int64_t dweight_stride;
    bool tma_out;
    int32_t m, n, k;        // dweight: m; dx: k (the others are the device's)
    int32_t tiles_m, tiles_n, strip;
    int32_t first_k, most_parts;  // dx: the first piece's k
};

template <int CG, int BN, typename T>
__global__ void __launch_bounds__(kTileThreads, 1) dweight_kernel(const __grid_constant__ GradArgs p) {
    tile_products<CG, BN, T>(
        &p.a, &p.b, false, false,
        [&] { return plan_rows<CG>(p.m, p.h.counted->padded, p.tiles_n, p.strip, true); },
        [&](uint32_t acc, const Part& part, char* staging, auto&& done) {
            const int row0 = part.row0, col0 = part.col0, cols = part.cols;
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
            done();
        });
}

// Parts in which dx's long sums are made side by side, at most `most`: its
// tiles are few, and parts fill the last wave, or the only one.  In units of a
// pipeline stage (0.36 us), a wave takes its share of k and four stages more;
// a part of m rows is written and read once.
template <int CG, int BN>
__device__ __forceinline__ int parts_of(int rows, int tiles_n, int k, int most) {
    const int tiles = (rows + kBM * CG - 1) / (kBM * CG) * tiles_n, workers = (int)gridDim.x / CG, kts = (k + kBK - 1) / kBK;
    const float traffic = (float)tiles * (kBM * CG * BN * 8 / 2.4e6f);  // of a part: 2.4 MB in a stage's time
    int best = 1;
    float least = 0.f;
    for (int s = 1; s <= most; ++s) {
        const float time = (float)((tiles * s + workers - 1) / workers) * ((float)kts / s + 4.f) + (s > 1 ? s * traffic : 0.f);
        if (s == 1 || time < least) {
            least = time;
            best = s;
        }
    }
    return best;
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
        [&] {
            // (every piece has the first one's parts; a last piece with less than a stage for each adds to the first)
            const int rows = p.h.counted->padded, parts = parts_of<CG, BN>(rows, p.tiles_n, p.first_k, p.most_parts);
            if (!p.add && blockIdx.x == 0 && threadIdx.x == 0) p.h.counted->parts = parts;
            return plan_rows<CG>(rows, p.k, p.tiles_n, p.strip, true, (p.k + kBK - 1) / kBK >= parts ? parts : 1);
        },
        [&](uint32_t acc, const Part& part, char*, auto&& done) {
            const int row0 = part.row0, col0 = part.col0, cols = part.cols;
            float* to = p.sums + (part.split * p.pitch + row0 + (threadIdx.x & 31)) * p.sums_stride;
            // (the sums' rows are as long as whole tiles)
            for (int c = 0; c < cols && col0 + c < p.n; c += 32) {
                uint32_t raw[32];
                tmem_ld32(acc + c, raw);
                tmem_ld_wait(raw);
                add_or_store(to + col0 + c, raw, p.add);
            }
            done();
        });
}

// dx of all rows: the sums of the parts, unscaled and rounded; 0 for rows that
// do not count.
template <typename T>
__global__ void __launch_bounds__(256) dx_round_kernel(const float* sums, int64_t pitch, int64_t sums_stride, HeadRows h,
                                                       T* dx, int64_t dx_stride, int64_t rows, int32_t cols, int pieces) {
    follow_stream();
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t r = item / pieces;
    const int c = ((int)(item - r * pieces) * 32 + (threadIdx.x & 31)) * 8;
    if (r >= rows || c >= cols) return;
    const int at = h.place[r];
    float x[8] = {};
    if (at >= 0) {
        const int parts = h.counted->parts;
        for (int s0 = 0; s0 < parts; s0 += 4) {  // four in flight
            float4 u[4], v[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                u[s] = v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (s0 + s >= parts) continue;
                const float4* from = reinterpret_cast<const float4*>(sums + ((s0 + s) * pitch + at) * sums_stride + c);
                u[s] = __ldcs(from);
                v[s] = __ldcs(from + 1);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                x[0] += u[s].x; x[1] += u[s].y; x[2] += u[s].z; x[3] += u[s].w;
                x[4] += v[s].x; x[5] += v[s].y; x[6] += v[s].z; x[7] += v[s].w;
            }
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
// What the statistics take that are joined together (8 bytes for 32 logits:
// 16384 rows of a vocabulary of 131072).  A piece more costs about 40 us, a join
// and a last wave: 65536 rows, 131072 x 512 7.23 ms with 256 MB, 7.02 with 512,
// 6.95 with 1024, 6.91 in one piece of 2.1 GB; nothing at k = 1024 (11.6 to 11.8).
constexpr int64_t kStatsBytes = 512ll << 20;

struct HeadLayout {
    int64_t counted, row, place, token, weight, g, lse, z_token, x, w, parts, run, joined, dz, sums, bytes;
    int64_t pitch;                   // rows, rounded up to whole tiles
    int64_t x_stride, w_stride, sums_stride;
    int64_t piece, pieces;           // columns of the vocabulary
    int64_t stats_piece;             // columns whose statistics are joined together
    bool keep;                       // the loss and the gradients of one piece: exponentials are kept for dz
    bool join;                       // few rows: their statistics are joined by the kernel that makes them
    int32_t most_parts;              // in which dx may be summed side by side
    bool big;                        // tiles on pairs of SMs
    HeadLayout(int64_t rows, int64_t vocab, int64_t k, bool copy_weight, bool forward, bool dx, bool dweight, int sms) {
        pitch = (rows + 255) / 256 * 256;
        // As for a linear layer: a 256 x 256 tile on two SMs takes as long as a
        // 128 x 128 tile on one, so the fewer waves win.
        const int64_t pairs = std::max(1, sms / 2);
        const int64_t t256 = (rows + 255) / 256 * ((vocab + 255) / 256), t128 = (rows + 127) / 128 * ((vocab + 127) / 128);
        big = rows > 128 && (t256 + pairs - 1) / pairs < (t128 + sms - 1) / sms;
        // (whole tiles on both sides: as many rows as columns of x, 256 of those or more, are one piece for any vocabulary)
        const int64_t width = k >= 256 && rows <= k ? pitch : k;
        const int64_t buffer = std::max(kPieceBytes, (vocab + 255) / 256 * 256 * width * 2);
        const int64_t most = std::max<int64_t>(256, buffer / (2 * pitch) / 256 * 256);
        pieces = (vocab + most - 1) / most;
        piece = ((vocab + pieces - 1) / pieces + 255) / 256 * 256;
        pieces = (vocab + piece - 1) / piece;
        // (32 rows of the pass over the kept exponentials are a row of its grid)
        keep = forward && (dx || dweight) && pieces == 1 && rows <= 32 * 65000;
        join = rows <= kJoinedRows;
        const int64_t most_stats = join ? vocab : std::max<int64_t>(256, kStatsBytes / (8 * pitch) * 32 / 256 * 256);
        const int64_t stats_pieces = (vocab + most_stats - 1) / most_stats;
        stats_piece = ((vocab + stats_pieces - 1) / stats_pieces + 255) / 256 * 256;
        // room for twice as many parts as fill a wave, each of 16 stages or more
        const int64_t edge = big ? 256 : 128, workers = big ? pairs : sms, kts = (std::min(piece, vocab) + kBK - 1) / kBK;
        const int64_t tiles = (rows + edge - 1) / edge * ((k + edge - 1) / edge);
        most_parts = (int32_t)std::max<int64_t>(1, std::min(std::min<int64_t>(16, kts / 16), 2 * workers / tiles));
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
        // kept exponentials need the statistics of all their logits
        parts = take(!forward || (join && !keep) ? 0 : pitch * slices(keep ? vocab : std::min(stats_piece, vocab)) * 8);
        run = take(forward && stats_piece < vocab ? pitch * 8 : 0);
        joined = take(forward && join ? (int64_t)kJoinedRows * sms * 8 : 0);
        dz = take(dx || dweight ? pitch * piece * 2 : 0);
        sums = take(dx ? most_parts * pitch * sums_stride * 4 : 0);
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
    // z = x W^T over columns [first, first + n) of the vocabulary, in tiles of `width` columns.
    int logits(LogitArgs& p, int64_t first, int64_t n, int width) const {
        p.h = h;
        p.pitch = at.pitch;
        p.n = (int32_t)n;
        p.k = a.k;
        p.first = (int32_t)first;
        p.tiles_n = (int32_t)((n + width - 1) / width);
        // Where L2 holds x beside all else, 8 columns of tiles at a time: a wave or two take them for all rows, and the
        // weight is read once.  dz of 1021 rows, 50021 x 1003, 76 us instead of 82 with strips that L2 holds, the logits
        // of 4096 rows, 131072 x 4096, 2.12 ms instead of 2.18 (4 and 16 columns are alike); of 8192 rows, whose x it
        // does not hold, 1.21 ms instead of 1.20.
        p.strip = strip_of(p.tiles_n, width, a.k);
        if (a.rows * a.k * 2 <= (40ll << 20)) p.strip = std::min(p.strip, 8);
        const char* b = static_cast<const char*>(w) + first * w_stride * 2;
        if (const int e = make_map(&p.a, a.dtype, ws + at.x, at.x_stride, at.pitch, a.k, kBM)) return e;
        return make_map(&p.b, a.dtype, b, w_stride, n, a.k, width / CG);
    }
    int forward() const {
        for (int64_t first = 0; first < a.vocab; first += at.stats_piece)
            if (const int e = statistics(first, std::min<int64_t>(at.stats_piece, a.vocab - first))) return e;
        if (!at.keep) return cudaSuccess;
        const float2* parts = reinterpret_cast<const float2*>(ws + at.parts);
        int64_t pitch = at.pitch, stride = at.piece;
        HeadRows rows = h;
        T* dz = reinterpret_cast<T*>(ws + at.dz);
        int32_t n = a.vocab;
        void* args[] = {&dz, &stride, &parts, &pitch, &rows, &n};
        const unsigned padded = (unsigned)std::max<int64_t>(64, (a.rows + 63) / 64 * 64);
        return launch_after((const void*)keep_kernel<T>, dim3((a.vocab + kKeepCols - 1) / kKeepCols, padded / kKeepRows), 256,
                            args, stream);
    }
    // Statistics of columns [first, first + n) of the vocabulary, joined with those before them.
    int statistics(int64_t first, int64_t n) const {
        LogitArgs p{};
        p.parts = reinterpret_cast<float2*>(ws + at.parts) + (at.keep ? HeadLayout::slices(first) * at.pitch : 0);
        p.keep = at.keep;
        if (at.keep)
            if (const int e = make_map(&p.out, a.dtype, ws + at.dz + first * 2, at.piece, at.pitch, n, 32, 32)) return e;
        void* args[] = {&p};
        int e;
        if (a.rows <= kBM) {
            // One row of tiles: reading the weight is what takes time, and tiles of
            // one width, at most 256, fill whole waves of SMs (32000 tokens: 143
            // tiles of 224 columns, not 250 of 128 in a wave and two thirds).
            const int64_t waves = ((n + 255) / 256 + sms - 1) / sms;
            p.columns = (int32_t)(((n + waves * sms - 1) / (waves * sms) + 31) / 32 * 32);
            p.join = at.join;
            p.joined = reinterpret_cast<float2*>(ws + at.joined);
            p.loss = a.loss;
            p.lse = a.lse;
            e = Head<1, 256, T>{a, at, h, ws, w, w_stride, sms, stream}.logits(p, first, n, p.columns);
            if (!e)
                e = launch_cluster((const void*)stats_kernel<1, 256, T>, args, std::min<int64_t>(p.tiles_n, sms),
                                   kTileThreads, TileShape<1, 256>::kSmem, 1, stream);
        } else {
            e = logits(p, first, n, BN);
            // (half tiles make at most twice as many units)
            if (!e) e = tiles((const void*)stats_kernel<CG, BN, T>, rows_of_tiles(a.rows) * p.tiles_n * 2, args);
        }
        return e || p.join ? e : join(p.parts, first, n);
    }
    int join(const float2* parts, int64_t first_column, int64_t n) const {
        int64_t pitch = at.pitch;
        int slices = (int)HeadLayout::slices(n);
        HeadRows rows = h;
        float *loss = a.loss, *lse = a.lse;
        float2* run = reinterpret_cast<float2*>(ws + at.run);
        bool first = first_column == 0, last = first_column + n == a.vocab;
        void* join_args[] = {&parts, &pitch, &slices, &rows, &loss, &lse, &run, &first, &last};
        // (few rows: 4 per CTA, a sector of each slice)
        const bool few = a.rows <= 1024;
        return launch_after(few ? (const void*)stats_join_kernel<4> : (const void*)stats_join_kernel<8>,
                            dim3((unsigned)((a.rows + (few ? 3 : 7)) / (few ? 4 : 8))), kJoinThreads, join_args, stream);
    }
    int gradients() const {
        for (int64_t first = 0; first < a.vocab; first += at.piece) {
            const int64_t n = std::min<int64_t>(at.piece, a.vocab - first);
            int e = cudaSuccess;
            if (!at.keep) {
                LogitArgs p{};
                e = make_map(&p.out, a.dtype, ws + at.dz, at.piece, at.pitch, n, 32, 32);
                void* args[] = {&p};
                if (!e) e = logits(p, first, n, BN);
                if (!e) e = tiles((const void*)dz_kernel<CG, BN, T>, rows_of_tiles(a.rows) * p.tiles_n * 2, args);
            }
            if (!e && a.dweight) e = dweight(first, n);
            if (!e && a.dx) e = dx(first, n);
            if (e) return e;
        }
        if (!a.dx) return cudaSuccess;
        const float* sums = reinterpret_cast<const float*>(ws + at.sums);
        int64_t pitch = at.pitch, sums_stride = at.sums_stride, stride = a.dx_stride, rows = a.rows;
        int pieces = (a.k + 255) / 256;
        int32_t cols = a.k;
        HeadRows hr = h;
        T* out = static_cast<T*>(a.dx);
        void* args[] = {&sums, &pitch, &sums_stride, &hr, &out, &stride, &rows, &cols, &pieces};
        const int64_t grid = (rows * pieces + 7) / 8;
        if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
        return launch_after((const void*)dx_round_kernel<T>, dim3((unsigned)grid), 256, args, stream);
    }
    int dweight(int64_t first, int64_t n) const {
        // (few rows: the larger tile where it takes fewer waves, for the output's sake: 100 rows, 131072 x 2048 146 us instead of 218)
        if constexpr (CG == 1) {
            const Head<2, 256, T> big{a, at, h, ws, w, w_stride, sms, stream};
            const int64_t small = rows_of_tiles(n) * ((a.k + BN - 1) / BN), large = big.rows_of_tiles(n) * ((a.k + 255) / 256);
            const int64_t pairs = std::max(1, sms / 2);
            if ((large + pairs - 1) / pairs < (small + sms - 1) / sms) return big.dweight(first, n);
        }
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
        p.first_k = (int32_t)std::min<int64_t>(at.piece, a.vocab);
        p.most_parts = at.most_parts;
        p.tiles_n = (a.k + BN - 1) / BN;
        p.strip = strip_of(p.tiles_n, BN, n);
        const char* b = static_cast<const char*>(w) + first * w_stride * 2;
        if (const int e = make_map(&p.a, a.dtype, ws + at.dz, at.piece, at.pitch, n, kBM)) return e;
        if (const int e = make_map(&p.b, a.dtype, b, w_stride, n, a.k, kBK)) return e;
        void* args[] = {&p};
        return tiles((const void*)dx_kernel<CG, BN, T>, rows_of_tiles(a.rows) * p.tiles_n * std::max(2, p.most_parts), args);
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
    auto run = [&](auto t) -> int {
        using T = decltype(t);
        HeadArgs all = a;
        T* out = reinterpret_cast<T*>(ws + at.x);
        int64_t out_stride = at.x_stride;
        int pieces = (a.k + 255) / 256;
        const int64_t padded = std::max<int64_t>(64, (a.rows + 63) / 64 * 64), grid = (padded * pieces + 7) / 8;
        if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
        if (a.rows <= kFewRows) {
            void* args[] = {&all, &h, &out, &out_stride, &pieces};
            if (const int e = launch_after((const void*)select_few_kernel<T>, dim3((unsigned)std::min<int64_t>(grid, 2 * sm_count)),
                                           kFewThreads, args, stream))
                return e;
        } else {
            void* select_args[] = {&all, &h};
            if (const int e = launch_after((const void*)select_kernel, dim3(1), kSelectThreads, select_args, stream)) return e;
            const T* x = static_cast<const T*>(a.x);
            int64_t stride = a.x_stride, rows = a.rows;
            int32_t cols = a.k;
            void* args[] = {&x, &stride, &rows, &cols, &out, &out_stride, &h, &pieces};
            if (const int e = launch_after((const void*)gather_kernel<T>, dim3((unsigned)grid), 256, args, stream)) return e;
        }
        auto products = [&](const auto& head) {
            int e = forward ? head.forward() : cudaSuccess;
            if (!e && (a.dx || a.dweight)) e = head.gradients();
            return e;
        };
        if (at.big) return products(Head<2, 256, T>{a, at, h, ws, w, w_stride, sm_count, stream});
        return products(Head<1, 128, T>{a, at, h, ws, w, w_stride, sm_count, stream});
    };
    return a.dtype == kBF16 ? run(__nv_bfloat16{}) : run(__half{});
}

int read_head_gave_up(unsigned* count) { return (int)cudaMemcpyFromSymbol(count, g_gave_up, sizeof(*count)); }

}  // namespace soma
