// Embedding lookup and its gradient (formulas in soma_ops.h).
//
// Forward: a warp copies a piece of a row, scaled, in 16-byte vectors of the
// output; a table's row that starts elsewhere in its 16-byte word is shifted
// into place.  HBM bound: rows read and written once.
//
// Backward: the tokens are sorted with their rows (stable, so that a token's
// rows rise), then every chunk of the sorted order adds its rows in fp32 and
// writes the tokens that lie wholly inside it; a token that passes over a
// chunk's border leaves partial sums, which a last kernel joins in order.  So
// no token is too frequent for one CTA, no atomic touches a gradient, and the
// same call gives the same bits.  While one cluster sorts, the launch's other
// CTAs zero the table, the rows with tokens too: that costs less than knowing
// which they are before the sort is done.
//
// Measured (GB300, 6786 GB/s copy; graph replays, a call takes 1 to 3 us more):
// 16384 tokens of 4096 bf16 looked up in 34.3 us; their gradient in a table of
// 32000 rows 72.2 us, of which zeroing beside the sort takes 38 (as long as a
// memset) and the sums 28 (5.5 TB/s), or 81 where each gradient goes to other
// memory than the one before (of that L2 still holds a part); 5003 tokens of
// 1003 fp32 added to a gradient 21.0 us, three dependent launches; 65536 tokens
// are sorted in 34 us.
#include <math.h>

#include <algorithm>
#include <utility>

#include "ops_device.cuh"
#include "ops_kernels.h"
#include "soma_ops.h"
#include "tcgen05.cuh"

namespace soma {
namespace {

__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Token of row r, or -1 where it is outside the vocabulary.
__device__ __forceinline__ int token_at(const TokenArgs& t, int64_t r, int vocab) {
    const int64_t at = t.length == t.stride ? r : r / t.length * t.stride + r % t.length;
    const int64_t v = t.type == SOMA_INDEX_I64 ? __ldg(static_cast<const long long*>(t.index) + at)
                                               : (int64_t)__ldg(static_cast<const int*>(t.index) + at);
    return v >= 0 && v < vocab ? (int)v : -1;
}

// ---- forward -------------------------------------------------------------------

constexpr int kFwdThreads = 128;
constexpr int kFwdDeep = 4;                   // vectors in flight per lane
constexpr int kFwdPiece = 32 * kFwdDeep;      // vectors of a row that one warp copies

template <typename T>
__global__ void __launch_bounds__(kFwdThreads) lookup_kernel(const __grid_constant__ EmbeddingArgs a, int pieces) {
    constexpr int kVec = 16 / sizeof(T);
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (kFwdThreads / 32) + (threadIdx.x >> 5);
    const int64_t r = item / pieces;
    if (r >= a.rows) return;
    const int piece = (int)(item - r * pieces);
    const int v = token_at(a.tokens, r, a.vocab);
    T* dst = static_cast<T*>(a.out) + r * a.out_stride;
    // elements before the first whole word of the output's row, and its whole words
    const int head = min(a.cols, (int)((16 - ((uintptr_t)dst & 15)) & 15) / (int)sizeof(T));
    const int words = (a.cols - head) / kVec;
    const T* table = static_cast<const T*>(a.table);
    const T* src = table + (int64_t)max(v, 0) * a.table_stride;
    if (piece == 0) {
        // the ends of the row, one element a lane
        const int ends = a.cols - words * kVec;
        if (lane < ends) {
            const int c = lane < head ? lane : words * kVec + lane;
            dst[c] = from_f32<T>(v < 0 ? 0.f : to_f32(src[c]) * a.scale);
        }
    }
    const int i0 = piece * kFwdPiece + lane;
    if (i0 - lane >= words) return;
    uint4* out = reinterpret_cast<uint4*>(dst + head);
    if (v < 0) {
        for (int q = 0; q < kFwdDeep; ++q)
            if (i0 + 32 * q < words) out[i0 + 32 * q] = make_uint4(0, 0, 0, 0);
        return;
    }
    const int phase = (int)((uintptr_t)(src + head) & 15);
    const uint4* in = reinterpret_cast<const uint4*>((uintptr_t)(src + head) - phase);
    // words that lie inside the table
    const uintptr_t end = (uintptr_t)(table + (int64_t)(a.vocab - 1) * a.table_stride + a.cols);
    uint4 u[kFwdDeep], w[kFwdDeep];
#pragma unroll
    for (int q = 0; q < kFwdDeep; ++q) {
        const int i = i0 + 32 * q;
        if (i >= words) break;
        const bool inside = (uintptr_t)(in + i) >= (uintptr_t)table && (uintptr_t)(in + i + (phase ? 2 : 1)) <= end;
        if (inside) {
            u[q] = __ldg(in + i);
            if (phase) w[q] = __ldg(in + i + 1);
        }
    }
#pragma unroll
    for (int q = 0; q < kFwdDeep; ++q) {
        const int i = i0 + 32 * q;
        if (i >= words) break;
        const bool inside = (uintptr_t)(in + i) >= (uintptr_t)table && (uintptr_t)(in + i + (phase ? 2 : 1)) <= end;
        float x[kVec];
        if (inside) {
            widen16(phase ? shifted<T>(u[q], w[q], phase) : u[q], x, T{});
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[e] = to_f32(src[head + i * kVec + e]);
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[e] *= a.scale;
        __stcs(out + i, narrow16(x, T{}));
    }
}

// ---- sorting the tokens ----------------------------------------------------------
//
// Least significant digit first, stable: a warp ranks its items 32 at a time,
// counting equal digits below each lane.  Tokens outside the vocabulary sort
// last, as `vocab`.

constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kMaxDigits = 512;
constexpr int kSortCtas = 8;                    // of the one-cluster sort, at most
constexpr int kSortShare = 11776;                // items of one of its CTAs, at most: 16 bytes each beside 36 KB of counts
constexpr int kSortTile = 8192;                 // items of a CTA of the many-launch sort

struct SortArgs {
    TokenArgs tokens;
    int64_t rows;
    int32_t vocab;
    int32_t digit_bits, passes;
    uint32_t* keys;       // [rows] sorted tokens
    uint32_t* order;      // [rows] their rows
    uint32_t* keys2;      // the many-launch sort's second buffers
    uint32_t* order2;
    uint32_t* counts;     // [digits][CTAs] of the many-launch sort
    int32_t share;        // items of a CTA
    char* zero;           // the table of gradients to zero: zero_rows rows (0: none) of zero_cols bytes, zero_stride apart
    int64_t zero_stride, zero_rows, zero_cols;
};

// Histograms of the warps' items; then `hist` holds for each warp and digit
// how many items of earlier warps have the digit, and total[] how many have it.
template <typename Key>
__device__ __forceinline__ void count_digits(uint32_t (*hist)[kMaxDigits], uint32_t* total, int n, int digits, Key key) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = (n + 32 * kSortWarps - 1) / (32 * kSortWarps) * 32;  // items of a warp
    for (int d = threadIdx.x; d < digits * kSortWarps; d += kSortThreads) hist[d / digits][d % digits] = 0;
    __syncthreads();
    for (int i = warp * per + lane; i < min(n, (warp + 1) * per); i += 32) atomicAdd(&hist[warp][key(i)], 1u);
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kSortThreads) {
        uint32_t sum = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = hist[w][d];
            hist[w][d] = sum;
            sum += c;
        }
        total[d] = sum;
    }
    __syncthreads();
}

// Hands item i, of digit key(i), to put(i, place): start[d] is the place of
// the CTA's first item of digit d.
template <typename Key, typename Put>
__device__ __forceinline__ void scatter_digits(uint32_t (*hist)[kMaxDigits], const uint32_t* start, int n, Key key, Put put) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = (n + 32 * kSortWarps - 1) / (32 * kSortWarps) * 32;
    const int end = min(n, (warp + 1) * per);
    for (int i0 = warp * per; i0 < end; i0 += 32) {
        const int i = i0 + lane;
        const bool on = i < end;
        const uint32_t d = on ? key(i) : 0xffffffffu;
        const uint32_t peers = __match_any_sync(0xffffffffu, d);
        uint32_t place = 0;
        if (on) place = start[d] + hist[warp][d] + __popc(peers & ((1u << lane) - 1));
        __syncwarp();
        if (on && lane == 31 - __clz(peers)) hist[warp][d] += __popc(peers);
        __syncwarp();
        if (on) put(i, place);
    }
}

// Exclusive sums over n <= kMaxDigits values, in place.
__device__ __forceinline__ void scan_digits(uint32_t* x, int n, uint32_t* scratch) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = threadIdx.x;
    static_assert(kMaxDigits == kSortThreads, "one digit per thread");
    const uint32_t own = d < n ? x[d] : 0;
    uint32_t sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += t;
    }
    if (lane == 31) scratch[warp] = sum;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += scratch[w];
    if (d < n) x[d] = before + sum - own;
    __syncthreads();
}

__device__ __forceinline__ int cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return (int)n;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster_u32x2(uint32_t addr, uint2 v) {
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}

// Zeroes `bytes` bytes (a multiple of 2) from p on, with the threads [at, at + 1, ...) of `step`.
__device__ __forceinline__ void zero_bytes(char* p, int64_t bytes, int64_t at, int64_t step) {
    const int64_t head = min(bytes, (int64_t)((16 - ((uintptr_t)p & 15)) & 15)), words = (bytes - head) / 16;
    for (int64_t i = at; i < (bytes - words * 16) / 2; i += step)
        *reinterpret_cast<uint16_t*>(p + (2 * i < head ? 2 * i : words * 16 + 2 * i)) = 0;
    uint4* body = reinterpret_cast<uint4*>(p + head);
#pragma unroll 4
    for (int64_t i = at; i < words; i += step) __stcs(body + i, make_uint4(0, 0, 0, 0));
}

constexpr int64_t kPage = 16384;  // bytes
constexpr int kZeroCtas = 8;      // per SM, one after the other

// CTA `at` of `ctas` zeroes its part of the table.
__device__ __forceinline__ void zero_table(const SortArgs& a, int at, int ctas) {
    if (a.zero_stride == a.zero_cols) {  // one long row, a page of it at a time
        const int64_t bytes = a.zero_rows * a.zero_cols;
        for (int64_t b = (int64_t)at * kPage; b < bytes; b += (int64_t)ctas * kPage)
            zero_bytes(a.zero + b, min(kPage, bytes - b), threadIdx.x, kSortThreads);
        return;
    }
    for (int64_t r = (int64_t)at * kSortWarps + (threadIdx.x >> 5); r < a.zero_rows; r += (int64_t)ctas * kSortWarps)
        zero_bytes(a.zero + r * a.zero_stride, a.zero_cols, threadIdx.x & 31, 32);
}

// The whole sort in one launch: the first cluster's CTAs hold `share` items
// each in shared memory and hand each other the items of a pass through it.
// The other clusters zero the table.
__global__ void __launch_bounds__(kSortThreads) cluster_sort_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ uint2 sort_smem[];  // token and row, so that an item moves in one store
    __shared__ uint32_t hist[kSortWarps][kMaxDigits];
    __shared__ uint32_t total[kMaxDigits], start[kMaxDigits], scratch[kSortWarps];
    launch_dependents();
    const int rank = cluster_rank(), ctas = cluster_size(), share = a.share;
    if ((int)blockIdx.x >= ctas) {
        zero_table(a, blockIdx.x - ctas, gridDim.x - ctas);
        return;
    }
    const int begin = rank * share, n = max(0, min(share, (int)a.rows - begin));
    uint2* items[2] = {sort_smem, sort_smem + share};
    for (int i = threadIdx.x; i < n; i += kSortThreads) {
        const int v = token_at(a.tokens, begin + i, a.vocab);
        items[0][i] = make_uint2(v < 0 ? a.vocab : v, begin + i);
    }
    __syncthreads();
    const int digits = 1 << a.digit_bits;
    for (int p = 0; p < a.passes; ++p) {
        const int from = p & 1, shift = p * a.digit_bits;
        auto key = [&](int i) { return items[from][i].x >> shift & (digits - 1); };
        count_digits(hist, total, n, digits, key);
        cluster_sync_all();  // every CTA's totals are there
        uint32_t all = 0, before = 0;
        const int d = threadIdx.x;
        if (d < digits) {
            uint32_t x[kSortCtas];
#pragma unroll
            for (int c = 0; c < kSortCtas; ++c) x[c] = c < ctas ? ld_cluster_u32(cluster_map(smem_addr(total + d), c)) : 0;
#pragma unroll
            for (int c = 0; c < kSortCtas; ++c) {
                if (c < rank) before += x[c];
                all += x[c];
            }
            start[d] = all;
        }
        __syncthreads();
        scan_digits(start, digits, scratch);
        if (d < digits) start[d] += before;
        __syncthreads();
        const bool last = p == a.passes - 1;
        scatter_digits(hist, start, n, key, [&](int i, uint32_t place) {
            const uint2 item = items[from][i];
            if (last) {
                a.keys[place] = item.x;
                a.order[place] = item.y;
            } else {
                const uint32_t c = place / share, at = place - c * share;
                st_cluster_u32x2(cluster_map(smem_addr(items[from ^ 1] + at), c), item);
            }
        });
        cluster_sync_all();  // the items have arrived; nobody reads this pass's totals any more
    }
}

// Zeroes the table, for the sort in many launches.
__global__ void __launch_bounds__(kSortThreads) zero_kernel(const __grid_constant__ SortArgs a) {
    zero_table(a, blockIdx.x, gridDim.x);
}

// The same in many launches, a pass in three: digits counted, places found,
// items moved.
__global__ void __launch_bounds__(kSortThreads) count_kernel(const __grid_constant__ SortArgs a, int pass) {
    __shared__ uint32_t hist[kSortWarps][kMaxDigits];
    __shared__ uint32_t total[kMaxDigits];
    const int64_t begin = (int64_t)blockIdx.x * kSortTile;
    const int n = (int)min((int64_t)kSortTile, a.rows - begin);
    const int digits = 1 << a.digit_bits, shift = pass * a.digit_bits;
    const uint32_t* keys = pass & 1 ? a.keys2 : a.keys;
    if (pass == 0) {
        for (int i = threadIdx.x; i < n; i += kSortThreads) {
            const int v = token_at(a.tokens, begin + i, a.vocab);
            a.keys[begin + i] = v < 0 ? a.vocab : v;
            a.order[begin + i] = (uint32_t)(begin + i);
        }
        __syncthreads();
    }
    count_digits(hist, total, n, digits, [&](int i) { return keys[begin + i] >> shift & (digits - 1); });
    for (int d = threadIdx.x; d < digits; d += kSortThreads) a.counts[(int64_t)d * gridDim.x + blockIdx.x] = total[d];
}

// Exclusive sums over all counts, in place, by one CTA.
__global__ void __launch_bounds__(kSortThreads) place_kernel(uint32_t* counts, int64_t n) {
    __shared__ uint32_t sums[kSortThreads], scratch[kSortWarps];
    uint32_t carry = 0;
    constexpr int kEach = 8;
    for (int64_t at = 0; at < n; at += kSortThreads * kEach) {
        uint32_t x[kEach], sum = 0;
        const int64_t i0 = at + threadIdx.x * kEach;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            x[k] = i0 + k < n ? counts[i0 + k] : 0;
            sum += x[k];
        }
        sums[threadIdx.x] = sum;
        __syncthreads();
        scan_digits(sums, kSortThreads, scratch);
        uint32_t before = carry + sums[threadIdx.x];
        if (threadIdx.x == kSortThreads - 1) scratch[0] = sums[threadIdx.x] + sum;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if (i0 + k < n) counts[i0 + k] = before;
            before += x[k];
        }
        __syncthreads();
        carry += scratch[0];
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kSortThreads) move_kernel(const __grid_constant__ SortArgs a, int pass) {
    __shared__ uint32_t hist[kSortWarps][kMaxDigits];
    __shared__ uint32_t start[kMaxDigits];
    const int64_t begin = (int64_t)blockIdx.x * kSortTile;
    const int n = (int)min((int64_t)kSortTile, a.rows - begin);
    const int digits = 1 << a.digit_bits, shift = pass * a.digit_bits;
    const uint32_t *keys = pass & 1 ? a.keys2 : a.keys, *order = pass & 1 ? a.order2 : a.order;
    uint32_t *to_keys = pass & 1 ? a.keys : a.keys2, *to_order = pass & 1 ? a.order : a.order2;
    auto key = [&](int i) { return keys[begin + i] >> shift & (digits - 1); };
    count_digits(hist, start, n, digits, key);
    for (int d = threadIdx.x; d < digits; d += kSortThreads) start[d] = a.counts[(int64_t)d * gridDim.x + blockIdx.x];
    __syncthreads();
    scatter_digits(hist, start, n, key, [&](int i, uint32_t place) {
        to_keys[place] = keys[begin + i];
        to_order[place] = order[begin + i];
    });
}

// ---- sums of the sorted rows -------------------------------------------------------

constexpr int kSumThreads = 128;
constexpr int kMostChunk = 64, kLeastChunk = 16;  // sorted positions of a CTA
constexpr int kSumDeep = 8;                       // rows in flight per thread

struct SumArgs {
    const uint32_t* keys;
    const uint32_t* order;
    float* partials;      // [chunks][2][cols]: of a chunk's first token, if it began earlier, and its last, if it goes on
    const void* dy;
    int64_t dy_stride;
    void* out;
    int64_t out_stride;
    int64_t rows;
    int32_t vocab, cols;
    int32_t chunk, chunks, col_blocks;  // chunks x col_blocks CTAs
    float scale;
};

// A thread's columns: a vector of kVec (kWhole: rows of dy and out start on
// 16-byte boundaries and hold whole vectors), else four columns kSumThreads
// apart (eight 16-bit ones took 164 registers).
template <typename T, bool kWhole>
struct Columns {
    static constexpr int kVec = kWhole ? 16 / sizeof(T) : 4;
    int c0, cols;
    __device__ __forceinline__ Columns(int block, int n) : cols(n) {
        c0 = kWhole ? (block * kSumThreads + (int)threadIdx.x) * kVec : block * kSumThreads * kVec + (int)threadIdx.x;
    }
    __device__ __forceinline__ int col(int e) const { return kWhole ? c0 + e : c0 + e * kSumThreads; }
    struct Raw {
        uint4 w;
        T x[kWhole ? 1 : kVec];
    };
    __device__ __forceinline__ void load(const T* row, Raw& r) const {
        if (kWhole) {
            if (c0 < cols) r.w = __ldcs(reinterpret_cast<const uint4*>(row + c0));
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (col(e) < cols) r.x[kWhole ? 0 : e] = row[col(e)];
        }
    }
    __device__ __forceinline__ void add(const Raw& r, float (&sum)[kVec]) const {
        if (kWhole) {
            float x[kVec];
            widen16(r.w, x, T{});
#pragma unroll
            for (int e = 0; e < kVec; ++e) sum[e] += x[e];
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) sum[e] += to_f32(r.x[kWhole ? 0 : e]);
        }
    }
    // out = scale * sum + before (a Raw of out, where kAdd)
    template <bool kAdd>
    __device__ __forceinline__ void store(T* row, const float (&sum)[kVec], float scale, const Raw& before) const {
        if (kWhole) {
            if (c0 >= cols) return;
            float x[kVec] = {};
            if (kAdd) widen16(before.w, x, T{});
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[e] = fmaf(sum[e], scale, x[e]);
            *reinterpret_cast<uint4*>(row + c0) = narrow16(x, T{});
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (col(e) < cols) row[col(e)] = from_f32<T>(fmaf(sum[e], scale, kAdd ? to_f32(before.x[kWhole ? 0 : e]) : 0.f));
        }
    }
    __device__ __forceinline__ void store_partial(float* row, const float (&sum)[kVec]) const {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            if (col(e) < cols) row[col(e)] = sum[e];
    }
};

template <typename T, bool kWhole, bool kAdd>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const __grid_constant__ SumArgs a) {
    __shared__ uint32_t keys[kMostChunk + 2], order[kMostChunk];
    launch_dependents();
    wait_for_previous();
    using C = Columns<T, kWhole>;
    const int chunk = (int)blockIdx.x / a.col_blocks;
    const C columns((int)blockIdx.x % a.col_blocks, a.cols);
    const int64_t begin = (int64_t)chunk * a.chunk;
    const int n = (int)min((int64_t)a.chunk, a.rows - begin);
    constexpr uint32_t kNone = 0xffffffffu;
    for (int i = threadIdx.x; i < n + 2; i += kSumThreads) {  // one neighbour on each side
        const int64_t at = begin + i - 1;
        keys[i] = at >= 0 && at < a.rows ? __ldcg(a.keys + at) : kNone;
        if (i < n) order[i] = __ldcg(a.order + begin + i);
    }
    __syncthreads();
    const T* dy = static_cast<const T*>(a.dy);
    auto out = [&](uint32_t key) { return static_cast<T*>(a.out) + (int64_t)key * a.out_stride; };
    float sum[C::kVec] = {};
    bool began_here = keys[0] != keys[1];
    for (int i0 = 0; i0 < n && keys[1 + i0] < (uint32_t)a.vocab; i0 += kSumDeep) {
        typename C::Raw raw[kSumDeep], before[kAdd ? kSumDeep : 1];
#pragma unroll
        for (int q = 0; q < kSumDeep; ++q) {
            const int i = i0 + q;
            if (i >= n || keys[1 + i] >= (uint32_t)a.vocab) break;  // (of a token outside the vocabulary nothing is read)
            columns.load(dy + (int64_t)order[i] * a.dy_stride, raw[q]);
            // what a token's sum is added to, where it ends (read now: one at a time they cost a latency each)
            if (kAdd && keys[1 + i] != keys[2 + i]) columns.load(out(keys[1 + i]), before[kAdd ? q : 0]);
        }
#pragma unroll
        for (int q = 0; q < kSumDeep; ++q) {
            const int i = i0 + q;
            if (i >= n) break;
            const uint32_t key = keys[1 + i];
            if (key >= (uint32_t)a.vocab) break;
            columns.add(raw[q], sum);
            const bool ends = key != keys[2 + i];
            if (!ends && i + 1 < n) continue;
            if (ends && began_here) columns.template store<kAdd>(out(key), sum, a.scale, before[kAdd ? q : 0]);
            else columns.store_partial(a.partials + ((int64_t)chunk * 2 + (began_here ? 1 : 0)) * a.cols, sum);
            began_here = true;
#pragma unroll
            for (int e = 0; e < C::kVec; ++e) sum[e] = 0.f;
        }
    }
}

// A token that began in a chunk and goes on after it: its partial sums from
// that chunk on, in order.
template <typename T, bool kWhole, bool kAdd>
__global__ void __launch_bounds__(kSumThreads) join_kernel(const __grid_constant__ SumArgs a) {
    launch_dependents();
    wait_for_previous();
    using C = Columns<T, kWhole>;
    const int chunk = (int)blockIdx.x / a.col_blocks, lane = threadIdx.x & 31;
    const int64_t begin = (int64_t)chunk * a.chunk, last = begin + a.chunk - 1;  // (there is a chunk after this one)
    const uint32_t key = __ldcg(a.keys + last), next = __ldcg(a.keys + last + 1);
    const uint32_t previous = begin > 0 ? __ldcg(a.keys + begin - 1) : ~key;
    if (key >= (uint32_t)a.vocab || next != key || previous == key) return;
    const C columns((int)blockIdx.x % a.col_blocks, a.cols);
    typename C::Raw before;
    T* out = static_cast<T*>(a.out) + (int64_t)key * a.out_stride;
    if (kAdd) columns.load(out, before);
    float sum[C::kVec];
    auto at = [&](int c, int which, int e) {
        return columns.col(e) < a.cols ? __ldcg(a.partials + ((int64_t)c * 2 + which) * a.cols + columns.col(e)) : 0.f;
    };
#pragma unroll
    for (int e = 0; e < C::kVec; ++e) sum[e] = at(chunk, 1, e);
    // the chunks after this one whose first key is the token, 32 of them looked at together
    for (int c0 = chunk + 1; c0 < a.chunks; c0 += 32) {
        const bool mine = c0 + lane < a.chunks && __ldcg(a.keys + (int64_t)(c0 + lane) * a.chunk) == key;
        const uint32_t same = __ballot_sync(0xffffffffu, mine);
        const int count = same == 0xffffffffu ? 32 : __ffs(~same) - 1;
        // eight at a time in flight (a token in 4200 of 65536 rows: 66 chunks, 27 us with four)
        for (int c = c0; c < c0 + count; c += 8) {
            float part[8][C::kVec];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
#pragma unroll
                for (int e = 0; e < C::kVec; ++e) part[k][e] = c + k < c0 + count ? at(c + k, 0, e) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
#pragma unroll
                for (int e = 0; e < C::kVec; ++e) sum[e] += part[k][e];
            }
        }
        if (count < 32) break;
    }
    columns.template store<kAdd>(out, sum, a.scale, before);
}

// ---- host side -------------------------------------------------------------------

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// Digits that the tokens and `vocab` itself need, in passes of at most 9 bits.
void plan_digits(SortArgs& s) {
    int bits = 1;
    while (((int64_t)1 << bits) <= s.vocab) ++bits;
    s.passes = (bits + 8) / 9;
    s.digit_bits = (bits + s.passes - 1) / s.passes;
}

bool one_cluster(int64_t rows) { return rows <= (int64_t)kSortCtas * kSortShare; }

// The workspace: sorted tokens and rows, partial sums, and what the
// many-launch sort needs.
struct Layout {
    int64_t keys, order, partials, keys2, order2, counts, bytes;
    int32_t chunk;
    int64_t chunks;
    Layout(int64_t rows, int64_t cols) {
        // Long chunks leave fewer partial sums; the CTAs of 1024 columns should still be six per SM.
        const int64_t blocks = (cols + 1023) / 1024;
        chunk = kMostChunk;
        while (chunk > kLeastChunk && (rows + chunk - 1) / chunk * blocks < 6 * 152) chunk /= 2;
        chunks = (rows + chunk - 1) / chunk;
        int64_t at = 0;
        auto take = [&](int64_t n) { const int64_t here = at; at += align256(n); return here; };
        keys = take(rows * 4);
        order = take(rows * 4);
        partials = take(chunks > 1 ? chunks * 2 * cols * 4 : 0);
        const bool many = !one_cluster(rows);
        keys2 = take(many ? rows * 4 : 0);
        order2 = take(many ? rows * 4 : 0);
        counts = take(many ? (rows + kSortTile - 1) / kSortTile * kMaxDigits * 4 : 0);
        bytes = at;
    }
};

int launch_after(const void* kernel, int64_t grid, int threads, void** args, void* stream) {
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelExC(&cfg, kernel, args);
}

int launch_sort(SortArgs& s, int sm_count, void* stream) {
    cudaStream_t st = (cudaStream_t)stream;
    plan_digits(s);
    const int64_t zero = s.zero_rows * s.zero_cols;
    // CTAs that zero: a page each at least, at most kZeroCtas per SM
    const int zeros = (int)std::min<int64_t>(kZeroCtas * sm_count, (zero + kPage - 1) / kPage);
    if (one_cluster(s.rows)) {
        // More CTAs sort faster (5003 rows in 11 us with eight, 23 with one), fewer
        // leave the zeroing more room: clusters of eight do not fill every SM.  So
        // as few as are done when the table is zeroed (about 9 us and 2.7 for each
        // 1000 rows of a CTA; 6.5 GB/ms), and one zeroing CTA per SM at a time,
        // which its shared memory sees to: 16384 tokens into 32000 x 4096 bf16 76 us
        // with clusters of two, 78 of four, 84 of eight or with three CTAs per SM.
        const double zeroed = (double)zero / 6.5e6;
        int ctas = 1;
        while (ctas < kSortCtas && ((int64_t)ctas * kSortShare < s.rows ||
                                    ((int64_t)ctas * 1024 < s.rows && 9 + 2.7e-3 * s.rows / ctas > zeroed)))
            ctas *= 2;
        s.share = (int32_t)((s.rows + ctas - 1) / ctas);
        const int smem = zeros ? std::max(s.share * 16, 100 << 10) : s.share * 16;
        if (const int e = allow_smem((const void*)cluster_sort_kernel, smem)) return e;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(ctas + (zeros + ctas - 1) / ctas * ctas);
        cfg.blockDim = dim3(kSortThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        void* args[] = {&s};
        return (int)cudaLaunchKernelExC(&cfg, (const void*)cluster_sort_kernel, args);
    }
    if (zeros) zero_kernel<<<zeros, kSortThreads, 0, st>>>(s);
    const int tiles = (int)((s.rows + kSortTile - 1) / kSortTile);
    if (s.passes & 1) {  // the last pass ends in the first buffers
        std::swap(s.keys, s.keys2);
        std::swap(s.order, s.order2);
    }
    for (int p = 0; p < s.passes; ++p) {
        count_kernel<<<tiles, kSortThreads, 0, st>>>(s, p);
        place_kernel<<<1, kSortThreads, 0, st>>>(s.counts, (int64_t)tiles << s.digit_bits);
        move_kernel<<<tiles, kSortThreads, 0, st>>>(s, p);
    }
    return (int)cudaGetLastError();
}

}  // namespace

int launch_embedding_fwd(const EmbeddingArgs& a, void* stream) {
    return with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        const int vectors = (a.cols + 16 / (int)sizeof(T) - 1) / (16 / (int)sizeof(T));
        int pieces = std::max(1, (vectors + kFwdPiece - 1) / kFwdPiece);
        const int64_t grid = (a.rows * pieces + kFwdThreads / 32 - 1) / (kFwdThreads / 32);
        if (grid > 0x7fffffff) return (int)cudaErrorInvalidConfiguration;
        lookup_kernel<T><<<(unsigned)grid, kFwdThreads, 0, (cudaStream_t)stream>>>(a, pieces);
        return (int)cudaGetLastError();
    });
}

int64_t embedding_bwd_workspace(int64_t rows, int64_t cols) { return Layout(rows, cols).bytes; }

int launch_embedding_bwd(const EmbeddingArgs& a, const void* dy, int64_t dy_stride, bool accumulate, void* workspace,
                         int sm_count, void* stream) {
    const Layout at(a.rows, a.cols);
    char* ws = static_cast<char*>(workspace);
    SortArgs s{};
    s.tokens = a.tokens;
    s.rows = a.rows;
    s.vocab = a.vocab;
    s.keys = reinterpret_cast<uint32_t*>(ws + at.keys);
    s.order = reinterpret_cast<uint32_t*>(ws + at.order);
    s.keys2 = reinterpret_cast<uint32_t*>(ws + at.keys2);
    s.order2 = reinterpret_cast<uint32_t*>(ws + at.order2);
    s.counts = reinterpret_cast<uint32_t*>(ws + at.counts);
    const int esize = a.dtype == kF32 ? 4 : 2;
    s.zero = static_cast<char*>(a.out);
    s.zero_rows = accumulate ? 0 : a.vocab;
    s.zero_cols = (int64_t)a.cols * esize;
    s.zero_stride = a.vocab == 1 ? s.zero_cols : a.out_stride * esize;
    SumArgs u{};
    u.keys = s.keys;
    u.order = s.order;
    if (const int e = launch_sort(s, sm_count, stream)) return e;
    return with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int kVec = 16 / sizeof(T);
        u.partials = reinterpret_cast<float*>(ws + at.partials);
        u.dy = dy;
        u.dy_stride = dy_stride;
        u.out = a.out;
        u.out_stride = a.out_stride;
        u.rows = a.rows;
        u.vocab = a.vocab;
        u.cols = a.cols;
        u.chunk = at.chunk;
        u.chunks = (int32_t)at.chunks;
        u.scale = a.scale;
        const bool whole = a.cols % kVec == 0 && (uintptr_t)dy % 16 == 0 && (uintptr_t)a.out % 16 == 0 &&
                           (a.rows == 1 || dy_stride % kVec == 0) && (a.vocab == 1 || a.out_stride % kVec == 0);
        const int block = kSumThreads * (whole ? kVec : 4);
        u.col_blocks = (a.cols + block - 1) / block;
        const void *sum, *join;
        if (accumulate) {
            sum = whole ? (const void*)sum_kernel<T, true, true> : (const void*)sum_kernel<T, false, true>;
            join = whole ? (const void*)join_kernel<T, true, true> : (const void*)join_kernel<T, false, true>;
        } else {
            sum = whole ? (const void*)sum_kernel<T, true, false> : (const void*)sum_kernel<T, false, false>;
            join = whole ? (const void*)join_kernel<T, true, false> : (const void*)join_kernel<T, false, false>;
        }
        void* args[] = {&u};
        const int e = launch_after(sum, (int64_t)u.chunks * u.col_blocks, kSumThreads, args, stream);
        if (e != cudaSuccess || u.chunks < 2) return e;
        return launch_after(join, (int64_t)(u.chunks - 1) * u.col_blocks, kSumThreads, args, stream);
    });
}

}  // namespace soma
