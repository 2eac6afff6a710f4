// Distillation loss from a teacher's top logits (formulas in soma_ops.h).
//
// A row's logits are streamed in 16-byte vectors: the forward pass reads them
// once (maximum and sum of exponentials together, in fp32), the backward pass
// reads them once and writes the gradient, and the one-call form reads a row
// twice: many long rows, where they are aligned, pass through a ring in shared
// memory that keeps most of a row for the second time; of other rows the second
// reading is from L2 as far as that holds the rows in progress.  One
// exponential and about six other instructions per element keep the bound
// with HBM.  The teacher's entries (at most 1024) live in shared memory; one
// warp works on them while the others stream.
//
// Measured (GB300, 6682 GB/s copy; 15 % of the rows do not count): 8192 x
// 131072 bf16 forward 285 us, 6405 GB/s; backward 639 us, 6225 GB/s; loss and
// gradient together 715 us, 5560 GB/s (914 us when the second pass re-read
// the row through L2, which the rows in progress overflow).  2048 x 50021
// bf16 backward, whose rows start anywhere, 103 us, 3668 GB/s: bound by the
// instructions that shift vectors on both sides (4987 GB/s for 50024).  Loss and
// gradient together of 2000 x 50021 fp16 133 us, of 2000 x 50024 95 us.
//
// A cluster of CTAs shares a row when there are fewer rows than CTAs that the
// device holds; the CTAs' maxima and sums are joined through distributed
// shared memory, in rank order.  Within a kernel, which thread takes which
// elements does not depend on where rows start in memory, so neither do the
// results.  Between the two kernels of the one-call form it does: the ring adds
// four vectors at a time, and the loss over more threads.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "mbarrier.cuh"
#include "ops_device.cuh"
#include "ops_kernels.h"
#include "soma_ops.h"

namespace soma {
namespace {

constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A maximum m and the sum of exp2((x - m) c) over what has been seen.  m
// starts at the lowest finite value, so that masked logits (-inf) add 0.
struct MaxSum {
    float m, s;
};
constexpr float kLowest = -3.402823466e38f;

__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
    const float m = fmaxf(a.m, b.m);
    return {m, a.s * exp2f((a.m - m) * c) + b.s * exp2f((b.m - m) * c)};
}

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float2 cluster_read(const float2* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
// Maximum; NaN if any x is.
__device__ __forceinline__ float larger(float a, float b) { return a > b || a != a ? a : b; }
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = larger(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

template <typename T>
__device__ __forceinline__ void take(MaxSum& a, const float (&x)[16 / sizeof(T)], float c) {
    constexpr int kVec = 16 / sizeof(T);
    float m = x[0];
#pragma unroll
    for (int i = 1; i < kVec; ++i) m = fmaxf(m, x[i]);
    if (m > a.m) {
        a.s *= exp2_fast((a.m - m) * c);
        a.m = m;
    }
    const float2 back = both(-a.m), cc = both(c);
#pragma unroll
    for (int i = 0; i < kVec; i += 2) {
        const float2 d = mul2(add2(make_float2(x[i], x[i + 1]), back), cc);
        a.s += exp2_fast(d.x) + exp2_fast(d.y);
    }
}

// Several vectors at once.
template <typename T, int kN>
__device__ __forceinline__ void take_many(MaxSum& a, const float (&x)[kN][16 / sizeof(T)], float c) {
    constexpr int kVec = 16 / sizeof(T);
    float m[kN];
#pragma unroll
    for (int q = 0; q < kN; ++q) {
        m[q] = x[q][0];
#pragma unroll
        for (int i = 1; i < kVec; ++i) m[q] = fmaxf(m[q], x[q][i]);
    }
#pragma unroll
    for (int q = 1; q < kN; ++q) m[0] = fmaxf(m[0], m[q]);
    if (m[0] > a.m) {
        a.s *= exp2_fast((a.m - m[0]) * c);
        a.m = m[0];
    }
    const float2 back = both(-a.m), cc = both(c);
    float2 s[kN];
#pragma unroll
    for (int q = 0; q < kN; ++q) {
        s[q] = both(0.f);
#pragma unroll
        for (int i = 0; i < kVec; i += 2) {
            const float2 d = mul2(add2(make_float2(x[q][i], x[q][i + 1]), back), cc);
            s[q] = add2(s[q], make_float2(exp2_fast(d.x), exp2_fast(d.y)));
        }
    }
#pragma unroll
    for (int q = 1; q < kN; ++q) s[0] = add2(s[0], s[q]);
    a.s += s[0].x + s[0].y;
}

// Maximum and sum of vectors [begin, end): vector i is thread i - begin mod
// kBlock's, in ascending order.
template <typename T, bool kKeep, int kBlock, bool kShift>
__device__ __forceinline__ MaxSum stream_max_sum(const RowReader<T, kKeep>& row, int begin, int end, float c) {
    constexpr int kVec = 16 / sizeof(T), kAhead = kShift ? 2 : 4;
    MaxSum a{kLowest, 0.f};
    int i = begin + threadIdx.x;
    float x[kVec];
    if (i < row.inner_begin && i < end) {
        row.gather(i, x);
        take<T>(a, x, c);
        i += kBlock;
    }
    const int inner = min(end, row.inner_end);
    uint4 u[kAhead], v[kShift ? kAhead : 1];
    for (; i + (kAhead - 1) * kBlock < inner; i += kAhead * kBlock) {
        row.template load<kShift, kAhead>(i, kBlock, u, v);
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            row.template widen<kShift>(u[q], v[kShift ? q : 0], x);
            take<T>(a, x, c);
        }
    }
    for (; i < inner; i += kBlock) {
        uint4 u1[1], v1[1];
        row.template load<kShift, 1>(i, kBlock, u1, v1);
        row.template widen<kShift>(u1[0], v1[0], x);
        take<T>(a, x, c);
    }
    for (; i < end; i += kBlock) {
        row.gather(i, x);
        take<T>(a, x, c);
    }
    return a;
}

// g q for one vector, q = exp(z / T - lse).
template <typename T>
__device__ __forceinline__ void scaled_softmax(float (&x)[16 / sizeof(T)], float inv_t, float lse, float g) {
    const float2 inv2 = both(inv_t), lse2 = both(-lse), log2 = both(kLog2e), g2 = both(g);
#pragma unroll
    for (int q = 0; q < 16 / (int)sizeof(T); q += 2) {
        const float2 d = mul2(fma2(make_float2(x[q], x[q + 1]), inv2, lse2), log2);
        const float2 e = mul2(make_float2(exp2_fast(d.x), exp2_fast(d.y)), g2);
        x[q] = e.x;
        x[q + 1] = e.y;
    }
}

// out = g q of vectors [begin, end).  Rows of logits and gradient that start
// on 16-byte boundaries go vector by vector; else whole warps take
// consecutive vectors together, as store_vector needs.
// ready() waits for what the first vector needs (lse, and for the others to
// be done with logits that the gradient replaces); the first loads are in
// flight meanwhile.
template <typename T, int kBlock, typename Ready>
__device__ __forceinline__ void stream_gradient(const RowReader<T, false>& row, T* out, int begin, int end, float inv_t,
                                                float g, Ready&& ready) {
    constexpr int kVec = 16 / sizeof(T);
    float x[kVec];
    const int out_phase = (int)((uintptr_t)out & 15);
    const int inner = min(end, row.inner_end);
    if (out_phase == 0 && row.phase == 0) {
        constexpr int kAhead = 4;
        uint4 u[kAhead], none[1];
        int i = begin + threadIdx.x;
        const bool full = i + (kAhead - 1) * kBlock < inner;
        if (full) row.template load<false, kAhead>(i, kBlock, u, none);
        const float lse = ready();
        for (bool loaded = true; i + (kAhead - 1) * kBlock < inner; i += kAhead * kBlock, loaded = false) {
            if (!loaded) row.template load<false, kAhead>(i, kBlock, u, none);
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                row.template widen<false>(u[q], none[0], x);
                scaled_softmax<T>(x, inv_t, lse, g);
                __stcs(reinterpret_cast<uint4*>(out) + i + q * kBlock, narrow16(x, T{}));
            }
        }
        for (; i < end; i += kBlock) {
            row.gather(i, x);
            scaled_softmax<T>(x, inv_t, lse, g);
            store_vector<T, true>(out, kVec * i, row.cols, 0, x);
        }
        return;
    }
    const float lse = ready();
    const int lane = threadIdx.x & 31;
    const int cols = min(row.cols, end * kVec);  // (a CTA stores nothing past its part of the row)
    int first = begin + (threadIdx.x & ~31);     // the warp's first vector
    auto general = [&] {
        row.gather(first + lane, x);
        scaled_softmax<T>(x, inv_t, lse, g);
        store_vector<T, false>(out, kVec * (first + lane), cols, out_phase, x);
        first += kBlock;
    };
    if (first < row.inner_begin && first < end) general();
    auto whole = [&](auto shift) {
        constexpr bool kShift = decltype(shift)::value;
        constexpr int kAhead = 2;
        for (; first + (kAhead - 1) * kBlock + 32 <= inner; first += kAhead * kBlock) {
            uint4 u[kAhead], v[kShift ? kAhead : 1];
            row.template load<kShift, kAhead>(first + lane, kBlock, u, v);
            float y[kAhead][kVec];
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                row.template widen<kShift>(u[q], v[kShift ? q : 0], y[q]);
                scaled_softmax<T>(y[q], inv_t, lse, g);
            }
#pragma unroll
            for (int q = 0; q < kAhead; ++q)
                store_vector<T, false>(out, kVec * (first + q * kBlock + lane), cols, out_phase, y[q]);
        }
    };
    if (row.phase) whole(std::true_type{});
    else whole(std::false_type{});
    while (first < end) general();
}

template <typename T, int kBlock>
__device__ __forceinline__ void stream_zeros(T* out, int begin, int end, int cols) {
    constexpr int kVec = 16 / sizeof(T);
    const float zero[kVec] = {};
    const int out_phase = (int)((uintptr_t)out & 15);
    for (int base = begin + (threadIdx.x & ~31); base < end; base += kBlock)
        store_vector<T, false>(out, kVec * (base + (threadIdx.x & 31)), min(cols, end * kVec), out_phase, zero);
}

// Teacher logit j of row r.
template <typename U>
__device__ __forceinline__ float teacher_at(const DistillArgs& a, int64_t r, int j) {
    return to_f32(static_cast<const U*>(a.teacher)[r * a.teacher_stride + j]);
}

// kBlock threads per CTA: few for short rows, of which an SM then holds many.
template <typename T, int PASS, int kBlock>
__global__ void __launch_bounds__(kBlock, 1536 / kBlock) distill_kernel(const __grid_constant__ DistillArgs a, int cluster) {
    constexpr int kVec = 16 / sizeof(T), kWarps = kBlock / 32;
    __shared__ float2 warp_part[kWarps];
    __shared__ float2 cta_part;
    __shared__ __align__(16) float p[SOMA_DISTILL_MAX_TOP], zt[SOMA_DISTILL_MAX_TOP];
    __shared__ __align__(16) int at[SOMA_DISTILL_MAX_TOP];
    __shared__ int any_entry;
    const int t = threadIdx.x, lane = t & 31;
    const int64_t r = blockIdx.x / cluster;
    const int rank = (int)(blockIdx.x % cluster);
    T* dz = static_cast<T*>(a.dlogits) + r * a.dlogits_stride;
    const float w = a.row_weight ? a.row_weight[r] : 1.f;
    // (a row of weight 0 does not count, whatever its grad_loss: an infinity or NaN would not give 0)
    const float scale = PASS == kDistillBackward && w != 0.f ? a.grad_loss[r] * w : w;

    // this CTA's vectors of the row
    const int vectors = (a.vocab + kVec - 1) / kVec;
    const int begin = (int)((int64_t)vectors * rank / cluster), end = (int)((int64_t)vectors * (rank + 1) / cluster);

    if (scale == 0.f) {  // (the same for all CTAs of the row)
        if (PASS != kDistillBackward && t == 0 && rank == 0) {
            a.loss[r] = 0.f;
            if (a.lse) a.lse[r] = 0.f;
        }
        if (PASS != kDistillForward) stream_zeros<T, kBlock>(dz, begin, end, a.vocab);
        return;
    }
    const T* z0 = static_cast<const T*>(a.logits);
    const T* z = z0 + r * a.logits_stride;

    // The teacher's entries: each thread's first one is loaded here and put
    // away by put_entries, with the student's logits at their places.
    if (t == 0) any_entry = 0;
    auto index_at = [&](int j) {
        return a.index_type == SOMA_INDEX_I64 ? static_cast<const int64_t*>(a.index)[r * a.index_stride + j]
                                              : (int64_t) static_cast<const int32_t*>(a.index)[r * a.index_stride + j];
    };
    auto logit_at = [&](int j) {
        return a.teacher_dtype == kF32    ? teacher_at<float>(a, r, j)
               : a.teacher_dtype == kBF16 ? teacher_at<__nv_bfloat16>(a, r, j)
                                          : teacher_at<__half>(a, r, j);
    };
    const int64_t first_index = t < a.top ? index_at(t) : -1;
    const float first_logit = t < a.top ? logit_at(t) : -INFINITY;
    auto put_entries = [&] {
        for (int j = t; j < (a.top + 3) / 4 * 4; j += kBlock) {
            const int64_t i = j >= a.top ? -1 : j == t ? first_index : index_at(j);
            const bool ok = i >= 0 && i < a.vocab;
            const float x = !ok ? -INFINITY : j == t ? first_logit : logit_at(j);
            at[j] = ok ? (int)i : -1;
            p[j] = x;
            zt[j] = ok ? to_f32(z[i]) : 0.f;
            if (x != -INFINITY) any_entry = 1;
        }
    };
    // The student's normalizer.
    float lse = 0.f;
    MaxSum mine{kLowest, 0.f};
    const float c = a.inv_temperature * kLog2e;
    __syncthreads();
    if (PASS == kDistillBackward) {
        lse = a.lse_in[r];
        put_entries();
    } else {
        const RowReader<T, PASS == kDistillLossGrad> row(z0, a.logits_stride, a.rows, r, a.vocab);
        mine = row.phase ? stream_max_sum<T, PASS == kDistillLossGrad, kBlock, true>(row, begin, end, c)
                         : stream_max_sum<T, PASS == kDistillLossGrad, kBlock, false>(row, begin, end, c);
        put_entries();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            mine = join(mine, {__shfl_xor_sync(0xffffffffu, mine.m, o), __shfl_xor_sync(0xffffffffu, mine.s, o)}, c);
        if (lane == 0) warp_part[t >> 5] = make_float2(mine.m, mine.s);
    }
    // What the CTAs of the row have to know of one another: lse, and that all
    // have read zt (dz may take the logits' place).
    auto ready = [&] {
        if (PASS == kDistillBackward) {
            if (cluster > 1) cluster_sync_all();
            else __syncthreads();
            return lse;
        }
        __syncthreads();
        // every warp joins the warps' parts, a lane each
        const float2 part = warp_part[lane % kWarps];
        mine = {part.x, part.y};
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1)
            mine = join(mine, {__shfl_xor_sync(0xffffffffu, mine.m, o), __shfl_xor_sync(0xffffffffu, mine.s, o)}, c);
        if (cluster > 1) {
            if (t == 0) cta_part = make_float2(mine.m, mine.s);
            cluster_sync_all();
            const float2 other = cluster_read(&cta_part, lane % cluster);
            mine = {other.x, other.y};
            for (int o = cluster / 2; o > 0; o >>= 1)
                mine = join(mine, {__shfl_xor_sync(0xffffffffu, mine.m, o), __shfl_xor_sync(0xffffffffu, mine.s, o)}, c);
        }
        return fmaf(mine.m, a.inv_temperature, logf(mine.s));
    };
    // The teacher's distribution, and the loss, by the first warp.
    auto teach = [&] {
        const bool any = any_entry != 0;
        float top = -INFINITY, total = 0.f, loss = 0.f;
        for (int j = lane; j < a.top; j += 32) top = larger(top, p[j]);
        top = warp_max(top);
        for (int j = lane; j < a.top; j += 32)
            if (p[j] != -INFINITY) total += expf((p[j] - top) * a.inv_temperature);
        total = warp_sum(total);
        const float log_total = logf(total);
        for (int j = lane; j < a.top; j += 32) {
            const float logp = (p[j] - top) * a.inv_temperature - log_total;
            const float pj = any && at[j] >= 0 ? expf(logp) : 0.f;
            if (pj != 0.f) loss += pj * (logp - fmaf(zt[j], a.inv_temperature, -lse));
            p[j] = pj;
        }
        if (PASS != kDistillBackward) {
            loss = warp_sum(loss);
            if (t == 0 && rank == 0) {
                a.loss[r] = any ? w * a.temperature * a.temperature * loss : 0.f;
                if (a.lse) a.lse[r] = lse;
            }
        }
    };
    if (PASS == kDistillForward) {
        lse = ready();
        if (t < 32) teach();
    } else {
        const float g = scale * a.temperature;
        const RowReader<T, false> row(z0, a.logits_stride, a.rows, r, a.vocab);
        stream_gradient<T, kBlock>(row, dz, begin, end, a.inv_temperature, g, [&] { return lse = ready(); });
        if (t < 32) teach();
        __syncthreads();
        if (any_entry == 0) {  // no teacher: what was just written goes back to 0
            stream_zeros<T, kBlock>(dz, begin, end, a.vocab);
        } else {
            for (int j = t; j < a.top; j += kBlock) {
                const int v = at[j];
                if (v < begin * kVec || v >= end * kVec) continue;
                float sum = 0.f;
                bool first = true;
                for (int i = 0; i < a.top; i += 4) {  // (p of the entries past top is -inf: never at v)
                    const int4 i4 = *reinterpret_cast<const int4*>(at + i);
                    const float4 p4 = *reinterpret_cast<const float4*>(p + i);
                    if (i4.x == v) { first &= i >= j; sum += p4.x; }
                    if (i4.y == v) { first &= i + 1 >= j; sum += p4.y; }
                    if (i4.z == v) { first &= i + 2 >= j; sum += p4.z; }
                    if (i4.w == v) { first &= i + 3 >= j; sum += p4.w; }
                }
                if (first) dz[v] = from_f32<T>(g * (exp2_fast(fmaf(zt[j], a.inv_temperature, -lse) * kLog2e) - sum));
            }
        }
    }
    if (cluster > 1 && PASS != kDistillBackward) cluster_sync_all();  // no CTA leaves while another may read its part
}

// ---- many rows: a persistent CTA per SM -----------------------------------------
//
// For loss and gradient together, a row passes through a ring of chunks in
// shared memory, filled by bulk copies.  The last chunks of the row stay in
// the ring from the first pass (maximum and sum) to the second (gradient), so
// that a row that fits is read once, from HBM; of a longer one, the first
// chunks are copied again, from L2.  Each chunk that the second pass frees is
// refilled at once, with the next row's: the copies never pause.  Sixteen
// warps compute, one fills the ring, four work on the teacher's entries.

constexpr int kRingBlock = 512;                 // computing threads
constexpr int kTeachers = 128;
constexpr int kRingThreads = kRingBlock + 32 + kTeachers;
constexpr int kEach = 4;                        // vectors of a chunk per computing thread
constexpr int kChunkVecs = kEach * kRingBlock;
constexpr int kSlotBytes = kChunkVecs * 16;
constexpr int kSlots = 6;

__device__ unsigned g_gave_up;  // threads that saw a bounded wait run out, on this device

// What the teachers know of a row: entries, their probabilities (then their
// logarithms), the student's logits there, and for the first entry of each
// place the sum of the probabilities at that place (-1 for a repeated one).
struct Lesson {
    __align__(16) int at[SOMA_DISTILL_MAX_TOP];
    __align__(16) float p[SOMA_DISTILL_MAX_TOP];
    float zt[SOMA_DISTILL_MAX_TOP], sum[SOMA_DISTILL_MAX_TOP];
};

// Rows that count are numbered 0, 1, ...; row k uses lesson, lse and barriers
// k % 2.  The teachers prepare row k + 1 while row k streams, and finish row
// k - 1 (loss and the gradient at its entries) before that.
struct RingShared {
    Lesson lesson[2];
    uint64_t full[kSlots], empty[kSlots];
    uint64_t taught[2];      // the row's lesson is ready, and zt is read
    uint64_t normalized[2];  // lse is known
    uint64_t done[2];        // the row's gradient is written
    float2 warp_part[2][kRingBlock / 32];
    float lse[2];
    float loss[kTeachers / 32];
    int any[2], gave_up;
};

// Chunk c of row r in memory.  Rows start on 16-byte boundaries; the words
// that hold a row's end are copied with it where they lie in the matrix's own
// span, and patched in where that ends first.
template <typename T>
struct Chunks {
    static constexpr int kVec = 16 / sizeof(T), kCols = kChunkVecs * kVec;
    const T* base;
    int64_t stride, rows;
    int cols, count;
    __device__ __forceinline__ const T* first(int64_t r, int c) const { return base + r * stride + (int64_t)c * kCols; }
    __device__ __forceinline__ int size(int c) const { return min(kCols, cols - c * kCols); }
    // The last row's last chunk, where it does not fill its last word.
    __device__ __forceinline__ bool cut(int64_t r, int c) const {
        return c == count - 1 && r == rows - 1 && cols % kVec != 0;
    }
    __device__ __forceinline__ void copy(int64_t r, int c, uint32_t slot, uint32_t bar) const {
        const uint32_t words = (uint32_t)(size(c) + (cut(r, c) ? 0 : kVec - 1)) / kVec;
        mbar_expect(bar, words * 16);
        if (words) bulk_load(slot, first(r, c), words * 16, bar);
    }
    __device__ __forceinline__ void patch(int64_t r, int c, char* slot, int t) const {
        const int n = size(c), whole = n / kVec * kVec;
        if (t < n - whole) reinterpret_cast<T*>(slot)[whole + t] = first(r, c)[whole + t];
    }
};

template <typename T>
__global__ void __launch_bounds__(kRingThreads) distill_ring_kernel(const __grid_constant__ DistillArgs a) {
    constexpr int kVec = 16 / sizeof(T), kWarps = kRingBlock / 32;
    extern __shared__ __align__(128) char dynamic[];
    RingShared& sh = *reinterpret_cast<RingShared*>(dynamic + kSlots * kSlotBytes);
    const int t = threadIdx.x, lane = t & 31;
    const Chunks<T> z{static_cast<const T*>(a.logits), a.logits_stride, a.rows, a.vocab,
                      (a.vocab + kChunkVecs * kVec - 1) / (kChunkVecs * kVec)};
    // chunks that do not stay in the ring until the second pass
    const int spilled = max(0, z.count - kSlots);
    const uint32_t full = smem_addr(sh.full), empty = smem_addr(sh.empty);
    const uint32_t taught = smem_addr(sh.taught), normalized = smem_addr(sh.normalized), done = smem_addr(sh.done);
    if (t == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, kWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(taught + 8 * i, kTeachers);
            mbar_init(normalized + 8 * i, 1);
            mbar_init(done + 8 * i, kWarps);
        }
        mbar_init_fence();
        sh.gave_up = 0;
    }
    __syncthreads();
    auto scale_of = [&](int64_t r) { return a.row_weight ? a.row_weight[r] : 1.f; };

    if (t >= kRingBlock && t < kRingBlock + 32) {  // fills the ring
        if (lane == 0) {
            int slot = 0;
            uint32_t parity = 1;  // a fresh barrier's previous phase counts as done
            float next = blockIdx.x < a.rows ? scale_of(blockIdx.x) : 0.f;
            for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
                const float scale = next;
                if (r + gridDim.x < a.rows) next = scale_of(r + gridDim.x);
                if (scale == 0.f) continue;
                for (int j = 0; j < z.count + spilled; ++j) {
                    mbar_wait(empty + 8 * slot, parity, &sh.gave_up);
                    z.copy(r, j < z.count ? j : j - z.count, smem_addr(dynamic + slot * kSlotBytes), full + 8 * slot);
                    if (++slot == kSlots) {
                        slot = 0;
                        parity ^= 1;
                    }
                }
            }
        }
    } else if (t >= kRingBlock + 32) {  // the teachers
        const int u = t - kRingBlock - 32;
        auto sync = [] { asm volatile("bar.sync 2, %0;" ::"n"(kTeachers) : "memory"); };
        constexpr int kMine = SOMA_DISTILL_MAX_TOP / kTeachers;
        auto next_row = [&](int64_t r) {  // the next row from r on that counts; the others' results
            for (; r < a.rows && scale_of(r) == 0.f; r += gridDim.x)
                if (u == 0) {
                    a.loss[r] = 0.f;
                    if (a.lse) a.lse[r] = 0.f;
                }
            return r;
        };
        // Row r into lesson b, up to its probabilities.
        auto prepare = [&](int64_t r, int b) {
            Lesson& l = sh.lesson[b];
            const T* row = z.first(r, 0);
            bool any = false;
            int64_t index[kMine];
#pragma unroll
            for (int q = 0; q < kMine; ++q) {
                const int j = q * kTeachers + u;
                index[q] = -1;
                if (j < a.top)
                    index[q] = a.index_type == SOMA_INDEX_I64
                                   ? static_cast<const int64_t*>(a.index)[r * a.index_stride + j]
                                   : static_cast<const int32_t*>(a.index)[r * a.index_stride + j];
            }
#pragma unroll
            for (int q = 0; q < kMine; ++q) {
                const int j = q * kTeachers + u;
                if (j >= (a.top + 3) / 4 * 4) break;
                const bool ok = index[q] >= 0 && index[q] < a.vocab;
                float x = -INFINITY;
                if (ok)
                    x = a.teacher_dtype == kF32    ? teacher_at<float>(a, r, j)
                        : a.teacher_dtype == kBF16 ? teacher_at<__nv_bfloat16>(a, r, j)
                                                   : teacher_at<__half>(a, r, j);
                l.zt[j] = ok ? to_f32(row[index[q]]) : 0.f;
                l.at[j] = ok ? (int)index[q] : -1;
                l.p[j] = x;
                any |= x != -INFINITY;
            }
            if (u == 0) sh.any[b] = 0;
            sync();
            if (any) sh.any[b] = 1;
            // every warp forms the same statistics; each thread then its own entries' p
            float top = -INFINITY, total = 0.f;
            for (int j = lane; j < a.top; j += 32) top = larger(top, l.p[j]);
            top = warp_max(top);
            for (int j = lane; j < a.top; j += 32)
                if (l.p[j] != -INFINITY) total += expf((l.p[j] - top) * a.inv_temperature);
            total = warp_sum(total);
            const float log_total = logf(total);
            sync();
            float logp[kMine];
#pragma unroll
            for (int q = 0; q < kMine; ++q) {
                const int j = q * kTeachers + u;
                logp[q] = -INFINITY;
                if (j >= a.top) break;
                if (sh.any[b] && l.at[j] >= 0) logp[q] = (l.p[j] - top) * a.inv_temperature - log_total;
                l.p[j] = expf(logp[q]);
            }
            sync();
            mbar_arrive(taught + 8 * b);  // zt is read and sh.any is set: the gradient may be written
#pragma unroll 1
            for (int j = u; j < a.top; j += kTeachers) {
                const int v = l.at[j];
                float sum = 0.f;
                bool first = v >= 0;
                for (int i = 0; i < a.top; i += 4) {  // (entries past top are at -1)
                    const int4 i4 = *reinterpret_cast<const int4*>(l.at + i);
                    const float4 p4 = *reinterpret_cast<const float4*>(l.p + i);
                    if (i4.x == v) { first &= i >= j; sum += p4.x; }
                    if (i4.y == v) { first &= i + 1 >= j; sum += p4.y; }
                    if (i4.z == v) { first &= i + 2 >= j; sum += p4.z; }
                    if (i4.w == v) { first &= i + 3 >= j; sum += p4.w; }
                }
                l.sum[j] = first ? sum : -1.f;  // (a NaN sum is not -1)
            }
            sync();  // (the probabilities make room for their logarithms)
#pragma unroll
            for (int q = 0; q < kMine; ++q)
                if (q * kTeachers + u < a.top) l.p[q * kTeachers + u] = logp[q];
        };
        // The k-th row that counts: its loss, and the gradient at its entries.
        auto finish = [&](int64_t r, int k) {
            const int b = k & 1;
            const uint32_t parity = (k >> 1) & 1;
            const Lesson& l = sh.lesson[b];
            mbar_wait(normalized + 8 * b, parity, &sh.gave_up);
            const float lse = sh.lse[b];
            float loss = 0.f;
            for (int j = u; j < a.top; j += kTeachers) {
                const float logp = l.p[j], p = expf(logp);
                if (p != 0.f) loss += p * (logp - fmaf(l.zt[j], a.inv_temperature, -lse));
            }
            loss = warp_sum(loss);
            if (lane == 0) sh.loss[u >> 5] = loss;
            sync();
            if (u == 0) {
                const float w = scale_of(r);
                loss = (sh.loss[0] + sh.loss[1]) + (sh.loss[2] + sh.loss[3]);
                a.loss[r] = sh.any[b] ? w * a.temperature * a.temperature * loss : 0.f;
                if (a.lse) a.lse[r] = lse;
            }
            const float g = scale_of(r) * a.temperature;
            mbar_wait(done + 8 * b, parity, &sh.gave_up);
            T* dz = static_cast<T*>(a.dlogits) + r * a.dlogits_stride;
            if (sh.any[b])
                for (int j = u; j < a.top; j += kTeachers)
                    if (l.sum[j] != -1.f)
                        dz[l.at[j]] = from_f32<T>(g * (exp2_fast(fmaf(l.zt[j], a.inv_temperature, -lse) * kLog2e) - l.sum[j]));
            sync();  // the lesson may go
        };
        int64_t r = next_row(blockIdx.x), before = 0;
        int k = 0;
        for (; r < a.rows; ++k) {
            prepare(r, k & 1);
            if (k > 0) finish(before, k - 1);
            before = r;
            r = next_row(r + gridDim.x);
        }
        if (k > 0) finish(before, k - 1);
    } else {
        const float c = a.inv_temperature * kLog2e;
        const int warp = t >> 5;
        int slot = 0, k = 0;
        uint32_t parity = 0;
        auto advance = [&] {
            if (++slot == kSlots) {
                slot = 0;
                parity ^= 1;
            }
        };
        auto release = [&](int s) {
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * s);
        };
        float next = blockIdx.x < a.rows ? scale_of(blockIdx.x) : 0.f;
        for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
            const float scale = next;
            if (r + gridDim.x < a.rows) next = scale_of(r + gridDim.x);
            T* dz = static_cast<T*>(a.dlogits) + r * a.dlogits_stride;
            if (scale == 0.f) {
                stream_zeros<T, kRingBlock>(dz, 0, (a.vocab + kVec - 1) / kVec, a.vocab);
                continue;
            }
            auto arrived = [&](int j) {  // chunk j is in the current slot
                mbar_wait(full + 8 * slot, parity, &sh.gave_up);
                if (z.cut(r, j)) {
                    z.patch(r, j, dynamic + slot * kSlotBytes, t);
                    fence_to_async();  // (before a later copy into the slot)
                    asm volatile("bar.sync 1, %0;" ::"n"(kRingBlock) : "memory");
                }
            };
            // Vector i of the chunk at `at`, of n elements; -inf past its end.
            auto vector = [&](const char* at, int i, int n, float (&x)[kVec]) {
                widen16(*reinterpret_cast<const uint4*>(at + i * 16), x, T{});
                if (kVec * (i + 1) > n) {
#pragma unroll
                    for (int q = 0; q < kVec; ++q)
                        if (kVec * i + q >= n) x[q] = -INFINITY;
                }
            };
            const int b = k & 1, first_slot = slot;
            MaxSum mine{kLowest, 0.f};
            for (int j = 0; j < z.count; ++j) {
                arrived(j);
                const int n = z.size(j);
                const char* at = dynamic + slot * kSlotBytes;
                if (n == Chunks<T>::kCols) {  // all of the thread's vectors at once
                    float x[kEach][kVec];
#pragma unroll
                    for (int q = 0; q < kEach; ++q) vector(at, t + q * kRingBlock, n, x[q]);
                    take_many<T>(mine, x, c);
                } else {
                    for (int i = t; i * kVec < n; i += kRingBlock) {
                        float x[kVec];
                        vector(at, i, n, x);
                        take<T>(mine, x, c);
                    }
                }
                if (j < spilled) release(slot);
                advance();
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                mine = join(mine, {__shfl_xor_sync(0xffffffffu, mine.m, o), __shfl_xor_sync(0xffffffffu, mine.s, o)}, c);
            if (lane == 0) sh.warp_part[b][warp] = make_float2(mine.m, mine.s);
            asm volatile("bar.sync 1, %0;" ::"n"(kRingBlock) : "memory");
            const float2 part = sh.warp_part[b][lane % kWarps];
            mine = {part.x, part.y};
#pragma unroll
            for (int o = kWarps / 2; o > 0; o >>= 1)
                mine = join(mine, {__shfl_xor_sync(0xffffffffu, mine.m, o), __shfl_xor_sync(0xffffffffu, mine.s, o)}, c);
            const float lse = fmaf(mine.m, a.inv_temperature, logf(mine.s));
            mbar_wait(taught + 8 * b, (k >> 1) & 1, &sh.gave_up);
            if (t == 0) {
                sh.lse[b] = lse;
                mbar_arrive(normalized + 8 * b);
            }
            const bool any = sh.any[b] != 0;
            const float g = scale * a.temperature;
            auto gradient = [&](int s, int j) {  // of chunk j in slot s
                const int n = z.size(j);
                const char* at = dynamic + s * kSlotBytes;
                T* out = dz + (int64_t)j * Chunks<T>::kCols;
                if (any && n == Chunks<T>::kCols) {
                    float x[kEach][kVec];
#pragma unroll
                    for (int q = 0; q < kEach; ++q) vector(at, t + q * kRingBlock, n, x[q]);
                    release(s);
#pragma unroll
                    for (int q = 0; q < kEach; ++q) scaled_softmax<T>(x[q], a.inv_temperature, lse, g);
#pragma unroll
                    for (int q = 0; q < kEach; ++q)
                        __stcs(reinterpret_cast<uint4*>(out) + t + q * kRingBlock, narrow16(x[q], T{}));
                    return;
                }
#pragma unroll 1
                for (int i = t; i * kVec < n; i += kRingBlock) {
                    float x[kVec];
                    vector(at, i, n, x);
                    scaled_softmax<T>(x, a.inv_temperature, lse, g);
#pragma unroll
                    for (int q = 0; q < kVec; ++q) x[q] = any ? x[q] : 0.f;
                    store_vector<T, true>(out, kVec * i, n, 0, x);
                }
                release(s);
            };
            // the chunks that stayed, then those copied again
            int s = (first_slot + spilled) % kSlots;
            for (int j = spilled; j < z.count; ++j) {
                gradient(s, j);
                if (++s == kSlots) s = 0;
            }
            for (int j = 0; j < spilled; ++j) {
                arrived(j);
                gradient(slot, j);
                advance();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(done + 8 * b);
            ++k;
        }
    }
    if (sh.gave_up) {
        atomicAdd(&g_gave_up, 1u);
        outlast_copies();
    }
}

template <typename T>
int launch_ring(const DistillArgs& a, int sm_count, cudaStream_t stream) {
    auto kernel = distill_ring_kernel<T>;
    const int smem = kSlots * kSlotBytes + (int)sizeof(RingShared);
    const int e = allow_smem((const void*)kernel, smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)std::min<int64_t>(a.rows, sm_count), kRingThreads, smem, stream>>>(a);
    return (int)cudaGetLastError();
}

// CTAs that share a row: enough to fill the device with few rows, each with
// at least 16 KB of logits.
int cluster_of(const DistillArgs& a, int64_t row_bytes, int64_t ctas) {
    int cluster = 1;
    while (cluster < kMaxCluster && row_bytes >= cluster * 2 * 16384 && a.rows * cluster * 2 <= ctas) cluster *= 2;
    return cluster;
}

template <typename T, int kBlock>
int launch_rows(const DistillArgs& a, DistillPass pass, int sm_count, cudaStream_t stream) {
    auto kernel = pass == kDistillForward    ? distill_kernel<T, kDistillForward, kBlock>
                  : pass == kDistillBackward ? distill_kernel<T, kDistillBackward, kBlock>
                                             : distill_kernel<T, kDistillLossGrad, kBlock>;
    int cluster = cluster_of(a, (int64_t)a.vocab * (int)sizeof(T), (int64_t)sm_count * (1536 / kBlock));
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kBlock);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // a grid holds 2^31 - 1 CTAs: longer lists of rows go in parts
    const int64_t most = 0x7fffffff / kMaxCluster;
    int e = cudaSuccess;
    for (int64_t r0 = 0; r0 < a.rows && e == cudaSuccess; r0 += most) {
        DistillArgs part = a;
        part.rows = std::min(a.rows - r0, most);
        if (r0 > 0) {
            part.logits = static_cast<const T*>(a.logits) + r0 * a.logits_stride;
            part.teacher = static_cast<const char*>(a.teacher) + r0 * a.teacher_stride * (a.teacher_dtype == kF32 ? 4 : 2);
            part.index = static_cast<const char*>(a.index) + r0 * a.index_stride * (a.index_type == SOMA_INDEX_I64 ? 8 : 4);
            if (a.row_weight) part.row_weight = a.row_weight + r0;
            if (a.grad_loss) part.grad_loss = a.grad_loss + r0;
            if (a.lse_in) part.lse_in = a.lse_in + r0;
            if (a.loss) part.loss = a.loss + r0;
            if (a.lse) part.lse = a.lse + r0;
            if (a.dlogits) part.dlogits = static_cast<T*>(a.dlogits) + r0 * a.dlogits_stride;
        }
        cfg.gridDim = dim3((unsigned)(part.rows * cluster));
        e = (int)cudaLaunchKernelEx(&cfg, kernel, part, cluster);
    }
    return e;
}

}  // namespace

int launch_distill(const DistillArgs& a, DistillPass pass, int sm_count, void* stream) {
    return with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        auto aligned = [](const void* p, int64_t stride) {
            return (uintptr_t)p % 16 == 0 && stride * (int64_t)sizeof(T) % 16 == 0;
        };
        // The ring for rows that start on 16-byte boundaries, are longer than 32
        // KB and come at least four to an SM: 4000 rows of 32000 fp32 take 168 to
        // 192 us with it and 214 without.  Unaligned rows would pay the shifting
        // with a third of the threads (2000 x 50021 fp16, all of which count: 144 us
        // without the ring, 239 when a ring for such rows was tried; 2000 x 50024 92).
        if (pass == kDistillLossGrad && a.rows >= 4 * sm_count && (int64_t)a.vocab * (int)sizeof(T) > 32768 &&
            aligned(a.logits, a.logits_stride) && aligned(a.dlogits, a.dlogits_stride))
            return launch_ring<T>(a, sm_count, (cudaStream_t)stream);
        // short rows: 16000 x 2000 bf16 in one call 89 us with 128 threads, 214 with 512
        if ((int64_t)a.vocab * (int)sizeof(T) <= 32768) return launch_rows<T, 128>(a, pass, sm_count, (cudaStream_t)stream);
        return launch_rows<T, 512>(a, pass, sm_count, (cudaStream_t)stream);
    });
}

int read_distill_gave_up(unsigned* count) { return (int)cudaMemcpyFromSymbol(count, g_gave_up, sizeof(*count)); }

}  // namespace soma
