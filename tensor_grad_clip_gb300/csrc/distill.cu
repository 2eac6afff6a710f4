// Distillation loss from a teacher's top logits (formulas in soma_ops.h).
//
// A row's logits are streamed in 16-byte vectors: the forward pass reads them
// once (maximum and sum of exponentials together, in fp32), the backward pass
// reads them once and writes the gradient, and the one-call form reads a row
// twice, the second time from L2, where the rows in progress all fit.  One
// exponential and about six other instructions per element keep the bound
// with HBM.  The teacher's entries (at most 1024) live in shared memory; one
// warp works on them while the others stream.
//
// A cluster of CTAs shares a row when there are fewer rows than CTAs that the
// device holds; the CTAs' maxima and sums are joined through distributed
// shared memory, in rank order.  Which thread takes which elements does not depend on where rows
// start in memory, so neither do the results.
#include <math.h>

#include <algorithm>

#include "mbarrier.cuh"
#include "ops_device.cuh"
#include "ops_kernels.h"
#include "soma_ops.h"

namespace soma {
namespace {

constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
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
            store_vector<T, true>(out, (int64_t)kVec * i, row.cols, 0, x);
        }
        return;
    }
    const float lse = ready();
    const int lane = threadIdx.x & 31;
    const int cols = min(row.cols, end * kVec);  // (a CTA of a cluster stores nothing past its part)
    for (int base = begin + (threadIdx.x & ~31); base < end; base += kBlock) {
        const int i = base + lane;
        if (base >= row.inner_begin && base + 32 <= inner) {
            uint4 u[1], v[1];
            if (row.phase) {
                row.template load<true, 1>(i, 0, u, v);
                row.template widen<true>(u[0], v[0], x);
            } else {
                row.template load<false, 1>(i, 0, u, v);
                row.template widen<false>(u[0], v[0], x);
            }
        } else {
            row.gather(i, x);
        }
        scaled_softmax<T>(x, inv_t, lse, g);
        store_vector<T, false>(out, (int64_t)kVec * i, cols, out_phase, x);
    }
}

template <typename T, int kBlock>
__device__ __forceinline__ void stream_zeros(T* out, int begin, int end, int cols) {
    constexpr int kVec = 16 / sizeof(T);
    const float zero[kVec] = {};
    const int out_phase = (int)((uintptr_t)out & 15);
    for (int base = begin + (threadIdx.x & ~31); base < end; base += kBlock)
        store_vector<T, false>(out, (int64_t)kVec * (base + (threadIdx.x & 31)), min(cols, end * kVec), out_phase, zero);
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
    const float scale = PASS == kDistillBackward ? a.grad_loss[r] * w : w;

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
// A row passes through a ring of chunks in shared memory, filled by bulk
// copies.  For loss and gradient together, the last chunks of the row stay in
// the ring from the first pass (maximum and sum) to the second (gradient), so
// that a row that fits is read once, from HBM; of a longer one, the first
// chunks are copied again, from L2.  Each chunk that the second pass frees is
// refilled at once, with the next row's: the copies never pause.  Sixteen
// warps compute, one fills the ring, four work on the teacher's entries.

constexpr int kRingBlock = 512;                 // computing threads
constexpr int kTeachers = 128;
constexpr int kRingThreads = kRingBlock + 32 + kTeachers;
constexpr int kChunkVecs = 1024;                // two vectors per computing thread
constexpr int kSlotBytes = kChunkVecs * 16 + 32;
constexpr int kSlots = 12;

__device__ int g_gave_up;  // a bounded wait ran out on this device

struct RingShared {
    uint64_t full[kSlots], empty[kSlots], taught, normalized, done;
    float2 warp_part[2][kRingBlock / 32];
    float lse;
    int any, gave_up;
    __align__(16) float p[SOMA_DISTILL_MAX_TOP];
    __align__(16) int at[SOMA_DISTILL_MAX_TOP];
};

// Chunk c of row r in memory.  The first and last words of the matrix's own
// span may not be whole: those are left out of the copy and patched.
template <typename T>
struct Chunks {
    static constexpr int kVec = 16 / sizeof(T), kCols = kChunkVecs * kVec;
    const T* base;
    int64_t stride, rows;
    int cols, count;
    __device__ __forceinline__ const T* first(int64_t r, int c) const { return base + r * stride + (int64_t)c * kCols; }
    __device__ __forceinline__ int size(int c) const { return min(kCols, cols - c * kCols); }
    __device__ __forceinline__ bool cut(int64_t r, int c) const {
        const uintptr_t s = (uintptr_t)first(r, c), e = s + (uintptr_t)size(c) * sizeof(T);
        return (s & ~(uintptr_t)15) < (uintptr_t)base ||
               ((e + 15) & ~(uintptr_t)15) > (uintptr_t)(base + (rows - 1) * stride + cols);
    }
    __device__ __forceinline__ void copy(int64_t r, int c, uint32_t slot, uint32_t bar) const {
        const uintptr_t s = (uintptr_t)first(r, c), e = s + (uintptr_t)size(c) * sizeof(T), a = s & ~(uintptr_t)15;
        uintptr_t lo = a, hi = (e + 15) & ~(uintptr_t)15;
        if (lo < (uintptr_t)base) lo += 16;
        if (hi > (uintptr_t)(base + (rows - 1) * stride + cols)) hi -= 16;
        const uint32_t bytes = hi > lo ? (uint32_t)(hi - lo) : 0;
        mbar_expect(bar, bytes);
        if (bytes) bulk_load(slot + (uint32_t)(lo - a), reinterpret_cast<const void*>(lo), bytes, bar);
    }
    // The elements of the chunk's first and last word, one by one.
    __device__ __forceinline__ void patch(int64_t r, int c, char* slot, int t) const {
        const T* from = first(r, c);
        T* to = reinterpret_cast<T*>(slot + ((uintptr_t)from & 15));
        const int n = size(c);
        if (t >= 2 * kVec) return;
        const int i = t < kVec ? t : n - 1 - (t - kVec);
        if (i >= 0 && i < n) to[i] = from[i];
    }
};

template <typename T, int PASS>
__global__ void __launch_bounds__(kRingThreads) distill_ring_kernel(const __grid_constant__ DistillArgs a) {
    constexpr int kVec = 16 / sizeof(T), kWarps = kRingBlock / 32, kPasses = kChunkVecs / kRingBlock;
    constexpr bool kBoth = PASS == kDistillLossGrad;
    extern __shared__ __align__(128) char dynamic[];
    RingShared& sh = *reinterpret_cast<RingShared*>(dynamic + kSlots * kSlotBytes);
    const int t = threadIdx.x, lane = t & 31;
    const Chunks<T> z{static_cast<const T*>(a.logits), a.logits_stride, a.rows, a.vocab,
                      (a.vocab + kChunkVecs * kVec - 1) / (kChunkVecs * kVec)};
    // chunks that do not stay in the ring until the second pass
    const int spilled = kBoth ? max(0, z.count - kSlots) : 0;
    const uint32_t full = smem_addr(sh.full), empty = smem_addr(sh.empty);
    const uint32_t taught = smem_addr(&sh.taught), normalized = smem_addr(&sh.normalized), done = smem_addr(&sh.done);
    if (t == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, kWarps);
        }
        mbar_init(taught, kTeachers);
        mbar_init(normalized, 1);
        mbar_init(done, kWarps);
        mbar_init_fence();
        sh.gave_up = 0;
    }
    __syncthreads();
    auto scale_of = [&](int64_t r) {
        const float w = a.row_weight ? a.row_weight[r] : 1.f;
        return kBoth ? w : a.grad_loss[r] * w;
    };

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
    } else if (t >= kRingBlock + 32) {  // the teacher's entries
        const int u = t - kRingBlock - 32;
        uint32_t parity = 0;
        auto sync = [] { asm volatile("bar.sync 2, %0;" ::"n"(kTeachers) : "memory"); };
        constexpr int kMine = SOMA_DISTILL_MAX_TOP / kTeachers;
        for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
            const float w = a.row_weight ? a.row_weight[r] : 1.f, scale = scale_of(r);
            if (scale == 0.f) {
                if (kBoth && u == 0) {
                    a.loss[r] = 0.f;
                    if (a.lse) a.lse[r] = 0.f;
                }
                continue;
            }
            const T* row = z.first(r, 0);
            float zt[kMine];  // the student's logits at this thread's entries
            bool any = false;
#pragma unroll
            for (int q = 0; q < kMine; ++q) {
                const int j = q * kTeachers + u;
                if (j >= (a.top + 3) / 4 * 4) break;
                int64_t i = -1;
                if (j < a.top)
                    i = a.index_type == SOMA_INDEX_I64 ? static_cast<const int64_t*>(a.index)[r * a.index_stride + j]
                                                       : static_cast<const int32_t*>(a.index)[r * a.index_stride + j];
                const bool ok = i >= 0 && i < a.vocab;
                float x = -INFINITY;
                zt[q] = 0.f;
                if (ok) {
                    x = a.teacher_dtype == kF32    ? teacher_at<float>(a, r, j)
                        : a.teacher_dtype == kBF16 ? teacher_at<__nv_bfloat16>(a, r, j)
                                                   : teacher_at<__half>(a, r, j);
                    zt[q] = to_f32(row[i]);
                }
                sh.at[j] = ok ? (int)i : -1;
                sh.p[j] = x;
                any |= x != -INFINITY;
            }
            if (u == 0) sh.any = 0;
            sync();
            if (any) sh.any = 1;
            sync();
            any = sh.any != 0;
            // every warp forms the same statistics; each thread then its own entries' p
            float top = -INFINITY, total = 0.f;
            for (int j = lane; j < a.top; j += 32) top = larger(top, sh.p[j]);
            top = warp_max(top);
            for (int j = lane; j < a.top; j += 32)
                if (sh.p[j] != -INFINITY) total += expf((sh.p[j] - top) * a.inv_temperature);
            total = warp_sum(total);
            const float log_total = logf(total);
            sync();
            float logp[kMine], p[kMine];
#pragma unroll
            for (int q = 0; q < kMine; ++q) {
                const int j = q * kTeachers + u;
                if (j >= a.top) break;
                logp[q] = (sh.p[j] - top) * a.inv_temperature - log_total;
                p[q] = any && sh.at[j] >= 0 ? expf(logp[q]) : 0.f;
                sh.p[j] = p[q];
            }
            sync();
            mbar_arrive(taught);  // zt is read and sh.any is set: the gradient may be written
            float sums[kMine];
            unsigned firsts = 0;
#pragma unroll
            for (int q = 0; q < kMine; ++q) {
                const int j = q * kTeachers + u;
                if (j >= a.top) break;
                const int v = sh.at[j];
                float sum = 0.f;
                bool first = v >= 0;
                for (int i = 0; i < a.top; i += 4) {  // (entries past top are at -1)
                    const int4 i4 = *reinterpret_cast<const int4*>(sh.at + i);
                    const float4 p4 = *reinterpret_cast<const float4*>(sh.p + i);
                    if (i4.x == v) { first &= i >= j; sum += p4.x; }
                    if (i4.y == v) { first &= i + 1 >= j; sum += p4.y; }
                    if (i4.z == v) { first &= i + 2 >= j; sum += p4.z; }
                    if (i4.w == v) { first &= i + 3 >= j; sum += p4.w; }
                }
                sums[q] = sum;
                firsts |= (unsigned)first << q;
            }
            float lse;
            if (kBoth) {
                mbar_wait(normalized, parity, &sh.gave_up);
                lse = sh.lse;
                float loss = 0.f;
#pragma unroll
                for (int q = 0; q < kMine; ++q)
                    if (q * kTeachers + u < a.top && p[q] != 0.f) loss += p[q] * (logp[q] - fmaf(zt[q], a.inv_temperature, -lse));
                loss = warp_sum(loss);
                sync();  // sh.p has been read by all
                if (lane == 0) sh.p[u >> 5] = loss;
                sync();
                if (u == 0) {
                    loss = (sh.p[0] + sh.p[1]) + (sh.p[2] + sh.p[3]);
                    a.loss[r] = any ? w * a.temperature * a.temperature * loss : 0.f;
                    if (a.lse) a.lse[r] = lse;
                }
            } else {
                lse = a.lse_in[r];
            }
            mbar_wait(done, parity, &sh.gave_up);
            T* dz = static_cast<T*>(a.dlogits) + r * a.dlogits_stride;
            const float g = scale * a.temperature;
#pragma unroll
            for (int q = 0; q < kMine; ++q)
                if (any && (firsts >> q & 1))
                    dz[sh.at[q * kTeachers + u]] =
                        from_f32<T>(g * (exp2_fast(fmaf(zt[q], a.inv_temperature, -lse) * kLog2e) - sums[q]));
            sync();  // sh.at has been read by all
            parity ^= 1;
        }
    } else {
        const float c = a.inv_temperature * kLog2e;
        const int warp = t >> 5;
        int slot = 0, turn = 0;
        uint32_t parity = 0, row_parity = 0;
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
        float next_lse = !kBoth && blockIdx.x < a.rows ? a.lse_in[blockIdx.x] : 0.f;
        for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
            const float scale = next;
            float lse = next_lse;
            if (r + gridDim.x < a.rows) {
                next = scale_of(r + gridDim.x);
                if (!kBoth) next_lse = a.lse_in[r + gridDim.x];
            }
            T* dz = static_cast<T*>(a.dlogits) + r * a.dlogits_stride;
            if (scale == 0.f) {
                stream_zeros<T, kRingBlock>(dz, 0, (a.vocab + kVec - 1) / kVec, a.vocab);
                continue;
            }
            const int phase = (int)((uintptr_t)z.first(r, 0) & 15), out_phase = (int)((uintptr_t)dz & 15);
            auto arrived = [&](int j) {  // chunk j is in the current slot
                mbar_wait(full + 8 * slot, parity, &sh.gave_up);
                if (z.cut(r, j)) {
                    z.patch(r, j, dynamic + slot * kSlotBytes, t);
                    fence_to_async();  // (before a later copy into the slot)
                    asm volatile("bar.sync 1, %0;" ::"n"(kRingBlock) : "memory");
                }
            };
            auto vector = [&](int s, int i, int n, float (&x)[kVec]) {  // vector i of a chunk of n elements
                const char* at = dynamic + s * kSlotBytes + i * 16;
                const uint4 u0 = *reinterpret_cast<const uint4*>(at);
                widen16(phase ? shifted<T>(u0, *reinterpret_cast<const uint4*>(at + 16), phase) : u0, x, T{});
                if (kVec * (i + 1) > n) {
#pragma unroll
                    for (int q = 0; q < kVec; ++q)
                        if (kVec * i + q >= n) x[q] = -INFINITY;
                }
            };
            const int first_slot = slot;
            if (kBoth) {
                MaxSum mine{kLowest, 0.f};
                for (int j = 0; j < z.count; ++j) {
                    arrived(j);
                    const int n = z.size(j);
#pragma unroll
                    for (int q = 0; q < kPasses; ++q) {
                        float x[kVec];
                        if ((t + q * kRingBlock) * kVec < n) {
                            vector(slot, t + q * kRingBlock, n, x);
                            take<T>(mine, x, c);
                        }
                    }
                    if (j < spilled) release(slot);
                    advance();
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    mine = join(mine, {__shfl_xor_sync(0xffffffffu, mine.m, o), __shfl_xor_sync(0xffffffffu, mine.s, o)}, c);
                if (lane == 0) sh.warp_part[turn][warp] = make_float2(mine.m, mine.s);
                asm volatile("bar.sync 1, %0;" ::"n"(kRingBlock) : "memory");
                const float2 part = sh.warp_part[turn][lane % kWarps];
                turn ^= 1;
                mine = {part.x, part.y};
#pragma unroll
                for (int o = kWarps / 2; o > 0; o >>= 1)
                    mine = join(mine, {__shfl_xor_sync(0xffffffffu, mine.m, o), __shfl_xor_sync(0xffffffffu, mine.s, o)}, c);
                lse = fmaf(mine.m, a.inv_temperature, logf(mine.s));
            }
            // the teachers are done with the row before, and have read what the gradient may replace
            mbar_wait(taught, row_parity, &sh.gave_up);
            if (kBoth && t == 0) {
                sh.lse = lse;
                mbar_arrive(normalized);
            }
            const float g = sh.any ? scale * a.temperature : 0.f;
            auto gradient = [&](int s, int j) {  // of chunk j in slot s
                const int n = z.size(j);
                T* out = dz + (int64_t)j * Chunks<T>::kCols;
#pragma unroll
                for (int q = 0; q < kPasses; ++q) {
                    const int i = t + q * kRingBlock, whole = (t & ~31) + q * kRingBlock;
                    if (whole * kVec >= n) break;  // (all lanes of a warp store together)
                    float x[kVec];
                    if (i * kVec < n) vector(s, i, n, x);
                    else
#pragma unroll
                        for (int k = 0; k < kVec; ++k) x[k] = -INFINITY;
                    scaled_softmax<T>(x, a.inv_temperature, lse, g);
                    if (g == 0.f) {
#pragma unroll
                        for (int k = 0; k < kVec; ++k) x[k] = 0.f;
                    }
                    if (out_phase == 0 && kVec * (i + 1) <= n) __stcs(reinterpret_cast<uint4*>(out) + i, narrow16(x, T{}));
                    else store_vector<T, false>(out, (int64_t)kVec * i, n, out_phase, x);
                }
                release(s);
            };
            if (kBoth) {
                // the chunks that stayed, then those copied again
                int s = (first_slot + spilled) % kSlots;
                for (int j = spilled; j < z.count; ++j) {
                    gradient(s, j);
                    if (++s == kSlots) s = 0;
                }
            }
            for (int j = 0; j < (kBoth ? spilled : z.count); ++j) {
                arrived(j);
                gradient(slot, j);
                advance();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(done);
            row_parity ^= 1;
        }
    }
    if (sh.gave_up) {
        g_gave_up = 1;
        outlast_copies();
    }
}

template <typename T>
int launch_ring(const DistillArgs& a, DistillPass pass, int sm_count, cudaStream_t stream) {
    auto kernel = pass == kDistillBackward ? distill_ring_kernel<T, kDistillBackward> : distill_ring_kernel<T, kDistillLossGrad>;
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
        if (pass != kDistillForward && a.rows >= 4 * sm_count && (int64_t)a.vocab * (int)sizeof(T) > 32768)
            return launch_ring<T>(a, pass, sm_count, (cudaStream_t)stream);
        if ((int64_t)a.vocab * (int)sizeof(T) <= 32768) return launch_rows<T, 128>(a, pass, sm_count, (cudaStream_t)stream);
        return launch_rows<T, 512>(a, pass, sm_count, (cudaStream_t)stream);
    });
}

int take_distill_gave_up(int* value) {
    int e = cudaMemcpyFromSymbol(value, g_gave_up, sizeof(int));
    if (e == cudaSuccess && *value) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_gave_up, &zero, sizeof(int));
    }
    return e;
}

}  // namespace soma
