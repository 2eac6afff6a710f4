// The fused update of tensors whose moments are held in 8 bits (layout and
// formulas in soma_opt.h, soma_opt_step8).
//
// A warp takes a block of 256 elements, eight per lane: it widens both
// moments with the block's two scales, runs the step's AdamW in fp32, finds
// the block's new largest moments with two warp reductions, and writes codes
// and scales back.  Nothing is read or written twice: with 16-bit gradients 14
// bytes an element (26 with fp32 moments) beside the 2 that the square-sum
// reads.
//
// Bound by HBM, closely followed by instruction issue (about 60 an element):
// 302 M elements with bf16 gradients and copies 969 us a step, 5.8 TB/s (786 us
// of it in this kernel, 6.1 TB/s).  Four CTAs of 64 registers per SM: 1035 us
// with three, 1023 with five; a first form with 126 registers and 80
// instructions an element took 1658 us.  The next block is prefetched into L2
// while one is worked on.
//
// e4m3 codes come from the fp32 bits: 2^-120 times an e4m3 value has that
// value's seven bits 20 places up, subnormal ones included, so that adding
// 20 random bits and dropping as many rounds up or down with the
// probabilities that make the mean exact.  Rounding to nearest would not do:
// with beta2 = 0.999 one step moves sqrt(v) by 0.05 %, where e4m3's steps are
// 6 to 12 %, and a second moment that moves against its block's largest (all
// that move with it are carried by the scale) would stay where it is.
#include <cuda_fp8.h>
#include <math.h>

#include "ops_device.cuh"
#include "soma_kernels.h"

namespace soma {
namespace {

constexpr int kWarps = kUpdate8Block / 32;
constexpr float kTop = 448.f;  // the largest e4m3 value

// 32 bits for the element at `low` (its index in its tensor, modulo 2^32) are
//   x = low ^ key;  x = (x ^ x >> 16) A;  x = (x ^ x >> 15) B;  x ^ x >> 16.
// A lane's eight elements differ in the lowest three bits of `low`, which
// x >> 16 drops: `mixed` = x ^ x >> 16 of the first of them serves all.
__device__ __forceinline__ uint32_t random_bits(uint32_t mixed, uint32_t i) {
    uint32_t x = (mixed ^ i) * 0x49a901a7u;
    x = (x ^ (x >> 15)) * 0x5fe29a0fu;
    return x ^ (x >> 16);
}
// For the element with this index, at a multiple of 8, and its group's step count.
__device__ __forceinline__ uint32_t random_mix(int64_t index, uint32_t step) {
    const uint32_t x = (uint32_t)index ^ ((uint32_t)(index >> 32) * 0xc4a8b3f7u + step * 0x9e3779b9u);
    return x ^ (x >> 16);
}

__device__ __forceinline__ float2 from_e4m3(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return __half22float2(__half2(h));
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN where either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float reciprocal_fast(float x) {  // within 2^-23; infinite for subnormal x
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Eight elements of a lane: gradients, weights, both moments as eight codes
// each; a missing element is 0 everywhere and stays 0.
struct Eight {
    float g[8], p[8];
    uint2 m, v;
};

// The largest of a warp's magnitudes; what is not a number is above everything.
__device__ __forceinline__ float warp_top(float x) {
    const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x) & 0x7fffffffu));
    return top < 0x1p-100f ? 0.f : top;
}

// The step on a block: weights, codes and the block's scales.  m, v and
// sqrt(v) are formed by the roundings that the formulas have, one for each
// operation (no fused ones), so that a plain program in fp32 finds the same
// codes; the weights' update is fused.
__device__ __forceinline__ void step_block(Eight& x, float& ms, float& vs, const GroupHp& h, float scale, uint32_t mixed) {
    float m[8], root[8], top_m = 0.f, top_v = 0.f;
    // (the reciprocal takes subnormal numbers for 0: where eps is one, which a
    // weight without moments is divided by, everything is 2^24 times as large)
    const float up = h.eps < 0x1p-126f ? 0x1p24f : 1.f;
    const float step_size = h.step_size * up, inv_sqrt_bc2 = h.inv_sqrt_bc2 * up, eps = h.eps * up;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 a = from_e4m3((i < 4 ? x.m.x : x.m.y) >> (8 * (i % 4)) & 0xffff);
        const float2 b = from_e4m3((i < 4 ? x.v.x : x.v.y) >> (8 * (i % 4)) & 0xffff);
        m[i] = a.x * ms; m[i + 1] = a.y * ms;
        root[i] = b.x * vs; root[i + 1] = b.y * vs;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float g = x.g[i] * scale;
        m[i] = __fadd_rn(__fmul_rn(m[i], h.beta1), __fmul_rn(g, h.one_minus_beta1));
        root[i] = sqrtf(__fadd_rn(__fmul_rn(__fmul_rn(root[i], root[i]), h.beta2),
                                  __fmul_rn(__fmul_rn(g, g), h.one_minus_beta2)));
        x.p[i] = fmaf(-step_size, m[i] * reciprocal_fast(fmaf(root[i], inv_sqrt_bc2, eps)), x.p[i] * h.decay);
        top_m = max_nan(top_m, fabsf(m[i]));
        top_v = max_nan(top_v, root[i]);
    }
    top_m = warp_top(top_m);
    top_v = warp_top(top_v);
    // |x| 448 / top 2^-120: the two factors together, but for a block so large
    // that the second would lose its bits
    float inv_m = top_m > 0.f ? __fmul_rn(__frcp_rn(top_m), kTop) : 0.f;
    float inv_v = top_v > 0.f ? __fmul_rn(__frcp_rn(top_v), kTop) : 0.f;
    if (top_m > 0x1p14f || top_v > 0x1p14f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m[i] = __fmul_rn(m[i], inv_m);
            root[i] = __fmul_rn(root[i], inv_v);
        }
        inv_m = inv_v = 1.f;
    }
    const float least = top_v > 0.f ? 0x1p-129f : 0.f;
    inv_m *= 0x1p-120f;
    inv_v *= 0x1p-120f;
    uint32_t mc[8], vc[8];  // codes in the upper byte
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // (448, the block's largest, and what rounding adds to it stay below the next code: 8 is left free)
        const uint32_t chance = random_bits(mixed, i);
        const uint32_t a = __float_as_uint(fabsf(m[i]) * inv_m) + ((chance << 4 & 0xffff0u) | 8u);
        mc[i] = (a << 4 & 0x7f000000u) | (__float_as_uint(m[i]) & 0x80000000u);
        // a second moment that is not 0 gets at least the first code: m / sqrt(v) has to stay bounded
        const float y = fmaxf(root[i] * inv_v, root[i] > 0.f ? least : 0.f);
        vc[i] = (__float_as_uint(y) + ((chance >> 12 & 0xffff0u) | 8u)) << 4;
    }
    auto pack = [](const uint32_t* c) {
        return __byte_perm(__byte_perm(c[0], c[1], 0x0073), __byte_perm(c[2], c[3], 0x0073), 0x5410);
    };
    x.m = make_uint2(pack(mc), pack(mc + 4));
    x.v = make_uint2(pack(vc), pack(vc + 4));
    ms = top_m * (1.f / kTop);
    vs = top_v * (1.f / kTop);
}

// A block of 256 elements whose buffers are aligned.
template <int GT>
__device__ __forceinline__ void whole_block(const Seg8& s, int e, const GroupHp& h, float scale, uint32_t step) {
    Eight x;
    const int block = e / kStateBlock;
    float ms = __ldcs(s.ms + block), vs = __ldcs(s.vs + block);
    if (GT == kF32) {
        const uint4* g = reinterpret_cast<const uint4*>(static_cast<const float*>(s.g) + e);
        widen16(__ldcs(g), x.g, float{});
        widen16(__ldcs(g + 1), x.g + 4, float{});
    } else {
        const uint4 g = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(s.g) + e));
        if (GT == kBF16) widen16(g, x.g, __nv_bfloat16{});
        else widen16(g, x.g, __half{});
    }
    float4* p = reinterpret_cast<float4*>(s.p + e);
    const float4 p0 = __ldcs(p), p1 = __ldcs(p + 1);
    x.m = __ldcs(reinterpret_cast<const uint2*>(s.m + e));
    x.v = __ldcs(reinterpret_cast<const uint2*>(s.v + e));
    x.p[0] = p0.x; x.p[1] = p0.y; x.p[2] = p0.z; x.p[3] = p0.w;
    x.p[4] = p1.x; x.p[5] = p1.y; x.p[6] = p1.z; x.p[7] = p1.w;
    step_block(x, ms, vs, h, scale, random_mix(s.first + e, step));
    __stcs(p, make_float4(x.p[0], x.p[1], x.p[2], x.p[3]));
    __stcs(p + 1, make_float4(x.p[4], x.p[5], x.p[6], x.p[7]));
    __stcs(reinterpret_cast<uint2*>(s.m + e), x.m);
    __stcs(reinterpret_cast<uint2*>(s.v + e), x.v);
    if (s.lowdt != kNone)
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(s.plow) + e),
               s.lowdt == kBF16 ? narrow16(x.p, __nv_bfloat16{}) : narrow16(x.p, __half{}));
    if ((threadIdx.x & 31) == 0) {
        __stcs(s.ms + block, ms);
        __stcs(s.vs + block, vs);
    }
}

// A block at a tensor's end, or of one whose buffers are not aligned: one
// element at a time.
__device__ __noinline__ void ragged_block(const Seg8& s, int e, const GroupHp& h, float scale, uint32_t step) {
    Eight x;
    const int n = min(8, s.len - e), block = e / kStateBlock;
    float ms = s.ms[block], vs = s.vs[block];
    uint32_t m[2] = {}, v[2] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x.p[i] = x.g[i] = 0.f;
        if (i >= n) continue;
        x.p[i] = s.p[e + i];
        x.g[i] = s.gdtype == kF32    ? static_cast<const float*>(s.g)[e + i]
                 : s.gdtype == kBF16 ? to_f32(static_cast<const __nv_bfloat16*>(s.g)[e + i])
                                     : to_f32(static_cast<const __half*>(s.g)[e + i]);
        m[i / 4] |= (uint32_t)s.m[e + i] << (8 * (i % 4));
        v[i / 4] |= (uint32_t)s.v[e + i] << (8 * (i % 4));
    }
    x.m = make_uint2(m[0], m[1]);
    x.v = make_uint2(v[0], v[1]);
    __syncwarp();  // all lanes have read the scales
    step_block(x, ms, vs, h, scale, random_mix(s.first + e, step));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= n) continue;
        s.p[e + i] = x.p[i];
        s.m[e + i] = (uint8_t)((i < 4 ? x.m.x : x.m.y) >> (8 * (i % 4)));
        s.v[e + i] = (uint8_t)((i < 4 ? x.v.x : x.v.y) >> (8 * (i % 4)));
        if (s.lowdt == kBF16) static_cast<__nv_bfloat16*>(s.plow)[e + i] = from_f32<__nv_bfloat16>(x.p[i]);
        else if (s.lowdt == kF16) static_cast<__half*>(s.plow)[e + i] = from_f32<__half>(x.p[i]);
    }
    if ((threadIdx.x & 31) == 0) {
        s.ms[block] = ms;
        s.vs[block] = vs;
    }
}

// L2 prefetch of what a lane reads of an aligned segment from element e on.
__device__ __forceinline__ void prefetch(const Seg8& s, int e) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(s.g) + (size_t)e * (s.gdtype == kF32 ? 4 : 2)));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(s.p + e));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(s.m + e));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(s.v + e));
}

// Blocks of segments before segment k of the chunk: one warp adds them up.
__device__ __forceinline__ void block_prefix(const Seg8* segs, int ns, int* before) {
    static_assert(kMaxSegsPerChunk == 64, "two segments per lane");
    if (threadIdx.x < 32) {
        const int l = threadIdx.x;
        auto blocks = [&](int k) { return k < ns ? (segs[k].len + kStateBlock - 1) / kStateBlock : 0; };
        const int b0 = blocks(2 * l), b1 = blocks(2 * l + 1);
        int sum = b0 + b1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, sum, o);
            if (l >= o) sum += t;
        }
        before[2 * l] = sum - b0 - b1;
        before[2 * l + 1] = sum - b1;
        if (l == 31) before[64] = sum;
    }
    __syncthreads();
}

template <bool kGraph, bool kGroupDiv>
__global__ void __launch_bounds__(kUpdate8Block, 4) update8_kernel(const __grid_constant__ Update8Args a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ __align__(16) Seg8 segs[kMaxSegsPerChunk];
    __shared__ int before[kMaxSegsPerChunk + 1];
    const int warp = threadIdx.x >> 5;
    const int c = a.t.nchunks - 1 - (int)blockIdx.x;  // the gradients that the square-sum read last come first
    const int b = __ldg(a.t.chunk_begin + c), ns = __ldg(a.t.chunk_begin + c + 1) - b;
    {
        constexpr int kWords = sizeof(Seg8) / sizeof(uint4);
        const uint4* src = reinterpret_cast<const uint4*>(a.t.segs + b);
        uint4* dst = reinterpret_cast<uint4*>(segs);
        for (int i = threadIdx.x; i < kWords * ns; i += kUpdate8Block) dst[i] = __ldg(src + i);
    }
    __syncthreads();
    block_prefix(segs, ns, before);
    // up to here only the tables were read
    const int lane8 = (threadIdx.x & 31) * 8;
    int k = 0, next = 0;  // segments of this warp's block and of its next one
    auto ahead = [&](int i) {
        if (i >= before[64]) return;
        while (i >= before[next + 1]) ++next;
        const int e = (i - before[next]) * kStateBlock + lane8;
        if (segs[next].aligned && e + 8 <= segs[next].len) prefetch(segs[next], e);
    };
    ahead(warp);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float scale1 = kGroupDiv ? 0.f : __ldcg(&a.res->scale);
    for (int i = warp; i < before[64]; i += kWarps) {
        while (i >= before[k + 1]) ++k;
        ahead(i + kWarps);
        const Seg8& s = segs[k];
        const GroupHp& h = kGraph ? a.dhp[s.group] : a.groups[s.group];
        const uint32_t step = kGraph ? (uint32_t)a.dgroups[s.group].step : a.step[s.group];
        const float scale = kGroupDiv ? __ldcg(a.gscale + s.group) : scale1;
        const int first = (i - before[k]) * kStateBlock, e = first + lane8;
        if (!s.aligned || first + kStateBlock > s.len) ragged_block(s, e, h, scale, step);
        else if (s.gdtype == kF32) whole_block<kF32>(s, e, h, scale, step);
        else if (s.gdtype == kBF16) whole_block<kBF16>(s, e, h, scale, step);
        else whole_block<kF16>(s, e, h, scale, step);
    }
}

}  // namespace

int launch_update8(const Update8Args& a, void* stream, bool graph, bool overlap, bool group_div) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.t.nchunks);
    cfg.blockDim = dim3(kUpdate8Block);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = overlap ? 1 : 0;
    cudaError_t e;
    if (graph && group_div) e = cudaLaunchKernelEx(&cfg, update8_kernel<true, true>, a);
    else if (graph) e = cudaLaunchKernelEx(&cfg, update8_kernel<true, false>, a);
    else if (group_div) e = cudaLaunchKernelEx(&cfg, update8_kernel<false, true>, a);
    else e = cudaLaunchKernelEx(&cfg, update8_kernel<false, false>, a);
    if (e != cudaSuccess) return (int)e;
    return (int)cudaGetLastError();
}

}  // namespace soma
