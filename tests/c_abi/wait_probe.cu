// The kernels' bounded wait (csrc/mbarrier.cuh) on a barrier whose phase ends,
// and on one that nothing arrives at.
#include "mbarrier.cuh"

using namespace soma;

// What a product may take per pipeline stage is at most a twentieth of its
// wait's limit: 0.36 us are measured with the SM to itself.
static_assert(product_limit(1 << 24) > 20ull * (1 << 24) * 360, "a long sum's wait ends before the sum");
static_assert(product_limit(172) < 1010000000ull, "a short sum's wait is about a second");

// out[0]: did thread 0's wait succeed; out[1]: thread 32's; out[2], out[3]: nanoseconds that they took.
__global__ void probe(int arrives, unsigned long long limit, long long* out) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int gave_up;
    if (threadIdx.x == 0) {
        gave_up = 0;
        mbar_init(smem_addr(&bar), 1);
        mbar_init_fence();
    }
    __syncthreads();
    if (threadIdx.x == 64 && arrives) mbar_arrive(smem_addr(&bar));
    if (threadIdx.x == 0 || threadIdx.x == 32) {
        const uint64_t start = global_ns();
        // thread 32's own limit is a second: it leaves when thread 0 has given up
        const bool ok = threadIdx.x == 0 ? mbar_wait(smem_addr(&bar), 0, &gave_up, limit)
                                         : mbar_wait(smem_addr(&bar), 0, &gave_up);
        out[threadIdx.x / 32] = ok;
        out[2 + threadIdx.x / 32] = (long long)(global_ns() - start);
    }
}

// Launches it and brings the four values back; returns the first CUDA error.
extern "C" int run_probe(int arrives, unsigned long long limit, long long* host) {
    long long* out = nullptr;
    int e = cudaMalloc(&out, 4 * sizeof *out);
    if (e) return e;
    probe<<<1, 96>>>(arrives, limit, out);
    e = cudaGetLastError();
    if (!e) e = cudaMemcpy(host, out, 4 * sizeof *out, cudaMemcpyDeviceToHost);
    cudaFree(out);
    return e;
}
