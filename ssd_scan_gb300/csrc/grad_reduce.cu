// grad_reduce.cu -- the last step of every parameter gradient: the sum over
// row blocks of the partial sums that the backward kernels leave in their
// workspace.
//
// One CTA per 32 columns and part k: rows of threads walk the blocks (128
// contiguous bytes per warp and block, about four blocks a thread), then meet in
// shared memory.  Launched while the kernel before it ends; 3 to 10 us, mostly
// latency (95 blocks of 8192 columns: 5 us for 3 MB).  No atomics: the order of the additions is fixed, so a gradient
// has the same bits on every run.  In fp32, as a tree: at most ~8 roundings on
// the way to a sum of a hundred terms (fp64 adds and conversions run at 1/64 of
// the rate here and took most of the kernel's time).
#include "backward.cuh"
#include "sm100.cuh"

namespace ssd {
namespace {

constexpr int kMaxRows = 32;

__global__ void __launch_bounds__(32 * kMaxRows) grad_reduce_kernel(GradReduceParams p)
{
    __shared__ float part[kMaxRows][32];
    // the partial sums; plain loads, as they were not there when this grid began
    sm100::griddep_wait();
    const int k = blockIdx.y;
    float* out = p.out[k];
    if (out == nullptr) return;
    const int lane = threadIdx.x & 31, rg = threadIdx.x >> 5, rows = blockDim.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float acc[4] = {};
    if (c < p.n) {
        const float* src = p.part + (size_t)k * p.n + c;
        const size_t step = (size_t)p.nk * p.n;
        for (int i = rg; i < p.nblk; i += 4 * rows)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j * rows < p.nblk) acc[j] += src[(size_t)(i + j * rows) * step];
    }
    part[rg][lane] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
    __syncthreads();
    for (int half = rows >> 1; half > 0; half >>= 1) {  // rows: a power of two
        if (rg < half) part[rg][lane] += part[rg + half][lane];
        __syncthreads();
    }
    if (rg == 0 && c < p.n) out[(size_t)c * p.stride[k]] = part[0][lane];
}

}  // namespace

cudaError_t launch_grad_reduce(const GradReduceParams& p, cudaStream_t st)
{
    if (p.n == 0 || p.nk == 0) return cudaSuccess;
    int rows = 1;
    while (rows < kMaxRows && 4 * rows < p.nblk) rows *= 2;
    void* args[] = {const_cast<GradReduceParams*>(&p)};
    return launch_after((const void*)grad_reduce_kernel, dim3((unsigned)((p.n + 31) / 32), (unsigned)p.nk), 32 * rows, 0, st, args);
}

}  // namespace ssd
