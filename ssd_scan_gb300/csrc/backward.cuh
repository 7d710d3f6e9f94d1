// backward.cuh -- launch parameters of the gradient kernels (the backward
// passes of the conv, the scan and the gated group RMSNorm).  Not part of the
// public ABI (see include/ssd.h).
#pragma once

#include "internal.cuh"

#include <cuda.h>

namespace ssd {

// ---- host side ----------------------------------------------------------------
// [batches][rows][cols] of 2-byte (bf16) or 4-byte (fp32) elements as boxes of
// box_cols x box_rows, with the 128-byte swizzle or none.
bool make_rows_map(CUtensorMap* m, const void* base, int elem, long long cols, long long rows, int batches,
                   int box_cols, int box_rows, bool swizzle);

// Launched to overlap the end of the kernel before it on the stream, which is
// one of this call's: the kernel waits for it before it reads its results.
inline cudaError_t launch_after(const void* fn, dim3 grid, int threads, size_t smem, cudaStream_t st, void** args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// softplus as in the forward, with the full-precision exponential: the fp32
// gradients keep the rounding of their own sums
__device__ __forceinline__ float softplus_full(float v) { return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))); }

// ---- sums over blocks of rows -------------------------------------------------
// out[k][c * stride[k]] = sum_{i < nblk} part[(i * nk + k) * n + c], added in
// a fixed order (the same bits on every run); out[k] null: skipped.
constexpr int kReduceMax = 9;
struct GradReduceParams {
    const float* part;
    int nblk, nk;
    int n;
    float* out[kReduceMax];
    int stride[kReduceMax];
};
cudaError_t launch_grad_reduce(const GradReduceParams& p, cudaStream_t st);

// ---- gated group RMSNorm --------------------------------------------------------
struct GatedNormBwdParams {
    long long rows;
    int C, G;
    float eps;
    const void* y;     // [rows, C] act
    const void* z;     // [rows, C] act
    const float* w;    // [C]
    const void* dout;  // [rows, C] act
    void* dy;          // [rows, C] act
    void* dz;          // [rows, C] act
    float* part;       // [nblk, C]: each row block's share of dweight
    int nblk;
};
// Row blocks of one call (the rows of dweight partial sums in the workspace).
int gated_norm_bwd_blocks(long long rows, int C, int G, bool bf16);
cudaError_t launch_gated_norm_bwd(const GatedNormBwdParams& p, bool bf16, cudaStream_t st);

// ---- conv1d + SiLU ----------------------------------------------------------------
struct ConvBwdParams {
    int B, S, C, W;
    const void* x;       // [B,S,C] act
    const float* w;      // [C,W]
    const float* bias;   // [C] or null
    const void* st_in;   // [B,W-1,C] act or null
    const void* dout;    // [B,S,C] act
    const void* dst_out; // [B,W-1,C] act or null
    void* dx;            // [B,S,C] act
    void* dst_in;        // [B,W-1,C] act or null
    float* part;         // [nblk, W + 1, C]: dw taps, then db
    int runs;            // CTAs along a sequence's rows
    unsigned* err;
    unsigned long long wait_ns;
};
int conv_bwd_runs(int S, bool bf16);  // per sequence; nblk = B * runs
cudaError_t launch_conv1d_bwd(const ConvBwdParams& p, bool bf16, cudaStream_t st);

// ---- the scan ------------------------------------------------------------------------
struct ScanBwdParams {
    int B, S, H, P, N, G;
    unsigned flags;
    const void* xbc;       // [B,S,Cdim] act, post-conv
    const float* dt;       // [B,S,H]
    const float* dt_bias;  // [H] or null
    const float* A;        // [H]
    const float* D;        // [H] or null
    const float* h0;       // [B,H,P,N] or null
    const void* dy;        // [B,S,H,P] act
    const float* dhS;      // [B,H,P,N] or null
    void* dxbc;            // [B,S,Cdim] act
    float* ddt;            // [B,S,H]
    float* dh0;            // [B,H,P,N] or null
    // workspace
    float* hin;            // [B,H,nc,P,N]: the state at each chunk's start
    float* lout;           // [B,H,nc,P,N]: the gradient of the state at each chunk's end
    float* part;           // [B*nc, 3, H]: dA, ddt_bias, dD
    float* decay;          // [B,H,nc]: a chunk's decay
    float* bcpart;         // [split][B,S,2*G*N]: shares of dB | dC (split > 1)
    int split;             // CTAs that share the heads of a (chunk, group)
};
// One CTA walks the heads of a (chunk, group); with few of those (`units`) a
// group's heads are split over CTAs whose shares of dB and dC are added
// afterwards.  The number of CTAs that takes least time, counted as waves of `slots` x
// (heads of a CTA + `setup` heads' worth of work that a CTA does once).  Split /
// not: 100 rows of 8 heads in 2 groups 21 / 27 us; in fp32 2 x 500 rows of them 58 / 101.
int scan_bwd_split(long long units, int heads, double setup, int slots);
int scan_bwd_simt_slots(int P, int N);
// The row-exact path's chunk length (0: this P, N not supported).
int scan_bwd_simt_chunk(int P, int N);
cudaError_t launch_scan_bwd_local(const ScanBwdParams& p, bool bf16, cudaStream_t st);
cudaError_t launch_scan_bwd_carry(const ScanBwdParams& p, cudaStream_t st);
cudaError_t launch_scan_bwd_simt(const ScanBwdParams& p, bool bf16, cudaStream_t st);
// dB | dC behind `lead` columns of dxbc, from `split` shares [split][rows][cols].
cudaError_t launch_scan_bwd_join(const float* part, void* dxbc, long long rows, int lead, int cols, int split, bool bf16,
                                 cudaStream_t st);

// Tensor-core path (bf16, P = 64, N = 128).
struct ScanBwdTcParams {
    int B, S, H, G;
    unsigned flags;
    const void* xbc;       // [B,S,Cdim] bf16, post-conv
    const float* dt;       // [B,S,H]
    const float* dt_bias;  // [H] or null
    const float* A;        // [H]
    const float* D;        // [H] or null
    const float* h0;       // [B,H,P,N] or null
    const void* dy;        // [B,S,H,P] bf16
    const float* dhS;      // [B,H,P,N] or null
    void* dxbc;            // [B,S,Cdim] bf16
    float* ddt;            // [B,S,H]
    float* dh0;            // [B,H,P,N] or null
    unsigned* err;
    unsigned long long wait_ns;
    // workspace
    float* vals;           // [B,H,nc]: row values of a chunk
    __nv_bfloat16* hin;    // [B,H,nc][2][P/8][N][8]: the state at each chunk's start, hi and lo
    __nv_bfloat16* lout;   // [B,H,nc][2][P/8][N][8]: the adjoint at each chunk's end
    float* part;           // [B*nc, 3, H]: dA, ddt_bias, dD
    float* bcpart;         // [split][B,S,2*G*N]: shares of dB | dC (split > 1)
    int split;             // CTAs that share the heads of a (chunk, group)
};
struct ScanBwdTcSizes {
    size_t vals, states, part, bcpart;  // bytes
    int split;
    size_t total() const { return vals + 2 * states + part + bcpart; }
};
bool scan_bwd_tc_supports(int P, int N);
ScanBwdTcSizes scan_bwd_tc_sizes(int B, int S, int H, int G);
// The three kernels of a call, and which of them were launched.
struct ScanBwdLaunched {
    bool rows, states, chunks;
};
cudaError_t launch_scan_bwd_tc(const ScanBwdTcParams& p, cudaStream_t st, ScanBwdLaunched* done);

}  // namespace ssd
