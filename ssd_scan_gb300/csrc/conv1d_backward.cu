// conv1d_backward.cu -- gradients of the causal depthwise conv1d + SiLU
// (conv1d.cu) over u = [conv state ; rows].
//
//   v_t = bias + sum_k w_k u_{t+k},  out_t = silu(v_t),  q = sigmoid(v_t)
//   dv_t = dout_t q (1 + v_t (1 - q))
//   du_j = sum_k w_k dv_{j-k}   (+ the new conv state's gradient on the last W-1 rows)
//   dw_k = sum_t dv_t u_{t+k},  dbias = sum_t dv_t
//
// HBM-bound: x and dout read, dx written.  A CTA is 64 channels x kRuns runs of
// consecutive rows; each warp asks for its run's tiles of x and dout by TMA at
// once (rows outside the sequence come as zeros), so that three resident CTAs keep
// some 200 KB of loads in flight per SM without holding registers for them.  A thread
// owns 2 channels and walks its run: the W-1 rows before a batch stay in
// registers, as do the du that later rows still add to, so v, dv and du of a row
// come out of one pass; W-1 rows behind the run are recomputed for the du they
// reach into.  The runs' shares of dw meet in shared memory, so the partial sums
// written for the final reduction are one set per CTA.
//
// Measured, 10,240 channels of 4 taps, bf16: 2 x 8192 rows 205 us (4.9 TB/s of the
// x, dout and dx bytes), 2048 rows 37 us with 4 of the final reduction.  With
// loads to registers, a batch ahead, they took 344 and 53.  No one thing bounds the 32
// us that the kernel takes of the 2048 rows: it issues 2.05 instructions a cycle of 4, of
// the cycles between a warp's instructions 2.2 wait for its tiles and 1.9 for the fp32
// pipe (19 packed multiply-adds a row and pair of channels), and DRAM is at 37 %.
// A CTA's rows are one sequence's, so sequences shorter than its 256 rows (fp32: 128)
// leave warps without work and add partial sums: 16,384 rows as 64 sequences take 201 us
// on the GPU, as 256 426, as 512 735, as 2048 3204.
#include "backward.cuh"
#include "sm100.cuh"

#include <type_traits>

namespace ssd {
namespace {

constexpr int V = 2;         // channels per thread
constexpr int kRuns = 8;     // runs per CTA, a warp each
constexpr int kBatch = 8;    // rows in registers at a time
constexpr int kBoxRows = 16; // rows of a TMA load
constexpr int kCols = 32 * V;
constexpr uint64_t kWaitNs = 2000000000ull;  // default bound on a wait
// rows per run: a tile of x and one of dout take 35 KB each
template <typename T> constexpr int kRun = sizeof(T) == 2 ? 32 : 16;
template <typename T> constexpr int kRows = kRun<T> * kRuns;  // of a CTA

template <typename T> struct ConvSmem {
    T x[kRows<T> + kBoxRows][kCols];  // from row T0 - (W-1) on
    T d[kRows<T> + kBoxRows][kCols];  // from row T0 on
    uint64_t full[kRuns + 1];         // a run's boxes; the last: the rows behind them
};

template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    typedef uint32_t raw;
    __device__ static raw load(const __nv_bfloat16* p) { return *reinterpret_cast<const uint32_t*>(p); }
    __device__ static float2 unpack(raw r) { return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r)); }
    __device__ static void store(__nv_bfloat16* p, float2 v)
    {
        *reinterpret_cast<__nv_bfloat162*>(p) = __float22bfloat162_rn(v);
    }
};
template <> struct Pair<float> {
    typedef float2 raw;
    __device__ static raw load(const float* p) { return *reinterpret_cast<const float2*>(p); }
    __device__ static float2 unpack(raw r) { return r; }
    __device__ static void store(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
};

__device__ __forceinline__ float2 bcast(float v) { return make_float2(v, v); }
__device__ __forceinline__ float ex2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_fast(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// dout silu'(v), through an exponential and a reciprocal (a few ulp: dw is an
// fp32 sum, which the forward's hardware tanh, 2^-11, would not serve)
__device__ __forceinline__ float2 dsilu(float2 v, float2 d)
{
    const float2 n = __fmul2_rn(v, bcast(-1.4426950408889634f));
    const float2 e = __fadd2_rn(make_float2(ex2_fast(n.x), ex2_fast(n.y)), bcast(1.0f));
    const float2 q = make_float2(rcp_fast(e.x), rcp_fast(e.y));
    const float2 t = __ffma2_rn(v, __ffma2_rn(q, bcast(-1.0f), bcast(1.0f)), bcast(1.0f));
    return __fmul2_rn(d, __fmul2_rn(q, t));
}

template <typename T, int W>
__global__ void __launch_bounds__(32 * kRuns, W <= 4 ? 3 : 2)
    conv1d_bwd_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_d,
                      const ConvBwdParams p)
{
    typedef Pair<T> PT;
    constexpr int M = kBatch + W - 1;  // rows a batch reads, and adds to
    extern __shared__ __align__(128) uint8_t smem_raw[];
    ConvSmem<T>& s = *reinterpret_cast<ConvSmem<T>*>(smem_raw);
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int b = blockIdx.z, T0 = blockIdx.y * kRows<T>, t0 = T0 + run * kRun<T>;
    if (threadIdx.x == 0) {
        for (int k = 0; k <= kRuns; ++k) sm100::mbar_init(&s.full[k], 1);
        sm100::fence_mbar_init();
    }
    sm100::griddep_launch_dependents();
    __syncthreads();
    if (lane == 0) {
        auto load = [&](uint64_t* bar, int at, int boxes) {
            sm100::mbar_arrive_expect_tx(bar, boxes * 2 * kBoxRows * kCols * sizeof(T));
            for (int k = 0; k < boxes; ++k, at += kBoxRows) {
                sm100::tma_load_3d(s.x[at], &map_x, bar, blockIdx.x * kCols, T0 - (W - 1) + at, b);
                sm100::tma_load_3d(s.d[at], &map_d, bar, blockIdx.x * kCols, T0 + at, b);
            }
        };
        load(&s.full[run], run * kRun<T>, kRun<T> / kBoxRows);
        if (run == kRuns - 1) load(&s.full[kRuns], kRows<T>, 1);
    }
    const int ch = blockIdx.x * kCols + lane * V;
    const bool on = ch < p.C;
    const int c0 = on ? ch : 0;
    const T* st = p.st_in ? static_cast<const T*>(p.st_in) + (size_t)b * (W - 1) * p.C + c0 : nullptr;
    const T* ds = p.dst_out ? static_cast<const T*>(p.dst_out) + (size_t)b * (W - 1) * p.C + c0 : nullptr;
    T* dsi = p.dst_in ? static_cast<T*>(p.dst_in) + (size_t)b * (W - 1) * p.C + c0 : nullptr;

    float2 w[W], dw[W], db = bcast(0.0f);
    const float2 bias = p.bias ? make_float2(__ldg(p.bias + c0), __ldg(p.bias + c0 + 1)) : bcast(0.0f);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        w[k] = make_float2(__ldg(p.w + (size_t)c0 * W + k), __ldg(p.w + (size_t)(c0 + 1) * W + k));
        dw[k] = bcast(0.0f);
    }
    // this run's tiles, and the rows of the next that it looks at
    const uint64_t wait = p.wait_ns ? p.wait_ns : kWaitNs;
    const bool ok = sm100::mbar_wait_ns(&s.full[run], 0, wait) && sm100::mbar_wait_ns(&s.full[run + 1], 0, wait);
    if (ok && on && t0 < p.S) {
        const T* xs = &s.x[run * kRun<T>][lane * V];  // row t0 - (W-1)
        const T* dr = &s.d[run * kRun<T>][lane * V];  // row t0
        // u[m], du[m]: row tb - (W-1) + m of [state ; rows]
        float2 u[M], du[M];
#pragma unroll
        for (int m = 0; m < W - 1; ++m) {
            u[m] = PT::unpack(PT::load(t0 == 0 && st ? st + (size_t)m * p.C : xs + m * kCols));
            du[m] = bcast(0.0f);
        }
        const unsigned C = (unsigned)p.C;
        T* ob = static_cast<T*>(p.dx) + ((size_t)b * p.S + t0) * C + c0 - (ptrdiff_t)(W - 1) * C;
        const int hot = ds ? p.S - (W - 1) : p.S;  // rows from here on take the slow way
        // dv of row tb + i, from u[i ..]; and into du
        auto row = [&](int i) {
            u[W - 1 + i] = PT::unpack(PT::load(xs + (W - 1 + i) * kCols));
            du[W - 1 + i] = bcast(0.0f);
            float2 v = bias;
#pragma unroll
            for (int k = 0; k < W; ++k) v = __ffma2_rn(w[k], u[i + k], v);
            // rows from S on have dout 0
            const float2 d = dsilu(v, PT::unpack(PT::load(dr + i * kCols)));
#pragma unroll
            for (int k = 0; k < W; ++k) du[i + k] = __ffma2_rn(w[k], d, du[i + k]);
            return d;
        };
        // the gradients of rows j0 .. j0 + n - 1
        auto out = [&](int j0, auto n) {
            if (j0 >= t0 && j0 + n <= hot) {
#pragma unroll
                for (int i = 0; i < n; ++i) PT::store(ob + (size_t)i * C, du[i]);
            } else {
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const int j = j0 + i;
                    if (j >= p.S || (j < t0 && t0 != 0)) continue;
                    float2 o = du[i];
                    if (ds != nullptr && j >= p.S - (W - 1))  // row j - (S - (W-1)) of the new state
                        o = __fadd2_rn(o, PT::unpack(PT::load(ds + (size_t)(j - (p.S - (W - 1))) * p.C)));
                    if (j >= 0) PT::store(ob + (size_t)i * C, o);
                    else if (dsi != nullptr) PT::store(dsi + (size_t)(j + W - 1) * p.C, o);
                }
            }
        };
#pragma unroll 1
        for (int tb = t0; tb < t0 + kRun<T>; tb += kBatch) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const float2 d = row(i);
                db = __fadd2_rn(db, d);
#pragma unroll
                for (int k = 0; k < W; ++k) dw[k] = __ffma2_rn(d, u[i + k], dw[k]);
            }
            // rows tb - (W-1) .. tb - (W-1) + kBatch - 1 have every dv they are read by
            out(tb - (W - 1), std::integral_constant<int, kBatch>());
            xs += kBatch * kCols;
            dr += kBatch * kCols;
            ob += (size_t)kBatch * C;
#pragma unroll
            for (int m = 0; m < W - 1; ++m) {
                u[m] = u[kBatch + m];
                du[m] = du[kBatch + m];
            }
        }
        // the rows behind, for what they add to the run's last rows
#pragma unroll
        for (int i = 0; i < W - 1; ++i) row(i);
        out(t0 + kRun<T> - (W - 1), std::integral_constant<int, W - 1>());
    }
    if (!ok) {
        atomicOr(p.err, kErrTimeout);
        // no copy of ours in flight when the CTA leaves (bounded)
        for (int k = 0; k <= kRuns; ++k) sm100::mbar_wait_ns(&s.full[k], 0, kWaitNs);
    }
    // this CTA's share of dw and dbias, in the x tile once all are done with it
    float2(*red)[W + 1][32] = reinterpret_cast<float2(*)[W + 1][32]>(s.x);
    static_assert(sizeof(s.x) >= sizeof(float2) * kRuns * (W + 1) * 32, "room for the shares");
    __syncthreads();
#pragma unroll
    for (int k = 0; k < W; ++k) red[run][k][lane] = dw[k];
    red[run][W][lane] = db;
    __syncthreads();
    for (int k = run; k <= W; k += kRuns) {
        float2 sum = red[0][k][lane];
#pragma unroll
        for (int r = 1; r < kRuns; ++r) sum = __fadd2_rn(sum, red[r][k][lane]);
        const size_t blk = (size_t)b * p.runs + blockIdx.y;
        if (on) *reinterpret_cast<float2*>(p.part + (blk * (W + 1) + k) * p.C + c0) = sum;
    }
}

template <typename T, int W> cudaError_t launch_w(const ConvBwdParams& p, const CUtensorMap& x, const CUtensorMap& d, cudaStream_t st)
{
    auto kern = conv1d_bwd_kernel<T, W>;
    static std::atomic<bool> done[kMaxDevices];
    const cudaError_t e = allow_smem((const void*)kern, sizeof(ConvSmem<T>), done);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((p.C + kCols - 1) / kCols), (unsigned)p.runs, (unsigned)p.B);
    kern<<<grid, 32 * kRuns, sizeof(ConvSmem<T>), st>>>(x, d, p);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_t(const ConvBwdParams& p, cudaStream_t st)
{
    if (p.C % V != 0) return cudaErrorInvalidValue;
    CUtensorMap x, d;
    const int e = sizeof(T);
    if (!make_rows_map(&x, p.x, e, p.C, p.S, p.B, kCols, kBoxRows, false) ||
        !make_rows_map(&d, p.dout, e, p.C, p.S, p.B, kCols, kBoxRows, false))
        return cudaErrorInvalidValue;
    switch (p.W) {
#define SSD_CONV_BWD_CASE(w) \
    case w: return launch_w<T, w>(p, x, d, st);
        SSD_CONV_BWD_CASE(1) SSD_CONV_BWD_CASE(2) SSD_CONV_BWD_CASE(3) SSD_CONV_BWD_CASE(4)
        SSD_CONV_BWD_CASE(5) SSD_CONV_BWD_CASE(6) SSD_CONV_BWD_CASE(7) SSD_CONV_BWD_CASE(8)
#undef SSD_CONV_BWD_CASE
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

int conv_bwd_runs(int S, bool bf16)
{
    const int rows = bf16 ? kRows<__nv_bfloat16> : kRows<float>;
    const int n = (int)(((long long)S + rows - 1) / rows);
    return n < 1 ? 1 : n;
}

cudaError_t launch_conv1d_bwd(const ConvBwdParams& p, bool bf16, cudaStream_t st)
{
    if (p.S == 0) {  // the state passes through
        const size_t n = (size_t)p.B * (p.W - 1) * p.C * (bf16 ? 2 : 4);
        if (p.dst_in == nullptr || n == 0) return cudaSuccess;
        return p.dst_out ? cudaMemcpyAsync(p.dst_in, p.dst_out, n, cudaMemcpyDeviceToDevice, st)
                         : cudaMemsetAsync(p.dst_in, 0, n, st);
    }
    return bf16 ? launch_t<__nv_bfloat16>(p, st) : launch_t<float>(p, st);
}

}  // namespace ssd
