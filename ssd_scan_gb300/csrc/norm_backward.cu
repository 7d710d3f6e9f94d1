// norm_backward.cu -- gradients of the gated group RMSNorm (norm.cu).
//
// With r = 1 / sqrt(mean_group y^2 + eps), n = y r, q = sigmoid(z):
//   out = silu(z) n w
//   dz  = dout n w q (1 + z (1 - q))
//   dn  = dout silu(z) w,  dy = r (dn - n mean_group(dn n))
//   dw  = sum over rows of dout silu(z) n
// Both group means come out of one pass: sum y^2 and sum dn y (mean(dn n) =
// r sum(dn y) / gs), so y, z and dout are read once and dy, dz written once.
// HBM-bound: 5 C elements a row.  Measured, 8192 channels in 8 groups, bf16: 2 x
// 8192 rows 248 us (5.4 TB/s), 2048 rows 39 us, 5 of them the final reduction.
//
// Groups of up to 64 vectors of 16 bytes (512 bf16 / 256 fp32 channels): one warp
// per (row, group), every vector held in registers from its load to its store; a
// warp walks rows and keeps its channels' share of dw in registers (at 64
// vectors, 16 groups, 16384 / 512 rows: 220 / 10 us; a CTA each 245 / 13).  Up to 512
// vectors: one CTA per (row, group), a vector a thread, the next row's loads in
// flight while this row's sums meet in shared memory.  Wider groups: one CTA per
// (row, group), which reads the rows a second time from L1/L2 and keeps dw in its
// row of the workspace (8192 rows, 512 vectors in 2 groups: 217 us, a vector a thread
// 128; 768 vectors: 164 against 186, 1024 vectors, 4096 rows: 111 against 125).
#include "backward.cuh"
#include "sm100.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 8;
constexpr int kWide = 512;  // threads of the wide-group kernel

// 16 bytes as pairs of fp32: the arithmetic is in packed pairs, which halves its
// instructions (48 an element one by one; the kernel was bound by them)
template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    __device__ static void unpack(uint4 r, float2* v)
    {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __bfloat1622float2(h[i]);
    }
    __device__ static uint4 pack(const float2* v)
    {
        uint4 r;
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&r);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __float22bfloat162_rn(v[i]);
        return r;
    }
};
template <> struct Vec<float> {
    static constexpr int n = 4;
    __device__ static void unpack(uint4 r, float2* v)
    {
        v[0] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
        v[1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
    }
    __device__ static uint4 pack(const float2* v)
    {
        return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
    }
};
// a vector's weights
template <int V> __device__ __forceinline__ void weights(const float* p, float2* w)
{
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(p) + i);
        w[2 * i] = make_float2(f.x, f.y);
        w[2 * i + 1] = make_float2(f.z, f.w);
    }
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
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
// sigmoid through one exponential and a reciprocal (a few ulp): dw and the
// fp32 outputs need more than the forward's hardware tanh (2^-11) gives
__device__ __forceinline__ float2 sigmoid2(float2 z)
{
    const float2 n = __fmul2_rn(z, both(-1.4426950408889634f));
    const float2 e = __fadd2_rn(make_float2(ex2_fast(n.x), ex2_fast(n.y)), both(1.0f));
    return make_float2(rcp_fast(e.x), rcp_fast(e.y));
}
// a vector's share of sum y^2 and of sum dn y; q = sigmoid(z)
template <int V>
__device__ __forceinline__ void sums(const float2* y, const float2* z, const float2* d, const float2* w, float2* q, float2& ss,
                                     float2& sd)
{
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        q[i] = sigmoid2(z[i]);
        ss = __ffma2_rn(y[i], y[i], ss);
        sd = __ffma2_rn(__fmul2_rn(__fmul2_rn(d[i], __fmul2_rn(z[i], q[i])), w[i]), y[i], sd);
    }
}
// its gradients; m = r^2 sum(dn y) / gs, to be multiplied by y (r times r sum(dn y)
// / gs, which is of dn's size: r^2 alone overflows for rows below 2^-64)
template <int V>
__device__ __forceinline__ void grads(const float2* y, const float2* z, const float2* d, const float2* w, const float2* q, float r,
                                      float m, float2* oy, float2* oz, float2* dw)
{
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const float2 silu = __fmul2_rn(z[i], q[i]), t = __fmul2_rn(d[i], silu), n = __fmul2_rn(y[i], both(r));
        oy[i] = __fmul2_rn(both(r), __ffma2_rn(both(-m), y[i], __fmul2_rn(t, w[i])));
        // q (1 + z (1 - q)) = q + silu (1 - q)
        const float2 g = __ffma2_rn(silu, __ffma2_rn(q[i], both(-1.0f), both(1.0f)), q[i]);
        oz[i] = __fmul2_rn(__fmul2_rn(__fmul2_rn(d[i], w[i]), n), g);
        dw[i] = __ffma2_rn(t, n, dw[i]);
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

__device__ __forceinline__ uint4 ld16(const void* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// K vectors per lane; grid (row blocks, G); warp w of block i walks rows
// i * kWarps + w, + gridDim.x * kWarps, ..
template <typename T, int K>
__global__ void __launch_bounds__(kWarps * 32) gated_norm_bwd_kernel(GatedNormBwdParams p)
{
    constexpr int V = Vec<T>::n, H = V / 2;
    __shared__ float acc[kWarps][32 * V * K];
    sm100::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = blockIdx.y, gs = p.C / p.G;
    const float inv = 1.0f / (float)gs;
    const float* w = p.w + (size_t)g * gs;
    float2 dw[K][H];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < H; ++i) dw[k][i] = both(0.0f);

    for (long long row = (long long)blockIdx.x * kWarps + warp; row < p.rows;
         row += (long long)gridDim.x * kWarps) {
        const size_t base = (size_t)row * p.C + (size_t)g * gs;
        uint4 ry[K], rz[K], rd[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = (k * 32 + lane) * V;
            const bool in = e < gs;
            ry[k] = in ? ld16(static_cast<const T*>(p.y) + base + e) : make_uint4(0, 0, 0, 0);
            rz[k] = in ? ld16(static_cast<const T*>(p.z) + base + e) : make_uint4(0, 0, 0, 0);
            rd[k] = in ? ld16(static_cast<const T*>(p.dout) + base + e) : make_uint4(0, 0, 0, 0);
        }
        float2 s2 = both(0.0f), d2 = both(0.0f), q[K][H];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = (k * 32 + lane) * V;
            if (e >= gs) continue;
            float2 y[H], z[H], d[H], wv[H];
            Vec<T>::unpack(ry[k], y);
            Vec<T>::unpack(rz[k], z);
            Vec<T>::unpack(rd[k], d);
            weights<V>(w + e, wv);
            sums<V>(y, z, d, wv, q[k], s2, d2);
        }
        const float ss = warp_sum(s2.x + s2.y), sd = warp_sum(d2.x + d2.y);
        const float r = rsqrtf(ss * inv + p.eps), m = r * (r * (sd * inv));
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = (k * 32 + lane) * V;
            if (e >= gs) continue;
            float2 y[H], z[H], d[H], wv[H], oy[H], oz[H];
            Vec<T>::unpack(ry[k], y);
            Vec<T>::unpack(rz[k], z);
            Vec<T>::unpack(rd[k], d);
            weights<V>(w + e, wv);
            grads<V>(y, z, d, wv, q[k], r, m, oy, oz, dw[k]);
            *reinterpret_cast<uint4*>(static_cast<T*>(p.dy) + base + e) = Vec<T>::pack(oy);
            *reinterpret_cast<uint4*>(static_cast<T*>(p.dz) + base + e) = Vec<T>::pack(oz);
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < H; ++i) {
            acc[warp][(k * 32 + lane) * V + 2 * i] = dw[k][i].x;
            acc[warp][(k * 32 + lane) * V + 2 * i + 1] = dw[k][i].y;
        }
    __syncthreads();
    for (int c = threadIdx.x; c < gs; c += kWarps * 32) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) s += acc[i][c];
        p.part[(size_t)blockIdx.x * p.C + (size_t)g * gs + c] = s;
    }
}

// A vector a thread: grid (row blocks, G), block i walks rows i, i + gridDim.x, ..
template <typename T, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, kMaxThreads == 256 ? 3 : 1) gated_norm_bwd_block_kernel(GatedNormBwdParams p)
{
    constexpr int V = Vec<T>::n, H = V / 2;
    __shared__ float part[2][2][kMaxThreads / 32];
    sm100::griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    const int g = blockIdx.y, gs = p.C / p.G;
    const float inv = 1.0f / (float)gs;
    const bool in = tid * V < gs;
    const size_t col = (size_t)g * gs + (in ? tid * V : 0);
    float2 w[H], dw[H];
    weights<V>(p.w + col, w);
#pragma unroll
    for (int i = 0; i < H; ++i) dw[i] = both(0.0f);
    uint4 ry, rz, rd;
    auto load = [&](long long row) {
        const size_t o = (size_t)row * p.C + col;
        const uint4 none = make_uint4(0, 0, 0, 0);
        ry = in ? ld16(static_cast<const T*>(p.y) + o) : none;
        rz = in ? ld16(static_cast<const T*>(p.z) + o) : none;
        rd = in ? ld16(static_cast<const T*>(p.dout) + o) : none;
    };
    load(blockIdx.x);
    int par = 0;
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, par ^= 1) {
        float2 y[H], z[H], d[H], q[H], s2 = both(0.0f), d2 = both(0.0f);
        Vec<T>::unpack(ry, y);
        Vec<T>::unpack(rz, z);
        Vec<T>::unpack(rd, d);
        if (row + gridDim.x < p.rows) load(row + gridDim.x);
        sums<V>(y, z, d, w, q, s2, d2);
        float ss = warp_sum(s2.x + s2.y), sd = warp_sum(d2.x + d2.y);
        if (lane == 0) {
            part[par][0][warp] = ss;
            part[par][1][warp] = sd;
        }
        __syncthreads();  // the next row writes the other half of part
        ss = sd = 0.0f;
        for (int i = 0; i < nw; ++i) {
            ss += part[par][0][i];
            sd += part[par][1][i];
        }
        const float r = rsqrtf(ss * inv + p.eps), m = r * (r * (sd * inv));
        float2 oy[H], oz[H];
        grads<V>(y, z, d, w, q, r, m, oy, oz, dw);
        if (in) {
            const size_t o = (size_t)row * p.C + col;
            *reinterpret_cast<uint4*>(static_cast<T*>(p.dy) + o) = Vec<T>::pack(oy);
            *reinterpret_cast<uint4*>(static_cast<T*>(p.dz) + o) = Vec<T>::pack(oz);
        }
    }
    if (in)
#pragma unroll
        for (int i = 0; i < H; i += 2)
            *reinterpret_cast<float4*>(p.part + (size_t)blockIdx.x * p.C + col + 2 * i) =
                make_float4(dw[i].x, dw[i].y, dw[i + 1].x, dw[i + 1].y);
}

// Wide groups: grid (row blocks, G), one CTA per (row, group) at a time.
template <typename T>
__global__ void __launch_bounds__(kWide) gated_norm_bwd_wide_kernel(GatedNormBwdParams p)
{
    constexpr int V = Vec<T>::n, H = V / 2;
    __shared__ float part[2][2][kWide / 32];
    sm100::griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = blockIdx.y, gs = p.C / p.G;
    const float inv = 1.0f / (float)gs;
    const float* w = p.w + (size_t)g * gs;
    float* dw = p.part + (size_t)blockIdx.x * p.C + (size_t)g * gs;
    // each thread touches only its own columns of dw, in every row
    for (int e = tid * V; e < gs; e += kWide * V)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[e + i] = 0.0f;
    int par = 0;
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, par ^= 1) {
        const size_t base = (size_t)row * p.C + (size_t)g * gs;
        float2 y[H], z[H], d[H], q[H], wv[H], s2 = both(0.0f), d2 = both(0.0f);
        auto load = [&](int e) {
            Vec<T>::unpack(ld16(static_cast<const T*>(p.y) + base + e), y);
            Vec<T>::unpack(ld16(static_cast<const T*>(p.z) + base + e), z);
            Vec<T>::unpack(ld16(static_cast<const T*>(p.dout) + base + e), d);
            weights<V>(w + e, wv);
        };
        for (int e = tid * V; e < gs; e += kWide * V) {
            load(e);
            sums<V>(y, z, d, wv, q, s2, d2);
        }
        float ss = warp_sum(s2.x + s2.y), sd = warp_sum(d2.x + d2.y);
        if (lane == 0) {
            part[par][0][warp] = ss;
            part[par][1][warp] = sd;
        }
        __syncthreads();  // the next row writes the other half of part
        ss = sd = 0.0f;
#pragma unroll
        for (int i = 0; i < kWide / 32; ++i) {
            ss += part[par][0][i];
            sd += part[par][1][i];
        }
        const float r = rsqrtf(ss * inv + p.eps), m = r * (r * (sd * inv));
        for (int e = tid * V; e < gs; e += kWide * V) {
            load(e);
            float2 oy[H], oz[H], sum[H];
#pragma unroll
            for (int i = 0; i < H; ++i) {
                q[i] = sigmoid2(z[i]);
                sum[i] = *reinterpret_cast<const float2*>(dw + e + 2 * i);
            }
            grads<V>(y, z, d, wv, q, r, m, oy, oz, sum);
            *reinterpret_cast<uint4*>(static_cast<T*>(p.dy) + base + e) = Vec<T>::pack(oy);
            *reinterpret_cast<uint4*>(static_cast<T*>(p.dz) + base + e) = Vec<T>::pack(oz);
#pragma unroll
            for (int i = 0; i < H; ++i) *reinterpret_cast<float2*>(dw + e + 2 * i) = sum[i];
        }
    }
}

enum class Form { kWarp, kBlock, kWide };
int vectors(int gs, bool bf16) { return gs / (bf16 ? 8 : 4); }  // of 16 bytes
Form form(int gs, bool bf16)
{
    const int n = vectors(gs, bf16);
    return n <= 64 ? Form::kWarp : (n <= 512 ? Form::kBlock : Form::kWide);
}

template <typename T> cudaError_t launch_t(const GatedNormBwdParams& p, bool bf16, cudaStream_t st)
{
    const dim3 grid((unsigned)p.nblk, (unsigned)p.G);
    const int gs = p.C / p.G, n = vectors(gs, bf16), threads = (n + 31) / 32 * 32;
    switch (form(gs, bf16)) {
        case Form::kWarp:
            if (n <= 32) gated_norm_bwd_kernel<T, 1><<<grid, kWarps * 32, 0, st>>>(p);
            else gated_norm_bwd_kernel<T, 2><<<grid, kWarps * 32, 0, st>>>(p);
            break;
        case Form::kBlock:
            if (threads <= 256) gated_norm_bwd_block_kernel<T, 256><<<grid, threads, 0, st>>>(p);
            else gated_norm_bwd_block_kernel<T, 512><<<grid, threads, 0, st>>>(p);
            break;
        case Form::kWide: gated_norm_bwd_wide_kernel<T><<<grid, kWide, 0, st>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace

int gated_norm_bwd_blocks(long long rows, int C, int G, bool bf16)
{
    // over all groups, as many blocks as run at a time, never more than there are
    // rows for.  A vector a thread: 640 threads an SM (2 x 8192 rows of 8 groups: 252
    // us; 512: 273, 768: 273, 1024: 310).
    const int n = vectors(C / G, bf16);
    long long per_sm = 2, most = rows;
    switch (form(C / G, bf16)) {
        case Form::kWarp: most = (rows + kWarps - 1) / kWarps; break;
        case Form::kBlock: per_sm = 640 / ((n + 31) / 32 * 32); break;
        case Form::kWide: break;
    }
    const long long want = (152 * (per_sm < 1 ? 1 : per_sm) + G - 1) / G;
    const long long b = want < most ? want : most;
    return b < 1 ? 1 : (int)b;
}

cudaError_t launch_gated_norm_bwd(const GatedNormBwdParams& p, bool bf16, cudaStream_t st)
{
    return bf16 ? launch_t<__nv_bfloat16>(p, bf16, st) : launch_t<float>(p, bf16, st);
}

}  // namespace ssd
