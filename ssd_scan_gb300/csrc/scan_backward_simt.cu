// scan_backward_simt.cu -- gradients of the SSD scan on the fp32 pipes, for
// fp32 activations and for the shapes the tensor-core path does not cover.
//
// Per (sequence, head), with a_t = min(dt_t A, 0), g_t = dL/dy_t, and the
// state's adjoint lam_t = g_t C_t^T + exp(a_{t+1}) lam_{t+1}:
//   dx_t = dt_t lam_t B_t + D g_t      dB_t = sum_h dt_t lam_t^T x_t
//   ddt_t = x_t . lam_t B_t + A da_t   dC_t = sum_h h_t^T g_t
//   da_t = exp(a_t) <lam_t, h_{t-1}>   dA = sum dt_t da_t   dD = sum g_t . x_t
//
// Three kernels.  scan_bwd_local_kernel: what every chunk of Q rows adds to the
// state behind it, sum_s w_s dt_s x_s B_s^T, and to the adjoint before it, sum_r
// u_r g_r C_r^T (one CTA each, u and w as below).
// scan_bwd_carry_kernel carries these over the chunks, a thread per state element,
// and leaves the state at the start and the adjoint at the end of every chunk.
// scan_bwd_simt_kernel takes one chunk of one group: with gamma the cumulative
// sum of a inside the chunk, u_r = exp(gamma_r), w_s = exp(gamma_Q - gamma_s),
// L[r,s] = exp(gamma_r - gamma_s) for s <= r, E = (C_r.B_s) L, and K = E (g_r.x_s),
//   dx_s = dt_s (sum_r E[r,s] g_r + w_s lam B_s) + D g_s
//   dC_r = sum_h (sum_s dt_s (g_r.x_s) L B_s + u_r h^T g_r)
//   dB_s = sum_h (sum_r dt_s (g_r.x_s) L C_r + dt_s w_s lam^T x_s)
//   da_t = sum_{r>=t>s} dt_s K[r,s] + sum_{r>=t} u_r g_r.h C_r
//          + sum_{s<t} dt_s w_s x_s.lam B_s + exp(gamma_Q) <lam, h>
// da_t is summed from the terms that cross row t: the shorter form, a running
// difference of g.y and x.dx, subtracts large terms that were rounded apart,
// and loses da where the decay is strong.
// Bound by shared memory and the fp32 pipes: every product is a small tile with
// its operands in shared memory.  Few chunks and groups: the heads of a group
// are split over CTAs, whose shares of dB and dC are added afterwards.  Measured, 2 x
// 500 rows of 8 heads in 2 groups, P = 64, N = 128, fp32: local 14 us, carry 10,
// chunks 40, sums 8; the call, whose launches overlap, 61 us.  The chunk kernel's shared-memory
// accesses are 44,000 passes an SM of its 75,000 cycles, its multiply-adds 16,000.
#include "backward.cuh"
#include "sm100.cuh"

namespace ssd {
namespace {

constexpr int kMaxQ = 32;      // rows of a chunk
constexpr int kThreads = 256;  // of the chunk kernel

__device__ __forceinline__ float dt_value(const ScanBwdParams& p, float raw, float bias)
{
    return (p.flags & kDtSoftplus) ? softplus_full(raw + bias) : raw;
}

// In place: each chunk's own contribution becomes the value before it on the walk.
__global__ void __launch_bounds__(256) scan_bwd_carry_kernel(ScanBwdParams p, int nc)
{
    sm100::griddep_launch_dependents();
    sm100::griddep_wait();  // the chunks' contributions
    const size_t pn = (size_t)p.P * p.N, total = (size_t)p.B * p.H * pn;
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    const bool back = blockIdx.y != 0;
    if (i >= total) return;
    const size_t bh = i / pn, e = i % pn;
    const float* init = back ? p.dhS : p.h0;
    float* v = (back ? p.lout : p.hin) + bh * nc * pn + e;
    const float* dec = p.decay + bh * nc;
    float st = init ? init[i] : 0.0f;
    constexpr int kAhead = 8;  // loads in flight
    for (int c0 = 0; c0 < nc; c0 += kAhead) {
        float d[kAhead], a[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int c = back ? nc - 1 - (c0 + k) : c0 + k;
            const bool on = c0 + k < nc;
            d[k] = on ? v[(size_t)c * pn] : 0.0f;
            a[k] = on ? dec[c] : 1.0f;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int c = back ? nc - 1 - (c0 + k) : c0 + k;
            if (c0 + k >= nc) break;
            v[(size_t)c * pn] = st;
            st = fmaf(a[k], st, d[k]);
        }
    }
    if (back && p.dh0 != nullptr) p.dh0[i] = st;
}

// By one warp, a lane per row of the chunk (Q <= 32): dt, and gamma as an fp64
// running sum.
__device__ __forceinline__ double row_gamma(const ScanBwdParams& p, size_t row0, int n, int h, float& raw, float& dt)
{
    const int lane = threadIdx.x & 31;
    raw = lane < n ? p.dt[(row0 + lane) * p.H + h] : 0.0f;
    dt = lane < n ? dt_value(p, raw, p.dt_bias ? p.dt_bias[h] : 0.0f) : 0.0f;
    double v = (double)fminf(dt * p.A[h], 0.0f);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// ---- products of tiles in shared memory -----------------------------------------------
//
// Rows of every array are an odd number of 16-byte units apart, so that eight
// rows read at once lie in different banks.  A warp has RM rows of the result,
// its lanes the columns n + 32 j or 4 n + 128 j .. + 3: the 16-byte loads of the
// rows are broadcasts (one pass over shared memory), those of the columns are
// 512 bytes (four), so 20 passes feed 4 x 4 x 4 multiply-adds a lane.  (With lanes as
// 4 x 8 a load of eight distinct vectors takes as many passes as one of 32:
// measured 3.1 a load, and the kernel 55 us instead of 50 before its copies
// became asynchronous.)

// floats from a row of `n` to the next
__host__ __device__ constexpr int row_stride(int n) { return 4 * (((n + 3) / 4) | 1); }

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float2 lo2(float4 v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi2(float4 v) { return make_float2(v.z, v.w); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// (fp32: the boundary states too, which the kernel before writes while this one is
// already there, so no read-only load)
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p)
{
    const uint2 r = __ldg(reinterpret_cast<const uint2*>(p));
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
// Rows of `cols` elements into shared memory, `n` of them there and zeros up to
// `rows`, in columns up to a multiple of four; by a warp a row, four rows a warp
// in flight.  vec: every row starts at a multiple of four elements, and has one.
// seen(r, k, v): what is stored for the elements k .. of row r.
template <typename T, typename F>
__device__ __forceinline__ void load_rows(float* dst, int ds, const T* src, size_t stride, int n, int rows, int cols, bool vec, F seen)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int k = 4 * lane; k < cols; k += 128) {
#pragma unroll 4
        for (int r = warp; r < rows; r += kThreads / 32) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const T* e = src + (size_t)r * stride + k;
            if (r < n) {
                if (vec) v = load4(e);
                else {
                    v.x = to_f32(e[0]);
                    if (k + 1 < cols) v.y = to_f32(e[1]);
                    if (k + 2 < cols) v.z = to_f32(e[2]);
                    if (k + 3 < cols) v.w = to_f32(e[3]);
                }
            }
            *reinterpret_cast<float4*>(dst + r * ds + k) = seen(r, k, v);
        }
    }
}
struct AsIs {
    __device__ float4 operator()(int, int, float4 v) const { return v; }
};
// ... as they are: fp32 rows as asynchronous copies, which `loaded` waits for
template <typename T>
__device__ __forceinline__ void load_rows(float* dst, int ds, const T* src, size_t stride, int n, int rows, int cols, bool vec)
{
    if (sizeof(T) == 4 && vec) {
        for (int k = 4 * (threadIdx.x & 31); k < cols; k += 128)
            for (int r = threadIdx.x >> 5; r < rows; r += kThreads / 32)
                // (no bytes read, and zeros written, behind the rows)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 (uint32_t)__cvta_generic_to_shared(dst + r * ds + k)),
                             "l"(src + (size_t)min(r, n - 1) * stride + k), "r"(r < n ? 16 : 0)
                             : "memory");
    } else {
        load_rows(dst, ds, src, stride, n, rows, cols, vec, AsIs());
    }
}
__device__ __forceinline__ void loaded() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// this thread's warp m and lane n
struct Lane {
    int m, n;
    __device__ Lane() : m(threadIdx.x >> 5), n(threadIdx.x & 31) {}
};

// four values in a row of an array, or as many as are left of it
__device__ __forceinline__ void put4(float* dst, const float (&v)[4], bool vec, int left)
{
    if (vec) {
        *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < left) dst[i] = v[i];
}
__device__ __forceinline__ void put4(__nv_bfloat16* dst, const float (&v)[4], bool vec, int left)
{
    if (vec) {
        __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
        *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(h);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < left) dst[i] = __float2bfloat16_rn(v[i]);
}

// done(m, n, sum_k a[m][k] b[n][k]) over `cols` columns; K a multiple of 4
template <int RM, int RN, typename FD>
__device__ __forceinline__ void mm_kk(Lane t, const float* a, int as, const float* b, int bs, int cols, int K, FD done)
{
    for (int n0 = 0; n0 < cols; n0 += 32 * RN) {
        float2 acc[RM][RN];
        const float* bp[RN];
#pragma unroll
        for (int j = 0; j < RN; ++j) {
            bp[j] = b + (size_t)min(n0 + t.n + 32 * j, cols - 1) * bs;
#pragma unroll
            for (int i = 0; i < RM; ++i) acc[i][j] = both(0.0f);
        }
#pragma unroll 2
        for (int k = 0; k < K; k += 4) {
            float4 av[RM], bv[RN];
#pragma unroll
            for (int i = 0; i < RM; ++i) av[i] = ld4(a + (RM * t.m + i) * as + k);
#pragma unroll
            for (int j = 0; j < RN; ++j) bv[j] = ld4(bp[j] + k);
#pragma unroll
            for (int i = 0; i < RM; ++i)
#pragma unroll
                for (int j = 0; j < RN; ++j)
                    acc[i][j] = __ffma2_rn(hi2(av[i]), hi2(bv[j]), __ffma2_rn(lo2(av[i]), lo2(bv[j]), acc[i][j]));
        }
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int j = 0; j < RN; ++j)
                if (n0 + t.n + 32 * j < cols) done(RM * t.m + i, n0 + t.n + 32 * j, acc[i][j].x + acc[i][j].y);
    }
}
template <int RM, typename FD>
__device__ __forceinline__ void mm_kk_by(Lane t, const float* a, int as, const float* b, int bs, int cols, int K, FD done)
{
    if (cols <= 32) mm_kk<RM, 1>(t, a, as, b, bs, cols, K, done);
    else mm_kk<RM, 2>(t, a, as, b, bs, cols, K, done);
}

// acc[i][j] += sum_k a(m, k) b[k][n] for four columns n = n0 + 4 t.n + 128 j at a
// time; kMajor: a[m][k] (K a multiple of 4), else a[k][m]
template <bool kMajor, int RM, int RJ>
__device__ __forceinline__ void mm_n(Lane t, const float* a, int as, const float* b, int bs, int n0, int cols, int K,
                                     float2 (&acc)[RM][RJ][2])
{
    const float* bp[RJ];
#pragma unroll
    for (int j = 0; j < RJ; ++j) bp[j] = b + min(n0 + 4 * t.n + 128 * j, (cols - 1) / 4 * 4);
    auto step = [&](const float (&av)[RM], int k) {
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
            if (n0 + 128 * j >= cols) break;
            const float4 bv = ld4(bp[j] + (size_t)k * bs);
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                acc[i][j][0] = __ffma2_rn(both(av[i]), lo2(bv), acc[i][j][0]);
                acc[i][j][1] = __ffma2_rn(both(av[i]), hi2(bv), acc[i][j][1]);
            }
        }
    };
    if (kMajor) {
#pragma unroll 1
        for (int k = 0; k < K; k += 4) {
            float4 v[RM];
#pragma unroll
            for (int i = 0; i < RM; ++i) v[i] = ld4(a + (RM * t.m + i) * as + k);
            float x[4][RM];
#pragma unroll
            for (int i = 0; i < RM; ++i) x[0][i] = v[i].x, x[1][i] = v[i].y, x[2][i] = v[i].z, x[3][i] = v[i].w;
#pragma unroll
            for (int q = 0; q < 4; ++q) step(x[q], k + q);
        }
    } else {
#pragma unroll 4
        for (int k = 0; k < K; ++k) {
            float x[RM];
            const float* r = a + (size_t)k * as + RM * t.m;
            if (RM == 2) {
                const float2 v = *reinterpret_cast<const float2*>(r);
                x[0] = v.x, x[1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < RM; i += 4) {
                    const float4 v = ld4(r + i);
                    x[i] = v.x, x[i + 1] = v.y, x[i + (RM > 2 ? 2 : 0)] = v.z, x[i + (RM > 2 ? 3 : 0)] = v.w;
                }
            }
            step(x, k);
        }
    }
}

// ---- what a chunk adds to the states --------------------------------------------------

// rows of x or g: whole blocks of 64 columns, of which those behind P are not used
__host__ __device__ constexpr int local_stride(int P) { return row_stride((P + 63) / 64 * 64); }

// grid: (sequence, direction, chunk) x head
template <typename T> __global__ void __launch_bounds__(kThreads, 4) scan_bwd_local_kernel(ScanBwdParams p, int Q)
{
    extern __shared__ __align__(16) float smem[];
    __shared__ float f[kMaxQ];
    sm100::griddep_launch_dependents();
    const int H = p.H, P = p.P, N = p.N, G = p.G, S = p.S;
    const int nc = (S + Q - 1) / Q, NS = row_stride(N), PS = local_stride(P);
    const int h = blockIdx.x % (unsigned)H;
    const unsigned bc = blockIdx.x / (unsigned)H;
    const int c = bc % nc, b = (bc / nc) >> 1;
    const bool back = (bc / nc & 1) != 0;  // lam rather than h
    const int g = h / (H / G), Cdim = H * P + 2 * G * N;
    const int t0 = c * Q, n = min(Q, S - t0), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* ms = smem;           // [Q][N]: B or C
    float* vs = ms + Q * NS;    // [Q][P]: x or g, by the row's factor
    const size_t row0 = (size_t)b * S + t0, unit = ((size_t)b * H + h) * nc + c;
    if (warp == 0) {
        float raw, dt;
        const double v = row_gamma(p, row0, n, h, raw, dt), vQ = __shfl_sync(0xffffffffu, v, 31);
        f[lane] = back ? expf((float)v) * (1.0f + (float)(v - (double)(float)v)) : expf((float)(vQ - v)) * dt;
        if (lane == 0 && !back) p.decay[unit] = expf((float)vQ) * (1.0f + (float)(vQ - (double)(float)vQ));
    }
    const T* m = static_cast<const T*>(p.xbc) + row0 * Cdim + H * P + (back ? G * N : 0) + g * N;
    load_rows(ms, NS, m, Cdim, n, n, N, ((N | (H * P)) & 3) == 0);
    __syncthreads();  // f
    const T* v = back ? static_cast<const T*>(p.dy) + (row0 * H + h) * P : static_cast<const T*>(p.xbc) + row0 * Cdim + h * P;
    load_rows(vs, PS, v, back ? (size_t)H * P : Cdim, n, n, P, (P & 3) == 0, [&](int r, int, float4 e) {
        return make_float4(e.x * f[r], e.y * f[r], e.z * f[r], e.w * f[r]);
    });
    loaded();
    __syncthreads();
    float* out = (back ? p.lout : p.hin) + unit * P * N;
    const Lane t;
    for (int q0 = 0; q0 < P; q0 += 64)
        for (int k0 = 0; k0 < N; k0 += 128) {
            float2 acc[8][1][2];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i][0][0] = acc[i][0][1] = both(0.0f);
            mm_n<false>(t, vs + q0, PS, ms, NS, k0, N, n, acc);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int q = q0 + 8 * t.m + i, k = k0 + 4 * t.n;
                const float o[4] = {acc[i][0][0].x, acc[i][0][0].y, acc[i][0][1].x, acc[i][0][1].y};
                if (q < P && k < N) put4(out + (size_t)q * N + k, o, (N & 3) == 0, N - k);
            }
        }
}

// ---- one chunk of one group ---------------------------------------------------------

// Rows of a chunk are padded to Q with zeros.
struct ChunkShape {
    int Q, PB;     // rows of a chunk, columns p of a state in shared memory at once
    size_t floats; // of shared memory
};
constexpr size_t kSmemFloats = 227 * 1024 / 4;
__host__ __device__ inline size_t chunk_smem_floats(int P, int N, int Q, int PB)
{
    // B, C; x, g, tmp; CB, F, E, K; row vectors; a block of a state
    return (size_t)2 * Q * row_stride(N) + (size_t)3 * Q * row_stride(P) + (size_t)4 * Q * row_stride(Q) + 10 * Q + 64 +
           (size_t)PB * row_stride(N);
}
// The longest chunk that fits, as the boundary states cost 2 P N floats per head
// and chunk; with it the fewest blocks of the state.
bool chunk_shape(int P, int N, ChunkShape* c)
{
    for (int Q = kMaxQ; Q >= 16; Q /= 2)
        for (int k = 1; k <= (P + 3) / 4; ++k) {
            const int PB = ((P + k - 1) / k + 3) / 4 * 4;
            if (PB < 16 && k > 1) break;
            const size_t f = chunk_smem_floats(P, N, Q, PB);
            if (f > kSmemFloats) continue;
            *c = {Q, PB, f};
            return true;
        }
    return false;
}

// NB: blocks of 128 columns n
template <typename T, int RM, int NB>
__global__ void __launch_bounds__(kThreads, NB == 1 ? 2 : 1) scan_bwd_simt_kernel(ScanBwdParams p, int PB)
{
    constexpr int Q = 8 * RM, QS = row_stride(Q), RJ = NB;
    extern __shared__ __align__(16) float smem[];
    const int c = blockIdx.x, g = blockIdx.y / p.split, sp = blockIdx.y % p.split, b = blockIdx.z;
    const int H = p.H, P = p.P, N = p.N, G = p.G, S = p.S, R = H / G;
    const int per = (R + p.split - 1) / p.split;
    const int Cdim = H * P + 2 * G * N, nc = (S + Q - 1) / Q;
    const int t0 = c * Q, n = min(Q, S - t0);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int NS = row_stride(N), PS = row_stride(P), N4 = (N + 3) / 4 * 4, P4 = (P + 3) / 4 * 4;
    const Lane t;
    sm100::griddep_launch_dependents();
    float* Bs = smem;             // [Q][N]
    float* Cs = Bs + Q * NS;
    float* xs = Cs + Q * NS;      // [Q][P]
    float* gs = xs + Q * PS;
    float* tmp = gs + Q * PS;
    float* CB = tmp + Q * PS;     // [r][s]
    float* F = CB + Q * QS;       // sum over heads of (g_r.x_s) L dt_s
    float* E = F + Q * QS;
    float* K = E + Q * QS;
    float* dts = K + Q * QS;      // [Q] each
    float* raw = dts + Q;
    float* u = raw + Q;
    float* w = u + Q;
    float* rho = w + Q;
    float* sig = rho + Q;
    float* kcol = sig + Q;
    float* krow = kcol + Q;
    float* gamh = krow + Q;       // gamma as a double-float pair
    float* gaml = gamh + Q;
    float* red = gaml + Q;        // [64]
    float* stage = red + 64;      // [PB][N]
    const T* xbc = static_cast<const T*>(p.xbc);
    const T* dy = static_cast<const T*>(p.dy);
    T* dxbc = static_cast<T*>(p.dxbc);

    const size_t row0 = (size_t)b * S + t0;
    const bool vecN = ((N | (H * P)) & 3) == 0, vecP = (P & 3) == 0;
    load_rows(Bs, NS, xbc + row0 * Cdim + H * P + g * N, Cdim, n, Q, N, vecN);
    load_rows(Cs, NS, xbc + row0 * Cdim + H * P + (G + g) * N, Cdim, n, Q, N, vecN);
    for (int i = tid; i < Q * QS; i += kThreads) F[i] = 0.0f;
    sm100::griddep_wait();  // the boundary states

    float2 dB[RM][RJ][2], dC[RM][RJ][2];
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < RJ; ++j) dB[i][j][0] = dB[i][j][1] = dC[i][j][0] = dC[i][j][1] = both(0.0f);
    // sum += f(row) * (rows of a) x (the staged block)
    auto add_rows = [&](float2(&sum)[RM][RJ][2], const float* a, int K, auto f) {
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
            float2 acc[RM][1][2];
#pragma unroll
            for (int i = 0; i < RM; ++i) acc[i][0][0] = acc[i][0][1] = both(0.0f);
            mm_n<true>(t, a, PS, stage, NS, 128 * j, N, K, acc);
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                const float2 k = both(f(RM * t.m + i));
                sum[i][j][0] = __ffma2_rn(k, acc[i][0][0], sum[i][j][0]);
                sum[i][j][1] = __ffma2_rn(k, acc[i][0][1], sum[i][j][1]);
            }
        }
    };
    // sum of a row of a times one of b, by the eight threads of a row
    constexpr int kPer = kThreads / Q;
    auto row_dot = [&](const float* a, const float* v, float* out) {
        const int r = tid / kPer;
        float sum = 0.0f;
        for (int q = 4 * (tid % kPer); q < P4; q += 4 * kPer) {
            const float4 x = ld4(a + r * PS + q), y = ld4(v + r * PS + q);
            sum = fmaf(x.x, y.x, sum);
            sum = fmaf(x.y, y.y, sum);
            sum = fmaf(x.z, y.z, sum);
            sum = fmaf(x.w, y.w, sum);
        }
#pragma unroll
        for (int d = kPer / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (tid % kPer == 0) out[r] = sum;
    };

    for (int hh = sp * per; hh < min(R, (sp + 1) * per); ++hh) {
        const int h = g * R + hh;
        const float Ah = p.A[h], Dh = p.D ? p.D[h] : 0.0f, bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
        const float* hin = p.hin + (((size_t)b * H + h) * nc + c) * P * N;
        const float* lam = p.lout + (((size_t)b * H + h) * nc + c) * P * N;
        float cross = 0.0f;
        for (int q0 = 0; q0 < P; q0 += PB) {
            __syncthreads();
            load_rows(stage, NS, lam + (size_t)q0 * N, N, P - q0, PB, N, (N & 3) == 0);  // rows behind P: zeros
            if (q0 == 0) {
                load_rows(xs, PS, xbc + row0 * Cdim + h * P, Cdim, n, Q, P, vecP);
                load_rows(gs, PS, dy + (row0 * H + h) * P, (size_t)H * P, n, Q, P, vecP);
                if (P4 > P)
                    for (int i = tid; i < Q * (P4 - P); i += kThreads) tmp[i / (P4 - P) * PS + P + i % (P4 - P)] = 0.0f;
                if (warp == 0) {
                    float rw, dt;
                    const double v = row_gamma(p, row0, n, h, rw, dt), vQ = __shfl_sync(0xffffffffu, v, 31);
                    if (lane < Q) {
                        raw[lane] = rw;
                        dts[lane] = dt;
                        gamh[lane] = (float)v;
                        gaml[lane] = (float)(v - (double)gamh[lane]);
                        u[lane] = expf((float)v) * (1.0f + gaml[lane]);
                        w[lane] = expf((float)(vQ - v));
                    }
                }
            }
            loaded();
            __syncthreads();
            if (hh == sp * per && q0 == 0)
                mm_kk<RM, 1>(t, Cs, NS, Bs, NS, Q, N4, [&](int r, int s, float v) { CB[r * QS + s] = v; });
            // lam B_s, its share of dx and of ddt; and of dB
            mm_kk_by<RM>(t, Bs, NS, stage, NS, min(PB, P - q0), N4,
                         [&](int s, int q, float v) { tmp[s * PS + q0 + q] = w[s] * v; });
            add_rows(dB, xs + q0, min(PB, P4 - q0), [&](int s) { return dts[s] * w[s]; });
        }
        // g_r . x_s, and with it everything of the pair (r, s) (the thread's own CB)
        mm_kk<RM, 1>(t, gs, PS, xs, PS, Q, P4, [&](int r, int s, float v) {
            const bool in = s <= r;
            const float L = in ? expf((gamh[r] - gamh[s]) + (gaml[r] - gaml[s])) : 0.0f;
            const float e = CB[r * QS + s] * L;
            if (in) F[r * QS + s] = fmaf(v * L, dts[s], F[r * QS + s]);
            E[r * QS + s] = in ? e : 0.0f;
            K[r * QS + s] = in ? e * v : 0.0f;
            if (r == s) rho[r] = v;  // g_r . x_r, for dD
        });
        for (int q0 = 0; q0 < P; q0 += PB) {
            __syncthreads();
            load_rows(stage, NS, hin + (size_t)q0 * N, N, P - q0, PB, N, (N & 3) == 0, [&](int q, int k, float4 v) {
                if (q0 + q < P) {  // <lam, h>
                    const float* l = lam + (size_t)(q0 + q) * N + k;
                    if ((N & 3) == 0) {
                        const float4 e = load4(l);
                        cross = fmaf(v.x, e.x, fmaf(v.y, e.y, fmaf(v.z, e.z, fmaf(v.w, e.w, cross))));
                    } else {
                        cross = fmaf(v.x, l[0], cross);
                        if (k + 1 < N) cross = fmaf(v.y, l[1], cross);
                        if (k + 2 < N) cross = fmaf(v.z, l[2], cross);
                        if (k + 3 < N) cross = fmaf(v.w, l[3], cross);
                    }
                }
                return v;
            });
            if (q0 == 0) {
                // dx
                for (int m0 = 0; m0 < P; m0 += 128) {
                    float2 acc[RM][1][2];
#pragma unroll
                    for (int i = 0; i < RM; ++i) acc[i][0][0] = acc[i][0][1] = both(0.0f);
                    mm_n<false>(t, E, QS, gs, PS, m0, P, Q, acc);
                    const int q = m0 + 4 * t.n;
#pragma unroll
                    for (int i = 0; i < RM; ++i) {
                        const int s = RM * t.m + i;
                        if (s >= n || q >= P) continue;
                        const float4 l = ld4(tmp + s * PS + q), d = ld4(gs + s * PS + q);
                        const float o[4] = {fmaf(dts[s], acc[i][0][0].x + l.x, Dh * d.x), fmaf(dts[s], acc[i][0][0].y + l.y, Dh * d.y),
                                            fmaf(dts[s], acc[i][0][1].x + l.z, Dh * d.z), fmaf(dts[s], acc[i][0][1].y + l.w, Dh * d.w)};
                        put4(dxbc + ((size_t)b * S + t0 + s) * Cdim + h * P + q, o, (P & 3) == 0 && (Cdim & 3) == 0, P - q);
                    }
                }
                // x . lam B over the row; below the diagonal the column sums of K, and in
                // its place the sums of dt_s K over the rows from r on
                row_dot(xs, tmp, sig);
                if (warp == 0) {
                    float d = lane < Q ? rho[lane] : 0.0f;
#pragma unroll
                    for (int m = 16; m > 0; m >>= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
                    if (lane == 0) red[32] = d;
                } else if (warp == 1 && lane < Q) {
                    const int s = lane;
                    float v[Q], k = 0.0f, suf = 0.0f;
#pragma unroll
                    for (int r = 0; r < Q; ++r) v[r] = K[r * QS + s];
#pragma unroll
                    for (int r = Q - 1; r >= 0; --r)
                        if (r > s) {
                            k += v[r];
                            suf = fmaf(dts[s], v[r], suf);
                            K[r * QS + s] = suf;
                        }
                    kcol[s] = k + K[s * QS + s];
                }
            }
            __syncthreads();
            // h C_r
            mm_kk_by<RM>(t, Cs, NS, stage, NS, min(PB, P - q0), N4, [&](int r, int q, float v) { tmp[r * PS + q0 + q] = v; });
            add_rows(dC, gs + q0, min(PB, P4 - q0), [&](int r) { return u[r]; });
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) cross += __shfl_xor_sync(0xffffffffu, cross, d);
        if (lane == 0) red[warp] = cross;
        __syncthreads();
        row_dot(gs, tmp, rho);
        {  // sum of dt_s K[r,s] over r >= t > s
            const int r = tid / kPer;
            float sum = 0.0f;
            for (int s = tid % kPer; s < r; s += kPer) sum += K[r * QS + s];
#pragma unroll
            for (int d = kPer / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (tid % kPer == 0) krow[r] = sum;
        }
        __syncthreads();
        if (warp == 0) {  // da over the chunk's rows, a lane per row
            const bool on = lane < n;
            const float dt = on ? dts[lane] : 0.0f, sg = on ? sig[lane] : 0.0f;
            float cr = lane < kThreads / 32 ? red[lane] : 0.0f;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) cr += __shfl_xor_sync(0xffffffffu, cr, d);
            cr *= u[n - 1];
            // inclusive sums behind and before
            float suf = on ? u[lane] * rho[lane] : 0.0f, pre = dt * sg;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const float x = __shfl_down_sync(0xffffffffu, suf, d), y = __shfl_up_sync(0xffffffffu, pre, d);
                if (lane + d < 32) suf += x;
                if (lane >= d) pre += y;
            }
            pre = __shfl_up_sync(0xffffffffu, pre, 1);
            if (lane == 0) pre = 0.0f;
            float dA = 0.0f, db = 0.0f;
            if (on) {
                // a decay clamped at 1 passes no gradient
                const float da = dt * Ah > 0.0f ? 0.0f : (suf + pre) + (krow[lane] + cr);
                float d = fmaf(Ah, da, kcol[lane] + sg);
                if (p.flags & kDtSoftplus) d *= 1.0f / (1.0f + expf(-(raw[lane] + bias)));
                p.ddt[((size_t)b * S + t0 + lane) * H + h] = d;
                dA = dt * da;
                db = p.flags & kDtSoftplus ? d : 0.0f;  // (dt_bias has no part in dt without)
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                dA += __shfl_xor_sync(0xffffffffu, dA, d);
                db += __shfl_xor_sync(0xffffffffu, db, d);
            }
            float* part = p.part + ((size_t)b * nc + c) * 3 * H + h;
            if (lane == 0) {
                part[0] = dA;
                part[H] = db;
                part[2 * H] = red[32];
            }
        }
    }
    __syncthreads();
    // the rows' own share of dC and dB, all heads of this CTA at once
    mm_n<true>(t, F, QS, Bs, NS, 0, N, Q, dC);
    mm_n<false>(t, F, QS, Cs, NS, 0, N, Q, dB);
    const bool vec = (N & 3) == 0 && ((H * P) & 3) == 0 && (Cdim & 3) == 0;
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const size_t row = (size_t)b * S + t0 + RM * t.m + i;
        if (RM * t.m + i >= n) continue;
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
            const int k = 4 * t.n + 128 * j;
            if (k >= N) continue;
#pragma unroll
            for (int m = 0; m < 2; ++m) {  // dB 0, dC 1
                const float2* v = m ? dC[i][j] : dB[i][j];
                const float o[4] = {v[0].x, v[0].y, v[1].x, v[1].y};
                const size_t col = (size_t)(m * G + g) * N + k;
                if (p.split == 1) put4(dxbc + row * Cdim + H * P + col, o, vec, N - k);
                else put4(p.bcpart + ((size_t)sp * p.B * S + row) * (2 * G * N) + col, o, vec, N - k);
            }
        }
    }
}

// The local kernel's limit, the same for every shape (the largest takes 78,848 bytes): a
// limit set to a call's own need would be lowered under the launch of another thread.
constexpr size_t kLocalSmem = 96 * 1024;

template <typename T> cudaError_t launch_local(const ScanBwdParams& p, int Q, cudaStream_t st)
{
    const size_t smem = sizeof(float) * (size_t)Q * (row_stride(p.N) + local_stride(p.P));
    auto kern = scan_bwd_local_kernel<T>;
    static std::atomic<bool> done[kMaxDevices];
    const cudaError_t e = allow_smem((const void*)kern, kLocalSmem, done);
    if (e != cudaSuccess) return e;
    const long long blocks = 2LL * p.B * (((long long)p.S + Q - 1) / Q) * p.H;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    kern<<<(unsigned)blocks, kThreads, smem, st>>>(p, Q);
    return cudaGetLastError();
}

template <typename T, int RM, int NB> cudaError_t launch_chunks_t(const ScanBwdParams& p, const ChunkShape& c, cudaStream_t st)
{
    static std::atomic<bool> done[kMaxDevices];
    auto kern = scan_bwd_simt_kernel<T, RM, NB>;
    const cudaError_t e = allow_smem((const void*)kern, kSmemFloats * 4, done);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((p.S + c.Q - 1) / c.Q), (unsigned)(p.G * p.split), (unsigned)p.B);
    int pb = c.PB;
    void* args[] = {const_cast<ScanBwdParams*>(&p), &pb};
    return launch_after((const void*)kern, grid, kThreads, c.floats * 4, st, args);
}
template <typename T> cudaError_t launch_chunks(const ScanBwdParams& p, cudaStream_t st)
{
    ChunkShape c;
    if (!chunk_shape(p.P, p.N, &c)) return cudaErrorInvalidValue;
    // N is a power of two up to 512, as the forward's; chunks have 16 rows only for head
    // sizes from 493 on, which go with N up to 64
    switch (c.Q + (p.N + 127) / 128) {
        case 33: return launch_chunks_t<T, 4, 1>(p, c, st);
        case 34: return launch_chunks_t<T, 4, 2>(p, c, st);
        case 36: return launch_chunks_t<T, 4, 4>(p, c, st);
        case 17: return launch_chunks_t<T, 2, 1>(p, c, st);
        default: return cudaErrorInvalidValue;
    }
}

// dB | dC from the shares of the CTAs that split a group's heads: whole rows of
// `cols` a CTA, V columns a thread
template <typename T, int V>
__global__ void __launch_bounds__(256) scan_bwd_join_kernel(const float* part, T* dxbc, long long rows, int lead, int cols, int split)
{
    sm100::griddep_launch_dependents();
    sm100::griddep_wait();  // the shares (plain loads: they were not there when this grid began)
    const int nv = cols / V, per = max(1, 256 / nv);
    const int r = threadIdx.x / nv;
    const long long row = (long long)blockIdx.x * per + r;
    if (r >= per || row >= rows) return;
    for (int k = V * (threadIdx.x - r * nv); k < cols; k += 256 * V) {
        const float* src = part + row * cols + k;
        float acc[V] = {};
#pragma unroll 4
        for (int m = 0; m < split; ++m, src += rows * cols) {
            if (V == 4) {
                const float4 v = ld4(src);
                acc[0] += v.x, acc[1] += v.y, acc[2] += v.z, acc[3] += v.w;
            } else {
                acc[0] += *src;
            }
        }
        T* dst = dxbc + row * ((long long)lead + cols) + lead + k;
        if (V == 4) {
            const float o[4] = {acc[0], acc[V > 1], acc[V > 2 ? 2 : 0], acc[V > 3 ? 3 : 0]};
            put4(dst, o, true, 4);
        } else {
            *dst = from_f32<T>(acc[0]);
        }
    }
}
template <typename T>
cudaError_t launch_join(const float* part, void* dxbc, long long rows, int lead, int cols, int split, cudaStream_t st)
{
    const bool vec = lead % 4 == 0 && cols % 4 == 0;
    const int nv = cols / (vec ? 4 : 1), per = nv < 256 ? 256 / nv : 1;
    const unsigned blocks = (unsigned)((rows + per - 1) / per);
    T* out = static_cast<T*>(dxbc);
    void* args[] = {&part, &out, &rows, &lead, &cols, &split};
    return launch_after(vec ? (const void*)scan_bwd_join_kernel<T, 4> : (const void*)scan_bwd_join_kernel<T, 1>, dim3(blocks), 256,
                        0, st, args);
}

}  // namespace

// CTAs of the chunk kernel that run at a time: two a SM where they fit
int scan_bwd_simt_slots(int P, int N)
{
    ChunkShape c;
    return chunk_shape(P, N, &c) && N <= 128 && c.floats * 4 <= 113 * 1024 ? 304 : 152;
}

int scan_bwd_simt_chunk(int P, int N)
{
    ChunkShape c;
    return scan_simt_supports(P, N) && chunk_shape(P, N, &c) ? c.Q : 0;
}

cudaError_t launch_scan_bwd_local(const ScanBwdParams& p, bool bf16, cudaStream_t st)
{
    const int Q = scan_bwd_simt_chunk(p.P, p.N);
    if (Q == 0) return cudaErrorInvalidValue;
    return bf16 ? launch_local<__nv_bfloat16>(p, Q, st) : launch_local<float>(p, Q, st);
}

cudaError_t launch_scan_bwd_carry(const ScanBwdParams& p, cudaStream_t st)
{
    const int Q = scan_bwd_simt_chunk(p.P, p.N);
    if (Q == 0) return cudaErrorInvalidValue;
    const size_t blocks = ((size_t)p.B * p.H * p.P * p.N + 255) / 256;
    if (blocks > 0x7fffffffu) return cudaErrorInvalidValue;
    int nc = (int)(((long long)p.S + Q - 1) / Q);
    void* args[] = {const_cast<ScanBwdParams*>(&p), &nc};
    return launch_after((const void*)scan_bwd_carry_kernel, dim3((unsigned)blocks, 2), 256, 0, st, args);
}

cudaError_t launch_scan_bwd_simt(const ScanBwdParams& p, bool bf16, cudaStream_t st)
{
    return bf16 ? launch_chunks<__nv_bfloat16>(p, st) : launch_chunks<float>(p, st);
}

int scan_bwd_split(long long units, int heads, double setup, int slots)
{
    long long best = -1;
    int split = 1;
    for (int k = 1; k <= heads && k <= 32; ++k) {
        const long long per = (heads + k - 1) / k;
        const int n = (int)((heads + per - 1) / per);  // CTAs that have heads
        const long long waves = (units * n + slots - 1) / slots;
        const long long t = (long long)(16 * waves * (per + setup)) + (n > 1 ? 16 : 0);
        if (best < 0 || t < best) {
            best = t;
            split = n;
        }
    }
    return split;
}

cudaError_t launch_scan_bwd_join(const float* part, void* dxbc, long long rows, int lead, int cols, int split, bool bf16,
                                 cudaStream_t st)
{
    return bf16 ? launch_join<__nv_bfloat16>(part, dxbc, rows, lead, cols, split, st)
                : launch_join<float>(part, dxbc, rows, lead, cols, split, st);
}

}  // namespace ssd
