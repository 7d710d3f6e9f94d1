// scan_backward_tc.cu -- gradients of the SSD scan on the 5th-generation tensor
// cores: bf16 activations, P = 64, N = 128, 128-row chunks.
//
// Notation as in scan_backward_simt.cu.  Inside a chunk, gamma = cumsum a,
// u_r = exp(gamma_r), w_s = exp(gamma_Q - gamma_s), L[s,r] = exp(gamma_r -
// gamma_s) for r >= s; h = the state at the chunk's start, lam = the adjoint at
// its end.  Three kernels:
//
// scan_bwd_rows_kernel: dt, gamma, u, w and what else depends on a row alone,
//   [b, h, chunk][kVals][128], a warp per (head, chunk): each value is computed
//   once, and read by the walks below and by every warp of a chunk's CTA.
// scan_bwd_states_tc_kernel: one CTA per (one or two heads, direction, sequence)
//   walks the chunks, forward for h, backward for lam; the fp32 state stays in
//   registers,
//     h <- exp(gamma_Q) h + sum_s w_s dt_s x_s B_s^T,
//     lam <- exp(gamma_Q) lam + sum_r u_r g_r C_r^T
//   (one 128x64x128 product a chunk and head), and leaves the value before each
//   chunk.
// scan_bwd_tc_kernel: one CTA per (chunk, group or part of one, sequence) walks the
//   group's heads, the B and C tiles in shared memory and CB^T in registers:
//     dM^T[s,r] = x_s . g_r                       A = x          B = g
//     Yo[r,p]   = C_r . h[.,p]                    A = C          B = h
//     Bl[s,p]   = B_s . lam[.,p]                  A = B          B = lam
//     dx[s,p]   = sum_r E^T[s,r] g[r,p]           A = E (TMEM)   B = g
//     dC[r,n]  += (u_r g_r) . h[n,.]              A = u o g      B = h
//     dB[s,n]  += (w_s dt_s x_s) . lam[n,.]       A = w dt o x   B = lam
//   with E^T = CB^T L dt_s, and over the heads F^T += dM^T L dt_s in registers;
//   at the end dB += F^T C and dC += F B.  dC and dB stay in TMEM throughout.
// The three overlap their launches, so one's prologue hides in the last one's end.
//
// Why this split.  The states are the only thing that runs through the chunks, so
// they get kernels of their own and the rest is parallel over chunks.  They
// cost 64 KB a head and chunk on the way to memory and as much on the way back,
// more than twice the bytes of x, g, B, C and their gradients; chunks of 256
// rows would halve that, and do not fit: the products of one head fill TMEM (512
// columns) and its operands shared memory (225 KB).
//
// Measured, 128 heads in 8 groups (us, rows / states / chunks): one sequence of
// 2048 rows 8 / 45 / 71, the call 121; 2 x 8192 rows 25 / 339 / 468, the call 830.
// The states kernel moves 128 KB between L2 and its SM a step, 6.4 TB/s in all,
// and its steps (5,500 cycles) are the product of 24 (1,500), the way of its result over
// TMEM to the next one's operands, and the scaling of rows between.  The chunk kernel is
// bound by the work around its products: 4.4 us a head, of which the tensor pipe is busy
// 1.2; the masks issue on every scheduler for a third of the time, the rest is the chain
// from one product's end over TMEM to the next one's operands.
//
// Precision.  x, g, B and C are bf16 already.  ddt, dA, ddt_bias, dD and the
// initial state's gradient are fp32.  The states are sums in fp32 registers of products
// that see all 24 bits of the scaled rows (three bf16, one product on each, the
// smallest first).  On their way to the chunks they are two bf16, hi + lo, 17 bits, in
// the bytes of one fp32, and each product with them runs on both: off by 2^-17 of an
// element at most.  K = E (g.x), whose sums da is made of, never leaves fp32.  Only what ends in
// a bf16 output takes single bf16 operands: E, F, u o g, w dt o x and, beside these two,
// the states.  Against 64 bits, in the 2-norm: ddt 4.5e-7, dA 4.6e-7 to 6e-7 and ddt_bias
// 5e-7 to 7e-7, more where the terms of a head cancel, the initial state's gradient
// 2.3e-7; all fp32 would be 1e-7 to 4e-7.  With two bf16 for the scaled rows as well ddt was
// 7.5e-7, dA 1.1e-6 to 2e-6 and the initial state's gradient 2.5e-6, at 117 us for the
// 2048 rows.  Three for the states on their way too, made from fp32 by the chunk kernel: 2.8e-7
// and 3.0e-7, and 154 us, as the products with them already take all of shared memory's
// bandwidth while they run.
//
// da_t sums the terms that cross row t, with no difference of large sums: in
// 32-row blocks, whole blocks of K below and left of t, partial row sums and
// column sums of the off-diagonal blocks, and inside the diagonal block the
// sum over r >= t > s, taken from suffix sums along r.
#include "backward.cuh"
#include "sm100.cuh"

#include <cudaTypedefs.h>

#include <atomic>
#include <cstddef>
#include <mutex>

namespace ssd {
namespace {

using namespace sm100;

constexpr int Q = 128;
constexpr int P = 64;
constexpr int N = 128;
constexpr uint64_t kWaitNs = 2000000000ull;  // default bound on a wait

constexpr uint32_t kIdQQ = idesc_bf16_f32(128, 128, false, false);  // both K-major
constexpr uint32_t kIdQP = idesc_bf16_f32(128, 64, false, true);    // B operand rows [k][p]
constexpr uint32_t idesc_state(int heads) { return idesc_bf16_f32(128, 64 * heads, true, true); }  // A = B^T, B operand rows [k][p]
constexpr uint32_t kIdFC = idesc_bf16_f32(128, 128, false, true);   // F^T C
constexpr uint32_t kIdFB = idesc_bf16_f32(128, 128, true, true);    // F B

__device__ __forceinline__ float ex2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// (hi, lo) += (bhi, blo), double-float (TwoSum then renormalise)
__device__ __forceinline__ void df_add(float& hi, float& lo, float bhi, float blo)
{
    const float s = hi + bhi;
    const float v = s - hi;
    float e = (hi - (s - v)) + (bhi - v);
    e += lo + blo;
    hi = s + e;
    lo = e - (hi - s);
}

// (hi, lo) * log2(e) as a double-float
__device__ __forceinline__ void df_to_log2(float hi, float lo, float& rh, float& rl)
{
    constexpr float kL = 1.4426950408889634f;  // log2(e) rounded to fp32
    constexpr float kLlo = 1.925963e-8f;       // log2(e) - kL
    const float p = hi * kL;
    float e = fmaf(hi, kL, -p);
    e += fmaf(hi, kLlo, lo * kL);
    rh = p + e;
    rl = e - (rh - p);
}

// 2^min(a - b, most) of double-floats: with the difference in fp32 alone the result
// would be off by half a step of it, 2e-6 of 2^60
__device__ __forceinline__ float exp2_diff(float ah, float al, float bh, float bl, float most)
{
    const float s = ah - bh, v = s - ah;
    const float e = ((ah - (s - v)) - (bh + v)) + (al - bl);  // what s left out
    const float t = s + e, r = e - (t - s);
    return t < most ? ex2_fast(t) * fmaf(r, 0.6931471806f, 1.0f) : ex2_fast(most);
}

__device__ __forceinline__ uint32_t pack2(float2 a)
{
    __nv_bfloat162 h = __float22bfloat162_rn(a);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t r)
{
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r));
}
__device__ __forceinline__ void unpack8(uint4 r, float2* f)
{
    f[0] = unpack2(r.x); f[1] = unpack2(r.y); f[2] = unpack2(r.z); f[3] = unpack2(r.w);
}
__device__ __forceinline__ uint4 pack8(const float2* f)
{
    return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}
// v = hi + lo in two bf16 each: off by at most 2^-17 of the value
__device__ __forceinline__ void split8(const float2* v, uint4& hi, uint4& lo)
{
    float2 r[4], h[4];
    hi = pack8(v);
    unpack8(hi, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = make_float2(v[i].x - h[i].x, v[i].y - h[i].y);
    lo = pack8(r);
}

// v = hi + mid + lo in bf16 each, a pair of them: all of v's 24 bits.  What the rounded hi
// leaves has 16 bits, whose upper and lower half are mid and lo.
__device__ __forceinline__ uint32_t upper2(float2 v) { return __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632); }
__device__ __forceinline__ void split2(float2 v, uint32_t& hi, uint32_t& mid, uint32_t& lo)
{
    hi = pack2(v);
    const float2 h = unpack2(hi), r = make_float2(v.x - h.x, v.y - h.y);
    mid = upper2(r);
    const float2 m = unpack2(mid);
    lo = upper2(make_float2(r.x - m.x, r.y - m.y));
}

// byte offset of 16-byte chunk j of row r in a SW128 tile of 64-element rows
__device__ __forceinline__ uint32_t chunk_off(int r, int j) { return (uint32_t)(r * 128 + (((j ^ r) & 7) << 4)); }
template <typename T> __device__ __forceinline__ T& at(void* base, uint32_t off)
{
    return *reinterpret_cast<T*>(reinterpret_cast<uint8_t*>(base) + off);
}

template <typename SM> __device__ __forceinline__ bool aborted(SM& s) { return *reinterpret_cast<volatile int*>(&s.abort) != 0; }
template <typename SM> __device__ __forceinline__ void set_abort(SM& s) { *reinterpret_cast<volatile int*>(&s.abort) = 1; }

// Bounded wait that also gives up once another thread has: at most `tries`
// suspended tries of about a microsecond each, then a last look.  Kept to a few
// instructions, as the chunk kernel lives off its instruction cache.
constexpr uint32_t kTryNs = 1000;
template <typename SM>
__device__ __forceinline__ bool wait_or_abort(SM& s, uint64_t* bar, uint32_t parity, uint32_t tries)
{
    while (!(tries ? mbar_try_wait_hint(bar, parity, kTryNs) : mbar_test(bar, parity))) {
        if (aborted(s)) return false;
        if (tries-- == 0) {
            set_abort(s);
            return false;
        }
    }
    return true;
}
// the tries that make up a bound in ns (0: the default)
__device__ __forceinline__ uint32_t wait_tries(unsigned long long ns)
{
    const unsigned long long n = (ns ? ns : kWaitNs) / kTryNs;
    return n > 0xfffffff0ull ? 0xfffffff0u : (uint32_t)n;
}
// ... by a whole warp, which gets one answer
template <typename SM>
__device__ __forceinline__ bool warp_wait(SM& s, uint64_t* bar, uint32_t parity, uint32_t tries)
{
    return __all_sync(0xffffffffu, wait_or_abort(s, bar, parity, tries));
}
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity, uint64_t t0)
{
    while (!mbar_test(bar, parity) && globaltimer_ns() - t0 < kWaitNs) __nanosleep(64);
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane)
{
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// ---- row values ---------------------------------------------------------------------

// of one (b, h, chunk): [kVals][128] floats, then four more.
//   kDt dt, kG2h / kG2l gamma (log2 units, double-float), kW w, kU u, kSg
//   ddt/d(raw dt), kV exp(gamma at the last row of s's 32-row block - gamma_s),
//   kUb + i: exp(gamma_r - gamma at block i's last row) for r from block i on
//   (1 or more inside the block, at most 2^60)
// then: D; bits of the diagonal blocks that decay by more than 2^60; A
enum { kDt, kG2h, kG2l, kW, kU, kSg, kV, kUb, kVals = kUb + 4 };
constexpr int kValStride = kVals * Q + 4;
// A diagonal block splits exp(gamma_r - gamma_s) at its last row when it decays
// by at most this (log2 units): both factors stay within 2^60.
constexpr float kSplitMaxLog2 = 60.0f;
constexpr int kRowHeads = 8;  // a warp each

__global__ void __launch_bounds__(32 * kRowHeads) scan_bwd_rows_kernel(ScanBwdTcParams p)
{
    __shared__ float raw[Q][kRowHeads + 1];
    griddep_launch_dependents();
    const int c = blockIdx.x, h0 = blockIdx.y * kRowHeads, b = blockIdx.z;
    const int nc = gridDim.x, lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int rows = min(Q, p.S - c * Q);
    for (int i = threadIdx.x; i < Q * kRowHeads; i += 32 * kRowHeads) {
        const int r = i / kRowHeads, m = i % kRowHeads;
        raw[r][m] = r < rows && h0 + m < p.H ? p.dt[((size_t)b * p.S + c * Q + r) * p.H + h0 + m] : 0.0f;
    }
    __syncthreads();
    const bool sp = (p.flags & kDtSoftplus) != 0;
    if (h0 + k < p.H) {
        const int h = h0 + k;
        const float Ah = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
        float dt[4], sg[4], gh[4], gl[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * lane + i;
            const float v = sp ? raw[r][k] + bias : raw[r][k];
            dt[i] = r < rows ? (sp ? softplus_full(v) : v) : 0.0f;
            sg[i] = sp ? 1.0f / (1.0f + expf(-v)) : 1.0f;
            gh[i] = fminf(dt[i] * Ah, 0.0f);
            gl[i] = 0.0f;
            if (i > 0) df_add(gh[i], gl[i], gh[i - 1], gl[i - 1]);
        }
        float th = gh[3], tl = gl[3];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const float oh = __shfl_up_sync(0xffffffffu, th, d), ol = __shfl_up_sync(0xffffffffu, tl, d);
            if (lane >= d) df_add(th, tl, oh, ol);
        }
        float eh = __shfl_up_sync(0xffffffffu, th, 1), el = __shfl_up_sync(0xffffffffu, tl, 1);
        if (lane == 0) eh = el = 0.0f;
        float oh[4], ol[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            df_add(gh[i], gl[i], eh, el);
            df_to_log2(gh[i], gl[i], oh[i], ol[i]);
        }
        const float qh = __shfl_sync(0xffffffffu, oh[3], 31), ql = __shfl_sync(0xffffffffu, ol[3], 31);
        float w[4], u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = exp2_diff(qh, ql, oh[i], ol[i], 0.0f);
            u[i] = exp2_diff(oh[i], ol[i], 0.0f, 0.0f, 0.0f);
        }
        float4* out = reinterpret_cast<float4*>(p.vals + (((size_t)b * p.H + h) * nc + c) * kValStride);
        out[kDt * 32 + lane] = make_float4(dt[0], dt[1], dt[2], dt[3]);
        out[kG2h * 32 + lane] = make_float4(oh[0], oh[1], oh[2], oh[3]);
        out[kG2l * 32 + lane] = make_float4(ol[0], ol[1], ol[2], ol[3]);
        out[kW * 32 + lane] = make_float4(w[0], w[1], w[2], w[3]);
        out[kU * 32 + lane] = make_float4(u[0], u[1], u[2], u[3]);
        out[kSg * 32 + lane] = make_float4(sg[0], sg[1], sg[2], sg[3]);
        int exact = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float fh = __shfl_sync(0xffffffffu, oh[0], 8 * k), fl = __shfl_sync(0xffffffffu, ol[0], 8 * k);
            const float mh = __shfl_sync(0xffffffffu, oh[3], 8 * k + 7), ml = __shfl_sync(0xffffffffu, ol[3], 8 * k + 7);
            if (!((fh - mh) + (fl - ml) <= kSplitMaxLog2)) exact |= 1 << k;
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = exp2_diff(oh[i], ol[i], mh, ml, kSplitMaxLog2);
            if ((lane >> 3) >= k) out[(kUb + k) * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
            if ((lane >> 3) == k) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = exp2_diff(mh, ml, oh[i], ol[i], 0.0f);
                out[kV * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
        if (lane == 0) out[kVals * 32] = make_float4(p.D ? p.D[h] : 0.0f, __int_as_float(exact), Ah, 0.0f);
    }
}

// ---- boundary states --------------------------------------------------------------------

// In the workspace a boundary state is two images, hi and lo, of the shared
// memory that the chunk kernel's products read it from: element (n, p) is
// number p % 8 of the 16 bytes at (p / 8) * kStatePitch + n * 16.  A thread that holds
// the row n then writes it with stores that are contiguous over the warp, and one
// untiled copy loads it.
constexpr int kStatePitch = N * 16;
constexpr int kStateBytes = N * P * 2;  // of one of the two

// kHeads heads of a group in a CTA, eight warps each: they share the B or C
// tiles, which halves that part of what the walk reads from L2, and one product
// serves both (128 columns keep the tensor pipe twice as busy as 64).  While a
// chunk's product runs, the value before it leaves and the next chunk's rows
// are scaled: 45 us for 2048 rows of 128 heads (with two planes of the scaled rows 42,
// and 49 with the two in turn).
// So x and g, and mid of the scaled rows, have stages.  B or C has two as well where
// there is room; otherwise it is asked for when the last product is done, some thousand
// cycles before the rows of the next are ready.
constexpr int kStX = 3;
template <int kHeads> struct __align__(1024) StSmem {
    static constexpr int kM = kHeads == 1 ? 2 : 1;
    __nv_bfloat16 M[kM][2][Q * 64];    // B or C tile [row][n], 2 panels of 64 n (TMA, SW128)
    struct {
        __nv_bfloat16 X[kStX][Q * 64]; // x or g tile [row][p]; scaled in place (hi)
        __nv_bfloat16 mid[2][Q * 64];  // the scaled rows' mid, by parity
        __nv_bfloat16 lo[Q * 64];      // ... and lo
    } hd[kHeads];
    uint64_t full_x[kStX], full_m[kM], ready, done;
    uint32_t tmem_base;
    int abort;
};
template <int kHeads> constexpr size_t kStSmemBytes = sizeof(StSmem<kHeads>) + 1024;
static_assert(kStSmemBytes<2> <= 232448, "shared memory per CTA");
static_assert(offsetof(StSmem<2>, hd) % 1024 == 0 && sizeof(StSmem<2>::hd[0]) % 1024 == 0, "tiles");

template <int kHeads>
__global__ void __launch_bounds__(256 * kHeads + 32, 1)
    scan_bwd_states_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_g,
                              const ScanBwdTcParams p)
{
    constexpr int kControl = 8 * kHeads, kM = StSmem<kHeads>::kM;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    StSmem<kHeads>& s =
        *reinterpret_cast<StSmem<kHeads>*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int h0 = blockIdx.x * kHeads, b = blockIdx.z;
    const bool back = blockIdx.y != 0;
    const int H = p.H, G = p.G, g = h0 / (H / G);  // kHeads divides the group's heads
    const int nc = (p.S + Q - 1) / Q;
    const uint32_t wlim = wait_tries(p.wait_ns);
    // the last product of a direction is needed only as the final value
    const int steps = back && p.dh0 != nullptr ? nc : nc - 1;
    auto chunk = [&](int i) { return back ? nc - 1 - i : i; };

    if (warp == kControl) {
        if (lane == 0) {
            for (int k = 0; k < kStX; ++k) mbar_init(&s.full_x[k], 1);
            for (int k = 0; k < kM; ++k) mbar_init(&s.full_m[k], 1);
            mbar_init(&s.ready, 8 * kHeads);
            mbar_init(&s.done, 1);
            s.abort = 0;
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(&s.tmem_base, 64 * kHeads);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = s.tmem_base;
    griddep_launch_dependents();

    if (warp == kControl) {
        const CUtensorMap* mx = back ? &map_g : &map_x;
        const int cm = H * P + (back ? G * N : 0) + g * N;
        int nx = 0, nm = 0, nd = 0;  // loads and commits issued
        auto load_x = [&]() {
            if (elect_one()) {
                const int k = nx % kStX;
                mbar_arrive_expect_tx(&s.full_x[k], kHeads * Q * 64 * 2);
                for (int m = 0; m < kHeads; ++m) tma_load_3d(s.hd[m].X[k], mx, &s.full_x[k], (h0 + m) * P, chunk(nx) * Q, b);
            }
            __syncwarp();
            ++nx;
        };
        auto load_m = [&]() {
            if (elect_one()) {
                uint64_t* bar = &s.full_m[nm % kM];
                mbar_arrive_expect_tx(bar, 2 * Q * 64 * 2);
                tma_load_3d(s.M[nm % kM][0], &map_x, bar, cm, chunk(nm) * Q, b);
                tma_load_3d(s.M[nm % kM][1], &map_x, bar, cm + 64, chunk(nm) * Q, b);
            }
            __syncwarp();
            ++nm;
        };
        while (nx < min(steps, kStX - 1)) load_x();
        while (nm < min(steps, kM)) load_m();
        bool ok = true;
        for (int i = 0; i < steps; ++i) {
            // the scaled rows; the last product has been taken out of TMEM by then, so
            // its stages are free
            if (!(ok = warp_wait(s, &s.ready, i & 1, wlim) && warp_wait(s, &s.full_m[i % kM], (i / kM) & 1, wlim))) break;
            tc_fence_after();
            const uint64_t dM = sdesc_sw128(smem_u32(s.M[i % kM]), Q * 128, 1024);
            const uint32_t lead = elect_one();
            // the heads side by side in one product: 64 columns each, a tile's
            // distance apart; the smallest plane first, as an addition cuts off bits of the sum
            auto side = [&](const void* tile) { return sdesc_sw128(smem_u32(tile), sizeof(s.hd[0]), 1024); };
            const uint64_t planes[3] = {side(s.hd[0].lo), side(s.hd[0].mid[i & 1]), side(s.hd[0].X[i % kStX])};
#pragma unroll
            for (int q = 0; q < 3; ++q)
#pragma unroll
                for (int m = 0; m < 8; ++m)
                    mma_bf16_ss_by(lead, tb, dM + 128 * m, planes[q] + 128 * m, idesc_state(kHeads), q + m > 0);
            mma_commit_by(elect_one(), &s.done);
            ++nd;
            if (nx < steps) load_x();
            if (nm < min(steps, i + 2)) {
                if (kM == 1 && !(ok = warp_wait(s, &s.done, i & 1, wlim))) break;
                load_m();
            }
        }
        if (!ok) set_abort(s);
        if (elect_one()) {
            // nothing of ours in flight when the CTA leaves (bounded waits)
            const uint64_t t0 = globaltimer_ns();
            if (nd > 0) drain(&s.done, (nd - 1) & 1, t0);
            for (int k = max(0, nx - kStX); k < nx; ++k) drain(&s.full_x[k % kStX], (k / kStX) & 1, t0);
            for (int k = max(0, nm - kM); k < nm; ++k) drain(&s.full_m[k % kM], (k / kM) & 1, t0);
        }
        __syncwarp();
    } else {
        // this thread's state: n = its TMEM lane, 32 columns p of its head
        auto& t = s.hd[warp >> 3];
        const int h = h0 + (warp >> 3), tid = threadIdx.x & 255;
        const int n = 32 * (warp & 3) + lane, p0 = 32 * ((warp >> 2) & 1);
        const int row = tid >> 1, j0 = 4 * (tid & 1);  // the row and 16-byte chunks it scales
        const uint32_t taddr = tb + 64 * (warp >> 3) + ((uint32_t)(32 * (warp & 3)) << 16) + p0;
        const float* init = back ? p.dhS : p.h0;
        const size_t sb = ((size_t)b * H + h) * P * N, unit = ((size_t)b * H + h) * nc;
        uint8_t* out = reinterpret_cast<uint8_t*>(back ? p.lout : p.hin) + unit * (2 * kStateBytes) +
                       (p0 >> 3) * kStatePitch + n * 16;
        float st[32];
        // (plain loads: dh0 may be the same memory, written by this thread at the end)
#pragma unroll
        for (int k = 0; k < 32; ++k) st[k] = init ? init[sb + (size_t)(p0 + k) * N + n] : 0.0f;
        const float* vals = p.vals + unit * kValStride;
        griddep_wait();  // the row values
        // the row's factor, and the chunk's decay
        auto factor = [&](int i) {
            const float* v = vals + (size_t)chunk(i) * kValStride;
            return back ? v[kU * Q + row] : v[kW * Q + row] * v[kDt * Q + row];
        };
        auto decay = [&](int i) { return vals[(size_t)chunk(i) * kValStride + kU * Q + Q - 1]; };  // exp(gamma_Q)
        // rows of chunk i by their factor: hi in place, mid to its stage, lo kept
        uint4 lo[4];
        auto scale = [&](int i, float f) -> bool {
            const int k = i % kStX;
            if (!warp_wait(s, &s.full_x[k], (i / kStX) & 1, wlim)) return false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t o = chunk_off(row, j0 + j);
                const uint4 x = at<uint4>(t.X[k], o);
                const float2 f2 = make_float2(f, f);
                uint4 hi, mid;
                split2(__fmul2_rn(unpack2(x.x), f2), hi.x, mid.x, lo[j].x);
                split2(__fmul2_rn(unpack2(x.y), f2), hi.y, mid.y, lo[j].y);
                split2(__fmul2_rn(unpack2(x.z), f2), hi.z, mid.z, lo[j].z);
                split2(__fmul2_rn(unpack2(x.w), f2), hi.w, mid.w, lo[j].w);
                at<uint4>(t.X[k], o) = hi;
                at<uint4>(t.mid[i & 1], o) = mid;
            }
            return true;
        };
        // lo, once no product reads the last one
        auto put = [&]() {
#pragma unroll
            for (int j = 0; j < 4; ++j) at<uint4>(t.lo, chunk_off(row, j0 + j)) = lo[j];
            fence_proxy_async_smem();
        };
        auto scaled = [&]() {
            tc_fence_before();  // the last step's TMEM loads
            warp_arrive(&s.ready, lane);
        };
        float fn = 0.0f, en = 0.0f;
        bool ok = true;
        if (steps > 0) {
            if ((ok = scale(0, factor(0)))) {
                put();
                scaled();
            }
            en = decay(0);
            if (steps > 1) fn = factor(1);
        }
        for (int i = 0; i < nc && ok; ++i) {
            // while the product of this chunk runs: the value before it leaves, and the
            // rows of the next are scaled
            uint8_t* o = out + (size_t)chunk(i) * (2 * kStateBytes);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float2 v2[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) v2[m] = make_float2(st[8 * k + 2 * m], st[8 * k + 2 * m + 1]);
                uint4 hi, l;
                split8(v2, hi, l);
                *reinterpret_cast<uint4*>(o + k * kStatePitch) = hi;
                *reinterpret_cast<uint4*>(o + kStateBytes + k * kStatePitch) = l;
            }
            if (i >= steps) break;
            const float e = en;
            const bool more = i + 1 < steps;
            if (more) {
                if (!(ok = scale(i + 1, fn))) break;
                en = decay(i + 1);
                if (i + 2 < steps) fn = factor(i + 2);
            }
            if (!(ok = warp_wait(s, &s.done, i & 1, wlim))) break;
            tc_fence_after();
            float d[32];
            tmem_ld32(taddr, d);
            if (more) put();
            tmem_ld_wait();
            if (more) scaled();
#pragma unroll
            for (int k = 0; k < 32; ++k) st[k] = fmaf(e, st[k], d[k]);
        }
        if (ok && back && p.dh0 != nullptr)
#pragma unroll
            for (int k = 0; k < 32; ++k) p.dh0[sb + (size_t)(p0 + k) * N + n] = st[k];
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kControl) {
        tc_fence_after();
        tmem_dealloc(tb, 64 * kHeads);
        if (lane == 0 && aborted(s)) atomicOr(p.err, kErrTimeout);
    }
}

// ---- one chunk of one group ---------------------------------------------------------------

// 16 warps and no more: a 17th would leave each thread 96 registers instead of
// 128, and the C.B and F blocks that a warp keeps take 64.  The code of the head
// loop is kept near 32 KB, rolled where that costs little: an SM fetches
// straight-line code beyond that at 5 bytes a cycle (measured: 1.2 cycles an
// instruction at 32 KB of loop, 3.1 at 64 KB), and the warps of this kernel run
// eight different pieces of it at a time.  Warp w works on TMEM lanes 32 (w % 4)..
// (a quarter's rows s), columns r of block w / 4.  Of the six warps whose
// block has r before s, and so no mask, one issues every load and product, one
// ends the last head's rows, and four take <lam, h>.
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kControlWarp = 3;   // TMA and MMA; its 16 columns go to the next two
constexpr int kRowWarp = 7;       // da of the last head
constexpr int kDotWarps = 4;      // <lam, h>: 1, 2, 6 and 11
constexpr int kDotChunks = N * P / 8 / 32 / kDotWarps;  // 16-byte chunks a lane takes
static_assert(32 * kDotWarps * kDotChunks == N * P / 8, "the whole state");
constexpr int kBusy = kWarps - 1; // warps that walk the heads

// TMEM columns (512 allocated)
constexpr uint32_t kColDM = 0;    // dM^T [s][r] by 32-column blocks; CB^T at first  128
                                  // then dx [s][p] over the first 64 of them and
                                  // E^T (bf16 pairs, [s][r/2]) over the other 64
constexpr uint32_t kColE = 64;
constexpr uint32_t kColBl = 128;  // Bl [s][p]                                         64
constexpr uint32_t kColYo = 192;  // Yo [r][p]                                         64
constexpr uint32_t kColDC = 256;  // dC [r][n]                                        128
constexpr uint32_t kColDB = 384;  // dB [s][n]                                        128

struct __align__(1024) BwSmem {
    __nv_bfloat16 C[2][Q * 64];   // C tile [r][n], 2 panels of 64 n (TMA, SW128)
    __nv_bfloat16 B[2][Q * 64];   // B tile [s][n]
    __nv_bfloat16 X[2][Q * 64];   // x tile [s][p] by head parity, then dx, stored from here
    __nv_bfloat16 Gr[2][Q * 64];  // g tile [r][p] by head parity; F^T [s][r] at the end
    // as in the workspace: 16-byte chunks of rows n, by 8 columns p
    __nv_bfloat16 Hh[N * 64];     // h, hi
    __nv_bfloat16 Hl[N * 64];     // ... lo, then u o g of rows r
    __nv_bfloat16 Lh[N * 64];     // lam, hi
    __nv_bfloat16 Ll[N * 64];     // ... lo, then w dt o x of rows s
    float vals[3][kValStride];  // row values of three heads in turn (bulk copies)
    // by head parity
    float rho[2][4][Q];    // by 16-column group: shares of Yo . g
    float sig[2][4][Q];    // by 16-column group: shares of Bl . x
    float krow[2][4][Q];   // [s block][r]: sum over the block's s of dt_s K; its own diagonal
                           // block instead the sum over r' >= r > s
    float kcol[2][4][Q];   // [r block][s]: sum over the block's r >= s of K
    float gx[2][kWarps];   // by warp: shares of the sum of g_s . x_s
    float cross[2][kDotWarps];  // shares of <lam, h>
    uint64_t full_bc, full_xg[2], full_h, full_l;           // TMA landed
    uint64_t cb, dmt, yo, bl, dx, dcb, fin;                 // MMA commits
    uint64_t cbread, erdy, uxrdy, dxrdy, frdy;              // warps -> control
    uint64_t dots, full_v[3];                               // <lam, h> taken; row values landed
    uint64_t dmread[4];                                     // by quarter: columns 64.. of dM^T read
    uint32_t tmem_base;
    int abort;
};
constexpr size_t kBwSmemBytes = sizeof(BwSmem) + 1024;
static_assert(kBwSmemBytes <= 232448, "shared memory per CTA");
static_assert(offsetof(BwSmem, X) % 1024 == 0 && offsetof(BwSmem, Hh) % 1024 == 0 && offsetof(BwSmem, vals) % 1024 == 0, "tile");
static_assert(offsetof(BwSmem, full_bc) % 8 == 0, "mbarriers");

// sums over the lanes of 16 values each: even lane l returns the sum of value
// l >> 1, bit by bit from the top (lane bit 4 picks value bit 3, ..)
__device__ __forceinline__ float lane_sums16(float* v, int lane)
{
#pragma unroll
    for (int half = 8, d = 16; half >= 1; half >>= 1, d >>= 1) {
        const bool up = (lane & d) != 0;
#pragma unroll
        for (int k = 0; k < half; ++k) {
            const float send = up ? v[k] : v[k + half];
            const float keep = up ? v[k + half] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, send, d);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

__device__ __forceinline__ float2 bcast(float v) { return make_float2(v, v); }

// 4 * `panels` products of 16 K elements each into D, by one lane of the warp.
// A K-major operand goes on by 64-element panels of 16 KB, an MN-major one by
// groups of 16 rows [k][..].
template <uint32_t kIdesc>
__device__ __forceinline__ void mma_run(uint32_t d, uint64_t a, uint64_t b, int panels, bool acc)
{
    constexpr uint64_t as = (kIdesc >> 15) & 1 ? 128 : 2, bs = (kIdesc >> 16) & 1 ? 128 : 2;
    constexpr uint64_t ap = as == 128 ? 512 : 1024, bp = bs == 128 ? 512 : 1024;
    const uint32_t lead = elect_one();
#pragma unroll 1
    for (int k = 0; k < panels; ++k, a += ap, b += bp)
#pragma unroll
        for (int m = 0; m < 4; ++m) mma_bf16_ss_by(lead, d, a + as * m, b + bs * m, kIdesc, acc || k + m > 0);
}
__device__ __forceinline__ void commit(uint64_t* bar) { mma_commit_by(elect_one(), bar); }

__global__ void __launch_bounds__(kThreads, 1)
    scan_bwd_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_g,
                       const __grid_constant__ CUtensorMap map_dx, const ScanBwdTcParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    BwSmem& s = *reinterpret_cast<BwSmem*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    // the same value in every lane as far as the compiler can see: the control
    // warp's descriptors then live in uniform registers
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int H = p.H, G = p.G, R = H / G, S = p.S;
    const int c = blockIdx.x, g = blockIdx.y / p.split, sp = blockIdx.y % p.split, b = blockIdx.z;
    const int nc = gridDim.x;
    const int per = (R + p.split - 1) / p.split;
    const int hbeg = g * R + sp * per, nh = min(per, R - sp * per);  // >= 1 head
    const int rows = min(Q, S - c * Q);
    const int Cdim = H * P + 2 * G * N;
    const uint32_t wlim = wait_tries(p.wait_ns);

    if (warp == 0) {
        if (lane == 0) {
            for (uint64_t* q : {&s.full_bc, &s.full_xg[0], &s.full_xg[1], &s.full_h, &s.full_l, &s.cb, &s.dmt, &s.yo,
                                &s.bl, &s.dx, &s.dcb, &s.fin, &s.full_v[0], &s.full_v[1], &s.full_v[2], &s.dmread[3]})
                mbar_init(q, 1);
            for (uint64_t* q : {&s.uxrdy, &s.dxrdy}) mbar_init(q, kBusy);
            mbar_init(&s.erdy, kBusy - 1);  // all but the row warp
            for (uint64_t* q : {&s.cbread, &s.frdy}) mbar_init(q, kWarps);
            mbar_init(&s.dots, kDotWarps);
            for (int k = 0; k < 3; ++k) mbar_init(&s.dmread[k], 2);
            s.abort = 0;
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(&s.tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    // all 512 columns are this CTA's, so the allocation starts at column 0
    const uint32_t tb = 0;
    if (s.tmem_base != 0) set_abort(s);

    // ---- control: the whole warp walks these steps, one lane issues every TMA
    // load and every MMA
    int nx = 0, ns = 0, nv = 0;  // loads issued: x and g, states, row values
    auto load_v = [&]() {
        const int k = nv % 3;
        if (elect_one()) {
            mbar_arrive_expect_tx(&s.full_v[k], kValStride * 4);
            bulk_load(s.vals[k], p.vals + (((size_t)b * H + hbeg + nv) * nc + c) * kValStride, kValStride * 4,
                      &s.full_v[k]);
        }
        ++nv;
    };
    auto load_xg = [&]() {
        if (elect_one()) {
            uint64_t* bar = &s.full_xg[nx & 1];
            mbar_arrive_expect_tx(bar, 2 * Q * 64 * 2);
            tma_load_3d(s.X[nx & 1], &map_x, bar, (hbeg + nx) * P, c * Q, b);
            tma_load_3d(s.Gr[nx & 1], &map_g, bar, (hbeg + nx) * P, c * Q, b);
        }
        ++nx;
    };
    // hi and lo of h and lam of head n; the next head's as far as L2
    auto load_states = [&](int n) {
        if (elect_one()) {
            const size_t o = (((size_t)b * H + hbeg + n) * nc + c) * (2 * N * P);
            mbar_arrive_expect_tx(&s.full_h, 2 * kStateBytes);
            bulk_load(s.Hh, p.hin + o, 2 * kStateBytes, &s.full_h);
            mbar_arrive_expect_tx(&s.full_l, 2 * kStateBytes);
            bulk_load(s.Lh, p.lout + o, 2 * kStateBytes, &s.full_l);
            if (n + 1 < nh) {
                const size_t o2 = o + (size_t)nc * (2 * N * P);
                bulk_prefetch(p.hin + o2, 2 * kStateBytes);
                bulk_prefetch(p.lout + o2, 2 * kStateBytes);
            }
        }
        ++ns;
    };
    // operand descriptors: K-major and MN-major ([k][64] rows) tiles
    auto km = [&](const void* t) { return sdesc_sw128(smem_u32(t), 16, 1024); };
    auto mn = [&](const void* t) { return sdesc_sw128(smem_u32(t), 8192, 1024); };
    auto mn2 = [&](const void* t) { return sdesc_sw128(smem_u32(t), Q * 128, 1024); };  // two panels of 64
    // a state, or rows in its layout: K = n, and K = p
    auto sn = [&](const void* t) { return sdesc_core(smem_u32(t), 128, kStatePitch); };
    auto spk = [&](const void* t) { return sdesc_core(smem_u32(t), kStatePitch, 128); };
    bool issued = false;  // some MMA was
    // rows times a state, its hi plane, then its lo
    auto mma_state = [&](uint32_t d, uint64_t a, uint64_t hi, uint64_t lo) {
        const uint32_t lead = elect_one();
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            const uint64_t ak = a + 1024 * (k & 1), bk = (k < 2 ? lo : hi) + 64 * (k & 1);
#pragma unroll
            for (int m = 0; m < 4; ++m) mma_bf16_ss_by(lead, d, ak + 2 * m, bk + 16 * m, kIdQP, k + m > 0);
        }
    };
    // scaled rows times a state's hi, both in its layout
    auto mma_rows = [&](uint32_t d, uint64_t a, uint64_t hi, bool acc) {
        const uint32_t lead = elect_one();
#pragma unroll
        for (int m = 0; m < 4; ++m)
            mma_bf16_ss_by(lead, d, a + 2 * kStatePitch / 16 * m, hi + 2 * kStatePitch / 16 * m, kIdQQ, acc || m > 0);
    };

    auto ctl_run = [&]() -> bool {
        const int cB = H * P + g * N, cC = cB + G * N;
        if (elect_one()) {
            mbar_arrive_expect_tx(&s.full_bc, 4 * Q * 64 * 2);
            tma_load_3d(s.B[0], &map_x, &s.full_bc, cB, c * Q, b);
            tma_load_3d(s.B[1], &map_x, &s.full_bc, cB + 64, c * Q, b);
            tma_load_3d(s.C[0], &map_x, &s.full_bc, cC, c * Q, b);
            tma_load_3d(s.C[1], &map_x, &s.full_bc, cC + 64, c * Q, b);
        }
        // step i: the products that end head i, and what head i + 1 begins with
        for (int i = -1; i < nh; ++i) {
            const bool next = i + 1 < nh;
            if (i >= 0) {
                // dx over the first columns of dM^T, E^T behind it
                if (!warp_wait(s, &s.erdy, i & 1, wlim)) return false;
                tc_fence_after();
                {
                    const uint64_t dG = mn(s.Gr[i & 1]);
                    const uint32_t lead = elect_one();
#pragma unroll 4
                    for (int k = 0; k < 8; ++k) mma_bf16_ts_by(lead, kColDM, kColE + 8 * k, dG + 128 * k, kIdQP, k > 0);
                    commit(&s.dx);
                }
                // dC and dB
                if (!warp_wait(s, &s.uxrdy, i & 1, wlim)) return false;
                tc_fence_after();
                mma_rows(kColDC, spk(s.Hl), spk(s.Hh), i > 0);
                mma_rows(kColDB, spk(s.Ll), spk(s.Lh), i > 0);
                commit(&s.dcb);
                if (!warp_wait(s, &s.dxrdy, i & 1, wlim)) return false;
            } else {
                load_xg();
                if (!warp_wait(s, &s.full_bc, 0, wlim)) return false;
                tc_fence_after();
                mma_run<kIdQQ>(kColDM, km(s.B), km(s.C), 2, false);
                commit(&s.cb);
                issued = true;
                if (!warp_wait(s, &s.cbread, 0, wlim)) return false;
            }
            if (next) {
                // dM^T, over the columns of the last head's dx
                if (!warp_wait(s, &s.full_xg[(i + 1) & 1], ((i + 1) >> 1) & 1, wlim)) return false;
                tc_fence_after();
                mma_run<kIdQQ>(kColDM, km(s.X[(i + 1) & 1]), km(s.Gr[(i + 1) & 1]), 1, false);
                commit(&s.dmt);
                // its states, once the products with the last head's are done
                if (i >= 0) {
                    if (!warp_wait(s, &s.dcb, i & 1, wlim)) return false;
                } else {
                    griddep_wait();  // the boundary states and row values
                    for (; nv < min(nh, 2);) load_v();
                }
                load_states(i + 1);
                if (!warp_wait(s, &s.full_h, (i + 1) & 1, wlim)) return false;
                tc_fence_after();
                mma_state(kColYo, km(s.C), sn(s.Hh), sn(s.Hl));
                commit(&s.yo);
                if (!warp_wait(s, &s.full_l, (i + 1) & 1, wlim)) return false;
                tc_fence_after();
                mma_state(kColBl, km(s.B), sn(s.Lh), sn(s.Ll));
                commit(&s.bl);
            }
            if (i >= 0) {
                if (elect_one()) {
                    tma_store_3d(&map_dx, s.X[i & 1], (hbeg + i) * P, c * Q, b);
                    bulk_commit();
                }
                __syncwarp();
                // the row warp has arrived for head i, so the values of head i - 1 have no
                // reader: those of head i + 2 take their place
                if (nv < nh) load_v();
            }
            if (nx < nh) {  // once dx has left x's tile (g's has no reader any more)
                if (elect_one()) bulk_wait_read_all();
                __syncwarp();
                load_xg();
            }
        }
        return true;
    };
    auto ctl_end = [&]() -> bool {
        if (!warp_wait(s, &s.frdy, 0, wlim)) return false;
        tc_fence_after();
        mma_run<kIdFC>(kColDB, km(s.Gr), mn2(s.C), 2, true);
        mma_run<kIdFB>(kColDC, mn2(s.Gr), mn2(s.B), 2, true);
        return true;
    };

    // ---- the row warp: da and ddt of a finished head
    auto rows_done = [&](int it) {
        const int q = it & 1, h = hbeg + it;
        const float* v = s.vals[it % 3];
        const float Ah = v[kVals * Q + 2];
        // this lane's rows 4l .. 4l + 3, of block j
        const int j = lane >> 3;
        auto ld4 = [&](const float* a, float* o) {
            const float4 f = *reinterpret_cast<const float4*>(a + 4 * lane);
            o[0] = f.x; o[1] = f.y; o[2] = f.z; o[3] = f.w;
        };
        // totals of K blocks (0,2), (0,3), (1,3)
        float t02 = s.krow[q][0][64 + lane], t03 = s.krow[q][0][96 + lane], t13 = s.krow[q][1][96 + lane];
#pragma unroll 1
        for (int d = 16; d > 0; d >>= 1) {
            t02 += __shfl_xor_sync(0xffffffffu, t02, d);
            t03 += __shfl_xor_sync(0xffffffffu, t03, d);
            t13 += __shfl_xor_sync(0xffffffffu, t13, d);
        }
        const float far = j == 1 ? t02 + t03 : (j == 2 ? t03 + t13 : 0.0f);  // K blocks below and left of block j
        float dt[4], rho[4] = {}, sig[4] = {}, ro[4] = {}, co[4] = {}, dg[4], cc[4], t4[4];
        ld4(v + kDt * Q, dt);
        ld4(s.krow[q][j], dg);
        ld4(s.kcol[q][j], cc);
#pragma unroll 1
        for (int m = 0; m < 4; ++m) {
            float a[4], d[4], e[4], f[4];
            ld4(s.rho[q][m], a);
            ld4(s.sig[q][m], d);
            ld4(s.krow[q][m], e);
            ld4(s.kcol[q][m], f);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                rho[k] += a[k];
                sig[k] += d[k];
                ro[k] += m < j ? e[k] : 0.0f;
                co[k] += m > j ? f[k] : 0.0f;
            }
        }
        ld4(v + kU * Q, t4);
#pragma unroll
        for (int k = 0; k < 4; ++k) rho[k] *= t4[k];
        ld4(v + kW * Q, t4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            sig[k] *= t4[k];
            cc[k] += co[k];
        }
        // over the rows behind: rho over the chunk, ro over the block (inclusive);
        // over the rows before: dt sig over the chunk, dt co over the block
        float sr[4], so[4], ps[4], pc[4];
        sr[3] = rho[3];
        so[3] = ro[3];
        ps[0] = pc[0] = 0.0f;
#pragma unroll
        for (int k = 1; k < 4; ++k) {
            sr[3 - k] = sr[4 - k] + rho[3 - k];
            so[3 - k] = so[4 - k] + ro[3 - k];
            ps[k] = fmaf(dt[k - 1], sig[k - 1], ps[k - 1]);
            pc[k] = fmaf(dt[k - 1], co[k - 1], pc[k - 1]);
        }
        float a = sr[0], bb = so[0], e = fmaf(dt[3], sig[3], ps[3]), f = fmaf(dt[3], co[3], pc[3]);
        const int l8 = lane & 7;
#pragma unroll 1
        for (int d = 1; d < 32; d <<= 1) {
            const float x = __shfl_down_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, e, d);
            if (lane + d < 32) a += x;
            if (lane >= d) e += y;
            if (d < 8) {
                const float z = __shfl_down_sync(0xffffffffu, bb, d), w = __shfl_up_sync(0xffffffffu, f, d);
                if (l8 + d < 8) bb += z;
                if (l8 >= d) f += w;
            }
        }
        float an = __shfl_down_sync(0xffffffffu, a, 1), en = __shfl_up_sync(0xffffffffu, e, 1);
        float bn = __shfl_down_sync(0xffffffffu, bb, 1), fn = __shfl_up_sync(0xffffffffu, f, 1);
        if (lane == 31) an = 0.0f;
        if (lane == 0) en = 0.0f;
        if (l8 == 7) bn = 0.0f;
        if (l8 == 0) fn = 0.0f;
        const float cr = ((s.cross[q][0] + s.cross[q][1]) + (s.cross[q][2] + s.cross[q][3])) * v[kU * Q + Q - 1];
        float dA = 0.0f, db = 0.0f, dd = lane < kWarps ? s.gx[q][lane] : 0.0f;
        ld4(v + kSg * Q, t4);
        float* out = p.ddt + ((size_t)b * S + c * Q + 4 * lane) * H + h;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float da = ((sr[k] + an) + (ps[k] + en)) + ((so[k] + bn) + (pc[k] + fn)) + ((dg[k] + far) + cr);
            if (dt[k] * Ah > 0.0f) da = 0.0f;  // a decay clamped at 1 passes no gradient
            const float d = fmaf(Ah, da, cc[k] + sig[k]) * t4[k];
            if (4 * lane + k < rows) {
                out[(size_t)k * H] = d;
                dA = fmaf(dt[k], da, dA);
                db += d;
            }
        }
#pragma unroll 1
        for (int d = 16; d > 0; d >>= 1) {
            dA += __shfl_xor_sync(0xffffffffu, dA, d);
            db += __shfl_xor_sync(0xffffffffu, db, d);
            dd += __shfl_xor_sync(0xffffffffu, dd, d);
        }
        if (!(p.flags & kDtSoftplus)) db = 0.0f;  // dt_bias has no part in dt then
        if (lane < 3) p.part[(((size_t)b * nc + c) * 3 + lane) * H + h] = lane == 0 ? dA : (lane == 1 ? db : dd);
        __syncwarp();
    };

    // ---- compute: TMEM lanes 32 i + lane; column block j
    const int i = warp & 3, j = warp >> 2;
    const int row = 32 * i + lane;  // s (or r, or n) of this thread
    const uint32_t tl = tb + ((uint32_t)(32 * i) << 16);
    float2 cb[16], facc[16];
    bool ok = true;
    if (warp == kControlWarp) {
        for (int k = 0; k < 2; ++k) s.rho[k][0][row] = s.sig[k][0][row] = s.gx[k][warp] = 0.0f;  // no share of its own
        if (lane == 0) mbar_arrive(&s.cbread);
        ok = ctl_run();
        if (!ok) {
            set_abort(s);
            // the walk may still run, and writes to the call's scratch and outputs: a CTA
            // that gave up early must not let the stream go on before it
            griddep_wait();
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) facc[k] = make_float2(0.0f, 0.0f);
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) facc[k] = make_float2(0.0f, 0.0f);
        ok = warp_wait(s, &s.cb, 0, wlim);
        if (ok) {
            tc_fence_after();
            tmem_ld32(tl + kColDM + 32 * j, reinterpret_cast<float*>(cb));
            tmem_ld_wait();
            // above the diagonal of a diagonal block, so that what it scales is 0
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                if (j == i && 2 * k < lane) cb[k].x = 0.0f;
                if (j == i && 2 * k + 1 < lane) cb[k].y = 0.0f;
            }
            tc_fence_before();
            warp_arrive(&s.cbread, lane);
        }
    }
    // this warp's 8-column chunks of a [row][64] tile (and of Yo, Bl, dx): two,
    // 2j and 2j + 1; in quarter 3, whose first warp is the control warp, two
    // warps take one of its chunks as a third
    const int chunks = i == 3 && (j == 1 || j == 2) ? 3 : 2;
    auto chunk = [&](int m) { return m < 2 ? 2 * j + m : j - 1; };
    // <lam, h>, the w-th quarter of it
    auto dots = [&](int it, int w) -> bool {
        if (!warp_wait(s, &s.full_h, it & 1, wlim) || !warp_wait(s, &s.full_l, it & 1, wlim)) return false;
        uint32_t o = 16 * (w * kDotChunks * 32 + lane);
        float2 acc[4] = {};
#pragma unroll 2
        for (int k = 0; k < kDotChunks; ++k, o += 16 * 32) {
            float2 a[4], d[4], e[4], f[4];
            unpack8(at<uint4>(s.Hh, o), a);
            unpack8(at<uint4>(s.Hl, o), d);
            unpack8(at<uint4>(s.Lh, o), e);
            unpack8(at<uint4>(s.Ll, o), f);
#pragma unroll
            for (int m = 0; m < 4; ++m) acc[m] = __ffma2_rn(__fadd2_rn(a[m], d[m]), __fadd2_rn(e[m], f[m]), acc[m]);
        }
        acc[0] = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
        float cross = acc[0].x + acc[0].y;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) cross += __shfl_xor_sync(0xffffffffu, cross, d);
        if (lane == 0) s.cross[it & 1][w] = cross;
        warp_arrive(&s.dots, lane);
        return true;
    };
    for (int it = 0; it <= nh && ok && warp != kControlWarp; ++it) {
        const int q = it & 1;
        // the row warp first finishes the last head (every warp's end of it was
        // waited for below), in one step more than there are heads
        if (warp == kRowWarp && it > 0) rows_done(it - 1);
        if (it == nh) break;
        const float* vals = s.vals[it % 3];
        if (!(ok = warp_wait(s, &s.full_v[it % 3], (it / 3) & 1, wlim))) break;
        if (j >= i && !(ok = warp_wait(s, &s.dmt, it & 1, wlim))) break;
        tc_fence_after();
        if (j < i) {
            if (warp != kRowWarp) {
                // ---- <lam, h> while the others mask
                if (!(ok = dots(it, warp == 6 ? 2 : (warp == 11 ? 3 : warp - 1)))) break;
                // r before s: E^T is zero there (warp 11: its quarter's others too)
                if (!(ok = warp_wait(s, &s.dmread[i], it & 1, wlim))) break;
                tc_fence_after();
                const uint32_t z[16] = {};
                tmem_st16(tl + kColE + 16 * j, z);
                if (i == 3) {
                    tmem_st16(tl + kColE, z);
                    tmem_st16(tl + kColE + 16, z);
                }
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(&s.erdy, lane);
            }
        } else {
            // ---- mask: E^T, F^T, K of block (s block i, r block j)
            const float dt = vals[kDt * Q + row];
            // the decay splits at the last row of block i; in a diagonal block with
            // too much of it, it is taken pair by pair instead
            const bool exact = j == i && ((__float_as_int(vals[kVals * Q + 1]) >> i) & 1);
            const float V = exact ? 1.0f : vals[kV * Q + row];
            const float Vd = V * dt;
            const float* U = vals + (kUb + i) * Q + 32 * j;
            float2 ccol = make_float2(0.0f, 0.0f);
            float suffix = 0.0f;
            uint32_t ep[2][8];  // E^T of the columns, as bf16 pairs
            float2 d[8];
            // factor(r): exp(gamma - ..) of the pair of columns r, r + 1
            auto off = [&](int hf, auto factor) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 u = factor(16 * hf + 2 * k), cu = cb[8 * hf + k];
                    const float2 t = __fmul2_rn(d[k], u), kp = __fmul2_rn(cu, t);
                    ccol = __fadd2_rn(ccol, kp);
                    facc[8 * hf + k] = __ffma2_rn(t, bcast(Vd), facc[8 * hf + k]);
                    ep[hf][k] = pack2(__fmul2_rn(__fmul2_rn(cu, u), bcast(Vd)));
                    d[k] = __fmul2_rn(kp, bcast(Vd));
                }
            };
            // Above the diagonal cb is 0, and so is dM here: factor would be up to 2^60
            // there, and dM beyond 2^68 times it no number.  L is formed before anything
            // is scaled, so it is at most 1 wherever dM counts.  (Multiplied in one after the
            // other, the factors took finite rows to NaN; that was 1 % faster, 118.6
            // us a call of 2048 rows of 128 heads against 120.2 at the time.)
            auto diagonal = [&](int hf, auto factor) {
#pragma unroll
                for (int k = 7; k >= 0; --k) {
                    const int r = 16 * hf + 2 * k;  // in the block, as lane is s
                    const float2 L = __fmul2_rn(factor(r), bcast(V)), e = __fmul2_rn(cb[8 * hf + k], L);
                    const float2 m = make_float2(r >= lane ? d[k].x : 0.0f, r + 1 >= lane ? d[k].y : 0.0f);
                    const float2 kp = __fmul2_rn(e, m);
                    ccol = __fadd2_rn(ccol, kp);
                    facc[8 * hf + k] = __ffma2_rn(__fmul2_rn(m, L), bcast(dt), facc[8 * hf + k]);
                    ep[hf][k] = pack2(__fmul2_rn(e, bcast(dt)));
                    // the sums over r' >= r, where r > s
                    const float sy = fmaf(kp.y, dt, suffix);
                    suffix = fmaf(kp.x, dt, sy);
                    d[k] = make_float2(r > lane ? suffix : 0.0f, r + 1 > lane ? sy : 0.0f);
                }
            };
            auto table = [&](int r) { return *reinterpret_cast<const float2*>(U + r); };
            auto pairs = [&](int r) {
                const float gh = vals[kG2h * Q + row], gl = vals[kG2l * Q + row];
                const float2 rh = *reinterpret_cast<const float2*>(&vals[kG2h * Q + 32 * j + r]);
                const float2 rl = *reinterpret_cast<const float2*>(&vals[kG2l * Q + 32 * j + r]);
                return make_float2(ex2_fast(fminf((rh.x - gh) + (rl.x - gl), 0.0f)),
                                   ex2_fast(fminf((rh.y - gh) + (rl.y - gl), 0.0f)));
            };
#pragma unroll
            for (int hf = 1; hf >= 0; --hf) {
                tmem_ld16(tl + kColDM + 32 * j + 16 * hf, reinterpret_cast<float*>(d));
                tmem_ld_wait();
                if (hf == 0 && j >= 2) {
                    tc_fence_before();
                    warp_arrive(&s.dmread[i], lane);
                }
                if (j > i) off(hf, table);
                else if (!exact) diagonal(hf, table);
                else diagonal(hf, pairs);
                if (hf == 0) {
                    // E^T goes over columns 64.., once they are read
                    if (!(ok = warp_wait(s, &s.dmread[i], it & 1, wlim))) break;
                    tc_fence_after();
                    tmem_st8(tl + kColE + 16 * j, ep[0]);
                    tmem_st8(tl + kColE + 16 * j + 8, ep[1]);
                    tmem_st_wait();
                    tc_fence_before();
                    warp_arrive(&s.erdy, lane);
                }
                const float sum = lane_sums16(reinterpret_cast<float*>(d), lane);
                if ((lane & 1) == 0) s.krow[q][i][32 * j + 16 * hf + (lane >> 1)] = sum;
            }
            if (!ok) break;
            s.kcol[q][j][row] = (ccol.x + ccol.y) * (j == i ? 1.0f : V);  // (a diagonal block's has it)
        }

        // ---- Yo . g, u o g over h's lo; Bl . x, w dt o x over lam's lo
        if (!(ok = warp_wait(s, &s.yo, it & 1, wlim) && warp_wait(s, &s.bl, it & 1, wlim) &&
                   warp_wait(s, &s.dots, it & 1, wlim)))
            break;
        tc_fence_after();
        const float wd = vals[kW * Q + row] * vals[kDt * Q + row];
        {
            const float u = vals[kU * Q + row];
            float2 dr = make_float2(0.0f, 0.0f), ds = dr, dg = dr;
#pragma unroll
            for (int m = 0; m < 3; ++m) {
                if (m >= chunks) break;
                float2 yo[4], bl[4], gv[4], xv[4];
                tmem_ld8(tl + kColYo + 8 * chunk(m), reinterpret_cast<float*>(yo));
                tmem_ld8(tl + kColBl + 8 * chunk(m), reinterpret_cast<float*>(bl));
                const uint32_t o = chunk_off(row, chunk(m));
                unpack8(at<uint4>(s.Gr[q], o), gv);
                unpack8(at<uint4>(s.X[q], o), xv);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    dr = __ffma2_rn(yo[k], gv[k], dr);
                    ds = __ffma2_rn(bl[k], xv[k], ds);
                    dg = __ffma2_rn(gv[k], xv[k], dg);
                    gv[k] = __fmul2_rn(gv[k], bcast(u));
                    xv[k] = __fmul2_rn(xv[k], bcast(wd));
                }
                const uint32_t so = chunk(m) * kStatePitch + row * 16;
                at<uint4>(s.Hl, so) = pack8(gv);
                at<uint4>(s.Ll, so) = pack8(xv);
            }
            s.rho[q][j][row] = dr.x + dr.y;
            s.sig[q][j][row] = ds.x + ds.y;
            float x = dg.x + dg.y;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
            if (lane == 0) s.gx[q][warp] = x;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(&s.uxrdy, lane);

        // ---- dx over x
        if (!(ok = warp_wait(s, &s.dx, it & 1, wlim))) break;
        tc_fence_after();
        {
            const float D = vals[kVals * Q];
#pragma unroll 1
            for (int m = 0; m < chunks; ++m) {
                float2 dx[4], bl[4], gv[4];
                tmem_ld8(tl + kColDM + 8 * chunk(m), reinterpret_cast<float*>(dx));
                tmem_ld8(tl + kColBl + 8 * chunk(m), reinterpret_cast<float*>(bl));
                const uint32_t o = chunk_off(row, chunk(m));
                unpack8(at<uint4>(s.Gr[q], o), gv);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    gv[k] = __ffma2_rn(gv[k], bcast(D), __ffma2_rn(bl[k], bcast(wd), dx[k]));
                at<uint4>(s.X[q], o) = pack8(gv);  // leaves with a TMA store
            }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(&s.dxrdy, lane);
        if (warp == kRowWarp) ok = warp_wait(s, &s.dxrdy, it & 1, wlim);
    }
    // ---- F^T in bf16 over the g tiles, once every warp is done reading them
    if (ok) ok = warp_wait(s, &s.dxrdy, (nh - 1) & 1, wlim);
    if (ok) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            if (j == i && 2 * k < lane) facc[k].x = 0.0f;
            if (j == i && 2 * k + 1 < lane) facc[k].y = 0.0f;
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) at<uint4>(s.Gr[j >> 1], chunk_off(row, 4 * (j & 1) + m)) = pack8(facc + 4 * m);
        fence_proxy_async_smem();
        warp_arrive(&s.frdy, lane);
    }
    if (warp == kControlWarp) {
        if (ok && !(ok = ctl_end())) set_abort(s);
        if (elect_one()) {
            // nothing of ours in flight when the CTA leaves (bounded waits)
            bulk_wait_all();
            const uint64_t t0 = globaltimer_ns();
            if (issued) {
                mma_commit(&s.fin);
                drain(&s.fin, 0, t0);
            }
            drain(&s.full_bc, 0, t0);
            for (int k = max(0, nx - 2); k < nx; ++k) drain(&s.full_xg[k & 1], (k >> 1) & 1, t0);
            if (ns > 0) {
                drain(&s.full_h, (ns - 1) & 1, t0);
                drain(&s.full_l, (ns - 1) & 1, t0);
            }
            for (int k = max(0, nv - 3); k < nv; ++k) drain(&s.full_v[k % 3], (k / 3) & 1, t0);
        }
    }
    __syncwarp();
    if (ok) ok = warp_wait(s, &s.fin, 0, wlim);
    if (ok) {
        tc_fence_after();
        // 32 of the N columns of dB (row s) and dC (row r)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            float v[32];
            tmem_ld32(tl + (m ? kColDC : kColDB) + 32 * j, v);
            tmem_ld_wait();
            if (row < rows) {
                if (p.split == 1) {
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.dxbc) + ((size_t)b * S + c * Q + row) * Cdim +
                                         H * P + (m * G + g) * N + 32 * j;
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        float2 f[4];
#pragma unroll
                        for (int n = 0; n < 4; ++n) f[n] = make_float2(v[k + 2 * n], v[k + 2 * n + 1]);
                        *reinterpret_cast<uint4*>(dst + k) = pack8(f);
                    }
                } else {
                    float* dst = p.bcpart + (((size_t)sp * p.B + b) * S + c * Q + row) * (2 * G * N) + (m * G + g) * N + 32 * j;
#pragma unroll
                    for (int k = 0; k < 32; k += 4) *reinterpret_cast<float4*>(dst + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tb, 512);
        if (lane == 0 && aborted(s)) atomicOr(p.err, kErrTimeout);
    }
}

// ---- host side ------------------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

bool encode_fn()
{
    std::call_once(g_encode_once, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return g_encode != nullptr;
}

// The arrays as tiles: x | B | C rows, dy, dxbc.
struct TcMaps {
    CUtensorMap x, g, dx;
};
bool make_maps(const ScanBwdTcParams& p, TcMaps* m)
{
    const long long Cdim = (long long)p.H * P + 2LL * p.G * N;
    auto map = [&](CUtensorMap* t, const void* base, long long cols) {
        return make_rows_map(t, base, 2, cols, p.S, p.B, 64, Q, true);
    };
    return map(&m->x, p.xbc, Cdim) && map(&m->g, p.dy, (long long)p.H * P) && map(&m->dx, p.dxbc, Cdim);
}

template <int kHeads> cudaError_t launch_states_t(const ScanBwdTcParams& p, TcMaps& m, cudaStream_t st)
{
    static std::atomic<bool> done[kMaxDevices];
    const void* kernel = (const void*)scan_bwd_states_tc_kernel<kHeads>;
    const cudaError_t e = allow_smem(kernel, kStSmemBytes<kHeads>, done);
    if (e != cudaSuccess) return e;
    void* args[] = {&m.x, &m.g, const_cast<ScanBwdTcParams*>(&p)};
    return launch_after(kernel, dim3(p.H / kHeads, 2, p.B), 256 * kHeads + 32, kStSmemBytes<kHeads>, st, args);
}

cudaError_t launch_states(const ScanBwdTcParams& p, TcMaps& m, cudaStream_t st)
{
    // two heads a CTA where that leaves a CTA for nearly every SM (the whole call: 2048
    // rows of 128 heads 121 us, one head a CTA 137; 4 x 1111 rows of 16 heads 59, one
    // head 53)
    const bool two = (p.H / p.G) % 2 == 0 && (long long)p.B * p.H >= 128;
    return two ? launch_states_t<2>(p, m, st) : launch_states_t<1>(p, m, st);
}

cudaError_t launch_chunks(const ScanBwdTcParams& p, TcMaps& m, cudaStream_t st)
{
    static std::atomic<bool> done[kMaxDevices];
    const cudaError_t e = allow_smem((const void*)scan_bwd_tc_kernel, kBwSmemBytes, done);
    if (e != cudaSuccess) return e;
    void* args[] = {&m.x, &m.g, &m.dx, const_cast<ScanBwdTcParams*>(&p)};
    return launch_after((const void*)scan_bwd_tc_kernel, dim3((p.S + Q - 1) / Q, p.G * p.split, p.B), kThreads, kBwSmemBytes,
                        st, args);
}

}  // namespace

bool make_rows_map(CUtensorMap* m, const void* base, int elem, long long cols, long long rows, int batches,
                   int box_cols, int box_rows, bool swizzle)
{
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batches};
    cuuint64_t strides[2] = {(cuuint64_t)(cols * elem), (cuuint64_t)(cols * elem) * (cuuint64_t)rows};
    cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1}, es[3] = {1, 1, 1};
    return encode_fn() &&
           g_encode(m, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
                    const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool scan_bwd_tc_supports(int P_, int N_) { return P_ == P && N_ == N; }

ScanBwdTcSizes scan_bwd_tc_sizes(int B, int S, int H, int G)
{
    auto r256 = [](size_t n) { return (n + 255) & ~(size_t)255; };
    const size_t nc = ((size_t)S + Q - 1) / Q, units = (size_t)B * H * nc;
    const int split = scan_bwd_split((long long)B * nc * G, H / G, 2.0, 152);
    ScanBwdTcSizes z;
    z.split = split;
    z.vals = r256(units * kValStride * 4);
    z.states = r256(units * 2 * N * P * 2);
    z.part = r256((size_t)B * nc * 3 * H * 4);
    z.bcpart = split > 1 ? r256((size_t)split * B * S * 2 * G * N * 4) : 0;
    return z;
}

cudaError_t launch_scan_bwd_tc(const ScanBwdTcParams& p, cudaStream_t st, ScanBwdLaunched* done)
{
    TcMaps m;
    if (!make_maps(p, &m)) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)((p.S + Q - 1) / Q), (unsigned)((p.H + kRowHeads - 1) / kRowHeads), (unsigned)p.B);
    scan_bwd_rows_kernel<<<grid, 32 * kRowHeads, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    done->rows = true;
    if ((e = launch_states(p, m, st)) != cudaSuccess) return e;
    done->states = true;
    if ((e = launch_chunks(p, m, st)) != cudaSuccess) return e;
    done->chunks = true;
    return cudaSuccess;
}

}  // namespace ssd
