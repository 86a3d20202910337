// la_block_norm.cuh -- the norms before and after a block with its gate and
// residual scale, per row of D channels:
//
//     n = x rsqrt(mean x^2 + eps) w_post      (n = x without w_post)
//     m = n act(gate)                         (m = n without gate)
//     h = residual + scale m
//     y = h rsqrt(mean h^2 + eps) w_pre       (no y without w_pre)
//
// and its backward, from dh and dy, with h computed again in fp32:
//
//     u = dy w_pre,  dH = dh + r_h (u - h r_h^2 mean(u h)),  dw_pre = sum dy h r_h
//     dresidual = dH,  dm = scale dH,  dgate = dm n act'(gate),  dn = dm act(gate)
//     dw_post = sum dn x r_x,  dx = r_x (dn w_post - x r_x^2 mean(dn w_post x))
//
// One pass: a row lives in the registers of a group of threads, 8 channels each (8 to
// 32 lanes, or a CTA for long rows); the row's sums are fp32 shuffles.  While a row is
// worked on the group's next two are on their way: aligned rows by asynchronous copies
// into places of shared memory that the thread that asks for them reads alone, so that
// no barrier stands between (gated heads, b4 n8192 32 x 128, forward and backward: 0.40 ms
// on one GB300, 0.45 with the next row in registers).  There the forward takes 139 us, 0.87
// of the copy rate, and the backward 255, 0.79; rows of 4096 with all parts, 16380 of them:
// 107 and 255, the backward bound by its sums over a CTA.  Above 4096 channels a thread
// holds 16 or 32 of a row and no longer keeps them all in registers (spill stores a
// thread, bf16 and fp32: backward to 8192 channels 488 and 984 bytes, to 16384 3240 and
// 3968; forward fp32 to 16384 2420).  All parts, 2^26 numbers a tensor, of the copy rate:
//     channels          1024  2048  4096  5120  7168  8192  12288  16384
//     bf16 forward      0.87  0.91  0.90  0.60  0.80  0.89  0.70   0.81
//     bf16 backward     0.67  0.64  0.61  0.33  0.45  0.50  0.13   0.16
//     fp32 forward      0.65  0.69  0.69  0.51  0.56  0.57  0.32   0.37
//     fp32 backward     0.57  0.41  0.52  0.26  0.33  0.36  0.15   0.19
// The weights' gradients are summed by each thread over
// the rows that it takes, then over a CTA's groups, then over CTAs by a last kernel:
// a fixed order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "la_f32x2.cuh"
#include "la_internal.h"

namespace la {
namespace {

// Eight channels as loaded.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
        return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
    }
};
template <> struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ float get(int i) const
    {
        const float4 &f = i < 4 ? a : b;
        return (i & 3) == 0 ? f.x : (i & 3) == 1 ? f.y : (i & 3) == 2 ? f.z : f.w;
    }
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// n: channels left of the row (8 or more: all eight).
template <bool VEC> __device__ __forceinline__ Raw<__nv_bfloat16> load8(const __nv_bfloat16 *p, int n)
{
    Raw<__nv_bfloat16> r{make_uint4(0, 0, 0, 0)};
    if (VEC) {
        if (n > 0)
            r.v = *reinterpret_cast<const uint4 *>(p);
    } else {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = i < n ? *reinterpret_cast<const uint16_t *>(p + i) : 0u;
        r.v = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16,
                         w[6] | w[7] << 16);
    }
    return r;
}
template <bool VEC> __device__ __forceinline__ Raw<float> load8(const float *p, int n)
{
    Raw<float> r{make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    if (VEC) {
        if (n > 0) {
            r.a = *reinterpret_cast<const float4 *>(p);
            r.b = *reinterpret_cast<const float4 *>(p + 4);
        }
    } else {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = i < n ? p[i] : 0.f;
        r.a = make_float4(w[0], w[1], w[2], w[3]);
        r.b = make_float4(w[4], w[5], w[6], w[7]);
    }
    return r;
}
template <bool VEC> __device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8], int n)
{
    if (VEC) {
        if (n > 0)
            *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]),
                                                       pack2(x[4], x[5]), pack2(x[6], x[7]));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                p[i] = __float2bfloat16_rn(x[i]);
    }
}
template <bool VEC> __device__ __forceinline__ void store8(float *p, const float (&x)[8], int n)
{
    if (VEC) {
        if (n > 0) {
            *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                p[i] = x[i];
    }
}
template <bool VEC>
__device__ __forceinline__ void weights8(const void *w, int bf16, int c, int n, float (&x)[8])
{
    if (bf16) {
        const Raw<__nv_bfloat16> r = load8<VEC>(static_cast<const __nv_bfloat16 *>(w) + c, n);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = r.get(i);
    } else {
        const Raw<float> r = load8<VEC>(static_cast<const float *>(w) + c, n);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = r.get(i);
    }
}

// act(z) and its slope.  bf16: by the approximate power of two and reciprocal (2^-21
// together, far below the rounding of the result; an infinite power gives 0).
template <typename T> __device__ __forceinline__ float sigmoid(float z)
{
    if (sizeof(T) == 2) {
        float e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
        return r;
    }
    return 1.f / (1.f + expf(-z));
}
template <typename T> __device__ __forceinline__ float act(float z, int kind)
{
    return kind == 0 ? z : kind == 1 ? sigmoid<T>(z) : z * sigmoid<T>(z);
}
template <typename T> __device__ __forceinline__ float act(float z, int kind, float &slope)
{
    slope = 1.f;
    if (kind == 0)
        return z;
    const float s = sigmoid<T>(z);
    if (kind == 1) {
        slope = s * (1.f - s);
        return s;
    }
    slope = s * (1.f + z * (1.f - s));
    return z * s;
}

// TPR threads a row (8, 16, 32, or a whole CTA of 128 to 512), NV times 8 channels
// each.
template <int TPR_, int NV_> struct Plan {
    static constexpr int TPR = TPR_, NV = NV_;
    static constexpr int CTA = TPR > 32 ? TPR : 256;
    static constexpr int GROUPS = CTA / TPR;
    static constexpr int WARPS = CTA / 32;
    // CTAs an SM at 128 registers a thread, and at 64 (the forward's are enough there)
    static constexpr int BLOCKS = 512 / CTA, FWD_BLOCKS = NV == 1 ? 1024 / CTA : 512 / CTA;
};

// Sums over the row's threads, in a fixed order.  turn: alternates, so that one
// barrier a sum is enough.
// TWO: x.y is wanted too.
template <typename PL, bool TWO = false>
__device__ __forceinline__ float2 row_sum(float2 x, float2 (*red)[PL::WARPS], int &turn)
{
#pragma unroll
    for (int m = 1; m < (PL::TPR < 32 ? PL::TPR : 32); m *= 2) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, m);
        if (TWO)
            x.y += __shfl_xor_sync(0xffffffffu, x.y, m);
    }
    if (PL::TPR > 32) {
        turn ^= 1;
        if ((threadIdx.x & 31) == 0)
            red[turn][threadIdx.x >> 5] = x;
        __syncthreads();
        // a warp's sum a lane (again and again where there are fewer), traded likewise
        x = red[turn][threadIdx.x & (PL::WARPS - 1)];
#pragma unroll
        for (int m = 1; m < PL::WARPS; m *= 2) {
            x.x += __shfl_xor_sync(0xffffffffu, x.x, m);
            if (TWO)
                x.y += __shfl_xor_sync(0xffffffffu, x.y, m);
        }
    }
    return x;
}

// The rows on their way: K tensors, NV times 8 channels a thread, AHEAD rows beside
// the one worked on: two, or one where two would take more than 128 KB, or (AHEAD 0,
// as for rows that are not aligned) the next one in registers.
template <typename T, typename PL, bool VEC, int K> struct Ring {
    static constexpr int UNITS = sizeof(Raw<T>) / 16;   // of 16 bytes
    static constexpr int ROW = K * PL::NV * UNITS * PL::CTA * 16;
    static constexpr int AHEAD = !VEC || 2 * ROW > 224 * 1024 ? 0 : 3 * ROW > 128 * 1024 ? 1 : 2;
    static constexpr size_t BYTES = AHEAD ? (size_t)(AHEAD + 1) * ROW : 0;
    // unit u of tensor k, part v in slot s: a thread's units lie CTA apart, so that
    // neighbours' are neighbours
    static __device__ __forceinline__ uint4 *place(uint4 *ring, int s, int k, int v, int u)
    {
        return ring + (((s * K + k) * PL::NV + v) * UNITS + u) * PL::CTA + threadIdx.x;
    }
    // n: channels left of the row; none: zeros
    static __device__ __forceinline__ void ask(uint4 *ring, int s, int k, int v, const T *p, int n)
    {
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const uint32_t to = (uint32_t)__cvta_generic_to_shared(place(ring, s, k, v, u));
            const int bytes = n > 0 ? 16 : 0;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                         "l"(reinterpret_cast<const char *>(p) + 16 * u), "r"(bytes)
                         : "memory");
        }
    }
    static __device__ __forceinline__ Raw<T> get(uint4 *ring, int s, int k, int v)
    {
        Raw<T> r;
        uint4 *w = reinterpret_cast<uint4 *>(&r);
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
            w[u] = *place(ring, s, k, v, u);
        return r;
    }
};
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until all but the youngest `younger` rows asked for are there
template <int younger> __device__ __forceinline__ void ring_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(younger) : "memory");
}

struct RowPlace {
    unsigned b, t, h, row;
};
// Where every tensor's rows lie a constant step apart (a.flat) nothing is divided.
__device__ __forceinline__ RowPlace row_place(const BlockNormArgs &a, unsigned row)
{
    if (a.flat)
        return {0u, 0u, 0u, row};
    const unsigned bt = row / (unsigned)a.H, b = bt / (unsigned)a.T;
    return {b, bt - b * (unsigned)a.T, row - bt * (unsigned)a.H, 0u};
}
template <typename T>
__device__ __forceinline__ T *at(const BlockNormArgs &a, const NormRows &x, const RowPlace &p)
{
    T *q = static_cast<T *>(const_cast<void *>(x.p));
    return a.flat ? q + p.row * x.step : q + p.b * x.s[0] + p.t * x.s[1] + p.h * x.s[2];
}

// Pair m of eight channels as loaded.
__device__ __forceinline__ F2 pair_of(const Raw<__nv_bfloat16> &r, int m)
{
    const uint32_t w = m == 0 ? r.v.x : m == 1 ? r.v.y : m == 2 ? r.v.z : r.v.w;
    return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ F2 pair_of(const Raw<float> &r, int m)
{
    const float4 &f = m < 2 ? r.a : r.b;
    return m & 1 ? f2(f.z, f.w) : f2(f.x, f.y);
}
template <bool VEC, typename T> __device__ __forceinline__ void store_pairs(T *p, const F2 (&x)[4], int n)
{
    float y[8];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const float2 u = un(x[m]);
        y[2 * m] = u.x;
        y[2 * m + 1] = u.y;
    }
    store8<VEC>(p, y, n);
}
__device__ __forceinline__ float sum_of(F2 x)
{
    const float2 u = un(x);
    return u.x + u.y;
}
template <typename T> __device__ __forceinline__ F2 act2(F2 z, int kind)
{
    const float2 u = un(z);
    return f2(act<T>(u.x, kind), act<T>(u.y, kind));
}

template <typename T, typename PL, bool VEC>
__global__ void __launch_bounds__(PL::CTA, PL::FWD_BLOCKS) block_norm_fwd_kernel(const BlockNormArgs a)
{
    constexpr int NV = PL::NV;
    __shared__ float2 red[2][PL::WARPS];
    int turn = 0;
    const int group = threadIdx.x / PL::TPR, me = threadIdx.x % PL::TPR;
    const float inv_d = 1.f / (float)a.D;
    const bool post = a.post, pre = a.pre, gated = a.gate.p, stream = a.residual.p;
    F2 wpost[NV][4], wpre[NV][4];       // this thread's channels, for all its rows
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * PL::TPR + me) * 8;
        float w[8];
        weights8<VEC>(post ? a.post : a.x.p, post ? a.w_bf16 : a.bf16, c, post ? a.D - c : 0, w);
#pragma unroll
        for (int m = 0; m < 4; ++m)     // the scale once and for all
            wpost[v][m] = mul2(f2(a.scale), post ? f2(w[2 * m], w[2 * m + 1]) : f2(1.f));
        weights8<VEC>(pre ? a.pre : a.x.p, pre ? a.w_bf16 : a.bf16, c, pre ? a.D - c : 0, w);
#pragma unroll
        for (int m = 0; m < 4; ++m)
            wpre[v][m] = f2(w[2 * m], w[2 * m + 1]);
    }
    Raw<T> x[NV], g[NV], r[NV];
    const int64_t step = (int64_t)gridDim.x * PL::GROUPS;
    int64_t row = (int64_t)blockIdx.x * PL::GROUPS + group;
    using R = Ring<T, PL, VEC, 3>;
    constexpr int AHEAD = R::AHEAD;
    extern __shared__ uint4 ring[];
    int slot = 0, ahead = AHEAD;        // slots of the row worked on, and of the one asked for
    auto load = [&](int64_t at_row, int s) {
        const bool live = at_row < a.rows;
        const RowPlace p = row_place(a, live ? (unsigned)at_row : 0u);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * PL::TPR + me) * 8, n = live ? a.D - c : 0;
            // past the row's end an address that is there
            const int cc = n > 0 ? c : 0;
            if constexpr (AHEAD > 0) {
                R::ask(ring, s, 0, v, at<const T>(a, a.x, p) + cc, n);
                if (gated)
                    R::ask(ring, s, 1, v, at<const T>(a, a.gate, p) + cc, n);
                if (stream)
                    R::ask(ring, s, 2, v, at<const T>(a, a.residual, p) + cc, n);
            } else {
                x[v] = load8<VEC>(at<const T>(a, a.x, p) + c, n);
                if (gated)
                    g[v] = load8<VEC>(at<const T>(a, a.gate, p) + c, n);
                if (stream)
                    r[v] = load8<VEC>(at<const T>(a, a.residual, p) + c, n);
            }
        }
        if constexpr (AHEAD > 0)
            ring_commit();
    };
    load(row, 0);
    if constexpr (AHEAD > 1)
        load(row + step, 1);
    for (int64_t first = (int64_t)blockIdx.x * PL::GROUPS; first < a.rows; first += step) {
        const bool live = row < a.rows;
        const RowPlace p = row_place(a, live ? (unsigned)row : 0u);
        F2 h[NV][4];
        F2 sx = f2(0.f), sh = f2(0.f);
        if constexpr (AHEAD > 0) {
            ring_wait<AHEAD - 1>();
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                x[v] = R::get(ring, slot, 0, v);
                g[v] = R::get(ring, slot, 1, v);
                r[v] = R::get(ring, slot, 2, v);
            }
            load(row + AHEAD * step, ahead);
            slot = slot == AHEAD ? 0 : slot + 1;
            ahead = ahead == AHEAD ? 0 : ahead + 1;
        }
        // n times the scale and the gate, but for the row's factor; what was loaded is
        // free for the next row's loads then
        F2 res[NV][4];
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const F2 u = pair_of(x[v], m);
                sx = fma2(u, u, sx);
                h[v][m] = mul2(u, wpost[v][m]);
                if (gated)
                    h[v][m] = mul2(h[v][m], act2<T>(pair_of(g[v], m), a.activation));
                res[v][m] = stream ? pair_of(r[v], m) : f2(0.f);
            }
        row += step;
        if (AHEAD == 0 && first + step < a.rows)
            load(row, 0);
        float rx = 1.f;
        if (post)
            rx = rsqrtf(row_sum<PL>(make_float2(sum_of(sx), 0.f), red, turn).x * inv_d + a.eps);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * PL::TPR + me) * 8, n = live ? a.D - c : 0;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                h[v][m] = fma2(h[v][m], f2(rx), res[v][m]);
                sh = fma2(h[v][m], h[v][m], sh);
            }
            store_pairs<VEC>(at<T>(a, a.h, p) + c, h[v], n);
        }
        if (!pre)
            continue;
        const float rh = rsqrtf(row_sum<PL>(make_float2(sum_of(sh), 0.f), red, turn).x * inv_d +
                                a.eps);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * PL::TPR + me) * 8, n = live ? a.D - c : 0;
#pragma unroll
            for (int m = 0; m < 4; ++m)
                h[v][m] = mul2(mul2(h[v][m], f2(rh)), wpre[v][m]);
            store_pairs<VEC>(at<T>(a, a.y, p) + c, h[v], n);
        }
    }
}

template <typename T, typename PL, bool VEC>
__global__ void __launch_bounds__(PL::CTA, PL::BLOCKS) block_norm_bwd_kernel(const BlockNormArgs a)
{
    constexpr int NV = PL::NV;
    __shared__ float2 red[2][PL::WARPS];
    int turn = 0;
    const int group = threadIdx.x / PL::TPR, me = threadIdx.x % PL::TPR;
    const float inv_d = 1.f / (float)a.D;
    const bool post = a.post, pre = a.pre, gated = a.gate.p, stream = a.residual.p && pre;
    F2 wpost[NV][4], wpre[NV][4], dpost[NV][4], dpre[NV][4];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * PL::TPR + me) * 8;
        float w[8];
        weights8<VEC>(post ? a.post : a.x.p, post ? a.w_bf16 : a.bf16, c, post ? a.D - c : 0, w);
#pragma unroll
        for (int m = 0; m < 4; ++m)
            wpost[v][m] = post ? f2(w[2 * m], w[2 * m + 1]) : f2(1.f);
        weights8<VEC>(pre ? a.pre : a.x.p, pre ? a.w_bf16 : a.bf16, c, pre ? a.D - c : 0, w);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            wpre[v][m] = f2(w[2 * m], w[2 * m + 1]);
            dpost[v][m] = dpre[v][m] = f2(0.f);
        }
    }
    Raw<T> x[NV], g[NV], r[NV], dh[NV], dy[NV];
    const int64_t step = (int64_t)gridDim.x * PL::GROUPS;
    int64_t row = (int64_t)blockIdx.x * PL::GROUPS + group;
    using R = Ring<T, PL, VEC, 5>;
    constexpr int AHEAD = R::AHEAD;
    extern __shared__ uint4 ring[];
    int slot = 0, ahead = AHEAD;
    auto load = [&](int64_t at_row, int s) {
        const bool live = at_row < a.rows;
        const RowPlace p = row_place(a, live ? (unsigned)at_row : 0u);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * PL::TPR + me) * 8, n = live ? a.D - c : 0;
            const int cc = n > 0 ? c : 0;
            if constexpr (AHEAD > 0) {
                R::ask(ring, s, 0, v, at<const T>(a, a.x, p) + cc, n);
                if (gated)
                    R::ask(ring, s, 1, v, at<const T>(a, a.gate, p) + cc, n);
                if (stream)
                    R::ask(ring, s, 2, v, at<const T>(a, a.residual, p) + cc, n);
                if (a.dh.p)
                    R::ask(ring, s, 3, v, at<const T>(a, a.dh, p) + cc, n);
                if (pre)
                    R::ask(ring, s, 4, v, at<const T>(a, a.dy, p) + cc, n);
            } else {
                x[v] = load8<VEC>(at<const T>(a, a.x, p) + c, n);
                if (gated)
                    g[v] = load8<VEC>(at<const T>(a, a.gate, p) + c, n);
                if (stream)
                    r[v] = load8<VEC>(at<const T>(a, a.residual, p) + c, n);
                dh[v] = load8<VEC>(at<const T>(a, a.dh, p) + c, a.dh.p ? n : 0);
                if (pre)
                    dy[v] = load8<VEC>(at<const T>(a, a.dy, p) + c, n);
            }
        }
        if constexpr (AHEAD > 0)
            ring_commit();
    };
    load(row, 0);
    if constexpr (AHEAD > 1)
        load(row + step, 1);
    for (int64_t first = (int64_t)blockIdx.x * PL::GROUPS; first < a.rows; first += step) {
        const bool live = row < a.rows;
        const RowPlace p = row_place(a, live ? (unsigned)row : 0u);
        // x and the gate as loaded, the gate's factor made where it is wanted (twice with
        // pre): registers are what the next row's loads need
        Raw<T> xc[NV], gc[NV];
        F2 d[NV][4];
        float rx = 1.f;
        if constexpr (AHEAD > 0) {
            ring_wait<AHEAD - 1>();
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                x[v] = R::get(ring, slot, 0, v);
                g[v] = R::get(ring, slot, 1, v);
                r[v] = R::get(ring, slot, 2, v);
                dh[v] = a.dh.p ? R::get(ring, slot, 3, v) : Raw<T>{};
                dy[v] = R::get(ring, slot, 4, v);
            }
            load(row + AHEAD * step, ahead);
            slot = slot == AHEAD ? 0 : slot + 1;
            ahead = ahead == AHEAD ? 0 : ahead + 1;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            xc[v] = x[v];
            gc[v] = g[v];
#pragma unroll
            for (int m = 0; m < 4; ++m)
                d[v][m] = pair_of(dh[v], m);
        }
        if (post) {
            F2 sx = f2(0.f);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const F2 t = pair_of(xc[v], m);
                    sx = fma2(t, t, sx);
                }
            rx = rsqrtf(row_sum<PL>(make_float2(sum_of(sx), 0.f), red, turn).x * inv_d + a.eps);
            // a group without a row: 0 times what eps 0 makes infinite is no 0
            rx = PL::GROUPS > 1 && !live ? 0.f : rx;
        }
        if (pre) {      // h again, and its two sums
            F2 h[NV][4], sh = f2(0.f), su = f2(0.f);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    h[v][m] = mul2(mul2(pair_of(xc[v], m), f2(rx * a.scale)), wpost[v][m]);
                    if (gated)
                        h[v][m] = mul2(h[v][m], act2<T>(pair_of(gc[v], m), a.activation));
                    if (stream)
                        h[v][m] = add2(h[v][m], pair_of(r[v], m));
                    sh = fma2(h[v][m], h[v][m], sh);
                    su = fma2(h[v][m], mul2(pair_of(dy[v], m), wpre[v][m]), su);
                }
            const float2 s = row_sum<PL, true>(make_float2(sum_of(sh), sum_of(su)), red, turn);
            const float rh = PL::GROUPS > 1 && !live ? 0.f : rsqrtf(s.x * inv_d + a.eps);
            const float mean = -s.y * inv_d * rh * rh;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const F2 y = pair_of(dy[v], m);
                    const F2 t = fma2(h[v][m], f2(mean), mul2(y, wpre[v][m]));
                    d[v][m] = fma2(t, f2(rh), d[v][m]);
                    dpre[v][m] = fma2(y, mul2(h[v][m], f2(rh)), dpre[v][m]);
                }
        }
        row += step;
        if (AHEAD == 0 && first + step < a.rows)
            load(row, 0);
        F2 sd = f2(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * PL::TPR + me) * 8, n = live ? a.D - c : 0;
            if (a.dresidual.p)
                store_pairs<VEC>(at<T>(a, a.dresidual, p) + c, d[v], n);
            F2 dg[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const F2 u = mul2(pair_of(xc[v], m), f2(rx));
                d[v][m] = mul2(d[v][m], f2(a.scale));
                if (gated) {
                    const float2 z = un(pair_of(gc[v], m));
                    float s0, s1;
                    const float f0 = act<T>(z.x, a.activation, s0);
                    const float f1 = act<T>(z.y, a.activation, s1);
                    dg[m] = mul2(mul2(d[v][m], f2(s0, s1)), mul2(u, wpost[v][m]));
                    d[v][m] = mul2(d[v][m], f2(f0, f1));
                }
                if (post) {
                    dpost[v][m] = fma2(d[v][m], u, dpost[v][m]);
                    d[v][m] = mul2(d[v][m], wpost[v][m]);
                    sd = fma2(d[v][m], u, sd);
                }
            }
            if (gated)
                store_pairs<VEC>(at<T>(a, a.dgate, p) + c, dg, n);
        }
        if (post) {
            const float mean = -row_sum<PL>(make_float2(sum_of(sd), 0.f), red, turn).x * inv_d * rx;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    d[v][m] = mul2(fma2(pair_of(xc[v], m), f2(mean), d[v][m]), f2(rx));
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * PL::TPR + me) * 8, n = live ? a.D - c : 0;
            store_pairs<VEC>(at<T>(a, a.dx, p) + c, d[v], n);
        }
    }
    // this CTA's part of the weights' gradients, [2][D]
    __shared__ float sums[PL::GROUPS > 1 ? PL::GROUPS : 1][PL::GROUPS > 1 ? PL::TPR * 8 + 8 : 1];
    for (int which = 0; which < 2; ++which) {
        if (!(which ? a.dpre : a.dpost))
            continue;
        float *to = a.partial + ((int64_t)blockIdx.x * 2 + which) * a.D;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = v * PL::TPR * 8;
            float w[8];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float2 t = un(which ? dpre[v][m] : dpost[v][m]);
                w[2 * m] = t.x;
                w[2 * m + 1] = t.y;
            }
            if (PL::GROUPS == 1) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c0 + me * 8 + i < a.D)
                        to[c0 + me * 8 + i] = w[i];
                continue;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sums[group][me * 8 + i] = w[i];
            __syncthreads();
            for (int c = threadIdx.x; c < PL::TPR * 8; c += PL::CTA) {
                float t = 0.f;
                for (int k = 0; k < PL::GROUPS; ++k)
                    t += sums[k][c];
                if (c0 + c < a.D)
                    to[c0 + c] = t;
            }
        }
    }
}

// One wave of CTAs (as many an SM as the launch bounds and shared memory let be; asking
// the runtime costs 5 us of a call), no more than there are rows for.
template <typename PL, int BLOCKS, typename K>
cudaError_t norm_launch(K kernel, size_t ring, const BlockNormArgs &a, int sms, cudaStream_t s,
                        int *ctas)
{
    if (ring > 32 * 1024) {     // with what the kernels have of their own above 48 KB
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ring);
        if (e != cudaSuccess)
            return e;
    }
    const int fit = (int)(228 * 1024 / (ring + 12 * 1024));
    const int per_sm = fit < 1 ? 1 : fit < BLOCKS ? fit : BLOCKS;
    const int64_t want = (a.rows + PL::GROUPS - 1) / PL::GROUPS;
    int64_t n = (int64_t)sms * per_sm;
    n = want < n ? want : n;
    if (n > NORM_MOST_CTAS && (a.dpost || a.dpre))
        n = NORM_MOST_CTAS;
    *ctas = (int)n;
    kernel<<<(unsigned)n, PL::CTA, ring, s>>>(a);
    note_launch();
    return cudaGetLastError();
}

template <bool BWD, typename T, typename PL>
cudaError_t norm_by_access(const BlockNormArgs &a, bool vec, int sms, cudaStream_t s, int *ctas)
{
    if constexpr (BWD)
        return vec ? norm_launch<PL, PL::BLOCKS>(block_norm_bwd_kernel<T, PL, true>,
                                                 Ring<T, PL, true, 5>::BYTES, a, sms, s, ctas)
                   : norm_launch<PL, PL::BLOCKS>(block_norm_bwd_kernel<T, PL, false>, 0, a, sms, s,
                                                 ctas);
    else
        return vec ? norm_launch<PL, PL::FWD_BLOCKS>(block_norm_fwd_kernel<T, PL, true>,
                                                     Ring<T, PL, true, 3>::BYTES, a, sms, s, ctas)
                   : norm_launch<PL, PL::FWD_BLOCKS>(block_norm_fwd_kernel<T, PL, false>, 0, a, sms,
                                                     s, ctas);
}

// Eight channels a thread: several rows a warp where rows are short, a CTA a row where
// they are longer than a warp's 256 channels.  (More channels a thread above 4096.)
template <bool BWD, typename T>
cudaError_t norm_by_width(const BlockNormArgs &a, bool vec, int sms, cudaStream_t s, int *ctas)
{
    const int chunks = (a.D + 7) / 8;
    if (chunks <= 8)
        return norm_by_access<BWD, T, Plan<8, 1>>(a, vec, sms, s, ctas);
    if (chunks <= 16)
        return norm_by_access<BWD, T, Plan<16, 1>>(a, vec, sms, s, ctas);
    if (chunks <= 32)
        return norm_by_access<BWD, T, Plan<32, 1>>(a, vec, sms, s, ctas);
    if (chunks <= 128)
        return norm_by_access<BWD, T, Plan<128, 1>>(a, vec, sms, s, ctas);
    if (chunks <= 256)
        return norm_by_access<BWD, T, Plan<256, 1>>(a, vec, sms, s, ctas);
    if (chunks <= 512)
        return norm_by_access<BWD, T, Plan<512, 1>>(a, vec, sms, s, ctas);
    if (chunks <= 1024)
        return norm_by_access<BWD, T, Plan<512, 2>>(a, vec, sms, s, ctas);
    return norm_by_access<BWD, T, Plan<512, 4>>(a, vec, sms, s, ctas);
}

}  // namespace
}  // namespace la
