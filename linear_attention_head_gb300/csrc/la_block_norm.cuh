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
// One pass: a row lives in the registers of a group of threads (8 to 32 lanes, or a
// CTA for long rows), as it was loaded, 16 bytes at a time; the row's sums are fp32
// shuffles.  Bytes bound it.  The weights' gradients are summed by each thread over
// the rows that it takes, then over a CTA's groups, then over CTAs by a last kernel:
// a fixed order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

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

// TPR threads a row (8, 16, 32, or a whole CTA of 256 or 512), NV times 8 channels
// each.
template <int TPR_, int NV_> struct Plan {
    static constexpr int TPR = TPR_, NV = NV_;
    static constexpr int CTA = TPR > 32 ? TPR : 256;
    static constexpr int GROUPS = CTA / TPR;
    static constexpr int WARPS = CTA / 32;
    static constexpr int CHANNELS = TPR * NV * 8;
};

// Sums over the row's threads, in a fixed order.  turn: alternates, so that one
// barrier a sum is enough.
template <typename PL>
__device__ __forceinline__ float2 row_sum(float2 x, float2 (*red)[PL::WARPS], int &turn)
{
#pragma unroll
    for (int m = 1; m < (PL::TPR < 32 ? PL::TPR : 32); m *= 2) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, m);
        x.y += __shfl_xor_sync(0xffffffffu, x.y, m);
    }
    if (PL::TPR > 32) {
        turn ^= 1;
        if ((threadIdx.x & 31) == 0)
            red[turn][threadIdx.x >> 5] = x;
        __syncthreads();
        x = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < PL::WARPS; ++w) {
            const float2 y = red[turn][w];
            x.x += y.x;
            x.y += y.y;
        }
    }
    return x;
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

template <typename T, typename PL, bool VEC>
__global__ void __launch_bounds__(PL::CTA) block_norm_fwd_kernel(const BlockNormArgs a)
{
    __shared__ float2 red[2][PL::WARPS];
    int turn = 0;
    const int group = threadIdx.x / PL::TPR, me = threadIdx.x % PL::TPR;
    const float inv_d = 1.f / (float)a.D;
    float post[PL::NV][8], pre[PL::NV][8];      // this thread's channels, for all its rows
#pragma unroll
    for (int v = 0; v < PL::NV; ++v) {
        const int c = (v * PL::TPR + me) * 8;
        if (a.post)
            weights8<VEC>(a.post, a.w_bf16, c, a.D - c, post[v]);
        if (a.pre)
            weights8<VEC>(a.pre, a.w_bf16, c, a.D - c, pre[v]);
    }
    for (int64_t first = (int64_t)blockIdx.x * PL::GROUPS; first < a.rows;
         first += (int64_t)gridDim.x * PL::GROUPS) {
        const bool live = first + group < a.rows;
        const RowPlace p = row_place(a, live ? (unsigned)(first + group) : 0u);
        Raw<T> x[PL::NV], g[PL::NV], r[PL::NV];
        float h[PL::NV][8];
#pragma unroll
        for (int v = 0; v < PL::NV; ++v) {
            const int c = (v * PL::TPR + me) * 8, n = live ? a.D - c : 0;
            x[v] = load8<VEC>(at<const T>(a, a.x, p) + c, n);
            if (a.gate.p)
                g[v] = load8<VEC>(at<const T>(a, a.gate, p) + c, n);
            if (a.residual.p)
                r[v] = load8<VEC>(at<const T>(a, a.residual, p) + c, n);
        }
        float rx = 1.f;
        if (a.post) {
            float2 s = make_float2(0.f, 0.f);
#pragma unroll
            for (int v = 0; v < PL::NV; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s.x = fmaf(x[v].get(i), x[v].get(i), s.x);
            rx = rsqrtf(row_sum<PL>(s, red, turn).x * inv_d + a.eps);
        }
        float2 sh = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < PL::NV; ++v) {
            const int c = (v * PL::TPR + me) * 8, n = live ? a.D - c : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float m = x[v].get(i);
                if (a.post)
                    m *= rx * post[v][i];
                if (a.gate.p)
                    m *= act<T>(g[v].get(i), a.activation);
                m *= a.scale;
                if (a.residual.p)
                    m += r[v].get(i);
                if (!VEC && i >= n)
                    m = 0.f;
                h[v][i] = m;
                sh.x = fmaf(m, m, sh.x);
            }
            store8<VEC>(at<T>(a, a.h, p) + c, h[v], n);
        }
        if (!a.pre)
            continue;
        const float rh = rsqrtf(row_sum<PL>(sh, red, turn).x * inv_d + a.eps);
#pragma unroll
        for (int v = 0; v < PL::NV; ++v) {
            const int c = (v * PL::TPR + me) * 8, n = live ? a.D - c : 0;
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = h[v][i] * rh * pre[v][i];
            store8<VEC>(at<T>(a, a.y, p) + c, y, n);
        }
    }
}

template <typename T, typename PL, bool VEC>
__global__ void __launch_bounds__(PL::CTA) block_norm_bwd_kernel(const BlockNormArgs a)
{
    __shared__ float2 red[2][PL::WARPS];
    int turn = 0;
    const int group = threadIdx.x / PL::TPR, me = threadIdx.x % PL::TPR;
    const float inv_d = 1.f / (float)a.D;
    float wpost[PL::NV][8] = {}, wpre[PL::NV][8] = {};
    for (int64_t first = (int64_t)blockIdx.x * PL::GROUPS; first < a.rows;
         first += (int64_t)gridDim.x * PL::GROUPS) {
        const bool live = first + group < a.rows;
        const RowPlace p = row_place(a, live ? (unsigned)(first + group) : 0u);
        Raw<T> x[PL::NV], g[PL::NV], r[PL::NV], dh[PL::NV], dy[PL::NV];
#pragma unroll
        for (int v = 0; v < PL::NV; ++v) {
            const int c = (v * PL::TPR + me) * 8, n = live ? a.D - c : 0;
            x[v] = load8<VEC>(at<const T>(a, a.x, p) + c, n);
            if (a.gate.p)
                g[v] = load8<VEC>(at<const T>(a, a.gate, p) + c, n);
            if (a.residual.p && a.pre)
                r[v] = load8<VEC>(at<const T>(a, a.residual, p) + c, n);
            dh[v] = load8<VEC>(at<const T>(a, a.dh, p) + c, a.dh.p ? n : 0);
            if (a.pre)
                dy[v] = load8<VEC>(at<const T>(a, a.dy, p) + c, n);
        }
        float rx = 1.f;
        if (a.post) {
            float2 s = make_float2(0.f, 0.f);
#pragma unroll
            for (int v = 0; v < PL::NV; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s.x = fmaf(x[v].get(i), x[v].get(i), s.x);
            rx = rsqrtf(row_sum<PL>(s, red, turn).x * inv_d + a.eps);
        }
        // h again, and its two sums
        float h[PL::NV][8], rh = 0.f, mean = 0.f;
        if (a.pre) {
            float2 s = make_float2(0.f, 0.f);
#pragma unroll
            for (int v = 0; v < PL::NV; ++v) {
                const int c = (v * PL::TPR + me) * 8, n = live ? a.D - c : 0;
                float w[8], u[8];
                if (a.post)
                    weights8<VEC>(a.post, a.w_bf16, c, n, w);
                weights8<VEC>(a.pre, a.w_bf16, c, n, u);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float m = x[v].get(i);
                    if (a.post)
                        m *= rx * w[i];
                    if (a.gate.p)
                        m *= act<T>(g[v].get(i), a.activation);
                    m *= a.scale;
                    if (a.residual.p)
                        m += r[v].get(i);
                    if (!VEC && i >= n)
                        m = 0.f;
                    h[v][i] = m;
                    s.x = fmaf(m, m, s.x);
                    s.y = fmaf(m, dy[v].get(i) * u[i], s.y);
                }
            }
            s = row_sum<PL>(s, red, turn);
            rh = rsqrtf(s.x * inv_d + a.eps);
            mean = s.y * inv_d * rh * rh;
        }
        // h turns into dn: the gradient before the gate and the scale
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < PL::NV; ++v) {
            const int c = (v * PL::TPR + me) * 8, n = live ? a.D - c : 0;
            float w[8], u[8], out[8];
            if (a.post)
                weights8<VEC>(a.post, a.w_bf16, c, n, w);
            if (a.pre)
                weights8<VEC>(a.pre, a.w_bf16, c, n, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float d = dh[v].get(i);
                if (a.pre) {
                    const float y = dy[v].get(i);
                    d += rh * (y * u[i] - h[v][i] * mean);
                    wpre[v][i] = fmaf(y, h[v][i] * rh, wpre[v][i]);
                }
                out[i] = d;
            }
            if (a.dresidual.p)
                store8<VEC>(at<T>(a, a.dresidual, p) + c, out, n);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float d = out[i] * a.scale;
                const float xi = x[v].get(i);
                if (a.gate.p) {
                    float slope;
                    const float f = act<T>(g[v].get(i), a.activation, slope);
                    out[i] = d * slope * (a.post ? xi * rx * w[i] : xi);
                    d *= f;
                }
                if (a.post) {
                    wpost[v][i] = fmaf(d, xi * rx, wpost[v][i]);
                    d *= w[i];
                    s.x = fmaf(d, xi, s.x);
                }
                h[v][i] = d;
            }
            if (a.gate.p)
                store8<VEC>(at<T>(a, a.dgate, p) + c, out, n);
        }
        const float mx = a.post ? row_sum<PL>(s, red, turn).x * inv_d * rx * rx : 0.f;
#pragma unroll
        for (int v = 0; v < PL::NV; ++v) {
            const int c = (v * PL::TPR + me) * 8, n = live ? a.D - c : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (a.post)
                    h[v][i] = rx * (h[v][i] - x[v].get(i) * mx);
            store8<VEC>(at<T>(a, a.dx, p) + c, h[v], n);
        }
    }
    // this CTA's part of the weights' gradients, [2][D]
    __shared__ float sums[PL::GROUPS > 1 ? PL::GROUPS : 1][PL::GROUPS > 1 ? PL::TPR * 8 + 8 : 1];
    for (int which = 0; which < 2; ++which) {
        if (!(which ? a.dpre : a.dpost))
            continue;
        float *to = a.partial + ((int64_t)blockIdx.x * 2 + which) * a.D;
#pragma unroll
        for (int v = 0; v < PL::NV; ++v) {
            const int c0 = v * PL::TPR * 8;
            if (PL::GROUPS == 1) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c0 + me * 8 + i < a.D)
                        to[c0 + me * 8 + i] = which ? wpre[v][i] : wpost[v][i];
                continue;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sums[group][me * 8 + i] = which ? wpre[v][i] : wpost[v][i];
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

// Rows a CTA takes at once, and the CTAs that one wave holds; a CTA more than there
// are rows for is not launched.
template <typename PL, typename K>
cudaError_t norm_launch(K kernel, const BlockNormArgs &a, int sms, cudaStream_t s, int *ctas)
{
    int per_sm = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, PL::CTA, 0);
    if (e != cudaSuccess)
        return e;
    const int64_t want = (a.rows + PL::GROUPS - 1) / PL::GROUPS;
    const int64_t wave = (int64_t)sms * (per_sm > 0 ? per_sm : 1);
    int64_t n = want < wave ? want : wave;
    if (n > NORM_MOST_CTAS && (a.dpost || a.dpre))
        n = NORM_MOST_CTAS;
    *ctas = (int)n;
    kernel<<<(unsigned)n, PL::CTA, 0, s>>>(a);
    note_launch();
    return cudaGetLastError();
}

template <bool BWD, typename T, typename PL>
cudaError_t norm_by_access(const BlockNormArgs &a, bool vec, int sms, cudaStream_t s, int *ctas)
{
    if constexpr (BWD)
        return vec ? norm_launch<PL>(block_norm_bwd_kernel<T, PL, true>, a, sms, s, ctas)
                   : norm_launch<PL>(block_norm_bwd_kernel<T, PL, false>, a, sms, s, ctas);
    else
        return vec ? norm_launch<PL>(block_norm_fwd_kernel<T, PL, true>, a, sms, s, ctas)
                   : norm_launch<PL>(block_norm_fwd_kernel<T, PL, false>, a, sms, s, ctas);
}

// The fewest threads that hold a row at 8 to 32 channels each: several rows a warp
// where rows are short, a CTA a row where a warp would hold more than 32 channels a
// lane (spills in the backward, and too few bytes in flight with few rows).
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
    if (chunks <= 64)
        return norm_by_access<BWD, T, Plan<32, 2>>(a, vec, sms, s, ctas);
    if (chunks <= 256)
        return norm_by_access<BWD, T, Plan<256, 1>>(a, vec, sms, s, ctas);
    if (chunks <= 512)
        return norm_by_access<BWD, T, Plan<256, 2>>(a, vec, sms, s, ctas);
    if (chunks <= 1024)
        return norm_by_access<BWD, T, Plan<512, 2>>(a, vec, sms, s, ctas);
    return norm_by_access<BWD, T, Plan<512, 4>>(a, vec, sms, s, ctas);
}

}  // namespace
}  // namespace la
