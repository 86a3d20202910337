// la_qk_rope.cu -- norms of queries and keys for each head with the position
// rotation in the same pass, and their backward.
//
//   y = R(n(x)), n(x) = x r w, r = rsqrt(mean x^2 + eps)
//   u = R^T(dy);  dx = r (z - x r^2 mean(z x)), z = u w;  dw = sum u x r
//
// Angles: inv_freq / 2 pi is kept as a 64-bit fixed-point fraction of a turn
// F, so position * F mod 2^64 is the angle's fraction of a turn, wrapped
// exactly, at every position; sin and cos of that fraction are taken in fp32.
// An fp32 product position * inv_freq would be off by 0.06 radians at
// position 10^6.
//
// One warp per row; the rotation's partner channel through shared memory.

#include <cstdint>

#include <cuda_bf16.h>

#include "la_internal.h"

namespace la {
namespace {

constexpr int WARPS = 8, PER = 8;   // channels per lane: D <= 256
constexpr int PARTS = 608;          // CTAs of the backward

__device__ __forceinline__ float ld(const void *p, int64_t i, int bf16)
{
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i])
                : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void st(void *p, int64_t i, float x, int bf16)
{
    if (bf16)
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
    else
        static_cast<float *>(p)[i] = x;
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int m = 16; m; m >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

__device__ __forceinline__ uint64_t turn_of(double inv_freq)
{
    double f = inv_freq * 0.15915494309189535;   // 1 / 2 pi
    f -= floor(f);
    return f >= 1.0 ? 0 : (uint64_t)(f * 18446744073709551616.0);
}

// The position of (batch row b, token t) on an axis.
__device__ __forceinline__ int64_t position(const RopeArgs &a, int axis, int b, int t)
{
    if (a.pos) {
        const int64_t i = axis * a.ps[0] + b * a.ps[1] + t * a.ps[2];
        return a.pos64 ? static_cast<const int64_t *>(a.pos)[i]
                       : (int64_t) static_cast<const int32_t *>(a.pos)[i];
    }
    int n = b, first = 0;
    if (a.cu) {
        int hi = a.N;   // the last n with cu[n] <= t
        n = 0;
        while (hi - n > 1) {
            const int m = (n + hi) / 2;
            if (a.cu[m] <= t)
                n = m;
            else
                hi = m;
        }
        first = a.cu[n];
    }
    return (int64_t)t - first + (a.offset ? a.offset[n] : 0);
}

// Rotates v (channel lane + 32 i of the row) by the token's angles, or back.
__device__ __forceinline__ void rotate(const RopeArgs &a, float (&v)[PER], float *row, int b,
                                       int t, bool back)
{
    const int lane = threadIdx.x % 32, half = a.R / 2;
    if (!a.R)
        return;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i)
        row[lane + 32 * i] = v[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int c = lane + 32 * i;
        if (c >= a.R)
            continue;
        const int j = a.interleaved ? c / 2 : (c < half ? c : c - half);
        const bool second = a.interleaved ? (c & 1) : c >= half;
        const int other = a.interleaved ? c ^ 1 : (second ? c - half : c + half);
        const uint64_t turns =
            (uint64_t)position(a, a.axis[j], b, t) * turn_of(a.inv_freq[j]);
        float sn, cs;
        sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &sn, &cs);
        if (second == back)
            sn = -sn;
        v[i] = v[i] * cs + row[other] * sn;
    }
}

__global__ void __launch_bounds__(WARPS * 32) rope_fwd(RopeArgs a)
{
    __shared__ float rows[WARPS][256];
    const int heads = a.t[0].heads + a.t[1].heads, lane = threadIdx.x % 32;
    const int64_t all = (int64_t)a.B * a.T * heads;
    for (int64_t i = (int64_t)blockIdx.x * WARPS + threadIdx.x / 32; i < all;
         i += (int64_t)gridDim.x * WARPS) {
        const int64_t tok = i / heads;
        int h = (int)(i % heads);
        const int b = (int)(tok / a.T), t = (int)(tok % a.T);
        const int w = h >= a.t[0].heads;
        const RopeTensor &q = a.t[w];
        h -= w ? a.t[0].heads : 0;
        float v[PER], ss = 0.f;
        const int64_t x0 = b * q.xs[0] + t * q.xs[1] + h * q.xs[2];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int c = lane + 32 * k;
            v[k] = c < a.D ? ld(q.x, x0 + c, a.bf16) : 0.f;
            ss += v[k] * v[k];
        }
        if (a.normalize) {
            const float r = 1.f / sqrtf(warp_sum(ss) / (float)a.D + a.eps);
#pragma unroll
            for (int k = 0; k < PER; ++k)
                if (lane + 32 * k < a.D)
                    v[k] *= r * (q.w ? ld(q.w, lane + 32 * k, a.w_bf16) : 1.f);
        }
        rotate(a, v, rows[threadIdx.x / 32], b, t, false);
        const int64_t y0 = b * q.ys[0] + t * q.ys[1] + h * q.ys[2];
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (lane + 32 * k < a.D)
                st(q.y, y0 + lane + 32 * k, v[k], a.bf16);
    }
}

__global__ void __launch_bounds__(WARPS * 32) rope_bwd(RopeArgs a)
{
    __shared__ float rows[WARPS][256];
    const int lane = threadIdx.x % 32, wp = threadIdx.x / 32;
    for (int w = 0; w < 2; ++w) {
        const RopeTensor &q = a.t[w];
        float dw[PER] = {};
        const int64_t all = (int64_t)a.B * a.T * q.heads;
        for (int64_t i = (int64_t)blockIdx.x * WARPS + wp; i < all;
             i += (int64_t)gridDim.x * WARPS) {
            const int64_t tok = i / q.heads;
            const int h = (int)(i % q.heads);
            const int b = (int)(tok / a.T), t = (int)(tok % a.T);
            float v[PER], x[PER], ss = 0.f, zx = 0.f;
            const int64_t d0 = b * q.dys[0] + t * q.dys[1] + h * q.dys[2];
            const int64_t x0 = b * q.xs[0] + t * q.xs[1] + h * q.xs[2];
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int c = lane + 32 * k;
                v[k] = c < a.D ? ld(q.dy, d0 + c, a.bf16) : 0.f;
                x[k] = a.normalize && c < a.D ? ld(q.x, x0 + c, a.bf16) : 0.f;
                ss += x[k] * x[k];
            }
            rotate(a, v, rows[wp], b, t, true);
            if (a.normalize) {
                const float r = 1.f / sqrtf(warp_sum(ss) / (float)a.D + a.eps);
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    dw[k] += v[k] * (x[k] * r);
                    if (lane + 32 * k < a.D)
                        v[k] *= q.w ? ld(q.w, lane + 32 * k, a.w_bf16) : 1.f;
                    zx += v[k] * x[k];
                }
                const float m = warp_sum(zx) / (float)a.D * (r * r);
#pragma unroll
                for (int k = 0; k < PER; ++k)
                    v[k] = r * (v[k] - x[k] * m);
            }
            const int64_t y0 = b * q.ys[0] + t * q.ys[1] + h * q.ys[2];
#pragma unroll
            for (int k = 0; k < PER; ++k)
                if (lane + 32 * k < a.D)
                    st(q.y, y0 + lane + 32 * k, v[k], a.bf16);
        }
        if (!q.dw)
            continue;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < PER; ++k)
            rows[wp][lane + 32 * k] = dw[k];
        __syncthreads();
        for (int c = threadIdx.x; c < a.D; c += WARPS * 32) {
            float sum = 0.f;
            for (int j = 0; j < WARPS; ++j)
                sum += rows[j][c];
            a.partial[((int64_t)w * gridDim.x + blockIdx.x) * a.D + c] = sum;
        }
        __syncthreads();
    }
}

// The weights' gradients from the CTAs' parts, in their order.
__global__ void __launch_bounds__(256) rope_dw(RopeArgs a, int parts)
{
    const RopeTensor &q = a.t[blockIdx.x];
    const int c = threadIdx.x;
    if (!q.dw || c >= a.D)
        return;
    float sum = 0.f;
    for (int j = 0; j < parts; ++j)
        sum += a.partial[((int64_t)blockIdx.x * parts + j) * a.D + c];
    st(q.dw, c, sum, a.w_bf16);
}

}  // namespace

size_t rope_partial_bytes(int D) { return (size_t)2 * PARTS * D * sizeof(float); }

cudaError_t rope_forward(const RopeArgs &a, cudaStream_t s)
{
    rope_fwd<<<PARTS, WARPS * 32, 0, s>>>(a);
    note_launch();
    return cudaGetLastError();
}

cudaError_t rope_backward(const RopeArgs &a, cudaStream_t s)
{
    rope_bwd<<<PARTS, WARPS * 32, 0, s>>>(a);
    note_launch();
    if (a.t[0].dw || a.t[1].dw) {
        rope_dw<<<2, 256, 0, s>>>(a, PARTS);
        note_launch();
    }
    return cudaGetLastError();
}

}  // namespace la
