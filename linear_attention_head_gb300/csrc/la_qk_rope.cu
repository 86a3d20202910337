// la_qk_rope.cu -- norms of queries and keys for each head with the position
// rotation in the same pass, and their backward.
//
//   y = R(n(x)), n(x) = x r w, r = rsqrt(mean x^2 + eps)
//   u = R^T(dy);  dx = r (z - x r^2 mean(z x)), z = u w;  dw = sum u x r
//
// Angles: inv_freq / 2 pi is kept as a 64-bit fixed-point fraction of a turn
// F, so position * F mod 2^64 is the angle's fraction of a turn, wrapped
// exactly, at every position; its upper 32 bits are kept (2^-32 of a turn), and
// sin and cos are taken of the remainder to the nearest quarter turn.  An fp32
// product position * inv_freq would be off by 0.06 radians at position 10^6.
//
// Bound: HBM, two accesses of a value forward and three backward (two without
// the norms).  A row (one head of one token) belongs to LPR lanes, 8 channels
// each, so that a lane's access is 16 or 32 bytes, a norm is a few shuffles and
// the rotation's partner channel one more.  A warp takes a token's heads one
// after the other: the 8 angles of a lane (25 instructions each) serve them all.

#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_bf16.h>

#include "la_internal.h"

namespace la {
namespace {

constexpr int V = 8;                           // channels per lane
constexpr int WARPS = 8, THREADS = WARPS * 32;
constexpr unsigned ALL = 0xffffffffu;

// ---- a lane's eight values ----------------------------------------------------

template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 r;
    __device__ void get(float (&v)[V]) const
    {
        const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ void set(const float (&v)[V])
    {
        unsigned w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const unsigned *>(&p);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Eight<float> {
    float4 a, b;
    __device__ void get(float (&v)[V]) const
    {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ void set(const float (&v)[V])
    {
        a = make_float4(v[0], v[1], v[2], v[3]);
        b = make_float4(v[4], v[5], v[6], v[7]);
    }
};
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// n of the lane's channels are there (VEC: 0 or all 8, 16-byte aligned).
template <typename T, bool VEC>
__device__ __forceinline__ void load(const T *p, int n, Eight<T> &x)
{
    if constexpr (VEC) {
        if (n)
            x = *reinterpret_cast<const Eight<T> *>(p);
    } else {
        float v[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            v[e] = e < n ? to_float(p[e]) : 0.f;
        x.set(v);
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store(T *p, int n, const float (&v)[V])
{
    if constexpr (VEC) {
        if (n) {
            Eight<T> x;
            x.set(v);
            *reinterpret_cast<Eight<T> *>(p) = x;
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < n)
                put(p + e, v[e]);
    }
}

template <int LPR> __device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int m = LPR / 2; m; m >>= 1)
        x += __shfl_xor_sync(ALL, x, m);
    return x;
}

__device__ __forceinline__ float weight(const void *w, int c, int bf16)
{
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[c])
                : static_cast<const float *>(w)[c];
}

// ---- angles ------------------------------------------------------------------

__device__ __forceinline__ uint64_t turn_of(double inv_freq)
{
    double f = inv_freq * 0.15915494309189535;   // 1 / 2 pi
    f -= floor(f);
    return f >= 1.0 ? 0 : (uint64_t)(f * 18446744073709551616.0);
}

// sin and cos of f / 2^32 of a turn: Taylor series of the remainder x to the
// nearest quarter turn (|x| <= pi / 4; the first terms left out are below 2^-28).
__device__ __forceinline__ void sincos_turn(unsigned f, float *sn, float *cs)
{
    const unsigned q = (f + 0x20000000u) >> 30;
    const float x = (float)(int)(f - (q << 30)) * 1.46291807926715968e-9f;   // 2 pi / 2^32
    const float x2 = x * x;
    float s = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f);
    s = fmaf(x2, s, 1.f / 120.f);
    s = fmaf(x2, s, -1.f / 6.f);
    s = fmaf(x2 * x, s, x);
    float c = fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f);
    c = fmaf(x2, c, -1.f / 720.f);
    c = fmaf(x2, c, 1.f / 24.f);
    c = fmaf(x2, c, -0.5f);
    c = fmaf(x2, c, 1.f);
    const float u = q & 1 ? c : s, v = q & 1 ? s : c;
    *sn = q & 2 ? -u : u;
    *cs = (q + 1) & 2 ? -v : v;
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

struct Table {
    uint64_t turn[128];
    uint8_t axis[128];
};

// Factors of the lane's channels: out = own * c + partner * s.  BACK: the
// rotation back.
template <bool BACK>
__device__ __forceinline__ void factors(const RopeArgs &a, const Table &tab, int b, int t, int c0,
                                        float (&cs)[V], float (&sn)[V])
{
    const int half = a.R / 2;
    int64_t pos[4] = {0, 0, 0, 0};
    if (a.R) {
        pos[0] = position(a, 0, b, t);
#pragma unroll
        for (int i = 1; i < 4; ++i)
            if (i < a.axes)
                pos[i] = position(a, i, b, t);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const int c = c0 + e;
        cs[e] = 1.f;
        sn[e] = 0.f;
        if (c >= a.R)
            continue;
        const int j = a.interleaved ? c / 2 : (c < half ? c : c - half);
        const bool second = a.interleaved ? (c & 1) : c >= half;
        int64_t p = pos[0];
        if (a.axes > 1) {
            const int ax = tab.axis[j];
            p = ax == 1 ? pos[1] : ax == 2 ? pos[2] : ax == 3 ? pos[3] : p;
        }
        sincos_turn((unsigned)((uint64_t)p * tab.turn[j] >> 32), &sn[e], &cs[e]);
        if (second == BACK)
            sn[e] = -sn[e];
    }
}

// v := v * cs + partner * sn.  The partner channel: in the lane itself
// (interleaved), in a lane of the row (VEC: the halves begin at whole lanes), or
// through the warp's rows in shared memory.
template <int LPR, bool VEC>
__device__ __forceinline__ void rotate(const RopeArgs &a, float (&v)[V], const float (&cs)[V],
                                       const float (&sn)[V], float *row)
{
    const int l = threadIdx.x % LPR, half = a.R / 2;
    if (!a.R)
        return;
    float p[V];
    if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            p[e] = v[e ^ 1];
    } else if (VEC) {
        const int d = half / V, from = l < d ? l + d : l - d;
#pragma unroll
        for (int e = 0; e < V; ++e)
            p[e] = __shfl_sync(ALL, v[e], from & (LPR - 1), LPR);
    } else {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < V; ++e)
            row[l * V + e] = v[e];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = l * V + e;
            p[e] = c < a.R ? row[c < half ? c + half : c - half] : 0.f;
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
        v[e] = fmaf(p[e], sn[e], v[e] * cs[e]);
}

// ---- kernels -------------------------------------------------------------------
// An item: a token's rows [block * rows, (block + 1) * rows) of q's and then
// k's.

struct Work {
    int64_t items;
    int blocks, rows;   // blocks of a token, rows of a block
};

template <typename T, int LPR, bool VEC, bool BACK>
__global__ void __launch_bounds__(THREADS, BACK ? 2 : 3) rope(const RopeArgs a, const Work wk)
{
    constexpr int SUBS = 32 / LPR, U = VEC ? (sizeof(T) == 2 ? 4 : 2) : 1;
    __shared__ Table tab;
    __shared__ float exchange[WARPS][32 * V];   // rows' partners, at the end the sums
    const int lane = threadIdx.x % 32, l = lane % LPR, sub = lane / LPR, warp = threadIdx.x / 32;
    const int c0 = l * V, n = max(0, min(V, a.D - c0));
    float *row = exchange[warp] + sub * LPR * V;
    for (int j = threadIdx.x; j < a.R / 2; j += THREADS) {
        tab.turn[j] = turn_of(a.inv_freq[j]);
        tab.axis[j] = a.axis[j];
    }
    __syncthreads();
    float dw[2][V] = {};
    const float inv_d = 1.f / (float)a.D;
    for (int64_t it = (int64_t)blockIdx.x * WARPS + warp; it < wk.items;
         it += (int64_t)gridDim.x * WARPS) {
        const int64_t tok = wk.blocks == 1 ? it : it / wk.blocks;
        const int r0 = (int)(it - tok * wk.blocks) * wk.rows;
        int b, t;
        if (tok <= 0xffffffffll) {
            b = (int)((unsigned)tok / (unsigned)a.T);
            t = (int)((unsigned)tok - (unsigned)b * (unsigned)a.T);
        } else {
            b = (int)(tok / a.T);
            t = (int)(tok - (int64_t)b * a.T);
        }
        float cs[V], sn[V];
        factors<BACK>(a, tab, b, t, c0, cs, sn);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const RopeTensor &q = a.t[which];
            const int base = which ? a.t[0].heads : 0;
            const int lo = max(r0 - base, 0), hi = min(r0 + wk.rows - base, q.heads);
            if (lo >= hi)
                continue;
            float w[V];
#pragma unroll
            for (int e = 0; e < V; ++e)
                w[e] = a.normalize && q.w && e < n ? weight(q.w, c0 + e, a.w_bf16) : 1.f;
            const T *xp = static_cast<const T *>(q.x) + b * q.xs[0] + t * q.xs[1] + c0;
            const T *gp = static_cast<const T *>(q.dy) + b * q.dys[0] + t * q.dys[1] + c0;
            T *yp = static_cast<T *>(q.y) + b * q.ys[0] + t * q.ys[1] + c0;
            const bool reads_x = !BACK || a.normalize;
            for (int h0 = lo; h0 < hi; h0 += SUBS * U) {
                Eight<T> xr[U], gr[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = h0 + u * SUBS + sub;
                    const int m = h < hi ? n : 0;
                    if (reads_x)
                        load<T, VEC>(xp + h * q.xs[2], m, xr[u]);
                    if (BACK)
                        load<T, VEC>(gp + h * q.dys[2], m, gr[u]);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (h0 + u * SUBS >= hi)
                        break;
                    const int h = h0 + u * SUBS + sub;
                    const int m = h < hi ? n : 0;
                    float v[V], x[V], r = 0.f;
                    if (reads_x) {
                        xr[u].get(x);
                        if (!m) {
#pragma unroll
                            for (int e = 0; e < V; ++e)
                                x[e] = 0.f;
                        }
                    }
                    if (a.normalize) {
                        float ss = 0.f;
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            ss = fmaf(x[e], x[e], ss);
                        r = rsqrtf(fmaf(row_sum<LPR>(ss), inv_d, a.eps));
                    }
                    if constexpr (!BACK) {
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            v[e] = a.normalize ? x[e] * r * w[e] : x[e];
                        rotate<LPR, VEC>(a, v, cs, sn, row);
                    } else {
                        gr[u].get(v);
                        if (!m) {
#pragma unroll
                            for (int e = 0; e < V; ++e)
                                v[e] = 0.f;
                        }
                        rotate<LPR, VEC>(a, v, cs, sn, row);
                        if (a.normalize) {
                            float zx = 0.f;
#pragma unroll
                            for (int e = 0; e < V; ++e) {
                                if (m)
                                    dw[which][e] = fmaf(v[e], x[e] * r, dw[which][e]);
                                v[e] *= w[e];
                                zx = fmaf(v[e], x[e], zx);
                            }
                            const float f = row_sum<LPR>(zx) * inv_d * (r * r);
#pragma unroll
                            for (int e = 0; e < V; ++e)
                                v[e] = r * fmaf(-x[e], f, v[e]);
                        }
                    }
                    store<T, VEC>(yp + h * q.ys[2], m, v);
                }
            }
        }
    }
    if constexpr (BACK) {
        // the CTA's part of the weights' gradients, summed in a fixed order
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            if (!a.t[which].dw)
                continue;
            __syncthreads();
#pragma unroll
            for (int e = 0; e < V; ++e)
                exchange[warp][lane * V + e] = dw[which][e];
            __syncthreads();
            for (int c = threadIdx.x; c < a.D; c += THREADS) {
                float sum = 0.f;
                for (int i = 0; i < WARPS * SUBS; ++i)
                    sum += exchange[i / SUBS][i % SUBS * LPR * V + c];
                a.partial[((int64_t)which * gridDim.x + blockIdx.x) * a.D + c] = sum;
            }
        }
    }
}

// The weights' gradients from the CTAs' parts: 32 channels a CTA, 32 slices of
// the parts side by side, then the slices in their order.
__global__ void __launch_bounds__(1024) rope_dw(const RopeArgs a, int parts)
{
    __shared__ float sums[32][33];
    const RopeTensor &q = a.t[blockIdx.y];
    if (!q.dw)
        return;
    const int lane = threadIdx.x % 32, slice = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    const int each = (parts + 31) / 32, lo = slice * each, hi = min(lo + each, parts);
    const float *p = a.partial + (int64_t)blockIdx.y * parts * a.D + c;
    float sum = 0.f;
    if (c < a.D) {
#pragma unroll 8
        for (int i = lo; i < hi; ++i)
            sum += p[(int64_t)i * a.D];
    }
    sums[slice][lane] = sum;
    __syncthreads();
    if (slice == 0 && c < a.D) {
        float all = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            all += sums[i][lane];
        if (a.w_bf16)
            put(static_cast<__nv_bfloat16 *>(q.dw) + c, all);
        else
            put(static_cast<float *>(q.dw) + c, all);
    }
}

// ---- launches --------------------------------------------------------------------

constexpr int MOST_CTAS = 512;   // of the backward: rope_partial_bytes

int sms()
{
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return 1;
    if (dev < 64 && (n = known[dev].load()) > 0)
        return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
        return 1;
    if (dev < 64)
        known[dev].store(n);
    return n;
}

bool wide(const void *p, const int64_t *st, int bf16)
{
    const int n = bf16 ? 8 : 4;
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && st[0] % n == 0 && st[1] % n == 0 &&
           st[2] % n == 0;
}

template <typename T, int LPR, bool VEC>
cudaError_t launch(bool back, const RopeArgs &a, cudaStream_t s)
{
    constexpr int SUBS = 32 / LPR, U = VEC ? (sizeof(T) == 2 ? 4 : 2) : 1;
    const int heads = a.t[0].heads + a.t[1].heads, most = std::min(sms() * (back ? 2 : 3), MOST_CTAS);
    // whole tokens to a warp, unless that leaves warps idle: then blocks of a
    // token's rows, of one round of a warp's loads at least
    Work wk;
    const int64_t tokens = (int64_t)a.B * a.T;
    const int64_t want = ((int64_t)most * WARPS + tokens - 1) / tokens;
    const int rounds = (heads + SUBS * U - 1) / (SUBS * U);
    wk.blocks = (int)std::min<int64_t>(std::max<int64_t>(want, 1), rounds);
    wk.rows = (rounds + wk.blocks - 1) / wk.blocks * (SUBS * U);
    wk.blocks = (heads + wk.rows - 1) / wk.rows;
    wk.items = tokens * wk.blocks;
    const int grid = (int)std::min<int64_t>((wk.items + WARPS - 1) / WARPS, most);
    if (back)
        rope<T, LPR, VEC, true><<<grid, THREADS, 0, s>>>(a, wk);
    else
        rope<T, LPR, VEC, false><<<grid, THREADS, 0, s>>>(a, wk);
    note_launch();
    if (back && (a.t[0].dw || a.t[1].dw)) {
        rope_dw<<<dim3((a.D + 31) / 32, 2), 1024, 0, s>>>(a, grid);
        note_launch();
    }
    return cudaGetLastError();
}

template <typename T, bool VEC> cudaError_t by_width(bool back, const RopeArgs &a, cudaStream_t s)
{
    if (a.D <= 64)
        return launch<T, 8, VEC>(back, a, s);
    if (a.D <= 128)
        return launch<T, 16, VEC>(back, a, s);
    return launch<T, 32, VEC>(back, a, s);
}

cudaError_t run(bool back, const RopeArgs &a, cudaStream_t s)
{
    // wide accesses: whole lanes of 16-byte aligned channels, the halves of the
    // rotation beginning at whole lanes
    bool vec = a.D % V == 0 && (a.interleaved || a.R % (2 * V) == 0);
    for (const RopeTensor &t : a.t) {
        if (!t.heads)
            continue;
        if (!back || a.normalize)
            vec &= wide(t.x, t.xs, a.bf16);
        if (back)
            vec &= wide(t.dy, t.dys, a.bf16);
        vec &= wide(t.y, t.ys, a.bf16);
    }
    if (a.bf16)
        return vec ? by_width<__nv_bfloat16, true>(back, a, s)
                   : by_width<__nv_bfloat16, false>(back, a, s);
    return vec ? by_width<float, true>(back, a, s) : by_width<float, false>(back, a, s);
}

}  // namespace

size_t rope_partial_bytes(int D) { return (size_t)2 * MOST_CTAS * D * sizeof(float); }

cudaError_t rope_forward(const RopeArgs &a, cudaStream_t s) { return run(false, a, s); }
cudaError_t rope_backward(const RopeArgs &a, cudaStream_t s) { return run(true, a, s); }

}  // namespace la
