// la_qk_rope.cuh -- norms of queries and keys for each head with the position
// rotation in the same pass, and their backward.
//
//   y = R(n(x)), n(x) = x r w, r = rsqrt(mean x^2 + eps)
//   u = R^T(dy);  dx = r (z - x r^2 mean(z x)), z = u w;  dw = sum u x r
//
// Angles: inv_freq / 2 pi is kept as a 64-bit fixed-point fraction of a turn
// F, so position * F mod 2^64 is the angle's fraction of a turn, whole turns
// wrapped exactly; F is within 2^-63, so the fraction within |position| 2^-63;
// its upper 32 bits are kept (2^-32 of a turn), and sin and cos are taken of the
// remainder to the nearest quarter turn.  An fp32 product position * inv_freq
// would be off by 0.06 radians at position 10^6.
//
// Bound: HBM, two accesses of a value forward and three backward (two without
// the norms).  A row (one head of one token) belongs to LPR lanes, 8 channels
// each, so that a lane's access is 16 or 32 bytes, a norm is a few shuffles and
// the rotation's partner channel one more.  A warp takes a token's heads one
// after the other: the 8 angles of a lane (25 instructions each) serve them all.

#pragma once

#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_bf16.h>

#include "la_f32x2.cuh"
#include "la_internal.h"

namespace la {
namespace {

constexpr int V = 8;                           // channels per lane
constexpr int WARPS = 8, THREADS = WARPS * 32;
// How a kernel rotates: not at all, halves or neighbours (wide accesses: dispatch,
// below, and rope_run), or as the arguments say, with any alignment.
enum { NONE, HALVES, NEIGHBOURS, ANY };
// Loads of a lane under way at once (bf16: 4 x 16 bytes, fp32: 2 x 32), and CTAs
// an SM, which bound the registers.  60000 tokens of 40 heads of 128, bf16,
// forward: 190 us with 4 CTAs, 199 with 3 (HBM's rate: 181); the rotation alone,
// 32760 tokens of 32 heads: 94 and 85 (79).
template <typename T, bool VEC> constexpr int rounds_of()
{
    return !VEC ? 1 : sizeof(T) == 2 ? 4 : 2;
}
constexpr int ctas_of(bool back, bool norm) { return back ? (norm ? 2 : 3) : (norm ? 4 : 3); }
constexpr unsigned ALL = 0xffffffffu;

// ---- a lane's eight values ----------------------------------------------------

struct Vals {
    F2 p[V / 2];
};
__device__ __forceinline__ Vals zeros()
{
    Vals v;
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
        v.p[i] = f2(0.f);
    return v;
}
__device__ __forceinline__ Vals operator*(const Vals &x, const Vals &y)
{
    Vals v;
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
        v.p[i] = mul2(x.p[i], y.p[i]);
    return v;
}
__device__ __forceinline__ Vals operator*(const Vals &x, float y)
{
    Vals v;
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
        v.p[i] = mul2(x.p[i], f2(y));
    return v;
}
__device__ __forceinline__ Vals fma(const Vals &x, const Vals &y, const Vals &z)
{
    Vals v;
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
        v.p[i] = fma2(x.p[i], y.p[i], z.p[i]);
    return v;
}
// s x + z
__device__ __forceinline__ Vals axpy(float s, const Vals &x, const Vals &z)
{
    Vals v;
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
        v.p[i] = fma2(f2(s), x.p[i], z.p[i]);
    return v;
}
// the sum of the products
__device__ __forceinline__ float dot(const Vals &x, const Vals &y)
{
    F2 s = mul2(x.p[0], y.p[0]);
#pragma unroll
    for (int i = 1; i < V / 2; ++i)
        s = fma2(x.p[i], y.p[i], s);
    const float2 f = un(s);
    return f.x + f.y;
}

template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 r;
    __device__ Vals get() const
    {
        const unsigned w[4] = {r.x, r.y, r.z, r.w};
        Vals v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v.p[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        return v;
    }
    __device__ void set(const Vals &v)
    {
        unsigned w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = un(v.p[i]);
            const __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
            w[i] = *reinterpret_cast<const unsigned *>(&p);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ void clear() { r = make_uint4(0, 0, 0, 0); }
    template <int LPR> __device__ Eight of_lane(int from) const
    {
        Eight x;
        x.r.x = __shfl_sync(ALL, r.x, from, LPR);
        x.r.y = __shfl_sync(ALL, r.y, from, LPR);
        x.r.z = __shfl_sync(ALL, r.z, from, LPR);
        x.r.w = __shfl_sync(ALL, r.w, from, LPR);
        return x;
    }
};
template <> struct Eight<float> {
    float4 a, b;
    __device__ Vals get() const
    {
        return Vals{{f2(a.x, a.y), f2(a.z, a.w), f2(b.x, b.y), f2(b.z, b.w)}};
    }
    __device__ void set(const Vals &v)
    {
        const float2 c = un(v.p[0]), d = un(v.p[1]), e = un(v.p[2]), f = un(v.p[3]);
        a = make_float4(c.x, c.y, d.x, d.y);
        b = make_float4(e.x, e.y, f.x, f.y);
    }
    __device__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    template <int LPR> __device__ Eight of_lane(int from) const
    {
        Eight x;
        x.a.x = __shfl_sync(ALL, a.x, from, LPR);
        x.a.y = __shfl_sync(ALL, a.y, from, LPR);
        x.a.z = __shfl_sync(ALL, a.z, from, LPR);
        x.a.w = __shfl_sync(ALL, a.w, from, LPR);
        x.b.x = __shfl_sync(ALL, b.x, from, LPR);
        x.b.y = __shfl_sync(ALL, b.y, from, LPR);
        x.b.z = __shfl_sync(ALL, b.z, from, LPR);
        x.b.w = __shfl_sync(ALL, b.w, from, LPR);
        return x;
    }
};
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// n of the lane's channels are there (VEC: 0 or all 8, 16-byte aligned); the
// others are 0.
template <typename T, bool VEC> __device__ __forceinline__ Eight<T> load(const T *p, int n)
{
    Eight<T> x;
    if constexpr (VEC) {
        x.clear();
        if (n)
            x = *reinterpret_cast<const Eight<T> *>(p);
    } else {
        float v[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            v[e] = e < n ? to_float(p[e]) : 0.f;
        x.set(Vals{{f2(v[0], v[1]), f2(v[2], v[3]), f2(v[4], v[5]), f2(v[6], v[7])}});
    }
    return x;
}
template <typename T, bool VEC> __device__ __forceinline__ void store(T *p, int n, const Vals &v)
{
    if constexpr (VEC) {
        if (n) {
            Eight<T> x;
            x.set(v);
            *reinterpret_cast<Eight<T> *>(p) = x;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 f = un(v.p[i]);
            if (2 * i < n)
                put(p + 2 * i, f.x);
            if (2 * i + 1 < n)
                put(p + 2 * i + 1, f.y);
        }
    }
}

template <int LPR> __device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int m = LPR / 2; m; m >>= 1)
        x += __shfl_xor_sync(ALL, x, m);
    return x;
}

// ---- angles ------------------------------------------------------------------

// A turn's fraction of x as 64-bit fixed point, to the nearest (whole turns wrap).
__device__ __forceinline__ uint64_t fixed_turn(double x)
{
    return (uint64_t)__double2ll_rn((x - rint(x)) * 18446744073709551616.0);
}
// inv_freq / 2 pi.  1 / 2 pi in two parts: the product with the first one and its
// rounding exactly, so that the fraction has all its 64 bits, which a far
// position multiplies up (one rounded fp64 product: 55 of them, 2^-25 of a turn
// at position 2^31).
__device__ __forceinline__ uint64_t turn_of(double inv_freq)
{
    constexpr double HI = 0x1.45f306dc9c883p-3, LO = -0x1.6b01ec5417056p-57;
    const double p = __dmul_rn(inv_freq, HI);   // (rounded by itself, in no fma)
    return fixed_turn(p) + fixed_turn(__fma_rn(inv_freq, LO, __fma_rn(inv_freq, HI, -p)));
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
    __align__(16) float w[2][256];   // the weights (ones where there are none)
};

// The channel that channel c is rotated with (itself where it is not rotated).
__device__ __forceinline__ int partner_channel(const RopeArgs &a, int c)
{
    const int half = a.R / 2;
    return c >= a.R ? c : a.interleaved ? c ^ 1 : c < half ? c + half : c - half;
}

// cos and sin of the token's angles, by the warp, into its shared memory.
__device__ __forceinline__ void angles(const RopeArgs &a, const Table &tab, int b, int t,
                                       float *cs, float *sn)
{
    if (!a.R)
        return;
    int64_t pos[4];
    pos[0] = position(a, 0, b, t);
#pragma unroll
    for (int i = 1; i < 4; ++i)
        pos[i] = i < a.axes ? position(a, i, b, t) : 0;
    __syncwarp();
    for (int j = threadIdx.x % 32; j < a.R / 2; j += 32) {
        int64_t p = pos[0];
        if (a.axes > 1) {
            const int ax = tab.axis[j];
            p = ax == 1 ? pos[1] : ax == 2 ? pos[2] : ax == 3 ? pos[3] : p;
        }
        sincos_turn((unsigned)((uint64_t)p * tab.turn[j] >> 32), sn + j, cs + j);
    }
    __syncwarp();
}

__device__ __forceinline__ Vals eight(const float *p)
{
    const float4 x = *reinterpret_cast<const float4 *>(p);
    const float4 y = *reinterpret_cast<const float4 *>(p + 4);
    return Vals{{f2(x.x, x.y), f2(x.z, x.w), f2(y.x, y.y), f2(y.z, y.w)}};
}

// Factors of the lane's channels: out = own * c + partner * s.  BACK: the
// rotation back.
template <int ROT, bool BACK>
__device__ __forceinline__ void factors(const RopeArgs &a, const float *cs, const float *sn, int c0,
                                        Vals *fc, Vals *fs)
{
    const int half = a.R / 2;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        fc->p[i] = f2(1.f);
        fs->p[i] = f2(0.f);
    }
    if (ROT == HALVES) {
        if (c0 < a.R) {
            const int j = c0 < half ? c0 : c0 - half;
            const float sign = (c0 >= half) == BACK ? -1.f : 1.f;
            *fc = eight(cs + j);
            *fs = eight(sn + j) * sign;
        }
    } else if (ROT != NONE) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const int c = c0 + 2 * i;
            if (c >= a.R)
                continue;
            if (ROT == NEIGHBOURS || a.interleaved) {
                const float s = sn[c / 2];
                fc->p[i] = f2(cs[c / 2]);
                fs->p[i] = BACK ? f2(s, -s) : f2(-s, s);
            } else {
                float k[2], s[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const bool second = c + u >= half;
                    const int j = second ? c + u - half : c + u;
                    k[u] = cs[j];
                    s[u] = second == BACK ? -sn[j] : sn[j];
                }
                fc->p[i] = f2(k[0], k[1]);
                fs->p[i] = f2(s[0], s[1]);
            }
        }
    }
}
// The partner channels' weights.
template <int ROT>
__device__ __forceinline__ Vals partner_weights(const RopeArgs &a, const float *w, int c0)
{
    Vals v;
    if constexpr (ROT == HALVES) {
        v = eight(w + (c0 >= a.R ? c0 : c0 < a.R / 2 ? c0 + a.R / 2 : c0 - a.R / 2));
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const int c = c0 + 2 * i;
            v.p[i] = ROT == NEIGHBOURS
                         ? f2(w[c + 1], w[c])
                         : f2(w[partner_channel(a, c)], w[partner_channel(a, c + 1)]);
        }
    }
    return v;
}

// The values of the partner channels: in the lane itself (interleaved), in a lane
// of the row (VEC: the halves begin at whole lanes), or through the warp's rows
// in shared memory.
__device__ __forceinline__ Vals swapped(const Vals &v)
{
    Vals r;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const float2 f = un(v.p[i]);
        r.p[i] = f2(f.y, f.x);
    }
    return r;
}
template <typename T, int LPR, int ROT>
__device__ __forceinline__ Vals partners(const RopeArgs &a, const Eight<T> &x, const Vals &v,
                                         int from, float *row)
{
    if (ROT == NEIGHBOURS || (ROT == ANY && a.interleaved))
        return swapped(v);
    if constexpr (ROT == HALVES)
        return x.template of_lane<LPR>(from).get();
    const int l = threadIdx.x % LPR;
    Vals r;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const float2 f = un(v.p[i]);
        row[l * V + 2 * i] = f.x;
        row[l * V + 2 * i + 1] = f.y;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
        r.p[i] = f2(row[partner_channel(a, l * V + 2 * i)],
                    row[partner_channel(a, l * V + 2 * i + 1)]);
    return r;
}

// Adds the partners' part to the rotated channels; the others keep what they
// are, whatever NaN or infinity stands in the row's rotated ones.
__device__ __forceinline__ void turn(const RopeArgs &a, int c0, const Vals &p, const Vals &s,
                                     Vals *v)
{
    if (a.R >= a.D) {
        *v = fma(p, s, *v);
        return;
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
        if (c0 + 2 * i < a.R)
            v->p[i] = fma2(p.p[i], s.p[i], v->p[i]);
}

// ---- kernels -------------------------------------------------------------------
// An item: a token's rows [block * rows, (block + 1) * rows) of q's and then
// k's.

struct Work {
    int64_t items;
    int blocks, rows;   // blocks of a token, rows of a block
    // the item's token (batch row, place) and first row
    __device__ __forceinline__ void at(const RopeArgs &a, int64_t it, int *b, int *t, int *r0) const
    {
        const int64_t tok = blocks == 1 ? it : it / blocks;
        *r0 = (int)(it - tok * blocks) * rows;
        if (tok <= 0xffffffffll) {
            *b = (int)((unsigned)tok / (unsigned)a.T);
            *t = (int)((unsigned)tok - (unsigned)*b * (unsigned)a.T);
        } else {
            *b = (int)(tok / a.T);
            *t = (int)(tok - (int64_t)*b * a.T);
        }
    }
};

// What a lane needs for the rows of one tensor of a token.
struct Lane {
    int c0, n;        // first channel, channels there are
    int from;         // the lane of the partner channels
    float inv_d;
    Vals fc, fs;      // forward: y = r (x fc + x' fs); backward: u = g fc + g' fs
    Vals w;           // backward: the weights
    float *row;
};

template <typename T, int LPR, bool BACK, bool NORM, int ROT>
__device__ __forceinline__ Vals one_row(const RopeArgs &a, const Lane &k, const Eight<T> &xr,
                                        const Eight<T> &gr, Vals *dw)
{
    const bool norm = ROT == ANY ? a.normalize : NORM;
    const bool rotates = ROT == ANY ? a.R > 0 : ROT != NONE;
    Vals x, v;
    float r = 1.f;
    if (!BACK || norm)
        x = xr.get();
    if (norm)
        r = rsqrtf(fmaf(row_sum<LPR>(dot(x, x)), k.inv_d, a.eps));
    if constexpr (!BACK) {
        v = x * k.fc;
        if (rotates)
            turn(a, k.c0, partners<T, LPR, ROT>(a, xr, x, k.from, k.row), k.fs, &v);
        if (norm)
            v = v * r;
    } else {
        const Vals g = gr.get();
        v = g * k.fc;
        if (rotates)
            turn(a, k.c0, partners<T, LPR, ROT>(a, gr, g, k.from, k.row), k.fs, &v);
        if (norm) {
            *dw = fma(v, x * r, *dw);
            v = v * k.w;
            const float f = row_sum<LPR>(dot(v, x)) * k.inv_d * (r * r) * -r;
            v = axpy(f, x, v * r);
        }
    }
    return v;
}

// bf16's backward with the norms holds too much to have enough loads under way in
// registers: a warp's rounds are copied to a ring in shared memory, each lane's
// values to a place of its own, so that nobody else is waited for.  60000 tokens
// of 40 heads of 128: 298 us (HBM's rate: 272), 335 from registers; 300 tokens:
// 11 us, 10.  fp32 from registers: 302 us (296) at 32768 tokens, 484 through the
// ring, whose copies are 16 bytes of a lane's 32.
template <typename T, bool BACK, bool NORM, int ROT> constexpr bool ringed()
{
    return BACK && NORM && ROT != ANY && sizeof(T) == 2;
}
// Bytes of a warp's round, and of one tensor's values of a row group in it.
constexpr int STAGES = 3, ROUND = 4096, PIECE = 512;
constexpr int RING_BYTES = WARPS * STAGES * ROUND;

__device__ __forceinline__ void slot_copy(uint32_t to, const void *from, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
                 "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ Eight<__nv_bfloat16> slot_load(uint32_t from)
{
    Eight<__nv_bfloat16> x;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.r.x), "=r"(x.r.y), "=r"(x.r.z), "=r"(x.r.w)
                 : "r"(from));
    return x;
}

// The rounds of a warp in the order that it takes them.
struct Ahead {
    using T = __nv_bfloat16;
    int64_t it;
    int which, h0, hi;
    const T *xp, *gp;

    // asks for the next round's values (none are left: for nothing)
    template <int SUBS, int U>
    __device__ __forceinline__ void next(const RopeArgs &a, const Work &wk, uint32_t to, int c0,
                                         int n, int sub)
    {
        while (h0 >= hi && it < wk.items) {
            if (++which == 2) {
                which = 0;
                it += (int64_t)gridDim.x * WARPS;
                if (it >= wk.items)
                    break;
            }
            const RopeTensor &q = a.t[which];
            int b, t, r0;
            wk.at(a, it, &b, &t, &r0);
            r0 -= which ? a.t[0].heads : 0;
            h0 = max(r0, 0);
            hi = min(r0 + wk.rows, q.heads);
            const int h = h0 + sub;
            xp = static_cast<const T *>(q.x) + b * q.xs[0] + t * q.xs[1] + h * q.xs[2] + c0;
            gp = static_cast<const T *>(q.dy) + b * q.dys[0] + t * q.dys[1] + h * q.dys[2] + c0;
        }
        if (it < wk.items) {
            const RopeTensor &q = a.t[which];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool there = n && h0 + u * SUBS + sub < hi;
                const T *x = there ? xp : static_cast<const T *>(q.x);
                const T *g = there ? gp : static_cast<const T *>(q.dy);
                slot_copy(to + 2 * u * PIECE, x, there);
                slot_copy(to + (2 * u + 1) * PIECE, g, there);
                xp += SUBS * q.xs[2];
                gp += SUBS * q.dys[2];
            }
            h0 += SUBS * U;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
};

template <typename T, int LPR, bool BACK, bool NORM, int ROT>
__global__ void __launch_bounds__(THREADS, ctas_of(BACK, NORM))
    rope(const RopeArgs a, const Work wk)
{
    constexpr bool VEC = ROT != ANY;
    constexpr int SUBS = 32 / LPR, U = rounds_of<T, VEC>();
    constexpr bool RING = ringed<T, BACK, NORM, ROT>();
    static_assert(!RING || (sizeof(Eight<T>) * 32 == PIECE && 2 * U * PIECE == ROUND), "ring");
    __shared__ Table tab;
    // a warp's cos and sin, ANY: then its rows' partners; at the end the sums
    __shared__ __align__(16) float exchange[WARPS][32 * V + (VEC ? 0 : 32 * V)];
    const int lane = threadIdx.x % 32, l = lane % LPR, sub = lane / LPR, warp = threadIdx.x / 32;
    const bool norm = VEC ? NORM : a.normalize;
    extern __shared__ __align__(16) uint8_t slots[];
    Lane k;
    k.c0 = l * V;
    k.n = max(0, min(V, a.D - k.c0));
    const int d = a.R / 2 / V;
    k.from = (l < d ? l + d : l - d) & (LPR - 1);
    k.inv_d = 1.f / (float)a.D;
    k.row = exchange[warp] + (VEC ? 0 : 32 * V) + sub * LPR * V;
    for (int j = threadIdx.x; j < a.R / 2; j += THREADS) {
        tab.turn[j] = turn_of(a.inv_freq[j]);
        tab.axis[j] = a.axis[j];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const void *w = a.t[i].w;
        const int c = threadIdx.x;
        tab.w[i][c] = !w || c >= a.D ? 1.f
                      : a.w_bf16     ? to_float(static_cast<const __nv_bfloat16 *>(w)[c])
                                     : static_cast<const float *>(w)[c];
    }
    __syncthreads();
    Vals dw[2] = {zeros(), zeros()};
    // RING: the warp's rounds, asked for STAGES - 1 ahead
    Ahead f;
    const uint32_t slot = RING ? (uint32_t)__cvta_generic_to_shared(slots) +
                                     warp * (STAGES * ROUND) + lane * 16
                               : 0;
    unsigned round = 0;
    if constexpr (RING) {
        f.it = (int64_t)blockIdx.x * WARPS + warp;
        f.which = -1;
        f.h0 = f.hi = 0;
        for (int i = 0; i < STAGES - 1; ++i)
            f.next<SUBS, U>(a, wk, slot + i * ROUND, k.c0, k.n, sub);
    }
    for (int64_t it = (int64_t)blockIdx.x * WARPS + warp; it < wk.items;
         it += (int64_t)gridDim.x * WARPS) {
        int b, t, r0;
        wk.at(a, it, &b, &t, &r0);
        float *cs = exchange[warp], *sn = cs + 128;
        bool known = ROT == NONE;   // the angles
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
            const RopeTensor &q = a.t[which];
            const int base = which ? a.t[0].heads : 0;
            const int lo = max(r0 - base, 0), hi = min(r0 + wk.rows - base, q.heads);
            if (lo >= hi)
                continue;
            const T *xp = static_cast<const T *>(q.x) + b * q.xs[0] + t * q.xs[1] + k.c0 +
                          (lo + sub) * q.xs[2];
            const T *gp = static_cast<const T *>(q.dy) + b * q.dys[0] + t * q.dys[1] + k.c0 +
                          (lo + sub) * q.dys[2];
            T *yp = static_cast<T *>(q.y) + b * q.ys[0] + t * q.ys[1] + k.c0 +
                    (lo + sub) * q.ys[2];
            const int64_t xd = SUBS * q.xs[2], gd = SUBS * q.dys[2], yd = SUBS * q.ys[2];
            Eight<T> xr[U], gr[U];
            auto fetch = [&](int h0) {   // a round's loads
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int m = h0 + u * SUBS + sub < hi ? k.n : 0;
                    if (!BACK || norm)
                        xr[u] = load<T, VEC>(xp, m);
                    if (BACK)
                        gr[u] = load<T, VEC>(gp, m);
                    xp += xd;
                    gp += gd;
                }
            };
            if constexpr (!RING)
                fetch(lo);   // on their way while the angles are formed
            if (!known) {
                angles(a, tab, b, t, cs, sn);
                known = true;
            }
            factors<ROT, BACK>(a, cs, sn, k.c0, &k.fc, &k.fs);
            if (norm) {
                const Vals w = eight(tab.w[which] + k.c0);
                if (BACK) {
                    k.w = w;
                } else {
                    k.fc = k.fc * w;
                    if (ROT != NONE)
                        k.fs = k.fs * partner_weights<ROT>(a, tab.w[which], k.c0);
                }
            }
            Vals sum = zeros();
            for (int h0 = lo;;) {
                uint32_t from = 0;
                if constexpr (RING) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
                    from = slot + round % STAGES * ROUND;
                    // (to the stage of the round before this one)
                    f.next<SUBS, U>(a, wk, slot + (round + STAGES - 1) % STAGES * ROUND,
                                             k.c0, k.n, sub);
                    ++round;
                }
                auto row = [&](int u) {
                    const int m = h0 + u * SUBS + sub < hi ? k.n : 0;
                    if constexpr (RING) {
                        xr[u] = slot_load(from + 2 * u * PIECE);
                        gr[u] = slot_load(from + (2 * u + 1) * PIECE);
                    }
                    const Vals before = sum;
                    const Vals y = one_row<T, LPR, BACK, NORM, ROT>(a, k, xr[u], gr[u], &sum);
                    if (BACK && !m)   // (with eps 0 a row that is not there has no finite norm)
                        sum = before;
                    store<T, VEC>(yp, m, y);
                    yp += yd;
                };
                // whole rounds without a branch: their rows' sums overlap then
                if (RING && h0 + SUBS * U <= hi) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        row(u);
                } else {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (h0 + u * SUBS >= hi)
                            break;
                        row(u);
                    }
                }
                h0 += SUBS * U;
                if (h0 >= hi)
                    break;
                if constexpr (!RING)
                    fetch(h0);
            }
            if (BACK && norm) {
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    if (which == 0)
                        dw[0].p[i] = add2(dw[0].p[i], sum.p[i]);
                    else
                        dw[1].p[i] = add2(dw[1].p[i], sum.p[i]);
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
            for (int i = 0; i < V / 2; ++i) {
                const float2 f = un(dw[which].p[i]);
                exchange[warp][lane * V + 2 * i] = f.x;
                exchange[warp][lane * V + 2 * i + 1] = f.y;
            }
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

// ---- launches --------------------------------------------------------------------

template <typename T, int LPR, bool BACK, bool NORM, int ROT>
cudaError_t launch(const RopeArgs &a, int sms, cudaStream_t s, int *parts)
{
    constexpr int SUBS = 32 / LPR, U = rounds_of<T, ROT != ANY>();
    const int heads = a.t[0].heads + a.t[1].heads;
    const int most = std::min(sms * ctas_of(BACK, NORM), ROPE_MOST_CTAS);
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
    *parts = (int)std::min<int64_t>((wk.items + WARPS - 1) / WARPS, most);
    constexpr int ring = ringed<T, BACK, NORM, ROT>() ? RING_BYTES : 0;
    constexpr auto kernel = rope<T, LPR, BACK, NORM, ROT>;
    if constexpr (ring > 0) {   // once per device
        static std::atomic<uint64_t> known;
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess)
            return e;
        if (dev > 63 || !(known.load() >> dev & 1)) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
            if (e != cudaSuccess)
                return e;
            if (dev < 64)
                known.fetch_or((uint64_t)1 << dev);
        }
    }
    kernel<<<*parts, THREADS, ring, s>>>(a, wk);
    note_launch();
    return cudaGetLastError();
}

template <typename T, bool BACK, bool NORM, int ROT>
cudaError_t by_width(const RopeArgs &a, int sms, cudaStream_t s, int *parts)
{
    if (a.D <= 64)
        return launch<T, 8, BACK, NORM, ROT>(a, sms, s, parts);
    if (a.D <= 128)
        return launch<T, 16, BACK, NORM, ROT>(a, sms, s, parts);
    return launch<T, 32, BACK, NORM, ROT>(a, sms, s, parts);
}

// vec: wide accesses, whole lanes of 16-byte aligned channels, the halves of the
// rotation beginning at whole lanes.
template <typename T, bool BACK>
cudaError_t rope_of(const RopeArgs &a, bool vec, int sms, cudaStream_t s, int *parts)
{
    if (!vec)
        return by_width<T, BACK, true, ANY>(a, sms, s, parts);
    if (!a.R)
        return by_width<T, BACK, true, NONE>(a, sms, s, parts);
    if (a.normalize)
        return a.interleaved ? by_width<T, BACK, true, NEIGHBOURS>(a, sms, s, parts)
                             : by_width<T, BACK, true, HALVES>(a, sms, s, parts);
    return a.interleaved ? by_width<T, BACK, false, NEIGHBOURS>(a, sms, s, parts)
                         : by_width<T, BACK, false, HALVES>(a, sms, s, parts);
}

}  // namespace
}  // namespace la
