// la_delta_token.cu -- the gated delta rule token by token, for every size and
// type: decoding (1 to 16 tokens against a carried state), fp32 tokens, and the
// widths and layouts that the chunked tensor-core kernels (la_delta_tc.cu) do
// not take.  Per sequence and value head, S a D x E state in fp32 registers,
//
//     S' = exp(g) S,   e = v - S'^T k,   S = S' + beta k e^T,   o = scale S^T q.
//
// Columns of S are independent of one another given k, so a warp owns whole
// columns (4 QW of them) and needs no other warp: 32 lanes = RG row groups of 16
// rows x QW column quads, a thread 16 x 4 numbers of S.  The sums over rows
// (S'^T k, S^T q) are RG-lane shuffles.  q, k, v and the gates of 8 (or 4)
// tokens at a time pass through shared memory as fp32.
//
// One token of b64 h32 d128 with the states in and out moves 270 MB: the states'
// bytes bound it, 51 us on one GB300, 0.79 of its copy rate.  All 64 numbers a thread are
// asked for at once, 16 bytes a lane.
//
// The backward takes three passes over the tokens and keeps no state:
//   1. forward, keeping e_t;
//   2. from last to first, K = dL/dS:  K += scale q do^T,  w = K^T k,
//      dv = beta w, dbeta = w . e, dk = K (beta e), K = exp(g) (K - k dv^T);
//   3. forward with the known e: dk -= S' dv, S = S' + beta k e^T,
//      dq = scale S do;
// and dg_t = sum over i >= t of (q_i . dq_i - v_i . dv_i) + <S_end, dS_end>: what
// scaling the state entering token t does, by the chain rule over all later
// tokens.  Sums over columns are joined over the warps of a CTA in shared memory
// and over CTAs (column tiles) by finish_kernel, in a fixed order.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "la_f32x2.cuh"
#include "la_internal.h"

namespace la {
namespace {

constexpr int ROWS = 16;        // of S, a thread
constexpr int WARPS = 4;
constexpr int RPAD = 20;        // floats a row group takes in shared memory: 4 groups read
                                // 16 bytes each from different banks

template <int RG> struct Shape {
    static constexpr int QW = 32 / RG;          // column quads a warp
    static constexpr int WCOLS = 4 * QW;        // columns a warp
    static constexpr int TW = WARPS * WCOLS;    // columns a CTA
    static constexpr int DP = RG * RPAD;
    static constexpr int TB = RG == 16 ? 4 : 8;     // tokens staged together (48 KB a CTA)
};

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f(float x) { return x; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float x)
{
    return __float2bfloat16_rn(x);
}

__device__ __forceinline__ float gate_at(const Tok &g, int bf16, int64_t row, int64_t t, int h)
{
    const int64_t at = row * g.sb + t * g.st + (int64_t)h * g.sh;
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(g.p)[at])
                : static_cast<const float *>(g.p)[at];
}

enum Mode { FWD, KEEP, BACK, AGAIN };   // KEEP, BACK, AGAIN: the backward's passes

struct Params {
    DeltaArgs a;
    int tiles;
    float *e, *dvf;             // [B][T][H][E] fp32: e_t, dv_t
    float *dqp, *dkp;           // [tiles][B][T][H][D] fp32
    float *dbp;                 // [tiles][B][T][H]
    float *end;                 // [tiles][N][H]: <S_end, dS_end>
};

struct Place {
    int n, h, tile;
    int64_t row, bos;
    int len;
};
__device__ __forceinline__ Place place(const DeltaArgs &a, int tiles)
{
    Place p;
    p.tile = blockIdx.x % tiles;
    const int64_t nh = blockIdx.x / tiles;
    p.h = (int)(nh % a.H);
    p.n = (int)(nh / a.H);
    if (a.cu) {
        p.row = 0;
        p.bos = a.cu[p.n];
        p.len = a.cu[p.n + 1] - (int)p.bos;
    } else {
        p.row = p.n;
        p.bos = 0;
        p.len = a.T;
    }
    return p;
}

// Sum over the lanes that hold the same columns.
template <int RG> __device__ __forceinline__ float4 over_rows(float4 x)
{
#pragma unroll
    for (int m = 32 / RG; m < 32; m *= 2) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, m);
        x.y += __shfl_xor_sync(0xffffffffu, x.y, m);
        x.z += __shfl_xor_sync(0xffffffffu, x.z, m);
        x.w += __shfl_xor_sync(0xffffffffu, x.w, m);
    }
    return x;
}

// x[r] summed over the warp's column quads: halves traded, so that lane quad qw ends
// with rows first .. first + ROWS / QW - 1, in x[0] ..
template <int RG> __device__ __forceinline__ int over_quads(float (&x)[ROWS], int qw)
{
    constexpr int QW = 32 / RG;
    int first = 0;
#pragma unroll
    for (int m = QW / 2, w = ROWS / 2; m >= 1; m /= 2, w /= 2) {
        const bool up = qw & m;
#pragma unroll
        for (int r = 0; r < ROWS / 2; ++r)
            if (r < w) {
                const float mine = up ? x[r + w] : x[r], other = up ? x[r] : x[r + w];
                x[r] = mine + __shfl_xor_sync(0xffffffffu, other, m);
            }
        first += up ? w : 0;
    }
    return first;
}

// The packed instructions do two columns at once.
template <int RG> __device__ __forceinline__ float4 dot_rows(const float4 (&S)[ROWS], const float *x)
{
    F2 u0 = f2(0.f), u1 = f2(0.f);
#pragma unroll
    for (int r4 = 0; r4 < ROWS; r4 += 4) {
        const float4 k = *reinterpret_cast<const float4 *>(x + r4);
        const float kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u0 = fma2(f2(S[r4 + j].x, S[r4 + j].y), f2(kk[j]), u0);
            u1 = fma2(f2(S[r4 + j].z, S[r4 + j].w), f2(kk[j]), u1);
        }
    }
    const float2 a = un(u0), b = un(u1);
    return over_rows<RG>(make_float4(a.x, a.y, b.x, b.y));
}

// S = f S + x y^T
__device__ __forceinline__ void rank_one(float4 (&S)[ROWS], float f, const float *x, float4 y)
{
    const F2 y0 = f2(y.x, y.y), y1 = f2(y.z, y.w), f0 = f2(f);
#pragma unroll
    for (int r4 = 0; r4 < ROWS; r4 += 4) {
        const float4 k = *reinterpret_cast<const float4 *>(x + r4);
        const float kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 a = un(fma2(f2(kk[j]), y0, mul2(f0, f2(S[r4 + j].x, S[r4 + j].y))));
            const float2 b = un(fma2(f2(kk[j]), y1, mul2(f0, f2(S[r4 + j].z, S[r4 + j].w))));
            S[r4 + j] = make_float4(a.x, a.y, b.x, b.y);
        }
    }
}

template <int RG, Mode M, typename T>
__global__ void __launch_bounds__(32 * WARPS, 4) delta_token_kernel(const Params P)
{
    using L = Shape<RG>;
    constexpr int TB = L::TB;
    const DeltaArgs &a = P.a;
    __shared__ __align__(16) float ks[TB][L::DP], qs[M == AGAIN ? 1 : TB][L::DP];
    // columns: v (FWD, KEEP), do (BACK, AGAIN); e and, in AGAIN, dv
    __shared__ __align__(16) float cs[TB][L::TW];
    __shared__ __align__(16) float es[M >= BACK ? TB : 1][L::TW], ds[M == AGAIN ? TB : 1][L::TW];
    __shared__ float decay[TB], betas[TB];
    __shared__ __align__(16) float red[M >= BACK ? 2 * TB : 1][M >= BACK ? WARPS : 1][RG * ROWS];
    __shared__ float redb[M == BACK ? TB : 1][WARPS];

    const Place p = place(a, P.tiles);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rg = lane / L::QW, qw = lane % L::QW;
    const int r0 = rg * ROWS;
    const int cl = warp * L::WCOLS + 4 * qw;        // column in the tile
    const int c0 = p.tile * L::TW;
    const int c = c0 + cl;
    const int64_t sbase = ((int64_t)p.n * a.H + p.h) * a.D * a.E;
    const int hq = p.h / a.q.hdiv;
    const bool vec = a.E % 4 == 0;

    float4 S[ROWS];
    const float *from = M == BACK ? a.dfin : a.init;
    const bool aligned = vec && (reinterpret_cast<uintptr_t>(from) & 15) == 0;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        S[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (from && r0 + r < a.D) {
            const float *src = from + sbase + (int64_t)(r0 + r) * a.E + c;
            if (aligned) {
                if (c < a.E)
                    S[r] = *reinterpret_cast<const float4 *>(src);
            } else {
                S[r].x = c < a.E ? src[0] : 0.f;
                S[r].y = c + 1 < a.E ? src[1] : 0.f;
                S[r].z = c + 2 < a.E ? src[2] : 0.f;
                S[r].w = c + 3 < a.E ? src[3] : 0.f;
            }
        }
    }

    const T *q = static_cast<const T *>(a.q.p), *k = static_cast<const T *>(a.k.p);
    const Tok &ctok = M >= BACK ? a.d_o : a.v;
    const T *cp = static_cast<const T *>(ctok.p);
    const int64_t tbase = (p.row * a.T + p.bos) * a.H + p.h;     // [B][T][H] index of token 0

    for (int b0 = 0; b0 < p.len; b0 += TB) {
        const int nb = min(TB, p.len - b0);
        // j-th processed token of the batch
        auto token = [&](int j) { return M == BACK ? p.len - 1 - (b0 + j) : b0 + j; };
        __syncthreads();
        for (int i = threadIdx.x; i < nb * RG * ROWS; i += 32 * WARPS) {
            const int j = i / (RG * ROWS), d = i % (RG * ROWS);
            const int64_t t = p.bos + token(j);
            const int at = (d / ROWS) * RPAD + d % ROWS;
            ks[j][at] = d < a.D ? to_f(k[p.row * a.k.sb + t * a.k.st + hq * a.k.sh + d]) : 0.f;
            if constexpr (M != AGAIN)
                if (M != KEEP)
                    qs[j][at] =
                        d < a.D ? a.scale * to_f(q[p.row * a.q.sb + t * a.q.st + hq * a.q.sh + d])
                                : 0.f;
        }
        for (int i = threadIdx.x; i < nb * L::TW; i += 32 * WARPS) {
            const int j = i / L::TW, x = i % L::TW;
            const int64_t t = p.bos + token(j);
            const bool in = c0 + x < a.E;
            cs[j][x] = in ? to_f(cp[p.row * ctok.sb + t * ctok.st + p.h * ctok.sh + c0 + x]) : 0.f;
            if constexpr (M >= BACK) {
                const int64_t at = (tbase + (int64_t)token(j) * a.H) * a.E + c0 + x;
                es[j][x] = in ? P.e[at] : 0.f;
                if constexpr (M == AGAIN)
                    ds[j][x] = in ? P.dvf[at] : 0.f;
            }
        }
        if (threadIdx.x < nb) {
            const int64_t t = p.bos + token(threadIdx.x);
            decay[threadIdx.x] = expf(gate_at(a.g, a.gate_bf16, p.row, t, p.h));
            betas[threadIdx.x] = gate_at(a.beta, a.gate_bf16, p.row, t, p.h);
        }
        __syncthreads();

        for (int j = 0; j < nb; ++j) {
            const int64_t tok = tbase + (int64_t)token(j) * a.H;     // [B][T][H] index
            const float f = decay[j], beta = betas[j];
            const float *kr = &ks[j][rg * RPAD];
            const float4 col = *reinterpret_cast<const float4 *>(&cs[j][cl]);
            if constexpr (M == FWD || M == KEEP) {
                const float4 u = dot_rows<RG>(S, kr);
                const float4 e = make_float4(fmaf(-f, u.x, col.x), fmaf(-f, u.y, col.y),
                                             fmaf(-f, u.z, col.z), fmaf(-f, u.w, col.w));
                rank_one(S, f, kr,
                         make_float4(beta * e.x, beta * e.y, beta * e.z, beta * e.w));
                float4 y = e;
                if constexpr (M == FWD)
                    y = dot_rows<RG>(S, &qs[j][rg * RPAD]);
                if (rg == 0) {
                    const float yy[4] = {y.x, y.y, y.z, y.w};
                    if constexpr (M == FWD) {
                        T *o = static_cast<T *>(a.o.p) + p.row * a.o.sb +
                               (p.bos + token(j)) * a.o.st + p.h * a.o.sh;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (c + i < a.E)
                                o[c + i] = from_f<T>(yy[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (c + i < a.E)
                                P.e[tok * a.E + c + i] = yy[i];
                    }
                }
            } else if constexpr (M == BACK) {
                const float4 e = *reinterpret_cast<const float4 *>(&es[j][cl]);
                rank_one(S, 1.f, &qs[j][rg * RPAD], col);
                const float4 w = dot_rows<RG>(S, kr);
                const float4 dv = make_float4(beta * w.x, beta * w.y, beta * w.z, beta * w.w);
                float dk[ROWS];
#pragma unroll
                for (int r = 0; r < ROWS; ++r)
                    dk[r] = beta * (S[r].x * e.x + S[r].y * e.y + S[r].z * e.z + S[r].w * e.w);
                const int rq = over_quads<RG>(dk, qw);
                float db = w.x * e.x + w.y * e.y + w.z * e.z + w.w * e.w;
#pragma unroll
                for (int m = 1; m < L::QW; m *= 2)
                    db += __shfl_xor_sync(0xffffffffu, db, m);
#pragma unroll
                for (int r = 0; r < ROWS / L::QW; ++r)
                    red[j][warp][r0 + rq + r] = dk[r];
                if (lane == 0)
                    redb[j][warp] = db;
                rank_one(S, 1.f, kr, make_float4(-dv.x, -dv.y, -dv.z, -dv.w));
#pragma unroll
                for (int r = 0; r < ROWS; ++r)
                    S[r] = make_float4(f * S[r].x, f * S[r].y, f * S[r].z, f * S[r].w);
                if (rg == 0) {
                    const float yy[4] = {dv.x, dv.y, dv.z, dv.w};
                    T *o = static_cast<T *>(a.dv.p) + p.row * a.dv.sb +
                           (p.bos + token(j)) * a.dv.st + p.h * a.dv.sh;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c + i < a.E) {
                            o[c + i] = from_f<T>(yy[i]);
                            P.dvf[tok * a.E + c + i] = yy[i];
                        }
                }
            } else {
                const float4 e = *reinterpret_cast<const float4 *>(&es[j][cl]);
                const float4 dv = *reinterpret_cast<const float4 *>(&ds[j][cl]);
                float dk[ROWS], dq[ROWS];
#pragma unroll
                for (int r = 0; r < ROWS; ++r)
                    dk[r] = -f * (S[r].x * dv.x + S[r].y * dv.y + S[r].z * dv.z + S[r].w * dv.w);
                rank_one(S, f, kr,
                         make_float4(beta * e.x, beta * e.y, beta * e.z, beta * e.w));
#pragma unroll
                for (int r = 0; r < ROWS; ++r)
                    dq[r] = a.scale * (S[r].x * col.x + S[r].y * col.y + S[r].z * col.z +
                                       S[r].w * col.w);
                const int rq = over_quads<RG>(dk, qw);
                over_quads<RG>(dq, qw);
#pragma unroll
                for (int r = 0; r < ROWS / L::QW; ++r) {
                    red[j][warp][r0 + rq + r] = dk[r];
                    red[TB + j][warp][r0 + rq + r] = dq[r];
                }
            }
        }
        if constexpr (M >= BACK) {
            __syncthreads();
            const int64_t part = (int64_t)p.tile * a.B * a.T * a.H;
            for (int i = threadIdx.x; i < nb * RG * ROWS; i += 32 * WARPS) {
                const int j = i / (RG * ROWS), d = i % (RG * ROWS);
                if (d >= a.D)
                    continue;
                const int64_t at = (part + tbase + (int64_t)token(j) * a.H) * a.D + d;
                float x = red[j][0][d] + red[j][1][d] + red[j][2][d] + red[j][3][d];
                if constexpr (M == AGAIN) {
                    x += P.dkp[at];     // BACK's part
                    P.dqp[at] = red[TB + j][0][d] + red[TB + j][1][d] + red[TB + j][2][d] +
                                red[TB + j][3][d];
                }
                P.dkp[at] = x;
            }
            if constexpr (M == BACK)
                if (threadIdx.x < nb)
                    P.dbp[part + tbase + (int64_t)token(threadIdx.x) * a.H] =
                        redb[threadIdx.x][0] + redb[threadIdx.x][1] + redb[threadIdx.x][2] +
                        redb[threadIdx.x][3];
        }
    }

    if constexpr (M == AGAIN) {     // <S_end, dS_end>
        float x = 0.f;
        if (a.dfin)
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                if (r0 + r < a.D) {
                    const float *d = a.dfin + sbase + (int64_t)(r0 + r) * a.E + c;
                    x += (c < a.E ? S[r].x * d[0] : 0.f) + (c + 1 < a.E ? S[r].y * d[1] : 0.f) +
                         (c + 2 < a.E ? S[r].z * d[2] : 0.f) + (c + 3 < a.E ? S[r].w * d[3] : 0.f);
                }
#pragma unroll
        for (int m = 1; m < 32; m *= 2)
            x += __shfl_xor_sync(0xffffffffu, x, m);
        __syncthreads();
        if (lane == 0)
            red[0][warp][0] = x;
        __syncthreads();
        if (threadIdx.x == 0)
            P.end[((int64_t)p.tile * a.N + p.n) * a.H + p.h] =
                red[0][0][0] + red[0][1][0] + red[0][2][0] + red[0][3][0];
        return;
    }
    float *to = M == FWD ? a.fin : M == BACK ? a.dinit : nullptr;
    if (!to)
        return;
    const bool out_vec = vec && (reinterpret_cast<uintptr_t>(to) & 15) == 0;
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
        if (r0 + r < a.D) {
            float *dst = to + sbase + (int64_t)(r0 + r) * a.E + c;
            if (out_vec) {
                if (c < a.E)
                    *reinterpret_cast<float4 *>(dst) = S[r];
            } else {
                if (c < a.E)
                    dst[0] = S[r].x;
                if (c + 1 < a.E)
                    dst[1] = S[r].y;
                if (c + 2 < a.E)
                    dst[2] = S[r].z;
                if (c + 3 < a.E)
                    dst[3] = S[r].w;
            }
        }
}

// A warp a (token, query/key head): dq and dk of its value heads and column tiles
// summed, dbeta, and each value head's term of dg's running sum (into dbp's tile 0).
template <typename T> __global__ void __launch_bounds__(128) finish_kernel(const Params P)
{
    const DeltaArgs &a = P.a;
    const int lane = threadIdx.x & 31;
    const int64_t tokens = (int64_t)a.B * a.T;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (id >= tokens * a.HK)
        return;
    const int hk = (int)(id % a.HK);
    const int64_t tok = id / a.HK;
    const int64_t b = tok / a.T, t = tok % a.T;
    const int group = a.H / a.HK;
    const T *q = static_cast<const T *>(a.q.p) + b * a.q.sb + t * a.q.st + hk * a.q.sh;
    float dq[8] = {}, dk[8] = {};
    for (int i = 0; i < group; ++i) {
        const int h = hk * group + i;
        const int64_t th = tok * a.H + h;
        float term = 0.f, db = 0.f;
        for (int x = 0; x < 8; ++x) {
            const int d = x * 32 + lane;
            if (d >= a.D)
                break;
            float sum = 0.f;
            for (int tile = 0; tile < P.tiles; ++tile) {
                const int64_t at = (tile * tokens * a.H + th) * a.D + d;
                sum += P.dqp[at];
                dk[x] += P.dkp[at];
            }
            dq[x] += sum;
            term = fmaf(to_f(q[d]), sum, term);
        }
        const T *v = static_cast<const T *>(a.v.p) + b * a.v.sb + t * a.v.st + h * a.v.sh;
        for (int c = lane; c < a.E; c += 32)
            term = fmaf(-to_f(v[c]), P.dvf[th * a.E + c], term);
        for (int m = 1; m < 32; m *= 2)
            term += __shfl_xor_sync(0xffffffffu, term, m);
        for (int tile = 0; tile < P.tiles; ++tile)
            db += P.dbp[tile * tokens * a.H + th];
        if (lane == 0) {
            static_cast<T *>(a.dbeta)[th] = from_f<T>(db);
            P.dbp[th] = term;
        }
    }
    T *odq = static_cast<T *>(a.dq.p) + b * a.dq.sb + t * a.dq.st + hk * a.dq.sh;
    T *odk = static_cast<T *>(a.dk.p) + b * a.dk.sb + t * a.dk.st + hk * a.dk.sh;
    for (int x = 0; x < 8; ++x) {
        const int d = x * 32 + lane;
        if (d >= a.D)
            break;
        odq[d] = from_f<T>(dq[x]);
        odk[d] = from_f<T>(dk[x]);
    }
}

// A warp a (sequence, head): dg as the running sum of the terms from the last
// token back.  The sum is kept in 64 bits: it runs over the whole sequence, and
// an error of an early (late) term stays in every dg before it.
template <typename T> __global__ void __launch_bounds__(128) dg_kernel(const Params P)
{
    const DeltaArgs &a = P.a;
    const int lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (id >= (int64_t)a.N * a.H)
        return;
    const int h = (int)(id % a.H), n = (int)(id / a.H);
    const int64_t bos = a.cu ? a.cu[n] : (int64_t)n * a.T;
    const int len = a.cu ? a.cu[n + 1] - (int)bos : a.T;
    double run = 0.0;
    for (int tile = 0; tile < P.tiles; ++tile)
        run += P.end[((int64_t)tile * a.N + n) * a.H + h];
    T *dg = static_cast<T *>(a.dg);
    for (int last = len - 1; last >= 0; last -= 32) {
        const int t = last - lane;
        double x = t >= 0 ? (double)P.dbp[(bos + t) * a.H + h] : 0.0;
        for (int m = 1; m < 32; m *= 2) {
            const double y = __shfl_up_sync(0xffffffffu, x, m);
            if (lane >= m)
                x += y;
        }
        if (t >= 0)
            dg[(bos + t) * a.H + h] = from_f<T>((float)(run + x));
        run += __shfl_sync(0xffffffffu, x, 31);
    }
}

int row_groups(int D) { return D <= 64 ? 4 : D <= 128 ? 8 : 16; }
int tiles_of(int D, int E)
{
    const int tw = WARPS * 4 * (32 / row_groups(D));
    return (E + tw - 1) / tw;
}

template <int RG, Mode M> cudaError_t launch(const Params &P, cudaStream_t s)
{
    const int64_t ctas = (int64_t)P.a.N * P.a.H * P.tiles;
    if (ctas > INT32_MAX)
        return cudaErrorNotSupported;
    if (P.a.bf16)
        delta_token_kernel<RG, M, __nv_bfloat16><<<(unsigned)ctas, 32 * WARPS, 0, s>>>(P);
    else
        delta_token_kernel<RG, M, float><<<(unsigned)ctas, 32 * WARPS, 0, s>>>(P);
    note_launch();
    return cudaGetLastError();
}
template <Mode M> cudaError_t launch_by_width(const Params &P, cudaStream_t s)
{
    switch (row_groups(P.a.D)) {
    case 4: return launch<4, M>(P, s);
    case 8: return launch<8, M>(P, s);
    default: return launch<16, M>(P, s);
    }
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// The backward's scratch; base null: its size alone.
size_t lay_out(Params &P, uint8_t *base)
{
    const DeltaArgs &a = P.a;
    const size_t th = (size_t)a.B * a.T * a.H;
    size_t at = 0;
    auto take = [&](float *&p, size_t floats) {
        p = reinterpret_cast<float *>(base + at);
        at += up(floats * sizeof(float));
    };
    take(P.e, th * a.E);
    take(P.dvf, th * a.E);
    take(P.dqp, th * a.D * P.tiles);
    take(P.dkp, th * a.D * P.tiles);
    take(P.dbp, th * P.tiles);
    take(P.end, (size_t)a.N * a.H * P.tiles);
    return at;
}

}  // namespace

cudaError_t delta_token_forward(const DeltaArgs &a, cudaStream_t s)
{
    if (a.N == 0)
        return cudaSuccess;
    Params P{};
    P.a = a;
    P.tiles = tiles_of(a.D, a.E);
    return launch_by_width<FWD>(P, s);
}

size_t delta_token_bwd_bytes(const DeltaArgs &a)
{
    Params P{};
    P.a = a;
    P.tiles = tiles_of(a.D, a.E);
    return lay_out(P, nullptr);
}

cudaError_t delta_token_backward(const DeltaArgs &a, cudaStream_t s)
{
    if (a.N == 0)
        return cudaSuccess;
    Params P{};
    P.a = a;
    P.tiles = tiles_of(a.D, a.E);
    lay_out(P, a.ws);
    cudaError_t e = launch_by_width<KEEP>(P, s);
    if (e == cudaSuccess)
        e = launch_by_width<BACK>(P, s);
    if (e == cudaSuccess)
        e = launch_by_width<AGAIN>(P, s);
    const int64_t rows = (int64_t)a.B * a.T * a.HK, chains = (int64_t)a.N * a.H;
    if (e != cudaSuccess || rows == 0)
        return e;
    if ((rows + 3) / 4 > INT32_MAX)
        return cudaErrorNotSupported;
    if (a.bf16)
        finish_kernel<__nv_bfloat16><<<(unsigned)((rows + 3) / 4), 128, 0, s>>>(P);
    else
        finish_kernel<float><<<(unsigned)((rows + 3) / 4), 128, 0, s>>>(P);
    note_launch();
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    if (a.bf16)
        dg_kernel<__nv_bfloat16><<<(unsigned)((chains + 3) / 4), 128, 0, s>>>(P);
    else
        dg_kernel<float><<<(unsigned)((chains + 3) / 4), 128, 0, s>>>(P);
    note_launch();
    return cudaGetLastError();
}

}  // namespace la
