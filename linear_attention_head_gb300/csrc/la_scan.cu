// la_scan.cu -- the gated linear recurrence, elementwise per (sequence, head,
// channel):
//     s_t = exp(g_t) s_{t-1} + x_t,   o_t = s_t
// and its backward.  With K_t = exp(g_t) G_t, G_t = dL/ds_t:
//     G_t = do_t + K_{t+1},   dx_t = G_t,   dg_t = K_t s_{t-1},
// K after the last token being the final state's gradient, K at the first
// token the initial state's.
//
// One thread per (sequence, channel) walks the sequence token by token.  The
// backward computes s_{t-1} again, a tile at a time from the state that
// entered the tile.

#include <cstdint>

#include <cuda_bf16.h>

#include "la_internal.h"

namespace la {
namespace {

template <typename T> __device__ __forceinline__ float ldt(const T *p);
template <> __device__ __forceinline__ float ldt<float>(const float *p) { return *p; }
template <> __device__ __forceinline__ float ldt<__nv_bfloat16>(const __nv_bfloat16 *p)
{
    return __bfloat162float(*p);
}
template <typename T> __device__ __forceinline__ void stt(T *p, float x);
template <> __device__ __forceinline__ void stt<float>(float *p, float x) { *p = x; }
template <> __device__ __forceinline__ void stt<__nv_bfloat16>(__nv_bfloat16 *p, float x)
{
    *p = __float2bfloat16_rn(x);
}

// exp(g).  Near 0 the decay is 1 + expm1(g) by its Taylor series (the next
// term, g^6 / 720, is below 2^-27 of 1 for |g| < 1/8): the last addition is
// the only rounding of the size of the result, and it has no preferred sign.
// expf's error, although below one unit in the last place, does, and a
// channel that remembers thousands of tokens adds it up once a token: 1.1e-5
// of the final state at 8192 tokens against 2e-6.  Larger |g| forget within a
// few tokens.
__device__ __forceinline__ float decay(float g)
{
    float p = fmaf(g, 1.f / 120.f, 1.f / 24.f);
    p = fmaf(g, p, 1.f / 6.f);
    p = fmaf(g, p, 0.5f);
    p = fmaf(g * g, p, g);
    return fabsf(g) < 0.125f ? 1.f + p : expf(g);
}

struct Seq {
    int64_t row, bos, len, p0;   // batch row, first token, tokens, first processing position
};

__device__ __forceinline__ Seq seq_of(const ScanArgs &a, int n)
{
    Seq s;
    if (a.cu) {
        s.row = 0;
        s.bos = a.cu[n];
        s.len = (int64_t)a.cu[n + 1] - s.bos;
        s.p0 = a.reverse ? (int64_t)a.T - a.cu[n + 1] : s.bos;
    } else {
        s.row = n;
        s.bos = 0;
        s.len = a.T;
        s.p0 = (int64_t)n * a.T;
    }
    return s;
}

__device__ __forceinline__ int64_t at(const ScanArgs &a, const Seq &s, int64_t j, int64_t sb,
                                      int64_t st)
{
    return s.row * sb + (s.bos + (a.reverse ? s.len - 1 - j : j)) * st;
}

template <typename T, typename TG> __global__ void __launch_bounds__(128) scan_fwd(ScanArgs a)
{
    const int64_t C = (int64_t)a.H * a.D;
    const unsigned parts = (unsigned)((C + 127) / 128);   // CTAs per sequence
    const int64_t c = (int64_t)(blockIdx.x % parts) * 128 + threadIdx.x;
    if (c >= C)
        return;
    const int n = (int)(blockIdx.x / parts), h = (int)(c / a.D), d = (int)(c % a.D);
    const Seq sq = seq_of(a, n);
    const T *x = static_cast<const T *>(a.x.p) + h * a.x.sh + d;
    const TG *g = static_cast<const TG *>(a.g.p) + h * a.g.sh + d;
    T *o = static_cast<T *>(a.o.p) + h * a.o.sh + d;
    float s = a.init ? a.init[n * C + c] : 0.f;
    for (int64_t j = 0; j < sq.len; ++j) {
        if (a.states && (sq.p0 + j) % SCAN_TILE == 0)
            a.states[(sq.p0 + j) / SCAN_TILE * C + c] = s;
        s = fmaf(decay(ldt(g + at(a, sq, j, a.g.sb, a.g.st))), s,
                 ldt(x + at(a, sq, j, a.x.sb, a.x.st)));
        if (a.o.p)
            stt(o + at(a, sq, j, a.o.sb, a.o.st), s);
    }
    if (a.fin)
        a.fin[n * C + c] = s;
}

template <typename T, typename TG> __global__ void __launch_bounds__(128) scan_bwd(ScanArgs a)
{
    const int64_t C = (int64_t)a.H * a.D;
    const unsigned parts = (unsigned)((C + 127) / 128);   // CTAs per sequence
    const int64_t c = (int64_t)(blockIdx.x % parts) * 128 + threadIdx.x;
    if (c >= C)
        return;
    const int n = (int)(blockIdx.x / parts), h = (int)(c / a.D), d = (int)(c % a.D);
    const Seq sq = seq_of(a, n);
    const T *x = static_cast<const T *>(a.x.p) + h * a.x.sh + d;
    const TG *g = static_cast<const TG *>(a.g.p) + h * a.g.sh + d;
    const T *d_o = static_cast<const T *>(a.d_o.p) + h * a.d_o.sh + d;
    T *dx = static_cast<T *>(a.dx.p) + h * a.dx.sh + d;
    TG *dg = static_cast<TG *>(a.dg.p) + h * a.dg.sh + d;
    float K = a.dfin ? a.dfin[n * C + c] : 0.f;
    float prev[SCAN_TILE];   // the states before the tile's tokens
    for (int64_t end = sq.len; end > 0;) {
        const int64_t tile = (sq.p0 + end - 1) / SCAN_TILE;
        int64_t begin = tile * SCAN_TILE - sq.p0;
        float s = begin >= 0 && a.states ? a.states[tile * C + c] : 0.f;
        if (begin <= 0) {
            begin = 0;
            s = a.init ? a.init[n * C + c] : 0.f;
        }
        for (int64_t j = begin; j < end; ++j) {
            prev[j - begin] = s;
            s = fmaf(decay(ldt(g + at(a, sq, j, a.g.sb, a.g.st))), s,
                     ldt(x + at(a, sq, j, a.x.sb, a.x.st)));
        }
        for (int64_t j = end - 1; j >= begin; --j) {
            const float G = ldt(d_o + at(a, sq, j, a.d_o.sb, a.d_o.st)) + K;
            K = decay(ldt(g + at(a, sq, j, a.g.sb, a.g.st))) * G;
            stt(dx + at(a, sq, j, a.dx.sb, a.dx.st), G);
            stt(dg + at(a, sq, j, a.dg.sb, a.dg.st), K * prev[j - begin]);
        }
        end = begin;
    }
    if (a.dinit)
        a.dinit[n * C + c] = K;
}

bool grid_of(const ScanArgs &a, unsigned *grid)
{
    const int64_t ctas = ((int64_t)a.H * a.D + 127) / 128 * a.N;
    *grid = (unsigned)ctas;
    return ctas <= 0x7fffffff;
}

}  // namespace

cudaError_t scan_forward(const ScanArgs &a, cudaStream_t s)
{
    unsigned grid;
    if (!grid_of(a, &grid))
        return cudaErrorNotSupported;
    if (a.bf16 && a.gate_bf16)
        scan_fwd<__nv_bfloat16, __nv_bfloat16><<<grid, 128, 0, s>>>(a);
    else if (a.bf16)
        scan_fwd<__nv_bfloat16, float><<<grid, 128, 0, s>>>(a);
    else
        scan_fwd<float, float><<<grid, 128, 0, s>>>(a);
    note_launch();
    return cudaGetLastError();
}

cudaError_t scan_backward(const ScanArgs &a, cudaStream_t s)
{
    unsigned grid;
    if (!grid_of(a, &grid))
        return cudaErrorNotSupported;
    if (a.bf16 && a.gate_bf16)
        scan_bwd<__nv_bfloat16, __nv_bfloat16><<<grid, 128, 0, s>>>(a);
    else if (a.bf16)
        scan_bwd<__nv_bfloat16, float><<<grid, 128, 0, s>>>(a);
    else
        scan_bwd<float, float><<<grid, 128, 0, s>>>(a);
    note_launch();
    return cudaGetLastError();
}

}  // namespace la
