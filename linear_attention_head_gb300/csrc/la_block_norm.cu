// la_block_norm.cu -- norms around a block with its gate and residual scale
// (la_block_norm.cuh): the choice of the kernel, and the weights' last sum.

#include "la_internal.h"

#include <cuda_bf16.h>

namespace la {
namespace {

// dw[c] = sum over the CTAs' parts: 32 channels a CTA, 16 warps sharing the parts,
// joined in order.
constexpr int SUM_WARPS = 16;
__global__ void __launch_bounds__(32 * SUM_WARPS) weights_sum_kernel(const float *partial, int ctas,
                                                                    int D, void *post, void *pre,
                                                                    int bf16)
{
    __shared__ float part[SUM_WARPS][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int which = blockIdx.y, c = blockIdx.x * 32 + lane;
    void *out = which ? pre : post;
    if (!out)
        return;
    float s = 0.f;
    if (c < D)
#pragma unroll 8
        for (int k = w; k < ctas; k += SUM_WARPS)
            s += partial[((int64_t)k * 2 + which) * D + c];
    part[w][lane] = s;
    __syncthreads();
    if (w != 0 || c >= D)
        return;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < SUM_WARPS; ++k)
        s += part[k][lane];
    if (bf16)
        static_cast<__nv_bfloat16 *>(out)[c] = __float2bfloat16_rn(s);
    else
        static_cast<float *>(out)[c] = s;
}

bool vec_rows(const NormRows &x, int e)
{
    if (!x.p)
        return true;
    const int m = 16 / e;
    return (reinterpret_cast<uintptr_t>(x.p) & 15) == 0 && x.s[0] % m == 0 && x.s[1] % m == 0 &&
           x.s[2] % m == 0;
}

// Whether x's rows in order (batch, token, head) are a constant step apart, and the step.
bool even_rows(const BlockNormArgs &a, NormRows &x)
{
    const int64_t n[3] = {a.B, a.T, a.H};
    int64_t step = 0, rows = 1;
    bool any = false;
    for (int i = 2; i >= 0; --i) {
        if (n[i] == 1)
            continue;
        if (!any)
            step = x.s[i];
        else if (x.s[i] != step * rows)
            return false;
        any = true;
        rows *= n[i];
    }
    x.step = step;
    return true;
}

}  // namespace

size_t block_norm_partial_bytes(int D) { return (size_t)NORM_MOST_CTAS * 2 * D * sizeof(float); }

cudaError_t block_norm_run(bool back, const BlockNormArgs &args, cudaStream_t s)
{
    BlockNormArgs a = args;
    int dev = 0, sms = 0, ctas = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    const int esz = a.bf16 ? 2 : 4;
    NormRows *rows[] = {&a.x, &a.gate, &a.residual, &a.h, &a.y, &a.dh, &a.dy, &a.dx,
                              &a.dgate, &a.dresidual};
    bool vec = a.D % 8 == 0;
    a.flat = 1;
    for (NormRows *r : rows) {
        vec = vec && vec_rows(*r, esz);
        a.flat = even_rows(a, *r) && a.flat;
    }
    for (const void *w : {a.post, a.pre})
        vec = vec && (reinterpret_cast<uintptr_t>(w) & 15) == 0;
    if (!back)
        return a.bf16 ? block_norm_fwd_bf16(a, vec, sms, s, &ctas)
                      : block_norm_fwd_f32(a, vec, sms, s, &ctas);
    e = a.bf16 ? block_norm_bwd_bf16(a, vec, sms, s, &ctas)
               : block_norm_bwd_f32(a, vec, sms, s, &ctas);
    if (e != cudaSuccess || !(a.dpost || a.dpre))
        return e;
    weights_sum_kernel<<<dim3((unsigned)(a.D + 31) / 32, 2), 32 * SUM_WARPS, 0, s>>>(
        a.partial, ctas, a.D, a.dpost, a.dpre, a.w_bf16);
    note_launch();
    return cudaGetLastError();
}

}  // namespace la
