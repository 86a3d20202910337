// la_qk_rope.cu -- the choice of a kernel for the norms and the rotation
// (la_qk_rope.cuh), and the last sum of the weights' gradients.

#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_bf16.h>

#include "la_internal.h"

namespace la {
namespace {

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
            static_cast<__nv_bfloat16 *>(q.dw)[c] = __float2bfloat16_rn(all);
        else
            static_cast<float *>(q.dw)[c] = all;
    }
}

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

}  // namespace

size_t rope_partial_bytes(int D) { return (size_t)2 * ROPE_MOST_CTAS * D * sizeof(float); }

cudaError_t rope_run(bool back, const RopeArgs &a, cudaStream_t s)
{
    // 8 channels a lane; without norms and rotation there is nothing but a copy,
    // which the kernel of any alignment does
    bool vec = a.D % 8 == 0 && (a.interleaved || a.R % 16 == 0) && (a.R || a.normalize);
    for (const RopeTensor &t : a.t) {
        if (!t.heads)
            continue;
        if (!back || a.normalize)
            vec &= wide(t.x, t.xs, a.bf16);
        if (back)
            vec &= wide(t.dy, t.dys, a.bf16);
        vec &= wide(t.y, t.ys, a.bf16);
    }
    int parts = 0;
    const int n = sms();
    cudaError_t e = back ? (a.bf16 ? rope_bwd_bf16(a, vec, n, s, &parts)
                                   : rope_bwd_f32(a, vec, n, s, &parts))
                         : (a.bf16 ? rope_fwd_bf16(a, vec, n, s, &parts)
                                   : rope_fwd_f32(a, vec, n, s, &parts));
    if (e != cudaSuccess || !back || !(a.t[0].dw || a.t[1].dw))
        return e;
    rope_dw<<<dim3((a.D + 31) / 32, 2), 1024, 0, s>>>(a, parts);
    note_launch();
    return cudaGetLastError();
}

}  // namespace la
