// la_qk_rope_bwd_bf16.cu -- the backward kernels of la_qk_rope.cuh for bf16 tokens (a file of
// their own: they compile side by side).
#include "la_qk_rope.cuh"

namespace la {

cudaError_t rope_bwd_bf16(const RopeArgs &a, bool vec, int sms, cudaStream_t s, int *parts)
{
    return rope_of<__nv_bfloat16, true>(a, vec, sms, s, parts);
}

}  // namespace la
