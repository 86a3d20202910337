// la_block_norm_fwd_bf16.cu -- the kernels of la_block_norm.cuh by direction and type.
#include "la_block_norm.cuh"

namespace la {

cudaError_t block_norm_fwd_bf16(const BlockNormArgs &a, bool vec, int sms, cudaStream_t s, int *ctas)
{
    return norm_by_width<false, __nv_bfloat16>(a, vec, sms, s, ctas);
}

}  // namespace la
