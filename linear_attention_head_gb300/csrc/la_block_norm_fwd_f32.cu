// la_block_norm_fwd_f32.cu -- the kernels of la_block_norm.cuh by direction and type.
#include "la_block_norm.cuh"

namespace la {

cudaError_t block_norm_fwd_f32(const BlockNormArgs &a, bool vec, int sms, cudaStream_t s, int *ctas)
{
    return norm_by_width<false, float>(a, vec, sms, s, ctas);
}

}  // namespace la
