// la_qk_rope_fwd_f32.cu -- the forward kernels of la_qk_rope.cuh for fp32 tokens (a file of
// their own: they compile side by side).
#include "la_qk_rope.cuh"

namespace la {

cudaError_t rope_fwd_f32(const RopeArgs &a, bool vec, int sms, cudaStream_t s, int *parts)
{
    return rope_of<float, false>(a, vec, sms, s, parts);
}

}  // namespace la
