// la_delta_tc.cu -- the gated delta rule in chunks on the tensor cores (none yet:
// every call runs token by token).
#include "la_internal.h"

namespace la {

bool delta_tc_sized(const DeltaArgs &) { return false; }
bool delta_tc_row_ok(const void *, const int64_t *, int, int, int) { return false; }
size_t delta_tc_saved_bytes(const DeltaArgs &) { return 0; }
size_t delta_tc_fwd_bytes(const DeltaArgs &, bool) { return 0; }
size_t delta_tc_bwd_bytes(const DeltaArgs &) { return 0; }
cudaError_t delta_tc_forward(const DeltaArgs &, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t delta_tc_backward(const DeltaArgs &, cudaStream_t) { return cudaErrorNotSupported; }

}  // namespace la
