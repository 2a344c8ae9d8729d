// Per-head norm with the position rotation for bfloat16 tensors.
#include "norm_rope.cuh"

namespace thd {

cudaError_t launch_norm_rope_bf16(const NormRopeParams& p, thd_norm_rope_form_t form, bool vec, int num_sms,
                                  cudaStream_t stream) {
  return norm_rope_type<__nv_bfloat16>(p, form, vec, num_sms, stream);
}

}  // namespace thd
