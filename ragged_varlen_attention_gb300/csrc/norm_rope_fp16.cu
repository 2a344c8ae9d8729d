// Per-head norm with the position rotation for float16 tensors.
#include "norm_rope.cuh"

namespace thd {

cudaError_t launch_norm_rope_fp16(const NormRopeParams& p, thd_norm_rope_form_t form, bool vec, int num_sms,
                                  cudaStream_t stream) {
  return norm_rope_type<__half>(p, form, vec, num_sms, stream);
}

}  // namespace thd
