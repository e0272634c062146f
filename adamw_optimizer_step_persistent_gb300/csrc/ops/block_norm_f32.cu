// Block norms, fp32 blocks.
#include "block_norm.cuh"

namespace fadam_ops {

fadam_status norm_forward_f32(const NormArgs& a, cudaStream_t stream) {
  return norm_forward<float, float>(a, stream);
}

fadam_status norm_backward_f32(const NormGradArgs& a, cudaStream_t stream) {
  return norm_backward<float, float>(a, stream);
}

}  // namespace fadam_ops
