// Block norms, f16 blocks.
#include "block_norm.cuh"

namespace fadam_ops {

fadam_status norm_forward_f16(const NormArgs& a, bool residual_f32, cudaStream_t stream) {
  return residual_f32 ? norm_forward<__half, float>(a, stream)
                      : norm_forward<__half, __half>(a, stream);
}

fadam_status norm_backward_f16(const NormGradArgs& a, bool residual_f32, cudaStream_t stream) {
  return residual_f32 ? norm_backward<__half, float>(a, stream)
                      : norm_backward<__half, __half>(a, stream);
}

}  // namespace fadam_ops
