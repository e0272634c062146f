// Block norms, bf16 blocks.
#include "block_norm.cuh"

namespace fadam_ops {

fadam_status norm_forward_bf16(const NormArgs& a, bool residual_f32, cudaStream_t stream) {
  return residual_f32 ? norm_forward<__nv_bfloat16, float>(a, stream)
                      : norm_forward<__nv_bfloat16, __nv_bfloat16>(a, stream);
}

fadam_status norm_backward_bf16(const NormGradArgs& a, bool residual_f32, cudaStream_t stream) {
  return residual_f32 ? norm_backward<__nv_bfloat16, float>(a, stream)
                      : norm_backward<__nv_bfloat16, __nv_bfloat16>(a, stream);
}

}  // namespace fadam_ops
