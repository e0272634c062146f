// Attention backward, fp16 instances.
#include "attention_backward.cuh"

namespace fadam_ops {
fadam_status attention_backward_f16(const BackwardMaps& maps, const AttentionArgs& g, cudaStream_t stream) {
  return backward_of<F16>(maps, g, stream);
}
}  // namespace fadam_ops
