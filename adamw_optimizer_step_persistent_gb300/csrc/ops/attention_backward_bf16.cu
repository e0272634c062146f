// Attention backward, bf16 instances.
#include "attention_backward.cuh"

namespace fadam_ops {
fadam_status attention_backward_bf16(const BackwardMaps& maps, const AttentionArgs& g, cudaStream_t stream) {
  return backward_of<BF16>(maps, g, stream);
}
}  // namespace fadam_ops
