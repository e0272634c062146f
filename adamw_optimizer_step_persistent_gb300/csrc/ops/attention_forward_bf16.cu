// Attention forward, bf16 instances.
#include "attention_forward.cuh"

namespace fadam_ops {
fadam_status attention_forward_bf16(const ForwardMaps& maps, const AttentionArgs& g, cudaStream_t stream) {
  return forward_of<BF16>(maps, g, stream);
}
}  // namespace fadam_ops
