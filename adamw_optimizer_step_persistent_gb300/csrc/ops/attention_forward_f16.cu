// Attention forward, fp16 instances.
#include "attention_forward.cuh"

namespace fadam_ops {
fadam_status attention_forward_f16(const ForwardMaps& maps, const AttentionArgs& g, cudaStream_t stream) {
  return forward_of<F16>(maps, g, stream);
}
}  // namespace fadam_ops
