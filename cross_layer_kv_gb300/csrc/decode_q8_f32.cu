// Decode over 8-bit caches in fp32 contexts.
#include "decode_q8_impl.cuh"

namespace fkv {

cudaError_t decode_q8_launch_f32(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t stream) {
  return q8_by_dim<float>(a, plan, stream);
}

}  // namespace fkv
