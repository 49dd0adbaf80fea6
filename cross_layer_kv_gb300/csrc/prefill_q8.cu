// Prefill over 8-bit caches: dispatch by head dimension and source count; the
// kernels of D = 64 and 80 (those of D = 96 and 128 compile beside them, in
// prefill_q8_96.cu).
#include "prefill_q8_impl.cuh"

namespace fkv {

cudaError_t prefill_q8_launch_96(const PrefillArgs& a, cudaStream_t stream);

cudaError_t prefill_q8_launch(const PrefillArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return a.nsrc == 2 ? q8p::launch<64, 2>(a, stream) : q8p::launch<64, 1>(a, stream);
    case 80: return a.nsrc == 2 ? q8p::launch<80, 2>(a, stream) : q8p::launch<80, 1>(a, stream);
    default: return prefill_q8_launch_96(a, stream);
  }
}

}  // namespace fkv
