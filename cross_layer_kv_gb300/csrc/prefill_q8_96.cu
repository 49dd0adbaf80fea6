// Prefill over 8-bit caches with D = 96 and 128.
#include "prefill_q8_impl.cuh"

namespace fkv {

cudaError_t prefill_q8_launch_96(const PrefillArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 96: return a.nsrc == 2 ? q8p::launch<96, 2>(a, stream) : q8p::launch<96, 1>(a, stream);
    case 128: return a.nsrc == 2 ? q8p::launch<128, 2>(a, stream) : q8p::launch<128, 1>(a, stream);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace fkv
