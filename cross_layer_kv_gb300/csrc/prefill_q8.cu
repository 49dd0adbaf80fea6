// Prefill over 8-bit caches: dispatch by head dimension and source count.
#include "prefill_q8_impl.cuh"

namespace fkv {
namespace {

template <int D>
cudaError_t by_src(const PrefillArgs& a, cudaStream_t stream) {
  return a.nsrc == 2 ? q8p::launch<D, 2>(a, stream) : q8p::launch<D, 1>(a, stream);
}

}  // namespace

cudaError_t prefill_q8_launch(const PrefillArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return by_src<64>(a, stream);
    case 80: return by_src<80>(a, stream);
    case 96: return by_src<96>(a, stream);
    case 128: return by_src<128>(a, stream);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace fkv
