// The tensor-core tree attention kernels for head dimension 64.
#include "tree_tc_impl.cuh"

namespace fkv {

void tree_tc_size_64(const TreeArgs& a, TreePlan* plan) { tree_tc_size<64>(a, plan); }

cudaError_t tree_tc_run_64(const TreeParams& p, const TreeArgs& a, const TreePlan& plan, cudaStream_t stream) {
  return tree_tc_run<64>(p, a, plan, stream);
}

}  // namespace fkv
