// Host side of fkv_tree_attn: which kernel runs a call, its workspace, and the
// parameters that the kernels share.
#include "tree_common.cuh"

namespace fkv {

cudaError_t tree_plan(const TreeArgs& a, int num_sms, TreePlan* plan) {
  if (!tree_tc_plan(a, num_sms, plan)) tree_simt_plan(a, num_sms, plan);
  // two partial records per range and row tile, then the arrival words
  plan->partial_bytes = (size_t)plan->ranges * 2 * plan->row_tiles *
                        tree_record_floats(plan->rows, a.head_dim) * sizeof(float);
  plan->workspace_bytes =
      plan->partial_bytes + (size_t)a.batch * a.kv_heads * plan->row_tiles * sizeof(unsigned long long);
  return cudaSuccess;
}

cudaError_t tree_launch(const TreeArgs& a, const TreePlan& plan, cudaStream_t stream) {
  TreeParams p{};
  for (int i = 0; i < 2; ++i) {
    p.k[i] = a.k[i];
    p.v[i] = a.v[i];
    p.a[i] = a.a[i];
    p.b[i] = a.b[i];
  }
  p.q = a.q;
  p.out = a.out;
  p.seq_lens = a.seq_lens;
  p.node_counts = a.node_counts;
  p.mask = a.mask;
  p.ws = static_cast<float*>(a.workspace);
  p.counters = reinterpret_cast<unsigned long long*>(static_cast<char*>(a.workspace) + plan.partial_bytes);
  p.status = a.status;
  p.wait_limit = a.wait_limit;
  p.B = a.batch;
  p.H = a.kv_heads;
  p.G = a.group;
  p.S_max = a.max_seq;
  p.T = a.T;
  p.words = (a.T + 63) / 64;
  p.window = a.window;
  p.ring = a.ring;
  p.row_tiles = plan.row_tiles;
  // an odd multiple keeps tags distinct and unlike the small numbers that a
  // recycled workspace may hold
  p.epoch = a.epoch * 0x9E3779B1u;
  p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  return plan.tensor ? tree_tc_launch(p, a, plan, stream) : tree_simt_launch(p, a, plan, stream);
}

}  // namespace fkv
