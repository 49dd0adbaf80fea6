// Host side of fkv_tree_attn: which kernel runs a call, its workspace, and the
// parameters that the kernels share.
#include "tc_device.cuh"
#include "tree_common.cuh"

namespace fkv {
namespace {

// The tensor-core kernels: bf16 and 4-bit caches.
bool tree_tc_plan(const TreeArgs& a, int num_sms, TreePlan* plan) {
  const int rows = a.group * a.T, nsrc = a.k[1] ? 2 : 1;
  plan->rows = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  if (plan->rows == 128 && (a.q4 || (nsrc == 2 && a.head_dim > 64))) plan->rows = 64;
  // fewer columns a CTA until the tiles that the products need fit beside them
  // (4-bit fused caches of 128 channels; batches of hundreds)
  for (;;) {
    plan->row_tiles = (rows + plan->rows - 1) / plan->rows;
    switch (a.head_dim) {
      case 64: tree_tc_size_64(a, plan); break;
      case 80: tree_tc_size_80(a, plan); break;
      case 96: tree_tc_size_96(a, plan); break;
      default: tree_tc_size_128(a, plan); break;
    }
    if (plan->slots > 0) break;
    if (plan->rows == 16) return false;
    plan->rows /= 2;
  }
  // one CTA an SM over ranges and row tiles; the device takes fewer ranges
  // where there are fewer key tiles
  plan->ranges = a.num_ctas > 0 ? a.num_ctas : num_sms / plan->row_tiles > 0 ? num_sms / plan->row_tiles : 1;
  plan->tensor = true;
  return true;
}

cudaError_t tree_tc_launch(const TreeParams& p, const TreeArgs& a, const TreePlan& plan, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return tree_tc_run_64(p, a, plan, stream);
    case 80: return tree_tc_run_80(p, a, plan, stream);
    case 96: return tree_tc_run_96(p, a, plan, stream);
    default: return tree_tc_run_128(p, a, plan, stream);
  }
}

}  // namespace

// Tensor maps of a bf16 plane: `planes` times `rows` rows of D elements.
bool tile_maps(TileMaps* m, const void* base, int D, int rows, long long planes) {
  static_assert(sizeof(CUtensorMap) == sizeof(m->full) && alignof(TileMaps) >= alignof(CUtensorMap), "tensor map");
  const size_t plane = (size_t)rows * D * 2;
  m->valid = make_map_box(reinterpret_cast<CUtensorMap*>(m->full), base, D, rows, planes, plane, 64,
                          kTreeKeyTile, CU_TENSOR_MAP_SWIZZLE_128B) &&
             make_map_box(reinterpret_cast<CUtensorMap*>(m->tail), base, D, rows, planes, plane, 64,
                          kTreeTailRows, CU_TENSOR_MAP_SWIZZLE_128B);
  return m->valid;
}

cudaError_t tree_plan(const TreeArgs& a, int num_sms, TreePlan* plan) {
  if (a.is_f32) tree_f32_plan(a, num_sms, plan);
  else if (!tree_tc_plan(a, num_sms, plan)) return cudaErrorNotSupported;
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
  return plan.tensor ? tree_tc_launch(p, a, plan, stream) : tree_f32_launch(p, a, plan, stream);
}

}  // namespace fkv
