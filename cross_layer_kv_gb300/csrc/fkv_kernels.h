// Host-visible launch interfaces of the FusedKV kernels (internal to the
// library; the public ABI is include/fusedkv.h).
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/fusedkv.h"

namespace fkv {

// Default limit of every bounded device wait (a context's wait-limit word
// starts here; only the failure-path tests lower it).
constexpr unsigned long long kWaitLimitNs = 1000000000ull;  // 1 s

// One decode attention call, after host validation.  Pointers are device
// pointers.  nsrc = 1: K from k[0], V from v[0] (vanilla or lite);
// nsrc = 2: fused, K = a0 (.) k[0] + a1 (.) k[1], V = b0 (.) v[0] + b1 (.) v[1].
struct DecodeArgs {
  const void* k[2];
  const void* v[2];
  const float* a[2];
  const float* b[2];
  const void* q;             // [B, H_q, D]
  void* out;                 // [B, H_q, D]
  const int32_t* seq_lens;   // [B]
  float* workspace;          // split partials
  int* status;               // device status word
  const unsigned long long* wait_limit;  // device word: limit of the bounded waits (ns)
  int batch, kv_heads, group, max_seq, head_dim;
  int nsrc;
  int is_f32;
  float softmax_scale;
  int num_ctas;              // split grid (0 = library default)
  int window;                // > 0: attend only to the last `window` rows
  int ring;                  // > 0: the source caches are rings of this many rows per
                             // unit (position t at row t % ring); 0: S_max rows, row = position
  unsigned epoch;            // distinct per call (tags the unit arrival counts)
  const float* k_scale[2];   // scales of 8-bit sources
  const float* v_scale[2];
  int device;
};

// Launch configuration the library picks for a decode call shape.
struct DecodePlan {
  int ctas;          // CTAs of the split kernel
  int warps_per_cta;
  size_t smem_bytes;
  size_t partial_bytes;    // split partials, then one 8-byte arrival word per unit
  size_t workspace_bytes;
};

// Plan (grid and workspace) for a shape; num_sms from the device.
cudaError_t decode_plan(const DecodeArgs& a, int num_sms, DecodePlan* plan);

// Launch the decode kernel on `stream`.
cudaError_t decode_launch(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t stream);

// Number of kernel launches one decode call makes (for launch accounting).
constexpr int kDecodeLaunchesPerCall = 1;

// Launch `kern` with programmatic stream serialization (see grid_dep_wait).
template <typename Kern, typename... Args>
cudaError_t launch_pdl(Kern kern, dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

struct AppendArgs {
  void* k_cache;
  void* v_cache;
  const void* k_new;
  const void* v_new;
  const int32_t* pos;
  int* status;
  int batch, kv_heads, max_seq, head_dim, T, elem_bytes;
  int ring;        // > 0: the cache is a ring of this many rows per unit (row = position % ring)
  float* k_scale;  // scales of an 8-bit cache
  float* v_scale;
};

cudaError_t append_launch(const AppendArgs& a, cudaStream_t stream);

// 4-bit caches: rows of q4_row_bytes(D) bytes (codes, then bf16 (scale, min)
// per group of kQ4Group channels, padded to 16 bytes).
constexpr int kQ4Group = 16;
__host__ __device__ constexpr int q4_row_bytes(int head_dim) {
  return (head_dim / 2 + head_dim / 4 + 15) / 16 * 16;
}
cudaError_t append_q4_launch(const AppendArgs& a, cudaStream_t stream);
cudaError_t decode_q4_launch(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t stream);
cudaError_t decode_q4_plan(const DecodeArgs& a, int num_sms, DecodePlan* plan);

// How a layer's cache holds its rows: elements of the context's type, 4-bit
// records, or 8-bit codes with scales.
enum CacheFormat { kCachePlain = 0, kCacheQ4 = 1, kCacheQ8 = 2 };

// 8-bit caches: e4m3 codes, and one fp32 scale per kQ8Block rows of a
// (sequence, KV head); a unit's scales are padded to whole 16-byte pieces.
constexpr int kQ8Block = 32;
constexpr int kQ8MinExp = -100, kQ8MaxExp = 119;   // of the scales that the append chooses
__host__ __device__ constexpr int q8_scale_cols(int rows) {
  return (rows / kQ8Block + (rows % kQ8Block ? 1 : 0) + 3) / 4 * 4;
}
cudaError_t append_q8_launch(const AppendArgs& a, cudaStream_t stream);
cudaError_t decode_q8_launch(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t stream);
cudaError_t decode_q8_plan(const DecodeArgs& a, int num_sms, DecodePlan* plan);

// One fkv_read_kv call, after host validation: sources and weights as in
// DecodeArgs.
struct ReadArgs {
  const void* k[2];
  const void* v[2];
  const float* a[2];
  const float* b[2];
  const float* k_scale[2];
  const float* v_scale[2];
  const int32_t* pos;   // [B]
  void* k_out;          // [B, H_kv, T, D]
  void* v_out;
  int* status;
  int batch, kv_heads, max_seq, head_dim, T;
  int nsrc, is_f32, format;
  int ring;
};
cudaError_t read_launch(const ReadArgs& a, cudaStream_t stream);

constexpr int kDevTimeoutBit = 2;  // must match kDevTimeout

struct PrefillArgs {
  const void* k[2];
  const void* v[2];
  const float* a[2];
  const float* b[2];
  const void* q;   // [B, H_q, S, D] bf16
  void* out;       // [B, H_q, S, D] bf16
  int* status;
  const unsigned long long* wait_limit;  // device word: limit of the bounded waits (ns)
  int batch, kv_heads, group, max_seq, head_dim, S;
  int q_start;     // cache position of query row 0 (0 for a whole prompt)
  int window;      // > 0: sliding window of that many positions
  int plane_rows;  // cache rows per (b, kv-head) unit (S_max, or a ring's rows)
  int ring;        // > 0: the caches are rings of that many rows (position t at row
                   // t % ring), a multiple of the kernel's key tile once positions wrap
  int nsrc;
  float softmax_scale;
  const float* k_scale[2];   // scales of 8-bit sources
  const float* v_scale[2];
  int device, num_sms;       // (8-bit caches: num_sms, how far a short chunk's keys are split)
};

// Returns cudaErrorNotSupported for shapes the tensor-core kernels do not
// cover.  One source (nsrc = 1) runs the 128-key kernel of prefill_wide.cu;
// two sources (fused) with D <= 96 the 112-key kernel of
// prefill_fused_wide.cu (Q in tensor memory), and with D = 128 the 64-key
// kernel of prefill.cu.
cudaError_t prefill_launch(const PrefillArgs& a, cudaStream_t stream);
cudaError_t prefill_wide_launch(const PrefillArgs& a, cudaStream_t stream);
cudaError_t prefill_fused_wide_launch(const PrefillArgs& a, cudaStream_t stream);
// Prefill over 8-bit caches, one source or two (prefill_q8_impl.cuh).
cudaError_t prefill_q8_launch(const PrefillArgs& a, cudaStream_t stream);

// What a kernel needs once per device before its first launch: its dynamic
// shared memory raised to `smem` bytes and, for kernels that split their
// registers by warpgroup, a launch allocation of at least `regs` registers
// (cudaErrorNotSupported otherwise).  One object per kernel; later calls are
// one load.
struct KernelReady {
  std::atomic<unsigned long long> devices{0};
  template <typename Kern>
  cudaError_t check(Kern kern, int device, int smem, int threads, int regs) {
    const unsigned long long bit = device >= 0 && device < 64 ? 1ull << device : 0;
    if (bit && (devices.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (regs > 0) {
      cudaFuncAttributes fa;
      e = cudaFuncGetAttributes(&fa, kern);
      if (e != cudaSuccess) return e;
      if ((long long)fa.numRegs * threads < regs) return cudaErrorNotSupported;
    }
    devices.fetch_or(bit, std::memory_order_release);
    return cudaSuccess;
  }
};

// Tensor maps of one bound bf16 plane as the tree kernels read it (boxes of a
// whole key tile and of a ragged tile's rows), made when the buffer is bound.
struct TileMaps {
  alignas(128) unsigned char full[128];
  alignas(128) unsigned char tail[128];
  bool valid;
};
bool tile_maps(TileMaps* m, const void* base, int D, int rows, long long planes);

// One fkv_tree_attn call, after host validation.
struct TreeArgs {
  const TileMaps* k_maps[2];   // of the sources (bf16 caches)
  const TileMaps* v_maps[2];
  int device;
  const void* k[2];          // second source null unless fused
  const void* v[2];
  const float* a[2];         // null for vanilla and lite
  const float* b[2];
  const void* q;             // [B, H_q, T, D]
  void* out;                 // [B, H_q, T, D]
  const int32_t* seq_lens;
  const int32_t* node_counts;      // may be null
  const unsigned long long* mask;  // [B, T, ceil(T / 64)]
  void* workspace;
  int* status;
  const unsigned long long* wait_limit;
  int batch, kv_heads, group, max_seq, head_dim, T;
  int is_f32, q4;
  int window, ring;
  int num_ctas;              // > 0: that many key ranges
  float softmax_scale;
  unsigned epoch;            // distinct per call
};

// Launch configuration of a tree attention call.
struct TreePlan {
  bool tensor;      // the tensor-core kernel (tree_tc_impl.cuh), else tree_f32.cu
  int slots;        // its key / value tile slots
  int raw_slots;    // its slots of 4-bit records
  int ranges;       // key ranges (grid.x)
  int rows;         // query rows per CTA
  int row_tiles;    // grid.y
  size_t smem_bytes;
  size_t partial_bytes;    // partials, then one 8-byte arrival word per unit and row tile
  size_t workspace_bytes;
};

cudaError_t tree_plan(const TreeArgs& a, int num_sms, TreePlan* plan);
cudaError_t tree_launch(const TreeArgs& a, const TreePlan& plan, cudaStream_t stream);

// The planes that one launch of compact or reorder moves rows in: the K or V
// caches of a layer, `rows` rows of row_bytes bytes per (sequence, KV head).
constexpr int kMovePlanes = 128;
struct MoveTable {
  void* plane[kMovePlanes];
  int rows[kMovePlanes];
  int row_bytes[kMovePlanes];
  int planes;
};

struct CompactArgs {
  const int32_t* pos;      // [B]
  const int32_t* idx;      // [B, A]
  const int32_t* counts;   // [B]
  int* status;
  int batch, kv_heads, max_seq, A;
  int min_rows;            // fewest rows of any bound layer's planes
  int cols;                // 16-byte columns per CTA (set by the launch)
};

struct ReorderArgs {
  const int32_t* src;        // [B]
  const int32_t* seq_lens;   // [B]
  int* status;
  const unsigned long long* wait_limit;
  int batch, kv_heads, max_seq, device;
};

constexpr int kMaxAccepted = 128;   // rows a sequence may compact in one call

cudaError_t compact_launch(const MoveTable& tb, CompactArgs a, cudaStream_t stream);
cudaError_t reorder_launch(const MoveTable& tb, const ReorderArgs& a, int num_sms,
                           cudaStream_t stream);

// The body of fkv_decode_attn (api.cu); clear_counts zeroes the call's unit
// arrival words on the stream before the launch.  Internal to the library.
__attribute__((visibility("hidden"))) fkv_status decode_attn_impl(
    fkv_ctx* c, const void* q, int layer, int mode, const int32_t* seq_lens, void* out,
    void* workspace, size_t workspace_bytes, void* stream, bool clear_counts);

}  // namespace fkv
