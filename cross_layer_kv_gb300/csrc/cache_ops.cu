// Moving cached rows: fkv_compact_rows (the accepted nodes of a drafted tree
// close up behind the committed prefix) and fkv_reorder_seqs (sequences become
// copies of others: forked beams, shared prompts).  Both move bytes, whatever
// the cache format, in every bound layer with one launch for up to
// kMovePlanes planes (K or V of a layer).
#include "fkv_device.cuh"
#include "fkv_kernels.h"

namespace fkv {
namespace {

// --- fkv_compact_rows ---------------------------------------------------------
//
// A unit is the rows of one (plane, sequence, KV head).  Row pos + j
// takes row pos + idx[j], j < count: a group of threads loads all of the
// unit's chunks (16 bytes each) into registers, meets, and stores them, so
// that any order of idx, with repeats, gives what the old rows held.  The call
// moves kilobytes to a few megabytes and is bound by the latency of its three
// dependent accesses (idx, load, store).  A group is a warp where the unit's
// chunks fit 8 a lane, else a CTA of 128 threads that splits wide rows by
// columns (a move keeps the column, so columns are independent).  Measured:
// 332M, 32 sequences, up to 5 rows 3.8 us on the device; 4B, 8 sequences, up
// to 12 rows of 18 layers 5.3 us; calls from Python one after another 6 to 7 us,
// the host's time.

constexpr int kMoveThreads = 128;
constexpr int kMoveItems = 8;   // chunks a thread holds

template <bool WARP>
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const __grid_constant__ MoveTable tb,
                                                               const CompactArgs a) {
  grid_dep_trigger();
  grid_dep_wait();
  constexpr int GS = WARP ? 32 : kMoveThreads;
  const int lane = WARP ? threadIdx.x & 31 : threadIdx.x;
  const long long unit = WARP ? (long long)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5)
                              : (long long)blockIdx.x;
  if (WARP && unit >= (long long)tb.planes * a.batch * a.kv_heads) return;
  // unit = (plane * B + b) * H + h
  const int h = (int)(unit % a.kv_heads);
  const long long r1 = unit / a.kv_heads;
  const int b = (int)(r1 % a.batch);
  const int pl = (int)(r1 / a.batch);
  const int rows = tb.rows[pl], chunks = tb.row_bytes[pl] / 16;
  const int c0 = WARP ? 0 : blockIdx.y * a.cols;
  const int cols = WARP ? chunks : min(a.cols, chunks - c0);
  if (!WARP && cols <= 0) return;
  const int count = a.counts[b], pos = a.pos[b];
  bool bad = count < 0 || count > a.A || count > a.min_rows || pos < 0 || pos > a.max_seq - count;
  const int items = bad ? 0 : count * cols;
  uint4* base = static_cast<uint4*>(tb.plane[pl]) + ((size_t)b * a.kv_heads + h) * rows * chunks + c0;
  uint4 x[kMoveItems];
  int to[kMoveItems];   // destination chunk; -1: none
#pragma unroll
  for (int k = 0; k < kMoveItems; ++k) {
    const int it = lane + k * GS;
    to[k] = -1;
    if (it < items) {
      const int j = it / cols, c = it - j * cols;
      const int from = a.idx[(size_t)b * a.A + j];
      if (from < 0 || from >= a.min_rows || from >= a.max_seq - pos) {
        bad = true;
      } else if (from != j) {
        // (pos + j) % rows is pos + j itself where the cache is no ring
        const size_t src = (size_t)((pos + from) % rows) * chunks + c;
        x[k] = base[src];
        to[k] = (pos + j) % rows;
      }
    }
  }
  const bool stop = WARP ? __any_sync(0xffffffffu, bad) : __syncthreads_or(bad);
  if (stop) {
    if (lane == 0 && pl == 0 && h == 0 && c0 == 0) flag_status(a.status, kDevBadArg);
    return;
  }
#pragma unroll
  for (int k = 0; k < kMoveItems; ++k)
    if (to[k] >= 0) base[(size_t)to[k] * chunks + (lane + k * GS) % cols] = x[k];
}

// --- fkv_reorder_seqs -----------------------------------------------------------
//
// new rows [0, len[b]) of b = old rows of src[b], in place, for any map src.
// A work item is one chunk of the same byte range of every sequence in one
// (layer, K or V, KV head) plane: the chunks of all sequences that are a
// source go to shared memory (bulk copies, one mbarrier a stage), and once all
// have landed each destination is written from its source's slot (bulk
// copies).  Items touch disjoint bytes, so cycles need no scratch memory, each
// source is read once and each destination written once: HBM traffic is the
// floor.  One warp per SM keeps the copy engines busy: 332M, 8 prompts of 4
// beams, up to 2048 rows 96 us (88% of the measured copy bandwidth), 4B, one
// prompt forked over 8192 rows 334 to 347 us (91 to 95%; 364 and 427 us on two other
// devices of the same kind).

constexpr int kReorderSmem = 200 * 1024;
constexpr int kReorderStages = 8;
constexpr int kReorderChunk = 16 * 1024;

__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

__global__ void __launch_bounds__(32) reorder_kernel(const __grid_constant__ MoveTable tb,
                                                     const ReorderArgs a) {
  extern __shared__ __align__(128) uint8_t stage_mem[];
  __shared__ uint64_t full[kReorderStages];
  __shared__ long long first_item[kMovePlanes + 1];
  __shared__ int head_items[kMovePlanes];
  uint8_t* meta = stage_mem + kReorderSmem;
  int* src_seq = reinterpret_cast<int*>(meta);   // [B] sequence of each slot
  int* src_len = src_seq + a.batch;              // [B] rows read of each slot
  int* dst_seq = src_len + a.batch;              // [B] destinations
  int* dst_slot = dst_seq + a.batch;             // [B] their source's slot
  int* dst_len = dst_slot + a.batch;             // [B] their rows
  int* need = dst_len + a.batch;                 // [B] rows needed of each sequence
  const int lane = threadIdx.x;
  const int B = a.batch;
  if (lane == 0) {
    for (int s = 0; s < kReorderStages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  grid_dep_trigger();
  for (int b = lane; b < B; b += 32) need[b] = 0;
  __syncwarp();
  grid_dep_wait();
  const unsigned long long wlim = wait_limit_ns(a.wait_limit);

  // destinations (src[b] names another sequence, with rows to copy) and the
  // rows each source has to give
  int ndst = 0, longest = 0;
  for (int base = 0; base < B; base += 32) {
    const int b = base + lane;
    int s = -1, len = 0;
    if (b < B) {
      s = a.src[b];
      len = a.seq_lens[b];
      if (s < -1 || s >= B || len < 0 || len > a.max_seq) {
        if (blockIdx.x == 0) flag_status(a.status, kDevBadArg);
        s = -1;
      }
      if (s == b) s = -1;
    }
    const bool mv = s >= 0 && len > 0;
    const unsigned m = __ballot_sync(0xffffffffu, mv);
    if (mv) {
      const int at = ndst + __popc(m & ((1u << lane) - 1));
      dst_seq[at] = b;
      dst_slot[at] = s;
      dst_len[at] = len;
      atomicMax(&need[s], len);
      longest = max(longest, len);
    }
    ndst += __popc(m);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  __syncwarp();
  int nsrc = 0;
  for (int base = 0; base < B; base += 32) {
    const int b = base + lane;
    const bool used = b < B && need[b] > 0;
    const unsigned m = __ballot_sync(0xffffffffu, used);
    if (used) {
      const int at = nsrc + __popc(m & ((1u << lane) - 1));
      src_seq[at] = b;
      src_len[at] = need[b];
      need[b] = at;   // from here on: the sequence's slot
    }
    nsrc += __popc(m);
  }
  __syncwarp();
  for (int i = lane; i < ndst; i += 32) dst_slot[i] = need[dst_slot[i]];
  __syncwarp();
  if (ndst == 0) return;

  // chunk bytes: two stages of all sources fit, and small calls still give
  // every CTA a few items
  long long bytes = 0;   // of one sequence's longest rows over all planes
  for (int i = lane; i < tb.planes; i += 32)
    bytes += (long long)a.kv_heads * min(longest, tb.rows[i]) * tb.row_bytes[i];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) bytes += __shfl_xor_sync(0xffffffffu, bytes, o);
  long long ch = kReorderSmem / 2 / nsrc;
  ch = min(ch, (long long)kReorderChunk);
  ch = min(ch, max(1024LL, bytes / (4LL * gridDim.x)));
  const int CH = (int)max(16LL, ch / 16 * 16);
  const int stage_bytes = nsrc * CH;
  const int NST = min(kReorderStages, kReorderSmem / stage_bytes);
  long long total = 0;   // items; each plane's first and its items a head
  for (int base = 0; base < tb.planes; base += 32) {
    const int i = base + lane;
    int per = 0;
    if (i < tb.planes) per = (int)(((long long)min(longest, tb.rows[i]) * tb.row_bytes[i] + CH - 1) / CH);
    long long incl = (long long)per * a.kv_heads;
    const long long own = incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (i < tb.planes) {
      head_items[i] = per;
      first_item[i] = total + incl - own;
    }
    total += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) first_item[tb.planes] = total;
  __syncwarp();

  // the plane (from `pl` on), the head's rows and the byte offset of an item
  auto locate = [&](long long item, int& pl, uint8_t*& head, long long& off) {
    while (item >= first_item[pl + 1]) ++pl;
    // (a plane's bytes are below 2^40 and its chunks, of 96 bytes at least,
    // below 2^34 for one head: 64-bit items, 32-bit chunks of a head)
    const long long per = head_items[pl], r = item - first_item[pl];
    const long long h = (r >> 31) == 0 ? (uint32_t)r / (uint32_t)per : r / per;
    head = static_cast<uint8_t*>(tb.plane[pl]) + (size_t)h * tb.rows[pl] * tb.row_bytes[pl];
    off = (r - h * per) * CH;
  };
  auto part = [&](int len, int pl, long long off) {
    const long long n = (long long)min(len, tb.rows[pl]) * tb.row_bytes[pl] - off;
    return (uint32_t)max(0LL, min(n, (long long)CH));
  };
  int load_pl = 0, store_pl = 0;
  auto load = [&](long long item, int st) {
    uint8_t* head;
    long long off;
    locate(item, load_pl, head, off);
    const size_t seq = (size_t)a.kv_heads * tb.rows[load_pl] * tb.row_bytes[load_pl];
    uint32_t sum = 0;
    for (int i = lane; i < nsrc; i += 32) sum += part(src_len[i], load_pl, off);
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) mbar_arrive_expect_tx(&full[st], sum);
    __syncwarp();
    for (int i = lane; i < nsrc; i += 32) {
      const uint32_t n = part(src_len[i], load_pl, off);
      if (n)
        bulk_g2s(stage_mem + (size_t)st * stage_bytes + (size_t)i * CH, head + src_seq[i] * seq + off,
                 n, &full[st], l2_policy_evict_first());
    }
  };

  const long long grid = gridDim.x;
  long long loaded = 0, done = 0;   // items of this CTA
  for (long long item = blockIdx.x; item < total && loaded < NST - 1; item += grid) load(item, (int)loaded++);
  bool ok = true;
  for (long long item = blockIdx.x; item < total; item += grid, ++done) {
    const int st = (int)(done % NST);
    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[st], (uint32_t)(done / NST) & 1u, wlim));
    if (!ok) {
      flag_status(a.status, kDevTimeout);
      break;
    }
    uint8_t* head;
    long long off;
    locate(item, store_pl, head, off);
    const size_t seq = (size_t)a.kv_heads * tb.rows[store_pl] * tb.row_bytes[store_pl];
    for (int i = lane; i < ndst; i += 32) {
      const uint32_t n = part(dst_len[i], store_pl, off);
      if (n)
        bulk_s2g(head + dst_seq[i] * seq + off,
                 stage_mem + (size_t)st * stage_bytes + (size_t)dst_slot[i] * CH, n);
    }
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    const long long next = blockIdx.x + loaded * grid;
    if (next < total) {
      // its stage was stored from one item ago: those reads are done
      asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      __syncwarp();
      load(next, (int)(loaded % NST));
      ++loaded;
    }
  }
  if (!ok)   // copies in flight land before the CTA exits
    for (long long k = done; k < loaded; ++k)
      (void)mbar_wait_bounded(&full[k % NST], (uint32_t)(k / NST) & 1u, kDrainLimitNs);
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

}  // namespace

cudaError_t compact_launch(const MoveTable& tb, CompactArgs a, cudaStream_t stream) {
  int chunks = 0;
  for (int i = 0; i < tb.planes; ++i) chunks = tb.row_bytes[i] / 16 > chunks ? tb.row_bytes[i] / 16 : chunks;
  const long long units = (long long)tb.planes * a.batch * a.kv_heads;
  if (a.A * chunks <= 32 * kMoveItems) {
    constexpr int W = kMoveThreads / 32;
    return launch_pdl(compact_kernel<true>, dim3((unsigned)((units + W - 1) / W)), dim3(kMoveThreads),
                      0, stream, tb, a);
  }
  a.cols = kMoveThreads * kMoveItems / a.A;
  if (a.cols > chunks) a.cols = chunks;
  return launch_pdl(compact_kernel<false>, dim3((unsigned)units, (unsigned)((chunks + a.cols - 1) / a.cols)),
                    dim3(kMoveThreads), 0, stream, tb, a);
}

cudaError_t reorder_launch(const MoveTable& tb, const ReorderArgs& a, int num_sms, cudaStream_t stream) {
  const size_t smem = kReorderSmem + (size_t)a.batch * 6 * sizeof(int);
  static KernelReady ready;
  const cudaError_t e = ready.check(reorder_kernel, a.device, kReorderSmem + 1024 * 6 * (int)sizeof(int), 32, 0);
  if (e != cudaSuccess) return e;
  return launch_pdl(reorder_kernel, dim3(num_sms), dim3(32), smem, stream, tb, a);
}

}  // namespace fkv
