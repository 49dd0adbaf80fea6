// fkv_tree_attn on the tcgen05 tensor cores (bf16 and 4-bit caches).
//
// A drafted tree gives a (sequence, KV head) unit G * T query rows, few
// against the cached keys, so the call is bound by reading the cache once.
// The products are taken transposed, keys as the 128 rows of the MMA and the
// query rows as its NC = 16 .. 128 columns: S^T = K Q^T, O^T = V^T P^T.  A
// thread of the softmax then owns a key, not a query row, so that all threads
// work however few query rows there are.
//
// Math.  Online softmax in base 2 with one reference m_c per column c; a tile
// keeps the reference unless a score exceeds it by more than 2^8 (P stays
// below 256, exact scaling), so the column maximum over the 128 threads is
// only taken on the first tile of a piece and when the scores grow.  Fused
// layers need no fused tile: S = K^1 (q a_1)^T + K^n (q a_n)^T accumulates in
// one product, and O = b_1 (V^1 P) + b_n (V^n P) keeps two accumulators (one of
// 128 lanes for both at 64 channels: 332M fused, T = 64, 228 -> 207 us).
// q a is split into two bf16 halves (exact to 2^-16; one half alone cost 1.5e-3
// of relative error in the output, as much as P), which doubles the score
// products of weighted layers, and P is rounded to bf16 as in the prefill
// kernels; sums are fp32.
//
// A CTA takes a contiguous range of key tiles of 128 rows (tree_common.cuh)
// and one tile of NC query rows:
//  * the producer warp loads K and V tiles by TMA (boxes of 128-byte rows) into
//    a ring of slots, in the order in which the MMAs read them: K_0, K_1, V_0,
//    K_2, V_1, ...;
//  * one warp issues S_j = K_j Q^T up to two tiles ahead (S has two buffers in
//    tensor memory), another O += V_j^T P_j: an MMA of these sizes costs its
//    issuer 40 to 48 clocks at 16 to 64 columns (64 at 128), as long as the
//    tensor pipe, so one issuer for both was the bound of small trees;
//  * two or four softmax warpgroups take a part of the columns each: scores
//    from tensor memory, P to shared memory as an MN-major operand (a thread writes its
//    key's columns, 16 bytes at a time, without bank conflicts).
// 4-bit caches: the producer copies a tile's records (one contiguous run) to a
// second ring, and two more warpgroups dequantise them into the slots, two
// values an instruction: a nibble pair under the exponent of 64 is 64 + code / 16
// in fp16, exactly; less 64, times 16 * scale, plus the minimum in one FMA is
// the record's value rounded once to fp16.  Queries and P are fp16 then too:
// each operand is off by 2^-11 of itself, so that the output's error is its own
// rounding's (bf16 operands gave twice that, 3.4e-3).  fp16's range is the price:
// keys and values up to 2^14 (16 * scale stays finite), beside an error of
// 3 * 2^-25 (scale, minimum and value, each below 2^-14); a query row that leaves
// it is held times a power of two.
// The pairs that fall out of a word are channels e and e + 4 of eight, so the
// tiles hold the channels in the order 0 4 1 5 2 6 3 7 and so do the queries; the
// epilogue undoes it.
//
// What bounds it (one GB300, against 6.78 TB/s of measured copy bandwidth; bytes
// are the cached rows once): HBM from 32 columns and 160-byte rows on (4B lite,
// T = 16: 2.0 GB in 300 us; 1.5B fused, T = 26: 3.2 GB in 460 us).  With 128
// columns the softmax's chain of short dependent steps (tensor-memory loads, a
// vote, exponentials, shared stores) beside instruction fetch: no pipe is near its
// limit (332M fused, T = 64: 0.82 GB in 206 us, 44% of the issue slots, 34% of
// the tensor pipe).  With 16 columns the end of a unit, which
// the ring's 192 KB of tiles hides only in part (332M lite, T = 8: 0.40 GB in
// 75 us, 26% of the slots); over 4-bit caches the dequantisation beside the
// softmax (332M fused, T = 16: 0.30 GB in 137 us, 54% of the slots); short calls
// their chain of prologue, first tile, merge (650M ring layer, T = 12: 18 us).
//
// Tiles with drafted rows, a window's edge or a ragged end are masked, and the
// value rows that nobody sees are zeroed in shared memory, since 0 * NaN is
// no 0.  A drafted value row that is not finite is zeroed too and its score
// made NaN, so that it stays with the nodes that see it.
#pragma once

#include <cfloat>
#include <cstring>
#include <type_traits>

#include <cuda_fp16.h>

#include "tc_device.cuh"
#include "tree_common.cuh"

namespace fkv {

// (an unnamed namespace: each unit has its own head dimension's kernels)
namespace {

constexpr int KT = kTreeKeyTile;
constexpr int DQ_THREADS = 256;       // dequantising threads (4-bit caches)
constexpr int DQ_GROUP = 64;          // of them that share a tile: four tiles are in work at a time
constexpr int MAX_RAW = 12;           // slots of records
constexpr int MAX_SLOTS = 12;
constexpr int TAIL_ROWS = kTreeTailRows;
constexpr int SMEM_LIMIT = 232448;
constexpr int SWB = 128;              // bytes of a swizzled row: 64 channels or columns
constexpr int SWC = SWB / 2;
constexpr float SLACK = 8.f;          // log2 growth of a score over its reference

template <int D, int NSRC, bool WGT, int NC, bool Q4>
struct TcCfg {
  static constexpr int CB = (D + SWC - 1) / SWC;         // 64-channel blocks
  static constexpr int SLOT = CB * KT * SWB;             // one K or V tile
  // the queries, or per source the high and low halves of query times weight
  // (over 4-bit caches one fp16, whose rounding is an eighth of bf16's)
  static constexpr int NQ = WGT && !Q4 ? 2 : 1;
  // How far the probabilities' exponents are raised (4-bit caches): 2^4 at the
  // reference, so that what fp16 loses below 2^-25 is below 2^-29 of a column's sum.
  static constexpr float RAISE = Q4 ? 4.f : 0.f;
  static constexpr int Q_BYTES = NSRC * NQ * CB * NC * SWB;
  static constexpr int P_BYTES = (NC + SWC - 1) / SWC * KT * SWB;
  static constexpr int NW = (NC + 31) / 32;              // 32-bit words of a column mask
  // V^T is read as 128 channels, 2 blocks from a slot on.  Two sources of 64
  // channels make one product: the blocks are their neighbouring slots, lanes
  // 0 .. 63 of the accumulator hold V^1 P, the others V^n P.  One source of 64
  // channels reads past its slot into what follows (rows that are not used;
  // the records behind 4-bit slots, else a block left free).
  static constexpr bool PAIR = NSRC == 2 && D == 64;
  static constexpr int NACC = PAIR ? 1 : NSRC;           // accumulators
  static constexpr int OVERRUN = Q4 || PAIR ? 0 : (2 - CB) * KT * SWB;
  // Softmax warpgroups, each with a part of the columns of every tile.  Four
  // from 64 columns on, where they hide each other's waits (332M fused, T = 64,
  // took a fifth less than with two); two below, which leaves them more registers and
  // shorter barriers, and for 4-bit caches, whose dequantising warpgroups take
  // the other threads.  (Two warpgroups with every second tile each, references
  // and accumulators of their own, gained 3% at 16 columns and lost 19% over
  // 4-bit caches.)
  static constexpr int NWG = NC <= 32 || Q4 ? 2 : 4;
  static constexpr int SM = NWG * 128;                   // softmax threads
  static constexpr int HC = NC / NWG;                    // columns of a softmax thread
  static constexpr int CH = HC < 16 ? HC : 16;           // of them in registers at a time
  static constexpr int PRODUCER_WARP = 4 * NWG, QK_WARP = PRODUCER_WARP + 1, PV_WARP = PRODUCER_WARP + 2;
  static constexpr int DQ_WARP = PRODUCER_WARP + 4;      // the first of the dequantising warps
  static constexpr int TMEM_USED = (2 + NACC) * NC;
  static constexpr int TMEM_COLS = TMEM_USED <= 32 ? 32 : TMEM_USED <= 64 ? 64 : TMEM_USED <= 128 ? 128
                                   : TMEM_USED <= 256 ? 256 : 512;
  static_assert(TMEM_USED <= 512, "tensor memory");
  // barriers and words, then the arrays of floats and masks
  static constexpr int BAR_BYTES = ((2 * MAX_SLOTS + 2 * MAX_RAW) * 8 + 11 * 8 + 7 * 4 + 127) / 128 * 128;
  static constexpr int ARRAY_BYTES = NC * 4 * 8 + kTreeMaxNodes * (16 + 4 + NW * 4) + (Q4 ? NC * 4 : 0);
  static constexpr int RAW = KT * q4_row_bytes(D);       // records of a tile
  // two P buffers where at least five tile slots remain beside them (4-bit
  // caches: the four that the dequantising groups need, with four of records
  // and the lengths of the largest batch)
  static constexpr int BESIDE = 3072 + Q_BYTES + BAR_BYTES + ARRAY_BYTES + OVERRUN + 2 * P_BYTES +
                                (Q4 ? (int)tree_seqs_bytes(1024) + 4 * RAW : 0);
  static constexpr int NPB = (SMEM_LIMIT - BESIDE) / SLOT >= (Q4 ? 4 : 5) ? 2 : 1;
  static constexpr int REF_OFF = Q_BYTES + NPB * P_BYTES + BAR_BYTES;
  __host__ __device__ static constexpr int ring_off(int B) {
    return (REF_OFF + ARRAY_BYTES + (int)tree_seqs_bytes(B) + 1023) / 1024 * 1024;
  }
  static constexpr int THREADS = SM + 128 + (Q4 ? DQ_THREADS : 0);
  // registers a thread: 168 at launch with 384 threads, 96 with 640; the
  // control (and dequantising) warpgroups give some up for the softmax:
  // 256 * 208 + 128 * 88 = 384 * 168, 512 * 104 + 128 * 64 = 640 * 96,
  // 256 * 128 + 128 * 64 + 256 * 80 = 640 * 96
  static constexpr int REGS_CONTROL = THREADS > 384 ? 64 : 88;
  static constexpr int REGS_SOFTMAX = Q4 ? 128 : NWG == 4 ? 104 : 208, REGS_DQ = 80;
  static constexpr int REGS_SPLIT =
      SM * REGS_SOFTMAX + 128 * REGS_CONTROL + (Q4 ? DQ_THREADS * REGS_DQ : 0);
};

struct TcMaps {
  CUtensorMap full[4];   // K first, K second, V first, V second: boxes of 128 rows
  CUtensorMap tail[4];   // boxes of TAIL_ROWS rows
};

// Sum or maximum over the warp's lanes of N values a lane; afterwards lane i
// holds the result of value i % N.  N = 8, 16 or 32.
template <int N, typename Op>
__device__ __forceinline__ float reduce_scatter(float* v, int lane, Op op) {
#pragma unroll
  for (int h = N / 2; h >= 1; h >>= 1) {
    const bool up = lane & h;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float give = up ? v[i] : v[i + h];
      const float keep = up ? v[i + h] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, h));
    }
  }
  float r = v[0];
#pragma unroll
  for (int h = N; h < 32; h <<= 1) r = op(r, __shfl_xor_sync(0xffffffffu, r, h));
  return r;
}

// All softmax threads.
template <int COUNT>
__device__ __forceinline__ void sm_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(COUNT) : "memory"); }

// Whether x holds in any thread of `count` threads that meet at barrier `id`.
__device__ __forceinline__ bool any_of(int id, int count, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}

// A wait that did not succeed at once: until the phase completes, another role
// gives up, or the limit passes.
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, unsigned long long limit,
                                     volatile int* abort_flag, int* status) {
  if (*abort_flag) return false;
  if (mbar_wait_bounded(bar, parity, limit)) return true;
  *abort_flag = 1;
  flag_status(status, kDevTimeout);
  return false;
}

// The 128 threads of softmax warpgroup wg.
__device__ __forceinline__ void wg_sync(int wg) { asm volatile("bar.sync %0, 128;" ::"r"(2 + wg) : "memory"); }

// Two floats as fp16 or bf16.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (F16) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// 2^n, |n| <= 126.
__device__ __forceinline__ float exp2_int(int n) { return __int_as_float((127 + n) << 23); }

// Slot (counted from a piece's first, in tiles of one tensor) of the values of
// tile i of a piece's n: the order is K_0, K_1, V_0, K_2, V_1, ..., K_n-1, V_n-2, V_n-1.
__device__ __forceinline__ int v_slot(int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 + 2 * i; }

template <int D, int NSRC, bool WGT, int NC, bool Q4>
__global__ void __launch_bounds__(TcCfg<D, NSRC, WGT, NC, Q4>::THREADS, 1)
    tree_tc_kernel(const __grid_constant__ TcMaps maps, const TreeParams p, const int nslots,
                   const int nraw) {
  using C = TcCfg<D, NSRC, WGT, NC, Q4>;
  constexpr int CB = C::CB, HC = C::HC, CH = C::CH, NACC = C::NACC, NW = C::NW, NPB = C::NPB;
  auto sm_sync = [] { sm_barrier<C::SM>(); };
  // Everything before the rings lies at offsets known at compile time, from a
  // pointer that the compiler sees is shared memory: addresses cost no
  // registers.  1024 bytes: the period of the 128-byte swizzle.
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sP = sQ + C::Q_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sP + NPB * C::P_BYTES);
  uint64_t* empty = full + MAX_SLOTS;
  uint64_t* raw_full = empty + MAX_SLOTS;
  uint64_t* raw_empty = raw_full + MAX_RAW;
  uint64_t* q_ready = raw_empty + MAX_RAW;
  uint64_t* s_full = q_ready + 1;   // [2]
  uint64_t* p_full = s_full + 2;    // [2]
  uint64_t* o_done = p_full + 2;    // [4]
  uint64_t* drain = o_done + 4;     // [2] an issuer's last products, after an abort
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* sm_issued = reinterpret_cast<int*>(tmem_slot + 2);
  int* merge_flag = sm_issued + 1;
  int* sm_span = merge_flag + 1;                               // [2] least and largest depth
  volatile int* sm_scaled = sm_span + 2;                       // one of them is not 1 (sCol)
  float* sRef = reinterpret_cast<float*>(smem + C::REF_OFF);   // [NC] negated reference
  float* sAlpha = sRef + NC;                                   // [NC] rescale, then weight
  int* sDepth = reinterpret_cast<int*>(sAlpha + NC);           // [NC] depth of the column's node
  int* sNode = sDepth + NC;                                    // [NC] node of the column, -1: none
  float* sWarp = reinterpret_cast<float*>(sNode + NC);         // [4][NC]
  unsigned long long* sMask = reinterpret_cast<unsigned long long*>(sWarp + 4 * NC);   // [nodes][2]
  int* sNodeDepth = reinterpret_cast<int*>(sMask + 2 * kTreeMaxNodes);   // [nodes]
  uint32_t* sVis = reinterpret_cast<uint32_t*>(sNodeDepth + kTreeMaxNodes);   // [nodes][NW]
  float* sCol = reinterpret_cast<float*>(sVis + kTreeMaxNodes * NW);   // [NC] powers of two of the query rows (4-bit)
  const TreeSeqs sq = tree_seqs(reinterpret_cast<int*>(sCol + (Q4 ? NC : 0)), p.B);
  uint8_t* sRing = smem + C::ring_off(p.B);
  uint8_t* sRaw = sRing + (size_t)nslots * C::SLOT;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rt = blockIdx.y;
  if (tid == 0) {
    for (int s = 0; s < nslots; ++s) {
      mbar_init(&full[s], Q4 ? DQ_GROUP / 32 : 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; Q4 && s < nraw; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], DQ_GROUP / 32);
    }
    mbar_init(q_ready, C::SM / 32);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], C::SM / 32);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&o_done[i], 1);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    *abort_flag = 0;
    *sm_issued = 0;
    *sm_scaled = 0;
    fence_mbar_init();
  }
  if (warp == C::QK_WARP) tmem_alloc(tmem_slot, C::TMEM_COLS);
  for (int c = tid; c < NC; c += C::THREADS) {
    const int row = rt * NC + c;
    sNode[c] = row < p.G * p.T ? row % p.T : -1;
  }
  if (!Q4 && warp == C::PRODUCER_WARP && lane < 8 && (lane & 1) < NSRC)
    tma_prefetch(lane < 4 ? &maps.full[lane] : &maps.tail[lane - 4]);
  grid_dep_trigger();
  grid_dep_wait();
  const unsigned long long wlim = wait_limit_ns(p.wait_limit);
  tc_fence_before();
  const TreeCut cut = tree_cut<__nv_bfloat16, D>(p, sq, KT, gridDim.x, 3);   // ends with a __syncthreads
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool active = (int)blockIdx.x < cut.ranges;
  TreeWalk walk;
  if (active) walk.begin(cut, sq.pre, p.B, p.H, blockIdx.x);

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (wlim != 0 && mbar_try_wait(bar, parity)) return true;
    return wait_on(bar, parity, wlim, abort_flag, p.status);
  };
  // the same by a whole warp, with one answer
  auto await = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (wlim != 0 && __all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_on(bar, parity, wlim, abort_flag, p.status));
  };
  // the value products of tile t are done
  auto products = [&](int t) { return await(&o_done[t & 3], (uint32_t)(t >> 2) & 1u); };
  auto slot_ptr = [&](int s) { return sRing + (size_t)s * C::SLOT; };

  if (active && warp >= C::PRODUCER_WARP && warp < C::DQ_WARP)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_CONTROL));
  if (active && warp == C::PRODUCER_WARP) {
    // ---------------- producer ----------------
    if (lane == 0) {
      const int nring = Q4 ? nraw : nslots;
      uint64_t* ring_empty = Q4 ? raw_empty : empty;
      const size_t plane = p.ring > 0 ? p.ring : p.S_max;
      int g = 0, sl = 0;   // slots filled; the next one
      uint32_t turn = 1;   // parity of its last release
      bool ok = true;
      TreePiece pc;
      while (ok && walk.next(sq.pre, p.B, p.H, pc)) {
        const TreeSeq s = tree_seq(p, sq.P[pc.b], sq.N[pc.b]);
        const int unit = pc.b * p.H + pc.h, n = pc.k1 - pc.k0;
        auto load = [&](int kv, const TreeTile& t) {
#pragma unroll
          for (int src = 0; src < NSRC; ++src) {
            if (g >= nring && !wait(&ring_empty[sl], turn)) return false;
            if constexpr (Q4) {
              const uint8_t* rec = static_cast<const uint8_t*>(kv ? p.v[src] : p.k[src]);
              const uint32_t bytes = t.cnt * q4_row_bytes(D);
              fence_proxy_async_smem();
              mbar_arrive_expect_tx(&raw_full[sl], bytes);
              bulk_g2s(sRaw + (size_t)sl * C::RAW, rec + (unit * plane + t.row) * q4_row_bytes(D), bytes,
                       &raw_full[sl], l2_policy_evict_first());
            } else {
              const int m = kv * 2 + src;
              uint8_t* dst = slot_ptr(sl);
              if (t.cnt == KT) {
                mbar_arrive_expect_tx(&full[sl], C::SLOT);
#pragma unroll
                for (int cb = 0; cb < CB; ++cb)
                  tma_load_3d(dst + cb * KT * SWB, &maps.full[m], cb * SWC, t.row, unit, &full[sl]);
              } else {
                const int boxes = (t.cnt + TAIL_ROWS - 1) / TAIL_ROWS;
                mbar_arrive_expect_tx(&full[sl], boxes * CB * TAIL_ROWS * SWB);
                for (int x = 0; x < boxes; ++x)
#pragma unroll
                  for (int cb = 0; cb < CB; ++cb)
                    tma_load_3d(dst + cb * KT * SWB + x * TAIL_ROWS * SWB, &maps.tail[m], cb * SWC,
                                t.row + x * TAIL_ROWS, unit, &full[sl]);
              }
            }
            ++g;
            if (++sl == nring) {
              sl = 0;
              turn ^= 1;
            }
          }
          return true;
        };
        // the keys of tile i + 1, then the values of tile i
        TreeTile t = tree_tile(p, s, pc.k0, KT);
        ok = load(0, t);
        for (int i = 0; ok && i < n; ++i) {
          TreeTile next = t;
          if (i + 1 < n) {
            next = tree_tile(p, s, pc.k0 + i + 1, KT);
            ok = load(0, next);
          }
          ok = ok && load(1, t);
          t = next;
        }
      }
      *sm_issued = g;
    }
  } else if (Q4 && active && warp >= C::DQ_WARP) {
    // ---------------- dequantisation ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_DQ));
    if constexpr (Q4) {
      constexpr int GR = D / kQ4Group, RB = q4_row_bytes(D);
      constexpr int GROUPS = DQ_THREADS / DQ_GROUP;
      const int t = (tid - C::DQ_WARP * 32) % DQ_GROUP;
      const __half2 bias = __floats2half2_rn(-64.f, -64.f);
      const long long total = (walk.t1 - walk.t) * 2 * NSRC;
      int sl = 0, r = 0;
      uint32_t turn = 1, rturn = 0;   // parities of the slot's last release and of the records' filling
      auto step = [&]() {
        if (++sl == nslots) {
          sl = 0;
          turn ^= 1;
        }
        if (++r == nraw) {
          r = 0;
          rturn ^= 1;
        }
      };
      // Both rings hold a multiple of GROUPS slots, so a slot stays with one
      // group and no phase of its barriers is awaited before the last is over.
      const int first = (tid - C::DQ_WARP * 32) / DQ_GROUP;
      for (int k = 0; k < first; ++k) step();
      for (long long g = first; g < total; g += GROUPS) {
        if (!await(&raw_full[r], rturn) || (g >= nslots && !await(&empty[sl], turn))) break;
        const uint8_t* rec = sRaw + (size_t)r * C::RAW;
        uint8_t* dst = slot_ptr(sl);
        auto eight = [&](int row, int ch, uint32_t w, __half2 sc, __half2 lo) {   // channels of a row
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t x = ((w >> (4 * e)) & 0x000f000fu) | 0x54005400u;
            const __half2 v = __hfma2(__hadd2(*reinterpret_cast<const __half2*>(&x), bias), sc, lo);
            o[e] = *reinterpret_cast<const uint32_t*>(&v);
          }
          *reinterpret_cast<uint4*>(dst + (ch >> 3) * KT * SWB + swz128(row, ch & 7)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        };
        // Four roles' loops share the instruction cache: 332M fused, T = 16, took
        // 137 us unrolled twice, 141 not at all, 152 four times, 169 eight times.
#pragma unroll 2
        for (int k = 0; k < KT * GR / DQ_GROUP; ++k) {   // a multiple: KT = 2 * DQ_GROUP
          const int it = t + k * DQ_GROUP;
          const int row = it / GR, gr = it - row * GR;
          const uint2 codes = *reinterpret_cast<const uint2*>(rec + row * RB + gr * 8);
          const uint32_t prm = *reinterpret_cast<const uint32_t*>(rec + row * RB + D / 2 + gr * 4);
          const __half2 both = __floats2half2_rn(bf16lo(prm) * 16.f, bf16hi(prm));
          const __half2 sc = __low2half2(both), lo = __high2half2(both);
          eight(row, gr * 2, codes.x, sc, lo);
          eight(row, gr * 2 + 1, codes.y, sc, lo);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[sl]);
          mbar_arrive(&raw_empty[r]);
        }
        for (int k = 0; k < GROUPS; ++k) step();
      }
    }
  } else if (active && (warp == C::QK_WARP || warp == C::PV_WARP)) {
    // ---------------- MMA issuers (the whole warp; one lane issues) ----------------
    constexpr uint32_t IDESC_QK = Q4 ? idesc_with_f16(idesc_bf16(KT, NC, false)) : idesc_bf16(KT, NC, false);
    constexpr uint32_t IDESC_PV = Q4 ? idesc_with_f16(idesc_bf16_tt(128, NC)) : idesc_bf16_tt(128, NC);
    const bool qk = warp == C::QK_WARP;
    // descriptors of slot 0 as K (K-major) and as V^T (MN-major), of Q and P
    const SDesc128 da = qk ? sdesc128(smem_u32(sRing), 16, 8 * SWB)
                           : sdesc128(smem_u32(sRing), KT * SWB, 8 * SWB);
    const SDesc128 db = qk ? sdesc128(smem_u32(sQ), 16, 8 * SWB)
                           : sdesc128(smem_u32(sP), KT * SWB, 8 * SWB);
    int sl = 0;          // next slot
    uint32_t turn = 0;   // parity of its filling
    auto skip = [&](int n) {
      sl += n;
      if (sl >= nslots) {
        sl -= nslots;
        turn ^= 1;
      }
    };
    int j = 0;   // tile of this CTA
    int piece = 0;
    bool ok = true;
    TreePiece pc;
    while (ok && walk.next(sq.pre, p.B, p.H, pc)) {
      const int n = pc.k1 - pc.k0;
      if (qk) {
        // S = K (q a)^T, both sources; its buffer is free once P of the tile
        // two before is written.  A slot's phase may only be awaited when the
        // one before it is known to be over: the slot of K_j held keys, or the
        // values of tile j - 3 at the latest.
        ok = await(q_ready, (uint32_t)piece & 1u);
        for (int i = 0; ok && i < n; ++i, ++j) {
          const uint32_t d = tmem + (j & 1) * NC;
          ok = (j < 2 || await(&p_full[j & 1], (uint32_t)((j - 2) >> 1) & 1u)) &&
               (j < 3 || products(j - 3));
#pragma unroll
          for (int src = 0; src < NSRC; ++src) {
            if (!ok || !await(&full[sl], turn)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (elect_one()) {
              const SDesc128 a{da.lo + (uint32_t)(sl * C::SLOT >> 4), da.hi};
#pragma unroll
              for (int part = 0; part < C::NQ; ++part)
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                  const uint64_t ad = a.at((k >> 2) * KT * SWB + (k & 3) * 32);
                  const uint64_t bd = db.at(((src * C::NQ + part) * CB + (k >> 2)) * NC * SWB + (k & 3) * 32);
                  if (src == 0 && part == 0 && k == 0) mma_bf16_t<false>(d, ad, bd, IDESC_QK);
                  else mma_bf16_t<true>(d, ad, bd, IDESC_QK);
                }
              if (src == NSRC - 1) mma_commit(&s_full[j & 1]);
              mma_commit(&empty[sl]);
            }
            __syncwarp();
            skip(1);
          }
          // the values of the tile before lie between K_i and K_i+1 (i > 0),
          // those of the last two behind the piece's last keys
          skip(i == n - 1 ? (n == 1 ? 1 : 2) * NSRC : i == 0 ? 0 : NSRC);
        }
      } else {
        const TreeSeq s = tree_seq(p, sq.P[pc.b], sq.N[pc.b]);
        skip((n == 1 ? 1 : 2) * NSRC);   // V_0 follows K_0 and K_1
        for (int i = 0; ok && i < n; ++i, ++j) {
          const int ks = i + 1 == n || p.ring > 0 ? (tree_tile(p, s, pc.k0 + i, KT).cnt + 15) / 16
                                                  : KT / 16;   // 16-key steps
          ok = await(&p_full[j & 1], (uint32_t)(j >> 1) & 1u);
          const SDesc128 b{db.lo + (NPB == 2 && (j & 1) ? C::P_BYTES >> 4 : 0), db.hi};
#pragma unroll
          for (int src = 0; src < NACC; ++src) {
            constexpr int SLOTS = C::PAIR ? 2 : 1;   // (a pair never wraps: both counts are even)
            ok = ok && await(&full[sl], turn) && (SLOTS == 1 || await(&full[sl + 1], turn));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              const SDesc128 a{da.lo + (uint32_t)(sl * C::SLOT >> 4), da.hi};
              const uint32_t d = tmem + (2 + src) * NC;
              mma_bf16(d, a.at(0), b.at(0), IDESC_PV, i > 0 ? 1u : 0u);
              if (ks == KT / 16) {
#pragma unroll
                for (int k = 1; k < KT / 16; ++k)
                  mma_bf16_t<true>(d, a.at(k * 16 * SWB), b.at(k * 16 * SWB), IDESC_PV);
              } else {
                for (int k = 1; k < ks; ++k)
                  mma_bf16_t<true>(d, a.at(k * 16 * SWB), b.at(k * 16 * SWB), IDESC_PV);
              }
              if (src == NACC - 1) mma_commit(&o_done[j & 3]);
              mma_commit(&empty[sl]);
              if (SLOTS == 2) mma_commit(&empty[sl + 1]);
            }
            __syncwarp();
            skip(SLOTS);
          }
          if (i + 2 < n) skip(NSRC);   // the keys of the tile after next
        }
      }
      ++piece;
    }
  } else if (active && warp < C::PRODUCER_WARP) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
    // ---------------- softmax ----------------
    const int wg = warp >> 2, quarter = warp & 3;
    const int key = quarter * 32 + lane;   // key of the tile; channel in the epilogue
    const int c0 = wg * HC;                // first column
    const int row = C::PAIR ? key & 63 : key;   // row of V^T; its channel:
    const int chan = Q4 ? (row & ~7) | (row & 1) << 2 | (row >> 1 & 3) : row;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16) + c0;
    auto fmaxop = [](float a, float b) { return fmaxf(a, b); };
    auto addop = [](float a, float b) { return a + b; };
    int base = 0, jt = 0;
    bool ok = true;
    TreePiece pc;
    while (walk.next(sq.pre, p.B, p.H, pc)) {
      const int P = sq.P[pc.b], N = sq.N[pc.b];
      const TreeSeq s = tree_seq(p, P, N);
      const size_t unit = (size_t)pc.b * p.H + pc.h;
      const int n = pc.k1 - pc.k0;
      const int rows = min(NC, p.G * p.T - rt * NC);

      // the piece's queries times the key weights, in the MMA's layout
      for (int it = tid; it < NC * (CB * 8); it += C::SM) {
        const int r = it / (CB * 8), ch = it - r * (CB * 8);   // 16-byte chunk of a row
        const int d = ch * 8;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (r < rows && d < D && (!Q4 || sNode[r] < N))
          w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                              (unit * p.G * p.T + rt * NC + r) * D + d);
        float f[8];
        unpack16<__nv_bfloat16>(w, f);
        auto place = [&](int src) { return sQ + src * C::NQ * CB * NC * SWB + (ch >> 3) * NC * SWB + swz128(r, ch & 7); };
        if constexpr (Q4) {
          // fp16, times a power of two where the row does not lie in its range
          float x[NSRC][8], top = 0.f;
#pragma unroll
          for (int src = 0; src < NSRC; ++src)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              x[src][e] = f[e];
              if (WGT && d < D) x[src][e] *= p.a[src][(size_t)pc.h * D + d + e];
              top = fmaxf(top, fabsf(x[src][e]));
            }
#pragma unroll
          for (int o = 1; o < CB * 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          // the row's largest is left in 2^-6 .. 2^14, else brought to 1 .. 2
          int ex = 0;
          if (top > 0.f && top < INFINITY && !(top >= 0.015625f && top <= 16384.f))
            ex = min(max((__float_as_int(top) >> 23) - 127, -126), 126);
          if (ch == 0) sCol[r] = exp2_int(ex);
          if (ex != 0) *sm_scaled = 1;
          const float down = exp2_int(-ex);
#pragma unroll
          for (int src = 0; src < NSRC; ++src) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)   // the order of the tiles' channels: 0 4 1 5 2 6 3 7
              o[e] = pack2<true>(x[src][e] * down, x[src][e + 4] * down);
            *reinterpret_cast<uint4*>(place(src)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        } else {
#pragma unroll
          for (int src = 0; src < NSRC; ++src) {
            uint8_t* dst = place(src);
            if constexpr (WGT) {
              uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
              if (d < D) {
                const float4* ap = reinterpret_cast<const float4*>(p.a[src] + (size_t)pc.h * D + d);
                const float4 a0 = ap[0], a1 = ap[1];
                const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float x0 = f[2 * e] * av[2 * e], x1 = f[2 * e + 1] * av[2 * e + 1];
                  const __nv_bfloat162 h2 = __floats2bfloat162_rn(x0, x1);
                  hi[e] = *reinterpret_cast<const uint32_t*>(&h2);
                  const __nv_bfloat162 l2 = __floats2bfloat162_rn(x0 - bf16lo(hi[e]), x1 - bf16hi(hi[e]));
                  lo[e] = *reinterpret_cast<const uint32_t*>(&l2);
                }
              }
              *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              *reinterpret_cast<uint4*>(dst + CB * NC * SWB) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            } else {
              *reinterpret_cast<uint4*>(dst) = w;
            }
          }
        }
      }
      // the nodes' masks and depths, then per drafted key the columns that see it
      if (tid < kTreeMaxNodes) {
        unsigned long long m0 = 0, m1 = 0;
        if (tid < N) {
          m0 = tree_mask_word(p, pc.b, tid, 0, N);
          if (p.words > 1) m1 = tree_mask_word(p, pc.b, tid, 1, N);
        }
        sMask[2 * tid] = m0;
        sMask[2 * tid + 1] = m1;
        sNodeDepth[tid] = max(__popcll(m0) + __popcll(m1), 1) - 1;
      }
      if (tid == 0) {
        sm_span[0] = kTreeMaxNodes;
        sm_span[1] = 0;
      }
      if (tid < NC) sRef[tid] = FLT_MAX;
      sm_sync();
      if (tid < NC) {
        const int i = sNode[tid];
        const int d = i >= 0 && i < N ? sNodeDepth[i] : 0;
        sDepth[tid] = d;
        if (i >= 0 && i < N) {
          atomicMin(&sm_span[0], d);
          atomicMax(&sm_span[1], d);
        }
      }
      {
        // a warp takes every STEP-th drafted key, its lanes 32 columns
        constexpr int STEP = 4 * C::NWG / NW;
        const int w = warp % NW, c = w * 32 + lane;
        const int node = c < NC ? sNode[c] : -1;
        const bool live = node >= 0 && node < N;
        const unsigned long long m0 = live ? sMask[2 * node] : 0ull, m1 = live ? sMask[2 * node + 1] : 0ull;
        const int floor = live && p.window > 0 ? sNodeDepth[node] - p.window : -1;
        for (int q = warp / NW; q < N; q += STEP) {
          const bool see = ((q < 64 ? m0 : m1) >> (q & 63) & 1) && sNodeDepth[q] > floor;
          const uint32_t v = __ballot_sync(0xffffffffu, see);
          if (lane == 0) sVis[q * NW + w] = v;
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
      sm_sync();
      const int least = sm_span[0], most = sm_span[1];
      const bool scaled = Q4 && *sm_scaled;

      // the piece's tiles that need masks: from `tail` on (drafted rows, a ragged
      // end), the ragged one before a ring's end, and up to `edge` (rows that the
      // window of a deep node has left: positions up to P + most - window)
      const int tA = (s.cntA + KT - 1) / KT;
      const int kept = P - s.start;   // committed rows
      const int tail = (kept < s.cntA ? kept / KT : tA + (kept - s.cntA) / KT) - pc.k0;
      const int seam = s.cntB > 0 ? tA - 1 - pc.k0 : -1;
      const int gone = p.window > 0 ? P + most - p.window - s.start : -1;   // last such row, from the start
      const int edge = gone < 0 ? 0 : (gone < s.cntA ? gone / KT + 1 : tA + (gone - s.cntA) / KT + 1) - pc.k0;

      float l[HC];
#pragma unroll
      for (int c = 0; c < HC; ++c) l[c] = 0.f;

      // A wait that runs out clears ok: the warp then goes through the piece's
      // remaining tiles without waiting, so that every barrier below keeps its
      // threads, and all leave together at the piece's end.
      for (int i = 0; i < n; ++i) {
        const int j = jt + i;
        ok = ok && await(&s_full[j & 1], (uint32_t)(j >> 1) & 1u);
        tc_fence_after();
        const uint32_t t_s = t_lane + (j & 1) * NC;
        if (Q4 && scaled) {
#pragma unroll 1
          for (int c = 0; c < HC; c += 8) {
            float v[8];
            tmem_ld8(t_s + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= sCol[c0 + c + e];
            tmem_st8(t_s + c, v);
          }
          tmem_wait_st();
        }
        // uniform over the CTA: rows that some column does not see
        const bool masked = i >= tail || i == seam || i < edge;
        TreeTile t{0, 0, KT};
        int q = 0;   // >= 0: drafted node q; else the key's distance from the drafted rows
        if (masked) {
          t = tree_tile(p, s, pc.k0 + i, KT);
          q = t.pos + key - P;
        }
        bool poison = false;
        if (masked) {
          // wait for the tile's values: unseen rows are zeroed, rows that are
          // not finite are noted
          // (once the products of the tile before are done, the slots' phases
          // before the awaited ones are known to be over)
          ok = ok && (i == 0 || products(j - 1));
          const int g0 = base + v_slot(i, n) * NSRC;
#pragma unroll
          for (int src = 0; src < NSRC; ++src) {
            const int g = g0 + src;
            ok = ok && await(&full[g % nslots], (uint32_t)(g / nslots) & 1u);
          }
          bool seen = false;
          constexpr uint32_t INF16 = Q4 ? 0x7c00u : 0x7f80u;   // exponents of fp16, bf16
          if (key < t.cnt) {
            if (q < 0) {
              seen = p.window == 0 || least < q + p.window;
            } else {
#pragma unroll
              for (int w = 0; w < NW; ++w) seen |= sVis[q * NW + w] != 0;
            }
            if (seen && ok && (q >= 0 || p.window > 0)) {
#pragma unroll 1
              for (int src = 0; src < NSRC; ++src) {
                const uint8_t* v = slot_ptr((g0 + src) % nslots);
#pragma unroll 1
                for (int ch = 0; ch < D / 8; ++ch) {
                  const uint4 x = *reinterpret_cast<const uint4*>(v + (ch >> 3) * KT * SWB + swz128(key, ch & 7));
                  const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    poison |= (xs[e] & INF16) == INF16 || (xs[e] & INF16 << 16) == INF16 << 16;
                }
              }
            }
          }
          sm_sync();   // every warpgroup has looked
          if (wg == 0 && ok && (!seen || poison) && key < (t.cnt + 15) / 16 * 16) {
#pragma unroll 1
            for (int src = 0; src < NSRC; ++src) {
              uint8_t* v = slot_ptr((g0 + src) % nslots);
#pragma unroll 1
              for (int ch = 0; ch < CB * 8; ++ch)
                *reinterpret_cast<uint4*>(v + (ch >> 3) * KT * SWB + swz128(key, ch & 7)) = make_uint4(0, 0, 0, 0);
            }
          }
        }
        // CH of this key's scores from column c0 + c on, -inf where a column does
        // not see it.  They are read again from tensor memory rather than kept:
        // 32 a thread beside its 32 sums spilled.
        float sv[CH];
        auto scores = [&](int c) {
          if constexpr (CH == 8) tmem_ld8(t_s + c, sv);
          else tmem_ld16(t_s + c, sv);
          tmem_wait_ld();
          if (masked) {
            const int first = c0 + c;
            const uint32_t vis =
                (key >= t.cnt ? 0u : q >= 0 ? sVis[q * NW + first / 32] : ~0u) >> (first & 31);
            const int reach = q < 0 && p.window > 0 ? q + p.window : kTreeMaxNodes;   // depths below it see the key
#pragma unroll
            for (int e = 0; e < CH; ++e) {
              const bool see = (vis >> e & 1u) && sDepth[first + e] < reach;
              sv[e] = !see ? -INFINITY : poison ? NAN : sv[e];
            }
          }
        };
        // score * scale - reference, and the largest of them
        auto shift = [&](int c) {
          float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < CH; e += 4) {
            const float4 r = *reinterpret_cast<const float4*>(sRef + c0 + c + e);   // negated references
            float x0 = r.x, x1 = r.y, x2 = r.z, x3 = r.w;
            fma2(x0, x1, sv[e], sv[e + 1], p.scale_log2, p.scale_log2);
            fma2(x2, x3, sv[e + 2], sv[e + 3], p.scale_log2, p.scale_log2);
            sv[e] = x0; sv[e + 1] = x1; sv[e + 2] = x2; sv[e + 3] = x3;
            top[0] = fmax3f(top[0], x0, x1);
            top[1] = fmax3f(top[1], x2, x3);
          }
          return fmaxf(top[0], top[1]);
        };
        // the first tile of a piece takes its maxima as references; later ones
        // keep them unless a score exceeds its own by more than the slack
        const bool first = i == 0;
        bool grow = first;
        if (!first) {
          float over = -INFINITY;
#pragma unroll
          for (int c = 0; c < HC; c += CH) {
            scores(c);
            over = fmaxf(over, shift(c));
          }
          grow = any_of(2 + wg, 128, over > SLACK);
        }
        if (grow) {
#pragma unroll
          for (int c = 0; c < HC; c += CH) {
            scores(c);
            const float m = reduce_scatter<CH>(sv, lane, fmaxop);
            if (lane < CH) sWarp[quarter * NC + c0 + c + lane] = m;
          }
          wg_sync(wg);
          if ((tid & 127) < HC) {
            const int c = c0 + (tid & 127);
            const float m = fmaxf(fmaxf(sWarp[c], sWarp[NC + c]), fmaxf(sWarp[2 * NC + c], sWarp[3 * NC + c]));
            const float old = -sRef[c], top = fmaxf(old, m * p.scale_log2 - C::RAISE);
            sAlpha[c] = fast_exp2(old - top);
            sRef[c] = -top;
          }
          // O holds every product before this tile once the last one is done
          ok = ok && (first || products(j - 1));
          tc_fence_after();
          wg_sync(wg);
          if (!first) {
#pragma unroll
            for (int c = 0; c < HC; c += 8) {
              float al[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                al[e] = sAlpha[c0 + c + e];
                l[c + e] *= al[e];
              }
#pragma unroll
              for (int src = 0; src < NACC; ++src) {
                const uint32_t to = t_lane + (2 + src) * NC + c;
                float o[8];
                tmem_ld8(to, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] *= al[e];
                tmem_st8(to, o);
              }
            }
            tmem_wait_st();
          }
        }

        // P of this key: 2^x, 16 bits
        const int pj = NPB == 2 ? j - 2 : j - 1;   // the tile whose products read the buffer last
        ok = ok && (pj < 0 || products(pj));
        uint8_t* pb = sP + (NPB == 2 ? (j & 1) * C::P_BYTES : 0);
#pragma unroll
        for (int c = 0; c < HC; c += CH) {
          if (HC > CH || grow) {
            scores(c);
            shift(c);
          }
#pragma unroll
          for (int h = 0; h < CH; h += 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = h; e < h + 8; e += 2) {
              const float e0 = fast_exp2(sv[e]), e1 = fast_exp2(sv[e + 1]);
              add2(l[c + e], l[c + e + 1], e0, e1);
              w[(e - h) / 2] = pack2<Q4>(e0, e1);
            }
            const int cc = c0 + c + h;
            *reinterpret_cast<uint4*>(pb + (cc >> 6) * KT * SWB + swz128(key, (cc & 63) >> 3)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        // one arrival a warp: 32 lanes on one barrier would be taken one by one
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&p_full[j & 1]);
      }
      // the sums of the columns over all keys, and the last products
      const int jl = jt + n - 1;
      ok = ok && products(jl);
      if (any_of(1, C::SM, !ok)) break;
      tc_fence_after();
      constexpr int RN = HC < 32 ? HC : 32;
#pragma unroll
      for (int b0 = 0; b0 < HC; b0 += RN) {
        const float m = reduce_scatter<RN>(l + b0, lane, addop);
        if (lane < RN) sWarp[quarter * NC + c0 + b0 + lane] = m;
      }
      sm_sync();
      const bool whole = n == pc.tiles;
      float* rec = p.ws + ((size_t)(2 * blockIdx.x + (pc.first ? 0 : 1)) * p.row_tiles + rt) *
                              tree_record_floats(NC, D);
      if (tid < NC) {
        const float sum = (sWarp[tid] + sWarp[NC + tid]) + (sWarp[2 * NC + tid] + sWarp[3 * NC + tid]);
        sAlpha[tid] = sum == 0.f ? 0.f : whole ? 1.f / sum : 1.f;
        if (!whole) {
          rec[NC * D + tid] = -sRef[tid];
          rec[NC * D + NC + tid] = sum;
        }
      }
      sm_sync();
      float bw[NACC];
#pragma unroll
      for (int src = 0; src < NACC; ++src) {
        bw[src] = 1.f;
        if (WGT && row < D) bw[src] = p.b[C::PAIR ? key >> 6 : src][(size_t)pc.h * D + chan];
      }
      float* pair = reinterpret_cast<float*>(sP) + wg * 64 * 9;   // (P is read; 9: no bank conflicts)
#pragma unroll 1
      for (int c = c0; c < c0 + HC; c += 8) {
        float o[NACC][8], x[8];
#pragma unroll
        for (int src = 0; src < NACC; ++src)
          tmem_ld8(t_lane - c0 + (2 + src) * NC + c, o[src]);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float w = sAlpha[c + e];
          float y = o[0][e];
          if constexpr (WGT) y *= bw[0];
          if constexpr (NACC == 2) y = fmaf(bw[1], o[1][e], y);
          x[e] = w == 0.f ? 0.f : w * y;
        }
        if constexpr (C::PAIR) {   // the second source's half joins the first's
          if (key >= 64) {
#pragma unroll
            for (int e = 0; e < 8; ++e) pair[row * 9 + e] = x[e];
          }
          wg_sync(wg);
          if (key < 64) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += pair[row * 9 + e];
          }
          wg_sync(wg);
        }
        if (key < D) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int cc = c + e;
            if (whole) {
              const int node = sNode[cc];
              if (node >= 0 && node < N)
                static_cast<__nv_bfloat16*>(p.out)[(unit * p.G * p.T + rt * NC + cc) * D + chan] =
                    __float2bfloat16_rn(x[e]);
            } else {
              rec[(size_t)cc * D + chan] = x[e];
            }
          }
        }
      }
      if (!whole)
        tree_publish<__nv_bfloat16, D, NC, C::SM>(p, cut, sq.pre, pc.b, pc.h, N, tid, merge_flag, sWarp,
                                                       sm_sync);
      if (tid == 0) *sm_scaled = 0;
      sm_sync();   // shared words are free for the next piece
      base += 2 * n * NSRC;
      jt += n;
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // no role may have awaited the last copies and products: let them finish
    if (warp == C::PRODUCER_WARP && lane == 0) {
      const int issued = *sm_issued, nring = Q4 ? nraw : nslots;
      uint64_t* ring_full = Q4 ? raw_full : full;
      for (int g = max(0, issued - nring); g < issued; ++g)
        (void)mbar_wait_bounded(&ring_full[g % nring], (uint32_t)(g / nring) & 1u, kDrainLimitNs);
    }
    if ((warp == C::QK_WARP || warp == C::PV_WARP) && elect_one()) {
      mma_commit(&drain[warp - C::QK_WARP]);
      (void)mbar_wait_bounded(&drain[warp - C::QK_WARP], 0, kDrainLimitNs);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
  }
  if (warp == C::QK_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Tile slots and shared memory of a configuration; 0 slots if it does not fit.
template <int D, int NSRC, bool WGT, int NC, bool Q4>
void size_tc(int B, TreePlan* plan) {
  using C = TcCfg<D, NSRC, WGT, NC, Q4>;
  const int fixed = 1024 + C::ring_off(B) + C::OVERRUN;
  int left = SMEM_LIMIT - fixed;
  plan->raw_slots = 0;
  if (Q4) {
    // records for at least a tile a group, the rest beside as many tile slots as
    // the MMAs need (and two tiles more where they are small)
    constexpr int GROUPS = DQ_THREADS / DQ_GROUP;
    const int want = C::SLOT <= 16384 ? 4 * NSRC : GROUPS;
    int raw = (left - want * C::SLOT) / C::RAW / GROUPS * GROUPS;
    raw = raw > MAX_RAW ? MAX_RAW : raw < GROUPS ? GROUPS : raw;
    plan->raw_slots = raw;
    left -= raw * C::RAW;
  }
  int slots = left > 0 ? left / C::SLOT : 0;
  if (slots > MAX_SLOTS) slots = MAX_SLOTS;
  if (Q4) slots = slots / (DQ_THREADS / DQ_GROUP) * (DQ_THREADS / DQ_GROUP);
  if (C::PAIR) slots &= ~1;
  if (slots < 2 * NSRC) slots = 0;
  plan->slots = slots;
  plan->smem_bytes = (size_t)fixed + (size_t)slots * C::SLOT + (size_t)plan->raw_slots * C::RAW;
}

template <int D, int NSRC, bool WGT, int NC, bool Q4>
cudaError_t launch_tc(const TreeParams& p, const TreeArgs& a, const TreePlan& plan, cudaStream_t stream) {
  TcMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  for (int i = 0; i < 4 && !Q4; ++i) {
    const TileMaps* m = i < 2 ? a.k_maps[i & 1] : a.v_maps[i & 1];
    if ((i & 1) >= NSRC) continue;
    if (!m || !m->valid) return cudaErrorInvalidValue;
    std::memcpy(&maps.full[i], m->full, sizeof(CUtensorMap));
    std::memcpy(&maps.tail[i], m->tail, sizeof(CUtensorMap));
  }
  using C = TcCfg<D, NSRC, WGT, NC, Q4>;
  auto kern = tree_tc_kernel<D, NSRC, WGT, NC, Q4>;
  // the softmax warpgroups' larger share of the registers has to fit the launch
  // allocation, or it would never be granted: refuse instead
  static KernelReady ready;
  const cudaError_t e = ready.check(kern, a.device, SMEM_LIMIT, C::THREADS, C::REGS_SPLIT);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(plan.ranges, plan.row_tiles), dim3(C::THREADS), plan.smem_bytes, stream, maps,
                    p, plan.slots, plan.raw_slots);
}

// Call f with the plan's sources, weights and columns and whether the caches
// are 4-bit as integral constants.
template <int D, typename F>
auto dispatch_tc(const TreeArgs& a, int rows, F f) {
  auto fmt = [&](auto ns, auto wt, auto nc) {
    // 4-bit caches take at most 64 columns: 128 registers a softmax thread
    if constexpr (decltype(nc)::value <= 64) {
      if (a.q4) return f(ns, wt, nc, std::true_type());
    }
    return f(ns, wt, nc, std::false_type());
  };
  auto cols = [&](auto ns, auto wt) {
    // two sources of more than 64 channels leave too little room for tiles
    // beside 128 columns
    constexpr bool wide = !(D > 64 && decltype(ns)::value == 2);
    switch (rows) {
      case 16: return fmt(ns, wt, std::integral_constant<int, 16>());
      case 32: return fmt(ns, wt, std::integral_constant<int, 32>());
      case 64: return fmt(ns, wt, std::integral_constant<int, 64>());
      default: return fmt(ns, wt, std::integral_constant<int, wide ? 128 : 64>());
    }
  };
  if (a.k[1]) return cols(std::integral_constant<int, 2>(), std::true_type());
  if (a.a[0]) return cols(std::integral_constant<int, 1>(), std::true_type());
  return cols(std::integral_constant<int, 1>(), std::false_type());
}

template <int D>
void tree_tc_size(const TreeArgs& a, TreePlan* plan) {
  dispatch_tc<D>(a, plan->rows, [&](auto ns, auto wt, auto nc, auto q4) {
    size_tc<D, decltype(ns)::value, decltype(wt)::value, decltype(nc)::value, decltype(q4)::value>(a.batch, plan);
  });
}

template <int D>
cudaError_t tree_tc_run(const TreeParams& p, const TreeArgs& a, const TreePlan& plan, cudaStream_t stream) {
  return dispatch_tc<D>(a, plan.rows, [&](auto ns, auto wt, auto nc, auto q4) {
    return launch_tc<D, decltype(ns)::value, decltype(wt)::value, decltype(nc)::value, decltype(q4)::value>(
        p, a, plan, stream);
  });
}

}  // namespace
}  // namespace fkv
