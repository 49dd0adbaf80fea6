// What the kernels of fkv_tree_attn share: the drafted sequences of a call,
// the cut of its key tiles into one range per CTA, and the merge of the
// partial results of a (sequence, KV head) unit that several ranges share.
//
// What a call computes: sequence b has P committed rows and N drafted nodes
// whose keys and values lie at positions P .. P + N - 1.  Node i of query
// head h sees every position t < P and position P + j where bit j of its mask
// word is set:
//     o_{h,i} = sum_t softmax_t(scale * q_{h,i} . K_t) V_t,  t visible to i,
// and 0 where nothing is visible.  With a window W the node's depth is
// d_i = max(popcount(mask_i), 1) - 1, its position P + d_i, and it sees the
// visible keys whose position (P + d_j for drafted node j) is above
// P + d_i - W.
#pragma once

#include <cfloat>
#include <cstdint>

#include "fkv_device.cuh"
#include "fkv_kernels.h"

namespace fkv {

constexpr int kTreeMaxNodes = 128;
constexpr int kTreeKeyTile = 128;    // keys per tile of the tensor-core kernels
constexpr int kTreeTailRows = 16;    // rows of the boxes of a ragged tile

struct TreeParams;
// tree_tc_impl.cuh, one unit per head dimension
void tree_tc_size_64(const TreeArgs& a, TreePlan* plan);
void tree_tc_size_80(const TreeArgs& a, TreePlan* plan);
void tree_tc_size_96(const TreeArgs& a, TreePlan* plan);
void tree_tc_size_128(const TreeArgs& a, TreePlan* plan);
cudaError_t tree_tc_run_64(const TreeParams&, const TreeArgs&, const TreePlan&, cudaStream_t);
cudaError_t tree_tc_run_80(const TreeParams&, const TreeArgs&, const TreePlan&, cudaStream_t);
cudaError_t tree_tc_run_96(const TreeParams&, const TreeArgs&, const TreePlan&, cudaStream_t);
cudaError_t tree_tc_run_128(const TreeParams&, const TreeArgs&, const TreePlan&, cudaStream_t);
void tree_f32_plan(const TreeArgs& a, int num_sms, TreePlan* plan);
cudaError_t tree_f32_launch(const TreeParams& p, const TreeArgs& a, const TreePlan& plan,
                            cudaStream_t stream);

struct TreeParams {
  const void* k[2];
  const void* v[2];
  const float* a[2];
  const float* b[2];
  const void* q;                   // [B, H_q, T, D]
  void* out;                       // [B, H_q, T, D]
  const int32_t* seq_lens;         // [B] committed rows
  const int32_t* node_counts;      // [B] drafted nodes, or null: T
  const unsigned long long* mask;  // [B, T, words]
  float* ws;                       // partials
  unsigned long long* counters;    // one arrival word per (b, kh, row tile)
  int* status;
  const unsigned long long* wait_limit;
  int B, H, G, S_max, T, words;
  int window, ring;
  int row_tiles;    // row tiles of a unit (grid.y)
  unsigned epoch;
  float scale_log2; // softmax scale * log2(e)
};

// What a CTA keeps of the sequences in shared memory (3 B + 1 words).
struct TreeSeqs {
  int* pre;   // [B + 1] key tiles of one head of the sequences before b
  int* P;     // [B] committed rows (-1: lengths out of range)
  int* N;     // [B] drafted nodes (0: nothing to do)
};
__host__ __device__ constexpr size_t tree_seqs_bytes(int B) { return (size_t)(3 * B + 1) * 4; }

__device__ __forceinline__ TreeSeqs tree_seqs(int* words, int B) {
  return TreeSeqs{words, words + B + 1, words + 2 * B + 1};
}

// One sequence of a call: its attended positions [start, n) lie in the cache
// rows as one run of cntA rows and, in a ring that wraps, a second of cntB.
struct TreeSeq {
  int P, N, start, cntA, cntB;
};

// The lengths of sequence b as the caller gave them; false if out of range.
__device__ __forceinline__ bool tree_lengths(const TreeParams& p, int b, int& P, int& N) {
  P = p.seq_lens[b];
  N = p.node_counts ? p.node_counts[b] : p.T;
  return P >= 0 && N >= 0 && N <= p.T && P <= p.S_max - N;
}

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int P, int N) {
  TreeSeq s{P, N, 0, 0, 0};
  if (N == 0) return s;
  const int n = P + N;
  if (p.window > 0 && P >= p.window) s.start = P - p.window + 1;
  int end = n;
  if (p.ring > 0) {
    const long long wrap = ((long long)s.start / p.ring + 1) * p.ring;
    if (wrap < n) end = (int)wrap;
  }
  s.cntA = end - s.start;
  s.cntB = n - end;
  return s;
}

__device__ __forceinline__ int tree_tiles(const TreeSeq& s, int KT) {
  return (s.cntA + KT - 1) / KT + (s.cntB + KT - 1) / KT;
}

// Tile k of a sequence: its first position and cache row, and its row count.
// A tile never crosses the end of a ring.
struct TreeTile {
  int pos, row, cnt;
};

__device__ __forceinline__ TreeTile tree_tile(const TreeParams& p, const TreeSeq& s, int k, int KT) {
  const int tA = (s.cntA + KT - 1) / KT;
  TreeTile t;
  if (k < tA) {
    t.pos = s.start + k * KT;
    t.cnt = min(KT, s.cntA - k * KT);
  } else {
    t.pos = s.start + s.cntA + (k - tA) * KT;
    t.cnt = min(KT, s.cntB - (k - tA) * KT);
  }
  t.row = p.ring > 0 ? t.pos % p.ring : t.pos;
  return t;
}

// Word w of node i's mask with the bits of nodes that do not exist cleared.
__device__ __forceinline__ unsigned long long tree_mask_word(const TreeParams& p, int b, int i,
                                                             int w, int N) {
  const unsigned long long m = p.mask[((size_t)b * p.T + i) * p.words + w];
  const int left = N - 64 * w;
  return left >= 64 ? m : left <= 0 ? 0ull : m & ((1ull << left) - 1);
}

__device__ __forceinline__ int tree_depth(const TreeParams& p, int b, int i, int N) {
  int c = 0;
  for (int w = 0; w < p.words; ++w) c += __popcll(tree_mask_word(p, b, i, w, N));
  return c > 1 ? c - 1 : 0;
}

// The cut: the tiles of all units, unit by unit, in `ranges` equal contiguous
// ranges.  Where ranges would be short (six tiles and fewer), a boundary within
// `snap` tiles of a unit's start or end moves there: on the tensor cores,
// writing, announcing and merging a partial takes as long as four to six tiles.
// Measured with snap = 0 and 3 (lite unless said): 32 units of 5 tiles 14.1 and
// 12.1 us, 64 of 6 19.5 and 11.5, 256 of 3 23.3 and 17.2, 32 of 12 27.2 and 18.6
// (fused 34.7 and 27.8), fused 128 of 7 25.4 and 16.3.  It loses where few units
// of dear tiles leave most CTAs without work: fused 16 units of 17 tiles 17.5 and
// 20.0 us, 16 of 10 19.6 and 20.8; lite units like these still gain (8 of 32
// tiles 20.6 and 18.7, 16 of 9 13.9 and 13.5), so the rule asks for neither the
// units nor the sources.  fp32 tiles take longer than a merge (snap = 0: 12.5 us
// a tiny call, 19.3 with 3).  Fills sq, and zeros the
// output of the sequences whose lengths are out of range; every thread of the
// CTA takes part.
struct TreeCut {
  long long total;
  int ranges;
  int snap;
};

template <typename E, int D>
__device__ __forceinline__ TreeCut tree_cut(const TreeParams& p, const TreeSeqs& sq, int KT,
                                            int max_ranges, int snap) {
  const bool first = blockIdx.x == 0 && blockIdx.y == 0;
  bool bad = false;
  for (int i = threadIdx.x; i < p.B; i += blockDim.x) {
    int P, N;
    if (!tree_lengths(p, i, P, N)) {
      bad = true;
      P = -1;
      N = 0;
    }
    sq.P[i] = P;
    sq.N[i] = N;
    sq.pre[i + 1] = tree_tiles(tree_seq(p, P, N), KT);
  }
  if (__syncthreads_or(bad) && first) {
    if (threadIdx.x == 0) flag_status(p.status, kDevBadArg);
    const size_t n = (size_t)p.H * p.G * p.T * D * sizeof(E) / 16;
    for (int b = 0; b < p.B; ++b) {
      if (sq.P[b] >= 0) continue;
      uint4* o = reinterpret_cast<uint4*>(p.out) + (size_t)b * n;
      for (size_t i = threadIdx.x; i < n; i += blockDim.x) o[i] = make_uint4(0, 0, 0, 0);
    }
  }
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int run = 0;
    for (int base = 0; base < p.B; base += 32) {
      int x = base + lane < p.B ? sq.pre[base + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (base + lane < p.B) sq.pre[base + lane + 1] = run + x;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) sq.pre[0] = 0;
  }
  __syncthreads();
  TreeCut c;
  c.total = (long long)p.H * sq.pre[p.B];
  c.ranges = (int)min((long long)max_ranges, c.total);
  c.snap = c.total <= 6ll * c.ranges ? snap : 0;
  return c;
}

// A run of tiles [k0, k1) of unit (b, h) inside a range.
struct TreePiece {
  int b, h, k0, k1, tiles;
  bool first;   // the range's first piece
};

// The first tile of a range, as cut.
__device__ __forceinline__ long long tree_bound(const TreeCut& c, const int* pre, int B, int H,
                                                long long range) {
  const long long t = range * c.total / c.ranges;
  if (c.snap == 0 || t >= c.total) return t;
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((long long)H * pre[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  const int n = pre[lo + 1] - pre[lo];
  const int k = (int)((t - (long long)H * pre[lo]) % n);   // of the unit's n tiles
  return k <= c.snap ? t - k : n - k <= c.snap ? t + n - k : t;
}

struct TreeWalk {
  long long t, t1;
  int b, h, k;
  bool first;

  __device__ __forceinline__ void begin(const TreeCut& c, const int* pre, int B, int H, int range) {
    t = tree_bound(c, pre, B, H, range);
    t1 = tree_bound(c, pre, B, H, range + 1);
    first = true;
    if (t >= t1) return;   // nothing is left of the range
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if ((long long)H * pre[mid + 1] > t) hi = mid; else lo = mid + 1;
    }
    const long long off = t - (long long)H * pre[lo];
    const int n = pre[lo + 1] - pre[lo];
    b = lo;
    h = (int)(off / n);
    k = (int)(off - (long long)h * n);
  }
  __device__ __forceinline__ bool next(const int* pre, int B, int H, TreePiece& pc) {
    if (t >= t1) return false;
    const int n = pre[b + 1] - pre[b];
    pc.b = b;
    pc.h = h;
    pc.k0 = k;
    pc.k1 = (int)min((long long)n, k + (t1 - t));
    pc.tiles = n;
    pc.first = first;
    first = false;
    t += pc.k1 - pc.k0;
    k = 0;
    if (++h == H) {
      h = 0;
      ++b;
      while (b < B && pre[b + 1] == pre[b]) ++b;
    }
    return true;
  }
};

// Partials.  A piece that is not its whole unit leaves (o, m, l) of its rows
// in the slot 2 * range (the range's first piece) or 2 * range + 1 (its last);
// a record is o[ROWS][D], m[ROWS], l[ROWS].
__host__ __device__ constexpr int tree_record_floats(int rows, int D) { return rows * (D + 2); }

// The ranges that hold tiles of unit (b, h), and the slot of one of them.
struct TreeUnit {
  long long first, last;   // ranges
  bool first_is_tail;      // the first range's piece is its last one
};

__device__ __forceinline__ TreeUnit tree_unit(const TreeCut& c, const int* pre, int B, int H, int b, int h) {
  const long long n = pre[b + 1] - pre[b];
  const long long u0 = (long long)H * pre[b] + h * n, u1 = u0 + n;
  // boundaries r * total / ranges up to `low` fall on u0 or before, those from
  // u1 - snap on on u1 or behind
  const long long low = u0 + min((long long)c.snap, n - 1);
  TreeUnit u;
  u.first = ((low + 1) * c.ranges + c.total - 1) / c.total - 1;
  u.last = max(u.first, ((u1 - c.snap) * c.ranges + c.total - 1) / c.total - 1);
  u.first_is_tail = tree_bound(c, pre, B, H, u.first) < u0;
  return u;
}

__device__ __forceinline__ void tree_store4(float* dst, const float* x) {
  *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void tree_store4(__nv_bfloat16* dst, const float* x) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
  *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                              *reinterpret_cast<const uint32_t*>(&hi));
}

// Announce a written partial of unit (b, h), row tile blockIdx.y; the CTA
// whose arrival completes the unit merges its pieces by their log-sum-exp
// weights into the output rows.  Called by NT threads (index tid) that `sync`
// brings together; all of them have written their part before.  scratch holds
// 2 * ROWS floats of shared memory.  A thread's items (four channels of a row)
// are loaded together, so a merge of P pieces takes about P trips to L2 (fewer
// where a thread has one or two items, whose loop is unrolled).
template <typename E, int D, int ROWS, int NT, typename Sync>
__device__ __forceinline__ void tree_publish(const TreeParams& p, const TreeCut& c, const int* pre,
                                             int b, int h, int N, int tid, int* flag, float* scratch,
                                             Sync sync) {
  const TreeUnit u = tree_unit(c, pre, p.B, p.H, b, h);
  const int P = (int)(u.last - u.first + 1);
  const int rt = blockIdx.y;
  __threadfence();
  sync();
  if (tid == 0) {
    unsigned long long* word = p.counters + ((size_t)b * p.H + h) * p.row_tiles + rt;
    const unsigned got = unit_arrive(word, p.epoch);
    if (got == 0) flag_status(p.status, kDevTimeout);
    // no arrival of this call can follow the last: clear the word, so that a
    // replay of this launch (the same epoch) starts at one
    if (got == (unsigned)P) *word = 0ull;
    *flag = got == (unsigned)P;
    __threadfence();
  }
  sync();
  if (!*flag) return;
  constexpr int REC = tree_record_floats(ROWS, D);
  constexpr int C4 = D / 4;
  constexpr int ITEMS = (ROWS * C4 + NT - 1) / NT;
  const int rows = min(ROWS, p.G * p.T - rt * ROWS);
  auto rec = [&](int i) {
    const long long slot = 2 * (u.first + i) + (i == 0 && u.first_is_tail ? 1 : 0);
    return p.ws + ((size_t)slot * p.row_tiles + rt) * REC + ROWS * D;   // its m; o lies before
  };
  float* sTop = scratch;
  float* sInv = scratch + ROWS;
  if (tid < ROWS) {
    float M = -FLT_MAX, L = 0.f;
#pragma unroll 4
    for (int i = 0; i < P; ++i) {
      const float m = __ldcg(rec(i) + tid), l = __ldcg(rec(i) + ROWS + tid);
      const float top = fmaxf(M, m);
      L = L * exp2f(M - top) + l * exp2f(m - top);
      M = top;
    }
    sTop[tid] = M;
    sInv[tid] = L == 0.f ? 0.f : 1.f / L;
  }
  sync();
  float acc[ITEMS][4];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[k][e] = 0.f;
#pragma unroll(ITEMS <= 2 ? 4 : 1)
  for (int i = 0; i < P; ++i) {
    const float* m = rec(i);
    const float* o = m - ROWS * D;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int it = tid + k * NT;
      if (it >= ROWS * C4) break;
      const int r = it / C4;
      const float w = exp2f(__ldcg(m + r) - sTop[r]);
      const float4 x = __ldcg(reinterpret_cast<const float4*>(o + it * 4));
      acc[k][0] = fmaf(w, x.x, acc[k][0]);
      acc[k][1] = fmaf(w, x.y, acc[k][1]);
      acc[k][2] = fmaf(w, x.z, acc[k][2]);
      acc[k][3] = fmaf(w, x.w, acc[k][3]);
    }
  }
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int it = tid + k * NT;
    if (it >= ROWS * C4) break;
    const int r = it / C4, d = (it - r * C4) * 4;
    const int row = rt * ROWS + r;
    if (r >= rows || row % p.T >= N) continue;
    const float inv = sInv[r];
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[k][e] = inv == 0.f ? 0.f : acc[k][e] * inv;
    tree_store4(static_cast<E*>(p.out) + (((size_t)b * p.H + h) * p.G * p.T + row) * D + d, acc[k]);
  }
}

}  // namespace fkv
