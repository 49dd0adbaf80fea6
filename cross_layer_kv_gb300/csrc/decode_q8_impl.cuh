// Decode attention over 8-bit caches (e4m3 codes, one scale per 32 rows of a
// KV head; q8_device.cuh).
//
// Every warp streams a contiguous range of the call's rows through a ring of
// its own (cp.async.bulk, one mbarrier a stage), as in decode_split_kernel.
// Ranges are cut at groups of 16 rows, counted from rows that are multiples of
// 16, so that a group has one key scale and one value scale; they come with
// the codes, in 16-byte pieces.
//
// A (sequence, KV head) unit that lies in one warp's range is finished by that
// warp.  Of the others a warp holds at most two, at its range's ends; these
// partials meet in shared memory once the CTA's warps are done, and only a unit
// that reaches into other CTAs goes through global memory, one partial a CTA.
// The last CTA of such a unit merges, with one warp where there are few
// partials and with all of them where there are many.  (A partial a warp, with
// every arrival and merge in global memory, as the other formats do it, costs
// 16 us on the smallest calls and 30 us on 128 units of 512 rows.)
//
// The products are warp-level matrix instructions (m16n8k16, fp16 operands,
// fp32 sums) on fragments that are converted in registers: e4m3 codes are
// exact in fp16 and two adjacent codes become one operand register in one
// instruction, so an element costs half an instruction to convert (and its
// share of a byte permute, for values) where scalar fp32 arithmetic costs
// three to five.  Nothing goes back to shared memory, which is why these are
// not tcgen05 products: their operands would have to be written there as fp16,
// twice the bytes that arrive.  332M Lite call (0.27 GB, 40 us at the measured
// copy rate): 78 us with scalar arithmetic, 50 with these; 4B fused call of
// full length (2.69 GB, 402 us): 549 us with 16 rows of values' products, 442
// with the transposed ones below, which take half the registers and products.
//
// Scores: S [16 x 8 keys] = Q [16 x 16 channels] . K^T.  Row g < G of Q is
// query head g of the group (times the key weights and a power of two), to
// fp16; row g + 8 is what that rounding left, to fp16 again: 22 bits of the
// query, at no cost, since the rows are there.
// Values: O^T [16 channels x 8] += V^T [16 x 16 keys] . P^T, whose column g is
// head g (a score's place in the first product is its weight's place in the
// second).  With the value scale r in the exponent, P' = p r = 2^(s + log2 r
// - M), no scale can take P' out of fp16's range (M is the running maximum of
// that sum, with a slack of 2^8 before O is rescaled); the softmax's sum takes
// P' / r.  P' is rounded to fp16, 2^-12, for bf16 outputs; fp32 contexts add a
// second product with what the rounding left.  Two value sources have one
// exponent, of the larger scale, and two P with the factors r_i / r.
//
// Fragment layout: lane 4 n + q holds channels [q D/4, (q + 1) D/4) of key n
// for the scores: contiguous bytes of a row, in which a step of 16 channels
// takes 4 of each lane (the channels' order is the same in Q, so any will do).
// For values, lane 4 n + q holds keys 2q, 2q+1, 2q+8, 2q+9 of the group and
// D/8 channels, contiguous bytes again, two to a product; a byte permute pairs
// two keys' codes.  Which row of the group a key index stands for is free too,
// and chosen so that the lanes of a load meet in few banks.
#pragma once

#include <type_traits>

#include "decode_impl.cuh"
#include "q8_device.cuh"

namespace fkv {

constexpr float kQ8Slack = 8.f;   // log2 growth of the running max tolerated before O is rescaled
constexpr float kQ8Bias = 7.f;    // P' < 2^15 and exact above 2^-31 of its frame

// Warps per CTA, ring stages per warp, groups of 16 rows per stage.
template <int D, int NSRC>
struct Q8Shape {
  static constexpr int W = NSRC == 1 ? 12 : 8;
  static constexpr int NS = 2;
  static constexpr int SB = NSRC == 1 ? 8192 : 12288;   // bytes of codes per stage
  static constexpr int GR0 = SB / (2 * NSRC * 16 * D);
  static constexpr int GROUPS = GR0 < 1 ? 1 : GR0;
};

template <int D, int NSRC>
struct Q8Cfg {
  using S = Q8Shape<D, NSRC>;
  static constexpr int TR = 16 * S::GROUPS;            // rows per tile
  static constexpr int TILE_BYTES = TR * D;            // codes of one plane's tile
  // scales of one plane's tile in whole 16-byte pieces (4 blocks each); a tile
  // that wraps in a ring has two such runs
  static constexpr int SCW = ((TR - 1) / (4 * kQ8Block) + 2) * 4;
  static constexpr int CODE_BYTES = 2 * NSRC * TILE_BYTES;
  static constexpr int STAGE_BYTES = CODE_BYTES + 2 * NSRC * 2 * SCW * 4;
  static_assert(TILE_BYTES % 16 == 0 && STAGE_BYTES % 16 == 0, "stages are read in 16-byte pieces");
};

struct Q8Params {
  SplitParams p;
  const float* ks[2];
  const float* vs[2];
  int G;
  int aux_bytes;
};

// d += a b: m16n8k16, fp16 operands, fp32 sums.
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t f16x2_of(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// (x, y) = hi + lo in fp16 pairs.
__device__ __forceinline__ void split_f16(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// N bytes of shared memory (a multiple of 4, aligned to the largest power of
// two that divides N, 16 at most) as words.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* src, uint32_t* w) {
  if constexpr (N % 16 == 0) {
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
      const uint4 q = reinterpret_cast<const uint4*>(src)[i];
      w[4 * i] = q.x;
      w[4 * i + 1] = q.y;
      w[4 * i + 2] = q.z;
      w[4 * i + 3] = q.w;
    }
  } else if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      const uint2 q = reinterpret_cast<const uint2*>(src)[i];
      w[2 * i] = q.x;
      w[2 * i + 1] = q.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = reinterpret_cast<const uint32_t*>(src)[i];
  }
}

// The codes of column n's channels in a row of values: D/8 of them, as
// (D + 31) / 32 words (the last one half used at D = 80).  D = 64, 128: bytes
// [n D/8, (n + 1) D/8); D = 80, 96: 8 of the first 64 channels and 2 or 4 of
// the rest.
template <int D>
__device__ __forceinline__ void load_value(const uint8_t* row, int n, uint32_t* w) {
  if constexpr (D == 128) {
    load_words<16>(row + n * 16, w);
  } else {
    load_words<8>(row + n * 8, w);
    if constexpr (D == 96) w[2] = *reinterpret_cast<const uint32_t*>(row + 64 + n * 4);
    if constexpr (D == 80) w[2] = *reinterpret_cast<const uint16_t*>(row + 64 + n * 2);
  }
}

// The channels of lane 4 n + q in the value products, in order: 8 (D = 128: 16)
// from n * 8 (n * 16) on, then D = 80, 96: 2 or 4 of those behind the 64th.
template <int D>
__device__ __forceinline__ int value_channel(int n, int k) {
  constexpr int main = D == 128 ? 16 : 8, rest = D / 8 - main;
  return k < main ? n * main + k : 64 + n * rest + (k - main);
}

__device__ __forceinline__ void store2(float* dst, float x, float y) {
  *reinterpret_cast<float2*>(dst) = make_float2(x, y);
}
__device__ __forceinline__ void store2(__nv_bfloat16* dst, float x, float y) {
  *reinterpret_cast<__nv_bfloat162*>(dst) = __floats2bfloat162_rn(x, y);
}

// log2, within 2^-22 (exact for powers of two).
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Count one arrival on a unit's word for call `epoch`; the count with this one
// (0 if the retry bound ran out).  One atomic addition where the word carries
// the epoch already.  A word with another epoch (whatever the workspace held)
// is replaced by the first to see it; an addition to it counts nowhere, and
// who made it arrives again.
__device__ __forceinline__ unsigned q8_arrive(unsigned long long* word, unsigned epoch) {
  const unsigned long long first = ((unsigned long long)epoch << 32) | 1ull;
#pragma unroll 1
  for (int i = 0; i < (1 << 16); ++i) {
    unsigned long long old = atomicAdd(word, 1ull);
    if ((unsigned)(old >> 32) == epoch) return (unsigned)old + 1u;
    ++old;
#pragma unroll 1
    for (int k = 0; k < (1 << 16) && (unsigned)(old >> 32) != epoch; ++k) {
      const unsigned long long prev = atomicCAS(word, old, first);
      if (prev == old) return 1u;
      old = prev;
    }
  }
  return 0;
}

// A warp's running combination of partials of G heads, lane = channel.
template <int D, int G>
struct Q8Acc {
  static constexpr int DPL = (D + 31) / 32;
  float M[G], L[G], o[G][DPL];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      M[g] = -FLT_MAX;
      L[g] = 0.f;
#pragma unroll
      for (int k = 0; k < DPL; ++k) o[g][k] = 0.f;
    }
  }
  // add a record (o[D], m, l per head); GLOBAL: read through L2, where other
  // SMs put it
  template <bool GLOBAL>
  __device__ __forceinline__ void add(const float* rec, int lane) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float* r = rec + g * partial_stride(D);
      const float m = GLOBAL ? __ldcg(r + D) : r[D], l = GLOBAL ? __ldcg(r + D + 1) : r[D + 1];
      const float top = fmaxf(M[g], m);
      const float a = exp2f(M[g] - top), b = exp2f(m - top);
      L[g] = L[g] * a + l * b;
#pragma unroll
      for (int k = 0; k < DPL; ++k) {
        const int d = lane + 32 * k;
        const float x = d < D ? (GLOBAL ? __ldcg(r + d) : r[d]) : 0.f;
        o[g][k] = o[g][k] * a + x * b;
      }
      M[g] = top;
    }
  }
  __device__ __forceinline__ void store(float* rec, int lane) const {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float* r = rec + g * partial_stride(D);
#pragma unroll
      for (int k = 0; k < DPL; ++k)
        if (lane + 32 * k < D) r[lane + 32 * k] = o[g][k];
      if (lane == 0) {
        r[D] = M[g];
        r[D + 1] = L[g];
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ void finish(T* out, int lane) const {   // out: the unit's G rows
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float inv = 1.f / L[g];
#pragma unroll
      for (int k = 0; k < DPL; ++k)
        if (lane + 32 * k < D) out[g * D + lane + 32 * k] = T(o[g][k] * inv);
    }
  }
};

constexpr int kQ8FewPartials = 6;   // merged by one warp

// What the warps of a CTA left: partials of units that cross warps (`head`:
// record of the unit that a warp's range starts inside, `tail`: of the one
// that it ends inside; unit numbers, -1: none), and the units that this CTA
// is the last to reach, for all its warps to merge.
struct Q8Shared {
  int* head;
  int* tail;
  int* merge;          // [2] units
  float* head_rec;     // [W][G] records
  uint8_t* ring;       // tails: at the start of each warp's ring
  size_t ring_bytes;   // of a warp
};

template <typename T, int D, int G>
__device__ __noinline__ void q8_tail(const SplitParams& p, const Q8Shared sh, int W, long long total,
                                     const int* lens, const int* pre) {
  constexpr int PS = partial_stride(D);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = p.H_kv;
  const long long grid = gridDim.x;
  const long long c0 = blockIdx.x * total / grid, c1 = (blockIdx.x + 1) * total / grid;   // the CTA's groups
  auto head_rec = [&](int w) { return sh.head_rec + (size_t)w * G * PS; };
  auto tail_rec = [&](int w) { return reinterpret_cast<const float*>(sh.ring + (size_t)w * sh.ring_bytes); };

  // a unit's groups [su, eu)
  auto unit_range = [&](int u, long long& su, long long& eu) {
    const int b = u / H, h = u - b * H;
    su = (long long)H * pre[b] + (long long)h * lens[b];
    eu = su + lens[b];
  };
  // chain of unit u from warp `w` on (from its tail, or its head)
  auto chain = [&](int u, int w, bool from_tail) {
    Q8Acc<D, G> acc;
    acc.clear();
    if (from_tail) acc.template add<false>(tail_rec(w), lane);
    for (int k = from_tail ? w + 1 : w; k < W; ++k)
      if (sh.head[k] == u) acc.template add<false>(head_rec(k), lane);
    long long su, eu;
    unit_range(u, su, eu);
    T* out = static_cast<T*>(p.out) + (size_t)u * G * D;
    if (su >= c0 && eu <= c1) {
      acc.finish(out, lane);
      return;
    }
    acc.store(p.ws + ((size_t)blockIdx.x + u) * G * PS, lane);
    const long long cf = ((su + 1) * grid - 1) / total, cl = (eu * grid - 1) / total;
    int need = (int)(cl - cf + 1);
    if (total < grid) {   // some CTAs have no groups
      need = 0;
      for (long long k = cf; k <= cl; k += 32) {
        const long long c = k + lane;
        need += __popc(__ballot_sync(0xffffffffu, c <= cl && c * total / grid < (c + 1) * total / grid));
      }
    }
    __threadfence();
    __syncwarp();
    unsigned arrived = 0;
    if (lane == 0) arrived = q8_arrive(p.counters + u, p.epoch);
    arrived = __shfl_sync(0xffffffffu, arrived, 0);
    if (arrived == 0) flag_status(p.status, lane == 0 ? kDevTimeout : 0);
    if (arrived != (unsigned)need) return;
    // No arrival of this call can follow: clear the word, so that a call with
    // the same epoch (a CUDA graph replaying this launch) starts at 1.
    if (lane == 0) p.counters[u] = 0ull;
    __threadfence();
    if (cl - cf + 1 <= kQ8FewPartials) {
      const int b = u / H;
      merge_unit<T, D, G, kQ8FewPartials>(p.ws, static_cast<T*>(p.out), u, cf, cl, grid, total, b,
                                          u - b * H, H, lane);
    } else if (lane == 0) {
      sh.merge[from_tail ? 1 : 0] = u;
    }
  };
  // the unit that the CTA starts inside belongs to its first warp with rows,
  // and the others to the warps that end inside them
  if (sh.head[warp] >= 0) {
    bool leads = true;
    for (int k = 0; k < warp; ++k)
      if (sh.head[k] == sh.head[warp] || sh.tail[k] == sh.head[warp]) leads = false;
    if (leads) chain(sh.head[warp], warp, false);
  }
  if (sh.tail[warp] >= 0) chain(sh.tail[warp], warp, true);
  __syncthreads();
  for (int i = 0; i < 2; ++i) {
    const int u = sh.merge[i];
    if (u < 0) continue;
    // all warps: each some of the unit's partials, then the first one theirs
    long long su, eu;
    unit_range(u, su, eu);
    const long long cf = ((su + 1) * grid - 1) / total, cl = (eu * grid - 1) / total;
    Q8Acc<D, G> acc;
    acc.clear();
    for (long long c = cf + warp; c <= cl; c += W)
      if (c * total / grid < (c + 1) * total / grid)
        acc.template add<true>(p.ws + ((size_t)c + u) * G * PS, lane);
    acc.store(head_rec(warp), lane);
    __syncthreads();
    if (warp == 0) {
      acc.clear();
      for (int k = 0; k < W; ++k) acc.template add<false>(head_rec(k), lane);
      acc.finish(static_cast<T*>(p.out) + (size_t)u * G * D, lane);
    }
    __syncthreads();
  }
}

template <typename T, int D, int NSRC>
__global__ void __launch_bounds__(Q8Shape<D, NSRC>::W * 32, 1) decode_q8_kernel(const Q8Params prm) {
  const SplitParams& p = prm.p;
  using Cfg = Q8Cfg<D, NSRC>;
  using S = typename Cfg::S;
  constexpr int GROUPS = S::GROUPS, SCW = Cfg::SCW;
  constexpr int TILE = Cfg::TILE_BYTES, STAGE = Cfg::STAGE_BYTES;
  constexpr int NS = S::NS, W = S::W;
  constexpr int PS = partial_stride(D);
  constexpr int KW = D / 16;          // words of codes a lane holds of a key; steps of 16 channels
  constexpr int VT = D / 16;          // value tiles of 16 channels, 2 of a lane's
  constexpr int VW = (D + 31) / 32;   // words of codes a lane holds of a value row
  const int G = prm.G;

  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (size_t)W * NS * STAGE);
  int* lens = reinterpret_cast<int*>(bars + W * NS);   // groups of 16 rows per sequence
  int* pre = lens + p.B;                               // their sums before a sequence
  int* first = pre + p.B + 1;                          // first attended row
  int* count = first + p.B;                            // attended rows
  Q8Shared sh;
  sh.head = count + p.B;
  sh.tail = sh.head + W;
  sh.merge = sh.tail + W;
  int* abort_flag = sh.merge + 2;
  sh.head_rec = reinterpret_cast<float*>(smem + (size_t)W * NS * STAGE + prm.aux_bytes);
  sh.ring = smem;
  sh.ring_bytes = (size_t)NS * STAGE;

  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < NS; ++s) mbar_init(&bars[warp * NS + s], 1);
    fence_mbar_init();
    sh.head[warp] = sh.tail[warp] = -1;
  }
  if (threadIdx.x == 0) sh.merge[0] = sh.merge[1] = -1, *abort_flag = 0;
  grid_dep_trigger();
  grid_dep_wait();
  const unsigned long long wlim = wait_limit_ns(p.wait_limit);

  for (int i = threadIdx.x; i < p.B; i += blockDim.x) {
    int L = p.seq_lens[i];
    if (L < 1 || L > p.S_max) {
      if (blockIdx.x == 0) flag_status(p.status, kDevBadArg);
      L = L < 0 ? 0 : (L > p.S_max ? p.S_max : L);
    }
    const int Le = p.window > 0 && L > p.window ? p.window : L;
    const int f = p.ring > 0 ? (L - Le) % p.ring : L - Le;   // (in a ring: its row)
    first[i] = f;
    count[i] = Le;
    lens[i] = Le > 0 ? (f % 16 + Le + 15) / 16 : 0;
  }
  __syncthreads();
  if (warp == 0) {
    int run = 0;
    for (int base = 0; base < p.B; base += 32) {
      const int x = base + lane < p.B ? lens[base + lane] : 0;
      int incl = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (base + lane < p.B) pre[base + lane] = run + incl - x;
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) pre[p.B] = run;
  }
  __syncthreads();

  const int H = p.H_kv;
  if (blockIdx.x == 0) {
    // sequences of length 0 have no rows and so no merging warp: zero output
    const int row_elems = H * G * D;
    for (int bb = 0; bb < p.B; ++bb) {
      if (lens[bb] != 0) continue;
      for (int i = threadIdx.x; i < row_elems; i += blockDim.x)
        static_cast<T*>(p.out)[(size_t)bb * row_elems + i] = T(0.f);
    }
  }
  // ranges of groups
  const long long total = (long long)H * pre[p.B];
  const long long N = (long long)gridDim.x * W;
  const long long w = (long long)blockIdx.x * W + warp;
  const long long r0 = w * total / N, r1 = (w + 1) * total / N;
  if (r0 < r1) {
  RowWalker walk;
  {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if ((long long)H * pre[mid + 1] > r0) hi = mid; else lo = mid + 1;
    }
    const long long off = r0 - (long long)H * pre[lo];
    const int L = lens[lo];
    walk.b = lo;
    walk.h = (int)(off / L);
    walk.t = (int)(off - (long long)walk.h * L);
    walk.r = r0;
    walk.r1 = r1;
  }
  RowWalker prod = walk;

  uint8_t* wring = smem + (size_t)warp * NS * STAGE;   // this warp's stages
  uint64_t* wbars = bars + warp * NS;
  const uint64_t policy = l2_policy_evict_first();
  const int plane_rows = p.ring > 0 ? p.ring : p.S_max;
  const size_t plane_codes = (size_t)plane_rows * D;            // bytes per unit
  const size_t plane_scales = (size_t)q8_scale_cols(plane_rows);

  // A tile of n groups from group t of sequence b: the row of its first one,
  // how many of its rows are read (the sequence's last rows may end inside a
  // group), and how many of those come before a ring's end (a whole number of
  // groups; the others follow from the ring's start).
  auto tile_rows = [&](int b, int t, int n, int& row0, int& nrows, int& n1) {
    const int lead = first[b] % 16;
    row0 = first[b] - lead + 16 * t;
    if (p.ring > 0 && row0 >= p.ring) row0 -= p.ring;
    nrows = min(16 * n, lead + count[b] - 16 * t);
    n1 = p.ring > 0 && row0 + nrows > p.ring ? p.ring - row0 : nrows;
  };

  auto issue = [&](int stage, int b, int h, int t, int n) {
    if (lane == 0) {
      uint8_t* dst = wring + (size_t)stage * STAGE;
      float* dsc = reinterpret_cast<float*>(dst + Cfg::CODE_BYTES);
      uint64_t* bar = &wbars[stage];
      const size_t u = (size_t)b * H + h;
      int row0, nrows, n1;
      tile_rows(b, t, n, row0, nrows, n1);
      const int n2 = nrows - n1;
      const int g0 = row0 / (4 * kQ8Block);                       // first 16-byte piece of scales
      const uint32_t sb1 = (uint32_t)((row0 + n1 - 1) / (4 * kQ8Block) - g0 + 1) * 16;
      const uint32_t sb2 = n2 > 0 ? (uint32_t)((n2 - 1) / (4 * kQ8Block) + 1) * 16 : 0;
      const uint32_t b1 = (uint32_t)n1 * D, b2 = (uint32_t)n2 * D;
      const size_t base = u * plane_codes, off = base + (size_t)row0 * D;
      const size_t sbase = u * plane_scales;
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(bar, (b1 + b2 + sb1 + sb2) * 2 * NSRC);
#pragma unroll
      for (int i = 0; i < 2 * NSRC; ++i) {
        const bool value = i >= NSRC;
        const int sidx = value ? i - NSRC : i;
        const uint8_t* src =
            static_cast<const uint8_t*>(value ? (sidx ? p.v1 : p.v0) : (sidx ? p.k1 : p.k0));
        const float* sc = value ? prm.vs[sidx] : prm.ks[sidx];
        bulk_g2s(dst + i * TILE, src + off, b1, bar, policy);
        bulk_g2s(dsc + i * 2 * SCW, sc + sbase + (size_t)g0 * 4, sb1, bar, policy);
        if (n2 > 0) {
          bulk_g2s(dst + i * TILE + b1, src + base, b2, bar, policy);
          bulk_g2s(dsc + (i * 2 + 1) * SCW, sc + sbase, sb2, bar, policy);
        }
      }
    }
  };

  int issued = 0;
#pragma unroll 1
  for (int s = 0; s < NS; ++s) {
    int tb, th, tt, tn;
    bool tl;
    if (!prod.next(lens, H, p.B, GROUPS, tb, th, tt, tn, tl)) break;
    issue(s, tb, th, tt, tn);
    ++issued;
  }

  const int n8 = lane >> 2, q4 = lane & 3;
  // Key index n of a group's first (second: + 8) eight stands for row
  // key_row(n): neighbours stay neighbours, so that score loads of two keys
  // are 2 D contiguous bytes, and the first keys 2q of the lanes q are even
  // and odd rows in turn, which halves the bank conflicts of value loads.
  const int krow = n8 ^ (n8 >> 1 & 1);
  const int vrow = 2 * q4 + (q4 & 1), vrow2 = vrow ^ 1;   // key_row(2q), key_row(2q + 1)

  uint32_t qf[NSRC][KW][4];    // Q fragments per source and step
  // O^T fragments: this lane's channels 2 i, 2 i + 1 of heads 2 q4 (elements
  // 0, 2) and 2 q4 + 1 (1, 3)
  float o[NSRC][VT][4];
  float c_row = 0.f;           // 2^-e of the head's query
  float m = -FLT_MAX, l = 0.f; // of head n8, this lane's keys
  bool fresh = true;
  bool whole = false;          // the range has the unit from its first group on
  int consumed = 0;

#pragma unroll 1
  for (;;) {
    int b, h, t0, n;
    bool last;
    if (!walk.next(lens, H, p.B, GROUPS, b, h, t0, n, last)) break;
    const int stage = consumed % NS;
    const uint32_t parity = (uint32_t)(consumed / NS) & 1u;

    if (fresh) {
      whole = t0 == 0;
      // head n8's query, channels [q4 D/4, + D/4), brought to [2^14, 2^15)
      const T* qp = static_cast<const T*>(p.q) + (((size_t)b * H + h) * G + n8) * D + q4 * (D / 4);
      float top = 0.f, x[D / 4];
#pragma unroll
      for (int e = 0; e < D / 4; ++e) {
        x[e] = n8 < G ? (float)qp[e] * p.qscale : 0.f;
        const float wmax = NSRC == 2 ? fmaxf(fabsf(p.a0[(size_t)h * D + q4 * (D / 4) + e]),
                                             fabsf(p.a1[(size_t)h * D + q4 * (D / 4) + e]))
                           : p.a0    ? fabsf(p.a0[(size_t)h * D + q4 * (D / 4) + e])
                                     : 1.f;
        top = fmaxf(top, fabsf(x[e]) * wmax);
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      int eq = 14 - ((int)(__float_as_uint(top) >> 23) - 127);
      eq = eq > 120 ? 120 : (eq < -120 ? -120 : eq);   // (2^eq and its inverse stay normal)
      const float f = __uint_as_float((uint32_t)(eq + 127) << 23);
      c_row = __uint_as_float((uint32_t)(127 - eq) << 23);
#pragma unroll
      for (int sidx = 0; sidx < NSRC; ++sidx) {
        const float* ap = sidx == 0 ? p.a0 : p.a1;
#pragma unroll
        for (int j = 0; j < KW; ++j) {
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[e] = x[4 * j + e];
            if (NSRC == 2 || ap) y[e] *= ap[(size_t)h * D + q4 * (D / 4) + 4 * j + e];
            y[e] *= f;
          }
          split_f16(y[0], y[1], qf[sidx][j][0], qf[sidx][j][1]);
          split_f16(y[2], y[3], qf[sidx][j][2], qf[sidx][j][3]);
        }
#pragma unroll
        for (int i = 0; i < VT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[sidx][i][e] = 0.f;
      }
      m = -FLT_MAX;
      l = 0.f;
      fresh = false;
    }

    // warp-uniform: every lane leaves, or none does (shuffles follow)
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&wbars[stage], parity, wlim))) {
      flag_status(p.status, kDevTimeout);
      // let every stage issued and not yet consumed land, this one included
      for (int k = consumed; k < issued; ++k)
        (void)mbar_wait_bounded(&wbars[k % NS], (uint32_t)(k / NS) & 1u, kDrainLimitNs);
      if (lane == 0) *abort_flag = 1;
      break;
    }

    int row0, nrows, n1;
    tile_rows(b, t0, n, row0, nrows, n1);
    const int skip = t0 == 0 ? first[b] % 16 : 0;   // rows of the first group before the first attended
    const uint8_t* st = wring + (size_t)stage * STAGE;
    const float* scales = reinterpret_cast<const float*>(st + Cfg::CODE_BYTES);

    // One tile.  EDGE: rows before `skip` or from nrows on are not attended, or
    // the tile wraps in a ring.
    auto tile = [&](auto edge) {
      constexpr bool EDGE = decltype(edge)::value;
      // where the scale of the tile's group gr lies in a plane's run of scales
      const int sc0 = row0 & (4 * kQ8Block - 1);
      auto scale_at = [&](int gr) {
        if (EDGE && 16 * gr >= n1) return SCW + (16 * gr - n1) / kQ8Block;
        return (sc0 + 16 * gr) / kQ8Block;
      };
      // scores in base 2 plus the group's value exponent: s[gr][2 half + e] is
      // key 2 q4 + e of the half
      float s[GROUPS][4], lv[GROUPS];
      float mt = -INFINITY;
#pragma unroll
      for (int gr = 0; gr < GROUPS; ++gr) {
        if (EDGE && 16 * gr >= nrows) {   // no such group in this tile
          s[gr][0] = s[gr][1] = s[gr][2] = s[gr][3] = -INFINITY;
          lv[gr] = 0.f;
          continue;
        }
        const int at = scale_at(gr);
        float vs = scales[NSRC * 2 * SCW + at];
        if constexpr (NSRC == 2) vs = fmaxf(vs, scales[(NSRC + 1) * 2 * SCW + at]);
        lv[gr] = fast_log2(vs);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[gr][e] = lv[gr];
#pragma unroll
        for (int sidx = 0; sidx < NSRC; ++sidx) {
          const float f = scales[sidx * 2 * SCW + at] * c_row;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t kw[KW];
            load_words<D / 4>(st + sidx * TILE + (16 * gr + 8 * half + krow) * D + q4 * (D / 4), kw);
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < KW; ++j) {
              uint32_t b0, b1;
              e4m3x4_to_f16(kw[j], b0, b1);
              mma16816(d, qf[sidx][j], b0, b1);
            }
            s[gr][2 * half] = fmaf(d[0] + d[2], f, s[gr][2 * half]);
            s[gr][2 * half + 1] = fmaf(d[1] + d[3], f, s[gr][2 * half + 1]);
          }
        }
        if constexpr (EDGE) {
          // keys 2 q4, 2 q4 + 1 of the halves are these rows of the group
          const int ra = 16 * gr + vrow, rb = 16 * gr + vrow2;
          if (ra < skip || ra >= nrows) s[gr][0] = -INFINITY;
          if (rb < skip || rb >= nrows) s[gr][1] = -INFINITY;
          if (ra + 8 < skip || ra + 8 >= nrows) s[gr][2] = -INFINITY;
          if (rb + 8 < skip || rb + 8 >= nrows) s[gr][3] = -INFINITY;
        }
        mt = fmaxf(mt, fmaxf(fmaxf(s[gr][0], s[gr][1]), fmaxf(s[gr][2], s[gr][3])));
      }
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
      const bool grow = mt > m + kQ8Slack;
      if (__any_sync(0xffffffffu, grow)) {
        const float m_new = grow ? mt : m;
        const float alpha = fast_exp2(m - m_new);
        l *= alpha;
        m = m_new;
        // of the heads whose O this lane holds
        const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * q4), a1 = __shfl_sync(0xffffffffu, alpha, 8 * q4 + 4);
#pragma unroll
        for (int sidx = 0; sidx < NSRC; ++sidx)
#pragma unroll
          for (int i = 0; i < VT; ++i) {
            o[sidx][i][0] *= a0;
            o[sidx][i][1] *= a1;
            o[sidx][i][2] *= a0;
            o[sidx][i][3] *= a1;
          }
      }

      // values
      const float off = kQ8Bias - m;
#pragma unroll
      for (int gr = 0; gr < GROUPS; ++gr) {
        if (EDGE && 16 * gr >= nrows) continue;
        float pv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pv[e] = fast_exp2(s[gr][e] + off);
        const float rv = fast_exp2(-lv[gr]);
        l = fmaf((pv[0] + pv[1]) + (pv[2] + pv[3]), rv, l);
#pragma unroll
        for (int sidx = 0; sidx < NSRC; ++sidx) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = pv[e];
          if constexpr (NSRC == 2) {
            const float ratio = scales[(NSRC + sidx) * 2 * SCW + scale_at(gr)] * rv;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] *= ratio;
          }
          uint32_t ph[2];
          [[maybe_unused]] uint32_t pl[2];
          if constexpr (sizeof(T) == 4) {
            split_f16(x[0], x[1], ph[0], pl[0]);
            split_f16(x[2], x[3], ph[1], pl[1]);
          } else {
            ph[0] = f16x2_of(x[0], x[1]);
            ph[1] = f16x2_of(x[2], x[3]);
          }
          uint32_t va[VW], vb[VW], vc[VW], vd[VW];   // keys 2q, 2q + 1, 2q + 8, 2q + 9
          const uint8_t* vt = st + (NSRC + sidx) * TILE + 16 * gr * D;
          load_value<D>(vt + vrow * D, n8, va);
          load_value<D>(vt + vrow2 * D, n8, vb);
          load_value<D>(vt + (vrow + 8) * D, n8, vc);
          load_value<D>(vt + (vrow2 + 8) * D, n8, vd);
          if constexpr (EDGE) {
            // rows that are not attended may hold anything: nothing times 0
            const int ra = 16 * gr + vrow, rb = 16 * gr + vrow2;
#pragma unroll
            for (int i = 0; i < VW; ++i) {
              if (ra < skip || ra >= nrows) va[i] = 0;
              if (rb < skip || rb >= nrows) vb[i] = 0;
              if (ra + 8 < skip || ra + 8 >= nrows) vc[i] = 0;
              if (rb + 8 < skip || rb + 8 >= nrows) vd[i] = 0;
            }
          }
#pragma unroll
          for (int i = 0; i < VT; ++i) {
            // channels 2 i, 2 i + 1 of both pairs of keys: bytes (a, b, a', b')
            const uint32_t sel = i & 1 ? 0x7362u : 0x5140u;
            uint32_t f[4];
            e4m3x4_to_f16(__byte_perm(va[i / 2], vb[i / 2], sel), f[0], f[1]);
            e4m3x4_to_f16(__byte_perm(vc[i / 2], vd[i / 2], sel), f[2], f[3]);
            mma16816(o[sidx][i], f, ph[0], ph[1]);
            if constexpr (sizeof(T) == 4) mma16816(o[sidx][i], f, pl[0], pl[1]);
          }
        }
      }
    };
    if (skip != 0 || nrows != 16 * GROUPS || n1 != nrows)
      tile(std::true_type{});
    else
      tile(std::false_type{});

    ++consumed;
    __syncwarp();
    // refill the stage just read with the warp's next tile
    {
      int tb, th, tt, tn;
      bool tl;
      if (prod.next(lens, H, p.B, GROUPS, tb, th, tt, tn, tl)) {
        issue(stage, tb, th, tt, tn);
        ++issued;
      }
    }

    if (last) {
      // the range's part of the unit is complete: finish the unit if that is
      // all of it, else leave a partial
      const int u = b * H + h;
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      const bool ends = t0 + n == lens[b];
      float* rec = whole ? reinterpret_cast<float*>(wring) : sh.head_rec + (size_t)warp * G * PS;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int head = 2 * q4 + e;
        const float inv = 1.f / __shfl_sync(0xffffffffu, l, 8 * q4 + 4 * e);
        if (head >= G) continue;
#pragma unroll
        for (int i = 0; i < VT; ++i) {
          const int c = value_channel<D>(n8, 2 * i);
          float x = o[0][i][e], y = o[0][i][e + 2];
          if (NSRC == 2 || p.b0) {
            const float2 w0 = *reinterpret_cast<const float2*>(p.b0 + (size_t)h * D + c);
            x *= w0.x;
            y *= w0.y;
          }
          if constexpr (NSRC == 2) {
            const float2 w1 = *reinterpret_cast<const float2*>(p.b1 + (size_t)h * D + c);
            x = fmaf(o[1][i][e], w1.x, x);
            y = fmaf(o[1][i][e + 2], w1.y, y);
          }
          if (whole && ends)
            store2(static_cast<T*>(p.out) + ((size_t)u * G + head) * D + c, x * inv, y * inv);
          else
            store2(rec + head * PS + c, x, y);
        }
      }
      if (!(whole && ends) && n8 < G && q4 == 0) {
        rec[n8 * PS + D] = m;
        rec[n8 * PS + D + 1] = l;
      }
      if (lane == 0 && !(whole && ends)) (whole ? sh.tail : sh.head)[warp] = u;
      fresh = true;
    }
  }
  }

  __syncthreads();
  if (*abort_flag) return;
  if (G == 1) q8_tail<T, D, 1>(p, sh, W, total, lens, pre);
  if (G == 2) q8_tail<T, D, 2>(p, sh, W, total, lens, pre);
  if (G == 4) q8_tail<T, D, 4>(p, sh, W, total, lens, pre);
}

// Shared memory behind the rings: barriers, lengths and the words of Q8Shared;
// then the records.
__host__ __device__ constexpr size_t q8_aux_bytes(int warps, int stages, int B) {
  return ((size_t)warps * stages * 8 + (size_t)(4 * B + 1 + 2 * warps + 3) * 4 + 15) / 16 * 16;
}

template <int D, int NSRC>
size_t q8_smem_bytes(int B, int G) {
  using S = Q8Shape<D, NSRC>;
  return (size_t)S::W * S::NS * Q8Cfg<D, NSRC>::STAGE_BYTES + q8_aux_bytes(S::W, S::NS, B) +
         (size_t)S::W * G * partial_stride(D) * sizeof(float);
}

template <typename T, int D, int NSRC>
cudaError_t launch_q8(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t stream) {
  Q8Params prm;
  SplitParams& sp = prm.p;
  sp.k0 = a.k[0];
  sp.k1 = a.k[1];
  sp.v0 = a.v[0];
  sp.v1 = a.v[1];
  sp.a0 = a.a[0];
  sp.a1 = a.a[1];
  sp.b0 = a.b[0];
  sp.b1 = a.b[1];
  sp.q = a.q;
  sp.out = a.out;
  sp.seq_lens = a.seq_lens;
  sp.ws = a.workspace;
  sp.counters = reinterpret_cast<unsigned long long*>(reinterpret_cast<char*>(a.workspace) +
                                                      plan.partial_bytes);
  sp.status = a.status;
  sp.wait_limit = a.wait_limit;
  sp.epoch = a.epoch;
  sp.B = a.batch;
  sp.H_kv = a.kv_heads;
  sp.S_max = a.max_seq;
  sp.window = a.window;
  sp.ring = a.ring;
  sp.qscale = a.softmax_scale * 1.4426950408889634f;
  for (int i = 0; i < 2; ++i) {
    prm.ks[i] = a.k_scale[i];
    prm.vs[i] = a.v_scale[i];
  }
  prm.G = a.group;
  prm.aux_bytes = (int)q8_aux_bytes(Q8Shape<D, NSRC>::W, Q8Shape<D, NSRC>::NS, a.batch);
  auto kern = decode_q8_kernel<T, D, NSRC>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan.smem_bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(plan.ctas), dim3(plan.warps_per_cta * 32), plan.smem_bytes, stream, prm);
}

template <typename T, int D>
cudaError_t q8_by_src(const DecodeArgs& a, const DecodePlan& pl, cudaStream_t s) {
  return a.nsrc == 2 ? launch_q8<T, D, 2>(a, pl, s) : launch_q8<T, D, 1>(a, pl, s);
}

template <typename T>
cudaError_t q8_by_dim(const DecodeArgs& a, const DecodePlan& pl, cudaStream_t s) {
  switch (a.head_dim) {
    case 64: return q8_by_src<T, 64>(a, pl, s);
    case 80: return q8_by_src<T, 80>(a, pl, s);
    case 96: return q8_by_src<T, 96>(a, pl, s);
    case 128: return q8_by_src<T, 128>(a, pl, s);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace fkv
