// Decode attention over 8-bit caches (e4m3 codes, one scale per 32 rows of a
// KV head; q8_device.cuh).
//
// Every warp streams a contiguous range of the call's rows through a ring of
// its own (cp.async.bulk, one mbarrier a stage), as in decode_split_kernel.
// Ranges are cut at groups of 16 rows, counted from rows that are multiples of
// 16, so that a group has one key scale and one value scale; they come with
// the codes, a lane holding one of the next tile's, since small bulk copies cost
// the copy engine as much as large ones.
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
// copy rate): 78 us with scalar arithmetic, 49 with these; 4B fused call of
// full length (2.69 GB, 402 us): 549 us with 16 rows of values' products, 418
// with the transposed ones below, which take half the registers and products.
//
// Scores: S [16 x 8 keys] = Q [16 x 16 channels] . K^T.  Row g < G of Q is
// query head g of the group (times the key weights and a power of two), to
// fp16; row g + 8 is what that rounding left, to fp16 again: 22 bits of the
// query, at no cost, since the rows are there.
// Values: O^T [16 channels x 8] += V^T [16 x 16 keys] . P^T, whose column g is
// head g (a score's place in the first product is its weight's place in the
// second).  With the value scale r in the exponent, P' = p 2^e = 2^(s + e - M),
// 2^(e - 1) < r <= 2^e, no scale can take P' out of fp16's range (M is the
// running maximum of that sum, rounded down to a whole number, with a slack of
// 2^8 before O is rescaled); the softmax's sum takes P' 2^-e, and the product
// P' (r 2^-e), which is P' itself where r is a power of two (appended rows).
// e - M is a whole number, so that a scale adds nothing to the score's rounding.
// (e stops at kQ8MinValue's; smaller scales take the rest with r 2^-e.)
// P' is rounded to fp16, 2^-12, for bf16 outputs; fp32 contexts add a
// second product with what the rounding left.  Two value sources have one
// exponent, of the larger scale, and two P with the factors r_i 2^-e, where a
// source's scales count times its largest weight (as a power of two, which the
// weights of the output are divided by): a source whose small weights make up
// for its large scales does not push the other out of fp16's range.  The query
// has a power of two for each source's key weights, too.
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
  static constexpr int CODE_BYTES = 2 * NSRC * TILE_BYTES;
  static constexpr int STAGE_BYTES = CODE_BYTES + (2 * NSRC * S::GROUPS * 4 + 15) / 16 * 16;   // and a scale for every plane and group
  static_assert(TILE_BYTES % 16 == 0, "stages are read in 16-byte pieces");
  static_assert(2 * NSRC * S::GROUPS <= 32, "a lane copies one of a tile's scales");
};

// Division by a number known at launch: floor(x / d) of 32-bit x.
struct Q8Div {
  unsigned long long m;   // ceil(2^64 / d); 0: d = 1
  unsigned d;
  static Q8Div of(unsigned d) { return {d > 1 ? ~0ull / d + 1 : 0, d}; }
  __device__ __forceinline__ unsigned operator()(unsigned x) const {
    return m ? (unsigned)__umul64hi(m, x) : x;
  }
};

struct Q8Params {
  SplitParams p;
  const float* ks[2];
  const float* vs[2];
  int G;
  int aux_bytes;
  Q8Div by_ctas, by_heads, by_ring;
};

// Copy 4 bytes to shared memory without waiting; and arrive on a barrier once
// this lane's copies so far have landed.
__device__ __forceinline__ void copy4_async(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// d += a b: m16n8k16, fp16 operands, fp32 sums.
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// N elements of global memory, aligned to the largest power of two that
// divides their bytes (16 at most), -> fp32.
template <int N>
__device__ __forceinline__ void load_floats(const float* src, float* f) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) unpack16<float>(reinterpret_cast<const uint4*>(src)[i], f + 4 * i);
}
template <int N>
__device__ __forceinline__ void load_floats(const __nv_bfloat16* src, float* f) {
  if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) unpack16<__nv_bfloat16>(reinterpret_cast<const uint4*>(src)[i], f + 8 * i);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint2 w = reinterpret_cast<const uint2*>(src)[i];
      f[4 * i] = bf16lo(w.x);
      f[4 * i + 1] = bf16hi(w.x);
      f[4 * i + 2] = bf16lo(w.y);
      f[4 * i + 3] = bf16hi(w.y);
    }
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

// Equal shares: part c of n has [start(c), start(c + 1)), start(c) = floor(c
// total / n), in 32-bit arithmetic (total < 2^32, n < 2^16).
struct Q8Split {
  Q8Div by;
  unsigned each, rest;
  __device__ __forceinline__ Q8Split(unsigned total, const Q8Div& parts) : by(parts) {
    each = by(total);
    rest = total - each * by.d;
  }
  __device__ __forceinline__ unsigned start(unsigned c) const { return c * each + by(c * rest); }
  // the part that holds group g
  __device__ __forceinline__ unsigned part(unsigned g, unsigned total) const {
    unsigned c = min((unsigned)__fdividef((float)g * (float)by.d, (float)total), by.d - 1);
    while (c > 0 && start(c) > g) --c;
    while (c + 1 < by.d && start(c + 1) <= g) ++c;
    return c;
  }
};

// A warp's combination of partials of one head (records o[D], m, l), lane =
// channel of o.
template <int D>
struct Q8Acc {
  static constexpr int DPL = (D + 31) / 32;
  float M, L, o[DPL];
  __device__ __forceinline__ void clear() {
    M = -FLT_MAX;
    L = 0.f;
#pragma unroll
    for (int k = 0; k < DPL; ++k) o[k] = 0.f;
  }
  // Add up to 32 records, rec(j) for the bits j of `members`: lane j takes
  // record j's m and l, so that the weights come in one step.  GLOBAL: read
  // through L2, where other SMs put them, several rows at a time.
  template <bool GLOBAL, typename Rec>
  __device__ __forceinline__ void add(unsigned members, Rec rec, int lane) {
    auto get = [](const float* p) { return GLOBAL ? __ldcg(p) : *p; };
    float m = -FLT_MAX, l = 0.f;
    if ((members >> lane) & 1u) {
      const float* r = rec(lane);
      m = get(r + D);
      l = get(r + D + 1);
    }
    const float top = fmaxf(M, warp_max(m)), old = fast_exp2(M - top);
    const float w = (members >> lane) & 1u ? fast_exp2(m - top) : 0.f;
    L = L * old + warp_sum(w * l);
    M = top;
#pragma unroll
    for (int k = 0; k < DPL; ++k) o[k] *= old;
    constexpr int AT = GLOBAL ? 4 : 2;
    while (members) {
      float wj[AT], x[AT][DPL];
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        const int j = members ? __ffs((int)members) - 1 : 0;
        wj[i] = __shfl_sync(0xffffffffu, w, j);
#pragma unroll
        for (int k = 0; k < DPL; ++k) x[i][k] = 0.f;
        if (members) {
          const float* r = rec(j);
#pragma unroll
          for (int k = 0; k < DPL; ++k)
            if (lane + 32 * k < D) x[i][k] = get(r + lane + 32 * k);
        }
        members &= members - 1;
      }
#pragma unroll
      for (int i = 0; i < AT; ++i)
#pragma unroll
        for (int k = 0; k < DPL; ++k) o[k] = fmaf(wj[i], x[i][k], o[k]);
    }
  }
  __device__ __forceinline__ void store(float* r, int lane) const {
#pragma unroll
    for (int k = 0; k < DPL; ++k)
      if (lane + 32 * k < D) r[lane + 32 * k] = o[k];
    if (lane == 0) {
      r[D] = M;
      r[D + 1] = L;
    }
  }
  template <typename T>
  __device__ __forceinline__ void finish(T* out, int lane) const {
    const float inv = 1.f / L;
#pragma unroll
    for (int k = 0; k < DPL; ++k)
      if (lane + 32 * k < D) out[lane + 32 * k] = T(o[k] * inv);
  }
};

constexpr int kQ8FewPartials = 8;   // merged by one warp
constexpr int kQ8Stopped = -2;      // Q8Shared::head of a warp that gave up

// What the warps of a CTA left: partials of units that cross warps (`head`:
// record of the unit that a warp's range starts inside, `tail`: of the one
// that it ends inside; unit numbers, -1: none), and the heads (unit * G + head)
// that this CTA is the last to reach, for all its warps to merge.
struct Q8Shared {
  int* head;
  int* tail;
  int* merge;          // [2][4], -1: none
  float* head_rec;     // [W][G] records
  uint8_t* ring;       // tails: at the start of each warp's ring
  unsigned ring_bytes; // of a warp
};

// [c0, c1): the CTA's groups; `split`: all CTAs' (not looked at where no unit
// crosses CTAs).  A warp takes a chain of partials and a head at a time.
template <typename T, int D, int W>
__device__ __forceinline__ void q8_tail(const SplitParams& p, const Q8Shared& sh, int G, unsigned total,
                                        const Q8Split& split, unsigned c0, unsigned c1,
                                        const int* pre) {
  constexpr int PS = partial_stride(D);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = p.H_kv;
  T* out = static_cast<T*>(p.out);
  const int my_head = lane < W ? sh.head[lane] : -1, my_tail = lane < W ? sh.tail[lane] : -1;
  // Chains: a tail with the heads that go on with its unit; and, of the unit
  // that the CTA starts inside, the first head and the others of it.
  const unsigned tails = __ballot_sync(0xffffffffu, my_tail >= 0);
  const unsigned heads = __ballot_sync(0xffffffffu, my_head >= 0);
  const int k0 = heads ? __ffs((int)heads) - 1 : 0;
  const int u0 = __shfl_sync(0xffffffffu, my_head, k0);
  const bool starts_inside = heads && !__any_sync(0xffffffffu, my_tail == u0);
  const int chains = __popc(tails) + (starts_inside ? 1 : 0);
  auto unit_range = [&](int u, unsigned& su, unsigned& eu) {   // its groups
    const int b = u / H, h = u - b * H;
    const int L = pre[b + 1] - pre[b];
    su = (unsigned)H * pre[b] + (unsigned)h * L;
    eu = su + L;
  };
  for (int task = warp; task < chains * G; task += W) {
    const int c = task / G, g = task - c * G;
    unsigned left = tails;
    for (int i = starts_inside ? 1 : 0; i < c; ++i) left &= left - 1;
    const bool from_tail = !starts_inside || c > 0;
    const int leader = from_tail ? __ffs((int)left) - 1 : -1;
    const int u = from_tail ? __shfl_sync(0xffffffffu, my_tail, leader) : u0;
    // (a warp that a unit goes through has no tail of it: a record a warp)
    const unsigned members = __ballot_sync(0xffffffffu, my_head == u) | (from_tail ? 1u << leader : 0u);
    Q8Acc<D> acc;
    acc.clear();
    acc.template add<false>(
        members,
        [&](int j) {
          const float* r = j == leader ? reinterpret_cast<const float*>(sh.ring + j * sh.ring_bytes)
                                       : sh.head_rec + j * G * PS;
          return r + g * PS;
        },
        lane);
    unsigned su, eu;
    unit_range(u, su, eu);
    if (su >= c0 && eu <= c1) {
      acc.finish(out + ((size_t)u * G + g) * D, lane);
      continue;
    }
    acc.store(p.ws + (((size_t)blockIdx.x + u) * G + g) * PS, lane);
    const unsigned cf = split.part(su, total), cl = split.part(eu - 1, total);
    int need = (int)(cl - cf + 1);
    if (total < split.by.d) {   // some CTAs have no groups
      need = 0;
      for (unsigned k = cf; k <= cl; k += 32) {
        const unsigned i = k + lane;
        need += __popc(__ballot_sync(0xffffffffu, i <= cl && split.start(i) < split.start(i + 1)));
      }
    }
    __threadfence();
    __syncwarp();
    unsigned arrived = 0;
    if (lane == 0) arrived = q8_arrive(p.counters + (size_t)u * G + g, p.epoch);
    arrived = __shfl_sync(0xffffffffu, arrived, 0);
    if (arrived == 0) flag_status(p.status, lane == 0 ? kDevTimeout : 0);
    if (arrived != (unsigned)need) continue;
    // No arrival of this call can follow: clear the word, so that a call with
    // the same epoch (a CUDA graph replaying this launch) starts at 1.
    if (lane == 0) p.counters[(size_t)u * G + g] = 0ull;
    __threadfence();
    if (cl - cf + 1 <= kQ8FewPartials) {
      const bool has = cf + lane <= cl && split.start(cf + lane) < split.start(cf + lane + 1);
      acc.clear();
      acc.template add<true>(
          __ballot_sync(0xffffffffu, has),
          [&](int j) { return p.ws + (((size_t)cf + j + u) * G + g) * PS; }, lane);
      acc.finish(out + ((size_t)u * G + g) * D, lane);
    } else if (lane == 0) {
      sh.merge[(from_tail ? 4 : 0) + g] = u;
    }
  }
  __syncthreads();
  for (int i = 0; i < 8; ++i) {
    const int u = sh.merge[i], g = i & 3;
    if (u < 0) continue;
    // all warps: each some of the head's partials, then the first one theirs
    unsigned su, eu;
    unit_range(u, su, eu);
    const unsigned cf = split.part(su, total), cl = split.part(eu - 1, total);
    Q8Acc<D> acc;
    acc.clear();
    for (unsigned base = cf; base <= cl; base += 32 * W) {
      const unsigned k = base + lane * W + warp;   // lane j's partial
      acc.template add<true>(
          __ballot_sync(0xffffffffu, k <= cl && split.start(k) < split.start(k + 1)),
          [&](int j) { return p.ws + (((size_t)base + j * W + warp + u) * G + g) * PS; }, lane);
    }
    acc.store(sh.head_rec + warp * PS, lane);
    __syncthreads();
    if (warp == 0) {
      acc.clear();
      acc.template add<false>((1u << W) - 1u, [&](int j) { return sh.head_rec + j * PS; }, lane);
      acc.finish(out + ((size_t)u * G + g) * D, lane);
    }
    __syncthreads();
  }
}

// Walk of a warp's range of groups, one tile at a time, crossing units.  pre:
// sums of the sequences' groups.
struct Q8Walker {
  unsigned r, r1;
  int b, h, t;
  __device__ __forceinline__ bool next(const int* pre, int H, int B, int most, int& tb, int& th, int& tt, int& tn,
                                       bool& last) {
    if (r >= r1) return false;
    const int L = pre[b + 1] - pre[b];
    const int seg = (int)min((unsigned)(L - t), r1 - r), n = min(most, seg);
    tb = b;
    th = h;
    tt = t;
    tn = n;
    last = n == seg;
    t += n;
    r += n;
    if (t == L) {
      t = 0;
      if (++h == H) {
        h = 0;
        ++b;
        while (r < r1 && b < B && pre[b + 1] == pre[b]) ++b;
      }
    }
    return true;
  }
};

// A CTA takes whole units where the busiest one then has at most these codes
// (bytes) more than an equal share: a merge through global memory costs 4 us,
// about what they take.  Both ways measured with 32, 128 and 160 units of 500 to
// 6000 rows, at 64, 96 and 128 channels, one source and two, bf16 and fp32
// contexts: whole units are 1.0 to 6.2 us faster in every call with up to 200 KB
// more on the busiest CTA, both are within 2.2 us of each other from there to 303
// KB, and split ones are 1.6 to 34 us faster from 320 KB on.  Us whole and split: 64
// channels, one source, 128 units of 2000 rows (40 KB) 11.4 and 16.7; 96, 32 of
// 1500 (227 KB) 11.9 and 13.1; 128, two sources, 128 of 3000 (243 KB) 50.5 and
// 49.9, of 4000 (323 KB) 64.4 and 61.2.
constexpr int kQ8Uneven = 230400;

template <typename T, int D, int NSRC>
__global__ void __launch_bounds__(Q8Shape<D, NSRC>::W * 32, 1) decode_q8_kernel(const Q8Params prm) {
  const SplitParams& p = prm.p;
  using Cfg = Q8Cfg<D, NSRC>;
  using S = typename Cfg::S;
  constexpr int GROUPS = S::GROUPS;
  constexpr int TILE = Cfg::TILE_BYTES, STAGE = Cfg::STAGE_BYTES;
  constexpr int NS = S::NS, W = S::W;
  constexpr int PS = partial_stride(D);
  constexpr int KW = D / 16;          // words of codes a lane holds of a key; steps of 16 channels
  constexpr int VT = D / 16;          // value tiles of 16 channels, 2 of a lane's
  constexpr int VW = (D + 31) / 32;   // words of codes a lane holds of a value row
  const int G = prm.G;

  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (size_t)W * NS * STAGE);
  int* len = reinterpret_cast<int*>(bars + W * NS);   // the sequences' lengths, clamped
  int* pre = len + p.B;                               // sums of their groups of 16 rows
  Q8Shared sh;
  sh.head = pre + p.B + 1;
  sh.tail = sh.head + W;
  sh.merge = sh.tail + W;
  sh.head_rec = reinterpret_cast<float*>(smem + (size_t)W * NS * STAGE + prm.aux_bytes);
  sh.ring = smem;
  sh.ring_bytes = NS * STAGE;

  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < NS; ++s) mbar_init(&bars[warp * NS + s], 33);   // a copy's bytes, and the lanes
    fence_mbar_init();
    sh.head[warp] = sh.tail[warp] = -1;
  }
  if (threadIdx.x < 8) sh.merge[threadIdx.x] = -1;
  // the parameters' cache lines, while the kernel ahead still runs
  asm volatile("" ::"r"(prm.by_heads.d), "r"(prm.G), "l"(prm.vs[0]), "r"(p.H_kv), "l"(p.out), "l"(p.ws));
  grid_dep_trigger();
  grid_dep_wait();
  const unsigned long long wlim = wait_limit_ns(p.wait_limit);

  // Lengths and their sums, by every warp for itself (all write the same
  // values): no warp waits for another.
  auto attended = [&](int L, int& f, int& rows) {   // first attended row (in a ring: its row), and how many
    rows = p.window > 0 && L > p.window ? p.window : L;
    f = L - rows;
    if (p.ring > 0) f -= (int)prm.by_ring(f) * p.ring;
  };
  int run = 0, longest = 0;
  for (int base = 0; base < p.B; base += 32) {
    const int i = base + lane;
    int L = 0, x = 0;
    if (i < p.B) {
      L = p.seq_lens[i];
      if (L < 1 || L > p.S_max) {
        if (blockIdx.x == 0 && warp == 0) flag_status(p.status, kDevBadArg);
        L = L < 0 ? 0 : (L > p.S_max ? p.S_max : L);
      }
      int f, rows;
      attended(L, f, rows);
      x = rows > 0 ? (int)(((unsigned)(f % 16) + rows + 15u) / 16) : 0;   // (rows may be 2^31 - 1)
    }
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (i < p.B) {
      len[i] = L;
      pre[i] = run + incl - x;
    }
    run += __shfl_sync(0xffffffffu, incl, 31);
    longest = max(longest, __reduce_max_sync(0xffffffffu, x));
  }
  if (lane == 0) pre[p.B] = run;
  __syncwarp();

  const int H = p.H_kv;
  if (blockIdx.x == 0) {
    // sequences of length 0 have no rows and so no merging warp: zero output
    const int row_elems = H * G * D;
    for (int bb = 0; bb < p.B; ++bb) {
      if (pre[bb + 1] != pre[bb]) continue;
      for (int i = threadIdx.x; i < row_elems; i += blockDim.x)
        static_cast<T*>(p.out)[(size_t)bb * row_elems + i] = T(0.f);
    }
  }
  // The CTA's groups [c0, c1): an equal share of all, or whole units where
  // these come to little more; and the warp's share of them.
  const unsigned total = (unsigned)H * run;
  const Q8Split split(total, prm.by_ctas);
  auto unit_start = [&](unsigned u) {
    const unsigned b = prm.by_heads(u);
    return b < (unsigned)p.B ? (unsigned)H * pre[b] + (u - b * H) * (pre[b + 1] - pre[b]) : total;
  };
  unsigned c0, c1;
  const Q8Split units((unsigned)p.B * H, prm.by_ctas);
  if ((units.each + (units.rest > 0 ? 1 : 0)) * longest <= split.each + kQ8Uneven / (16 * 2 * NSRC * D)) {
    c0 = unit_start(units.start(blockIdx.x));
    c1 = unit_start(units.start(blockIdx.x + 1));
  } else {
    c0 = split.start(blockIdx.x);
    c1 = split.start(blockIdx.x + 1);
  }
  const unsigned share = (c1 - c0) / W, odd = (c1 - c0) % W;   // the first `odd` warps take one more
  const unsigned r0 = c0 + warp * share + min((unsigned)warp, odd), r1 = r0 + share + ((unsigned)warp < odd ? 1 : 0);
  if (r0 < r1) {
  Q8Walker walk;
  {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if ((unsigned)H * pre[mid + 1] > r0) hi = mid; else lo = mid + 1;
    }
    const unsigned off = r0 - (unsigned)H * pre[lo];
    const unsigned L = pre[lo + 1] - pre[lo];
    walk.b = lo;
    walk.h = (int)(off / L);
    walk.t = (int)(off - walk.h * L);
    walk.r = r0;
    walk.r1 = r1;
  }
  Q8Walker prod = walk;

  uint8_t* wring = smem + (size_t)warp * NS * STAGE;   // this warp's stages
  uint64_t* wbars = bars + warp * NS;
  const uint64_t policy = l2_policy_evict_first();
  const int plane_rows = p.ring > 0 ? p.ring : p.S_max;
  const size_t plane_codes = (size_t)plane_rows * D;            // bytes per unit
  const size_t plane_scales = (size_t)q8_scale_cols(plane_rows);

  // A tile of n groups from group t of sequence b: the row of its first one,
  // how many of its rows are read (the sequence's last rows may end inside a
  // group), how many of those come before a ring's end (a whole number of
  // groups; the others follow from the ring's start), and how many come before
  // the first attended one.
  auto tile_rows = [&](int b, int t, int n, int& row0, int& nrows, int& n1, int& skip) {
    int f, rows;
    attended(len[b], f, rows);
    const int lead = f % 16;
    row0 = f - lead + 16 * t;
    if (p.ring > 0 && row0 >= p.ring) row0 -= p.ring;
    nrows = min(16 * n, lead + rows - 16 * t);
    skip = t == 0 ? lead : 0;
    n1 = p.ring > 0 && nrows > p.ring - row0 ? p.ring - row0 : nrows;
  };

  // This lane's scale of a tile: of plane lane / GROUPS (key sources, then
  // value sources) and group lane % GROUPS.
  const float* my_scales = nullptr;
#pragma unroll
  for (int i = 0; i < 2 * NSRC; ++i)
    if (lane / GROUPS == i) my_scales = i >= NSRC ? prm.vs[i % NSRC] : prm.ks[i % NSRC];

  auto issue = [&](int stage, int b, int h, int t, int n) {
    uint8_t* dst = wring + (size_t)stage * STAGE;
    uint64_t* bar = &wbars[stage];
    const size_t u = (size_t)b * H + h;
    int row0, nrows, n1, before;
    tile_rows(b, t, n, row0, nrows, n1, before);
    if (lane == 0) {
      const uint32_t b1 = (uint32_t)n1 * D, b2 = (uint32_t)(nrows - n1) * D;
      const size_t base = u * plane_codes, off = base + (size_t)row0 * D;
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(bar, (b1 + b2) * 2 * NSRC);
#pragma unroll
      for (int i = 0; i < 2 * NSRC; ++i) {
        const int sidx = i % NSRC;
        const uint8_t* src =
            static_cast<const uint8_t*>(i >= NSRC ? (sidx ? p.v1 : p.v0) : (sidx ? p.k1 : p.k0));
        bulk_g2s(dst + i * TILE, src + off, b1, bar, policy);
        if (b2) bulk_g2s(dst + i * TILE + b1, src + base, b2, bar, policy);
      }
    }
    const int gr = lane % GROUPS;
    if (my_scales && gr < n) {
      int row = row0 + 16 * gr;
      if (p.ring > 0 && row >= p.ring) row -= p.ring;
      copy4_async(dst + Cfg::CODE_BYTES + lane * 4, my_scales + u * plane_scales + row / kQ8Block);
    }
    arrive_after_copies(bar);
  };

  int issued = 0;
#pragma unroll 1
  for (int s = 0; s < NS; ++s) {
    int tb, th, tt, tn;
    bool tl;
    if (!prod.next(pre, H, p.B, GROUPS, tb, th, tt, tn, tl)) break;
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
  float c_row[NSRC];           // 2^-e of the head's query times a source's key weights
  // what a source's value scales are multiplied by: its largest value weight over
  // the larger source's, as powers of two (below 2^-126: 0)
  [[maybe_unused]] float gv[2] = {1.f, 1.f};
  float m = -FLT_MAX, l = 0.f; // of head n8, this lane's keys
  bool fresh = true;
  bool whole = false;          // the range has the unit from its first group on
  int consumed = 0;

#pragma unroll 1
  for (;;) {
    int b, h, t0, n;
    bool last;
    if (!walk.next(pre, H, p.B, GROUPS, b, h, t0, n, last)) break;
    const int stage = consumed % NS;
    const uint32_t parity = (uint32_t)(consumed / NS) & 1u;

    if (fresh) {
      whole = t0 == 0;
      // head n8's query, channels [q4 D/4, + D/4), times the source's key weights,
      // brought to [2^14, 2^15)
      float x[D / 4], wk[NSRC][D / 4];
#pragma unroll
      for (int e = 0; e < D / 4; ++e) x[e] = 0.f;
      if (n8 < G)
        load_floats<D / 4>(static_cast<const T*>(p.q) + (((size_t)b * H + h) * G + n8) * D + q4 * (D / 4), x);
      [[maybe_unused]] float wv[2][(D + 31) / 32];
      if constexpr (NSRC == 2) {
#pragma unroll
        for (int sidx = 0; sidx < 2; ++sidx)
#pragma unroll
          for (int k = 0; k < (D + 31) / 32; ++k)
            wv[sidx][k] = lane + 32 * k < D ? (sidx ? p.b1 : p.b0)[(size_t)h * D + lane + 32 * k] : 0.f;
      }
#pragma unroll
      for (int sidx = 0; sidx < NSRC; ++sidx) {
        const float* ap = sidx == 0 ? p.a0 : p.a1;
        if (NSRC == 2 || ap) {
          load_floats<D / 4>(ap + (size_t)h * D + q4 * (D / 4), wk[sidx]);
        } else {
#pragma unroll
          for (int e = 0; e < D / 4; ++e) wk[sidx][e] = 1.f;
        }
#pragma unroll
        for (int e = 0; e < D / 4; ++e) {
          wk[sidx][e] *= x[e] * p.qscale;
        }
      }
      if constexpr (NSRC == 2) {
        uint32_t e[2];   // the largest weights' exponents
#pragma unroll
        for (int sidx = 0; sidx < 2; ++sidx) {
          uint32_t most = 0;
#pragma unroll
          for (int k = 0; k < (D + 31) / 32; ++k) {
            const uint32_t u = __float_as_uint(fabsf(wv[sidx][k]));
            if (u < 0x7f800000u) most = max(most, u);
          }
          e[sidx] = __reduce_max_sync(0xffffffffu, most) >> 23;
        }
#pragma unroll
        for (int sidx = 0; sidx < 2; ++sidx) {
          const uint32_t below = max(e[0], e[1]) - e[sidx];
          gv[sidx] = below > 126 ? 0.f : __uint_as_float((127 - below) << 23);
        }
      }
#pragma unroll
      for (int sidx = 0; sidx < NSRC; ++sidx) {
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < D / 4; ++e) top = fmaxf(top, fabsf(wk[sidx][e]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int eq = 14 - ((int)(__float_as_uint(top) >> 23) - 127);
        eq = eq > 120 ? 120 : (eq < -120 ? -120 : eq);   // (2^eq and its inverse stay normal)
        const float f = __uint_as_float((uint32_t)(eq + 127) << 23);
        c_row[sidx] = __uint_as_float((uint32_t)(127 - eq) << 23);
#pragma unroll
        for (int j = 0; j < KW; ++j) {
          const float* y = wk[sidx] + 4 * j;
          split_f16(y[0] * f, y[1] * f, qf[sidx][j][0], qf[sidx][j][1]);
          split_f16(y[2] * f, y[3] * f, qf[sidx][j][2], qf[sidx][j][3]);
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
      if (lane == 0) sh.head[warp] = kQ8Stopped;
      break;
    }

    int row0, nrows, n1, skip;   // skip: rows of the first group before the first attended
    tile_rows(b, t0, n, row0, nrows, n1, skip);
    const uint8_t* st = wring + (size_t)stage * STAGE;
    const float* scales = reinterpret_cast<const float*>(st + Cfg::CODE_BYTES);

    // A whole tile (EDGE false), or its group g0, of whose rows those before
    // `skip` and from `nrows` on are not attended.
    auto tile = [&](auto edge, int g0, int skip, int nrows) {
      constexpr bool EDGE = decltype(edge)::value;
      constexpr int NG = EDGE ? 1 : GROUPS;
      const uint8_t* codes = st + 16 * g0 * D;
      // scale of plane i (key sources, then value sources), group g0 + gr
      auto scale = [&](int i, int gr) { return scales[i * GROUPS + g0 + gr]; };
      // scores in base 2: s[gr][2 half + e] is key 2 q4 + e of the half; and
      // the groups' value exponents
      float s[NG][4], ev[NG], rv[NG];   // rv: 2^-ev
      float mt = -INFINITY;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        float vs = scale(NSRC, gr);
        if constexpr (NSRC == 2) vs = fmaxf(vs * gv[0], scale(NSRC + 1, gr) * gv[1]);
        ceil_log2(fmaxf(vs, kQ8MinValue), ev[gr], rv[gr]);
#pragma unroll
        for (int sidx = 0; sidx < NSRC; ++sidx) {
          const float f = scale(sidx, gr) * c_row[sidx];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t kw[KW];
            load_words<D / 4>(codes + sidx * TILE + (16 * gr + 8 * half + krow) * D + q4 * (D / 4), kw);
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < KW; ++j) {
              uint32_t b0, b1;
              e4m3x4_to_f16(kw[j], b0, b1);
              mma16816(d, qf[sidx][j], b0, b1);
            }
            s[gr][2 * half] = sidx == 0 ? (d[0] + d[2]) * f : fmaf(d[0] + d[2], f, s[gr][2 * half]);
            s[gr][2 * half + 1] = sidx == 0 ? (d[1] + d[3]) * f : fmaf(d[1] + d[3], f, s[gr][2 * half + 1]);
          }
        }
        if constexpr (EDGE) {
          // keys 2 q4, 2 q4 + 1 of the halves are these rows of the group
          const int ra = vrow, rb = vrow2;
          if (ra < skip || ra >= nrows) s[gr][0] = -INFINITY;
          if (rb < skip || rb >= nrows) s[gr][1] = -INFINITY;
          if (ra + 8 < skip || ra + 8 >= nrows) s[gr][2] = -INFINITY;
          if (rb + 8 < skip || rb + 8 >= nrows) s[gr][3] = -INFINITY;
        }
        mt = fmaxf(mt, fmaxf(fmaxf(s[gr][0], s[gr][1]), fmaxf(s[gr][2], s[gr][3])) + ev[gr]);
      }
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
      const bool grow = mt > m + kQ8Slack;
      if (__any_sync(0xffffffffu, grow)) {
        const float m_new = grow ? floorf(mt) : m;
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
      for (int gr = 0; gr < NG; ++gr) {
        float pv[4];
        const float add = ev[gr] + off;
#pragma unroll
        for (int e = 0; e < 4; ++e) pv[e] = fast_exp2(s[gr][e] + add);
        l = fmaf((pv[0] + pv[1]) + (pv[2] + pv[3]), rv[gr], l);
#pragma unroll
        for (int sidx = 0; sidx < NSRC; ++sidx) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = pv[e];
          const float ratio = (NSRC == 2 ? scale(NSRC + sidx, gr) * gv[sidx] : scale(NSRC, gr)) * rv[gr];
          if (NSRC == 2 || ratio != 1.f) {
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
          const uint8_t* vt = codes + (NSRC + sidx) * TILE + 16 * gr * D;
          load_value<D>(vt + vrow * D, n8, va);
          load_value<D>(vt + vrow2 * D, n8, vb);
          load_value<D>(vt + (vrow + 8) * D, n8, vc);
          load_value<D>(vt + (vrow2 + 8) * D, n8, vd);
          if constexpr (EDGE) {
            // rows that are not attended may hold anything: nothing times 0
            const int ra = vrow, rb = vrow2;
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
    if (skip == 0 && nrows == 16 * GROUPS) {
      tile(std::false_type{}, 0, 0, 16 * GROUPS);
    } else {
#pragma unroll 1
      for (int g0 = 0; g0 < n; ++g0) tile(std::true_type{}, g0, skip - 16 * g0, nrows - 16 * g0);
    }

    ++consumed;
    __syncwarp();
    // refill the stage just read with the warp's next tile
    {
      int tb, th, tt, tn;
      bool tl;
      if (prod.next(pre, H, p.B, GROUPS, tb, th, tt, tn, tl)) {
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
      const bool ends = t0 + n == pre[b + 1] - pre[b];
      float* rec = whole ? reinterpret_cast<float*>(wring) : sh.head_rec + (size_t)warp * G * PS;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int head = 2 * q4 + e;
        // (1 / gv; 0: a finite one, times sums of zeros)
        [[maybe_unused]] const float ug[2] = {__uint_as_float((254u << 23) - __float_as_uint(gv[0])),
                                              __uint_as_float((254u << 23) - __float_as_uint(gv[1]))};
        const float inv = 1.f / __shfl_sync(0xffffffffu, l, 8 * q4 + 4 * e);
        if (head >= G) continue;
#pragma unroll
        for (int i = 0; i < VT; ++i) {
          const int c = value_channel<D>(n8, 2 * i);
          float x = o[0][i][e], y = o[0][i][e + 2];
          if (NSRC == 2 || p.b0) {
            const float2 w0 = *reinterpret_cast<const float2*>(p.b0 + (size_t)h * D + c);
            x *= NSRC == 2 ? w0.x * ug[0] : w0.x;
            y *= NSRC == 2 ? w0.y * ug[0] : w0.y;
          }
          if constexpr (NSRC == 2) {
            const float2 w1 = *reinterpret_cast<const float2*>(p.b1 + (size_t)h * D + c);
            x = fmaf(o[1][i][e], w1.x * ug[1], x);
            y = fmaf(o[1][i][e + 2], w1.y * ug[1], y);
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
  if (__any_sync(0xffffffffu, lane < W && sh.head[lane] == kQ8Stopped)) return;   // a wait ran out
  q8_tail<T, D, W>(p, sh, G, total, split, c0, c1, pre);
}

// Shared memory behind the rings: barriers, lengths and the words of Q8Shared;
// then the records.
__host__ __device__ constexpr size_t q8_aux_bytes(int warps, int stages, int B) {
  return ((size_t)warps * stages * 8 + (size_t)(2 * B + 1 + 2 * warps + 8) * 4 + 15) / 16 * 16;
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
  prm.by_ctas = Q8Div::of((unsigned)plan.ctas);
  prm.by_heads = Q8Div::of((unsigned)a.kv_heads);
  prm.by_ring = Q8Div::of((unsigned)(a.ring > 0 ? a.ring : 1));
  prm.aux_bytes = (int)q8_aux_bytes(Q8Shape<D, NSRC>::W, Q8Shape<D, NSRC>::NS, a.batch);
  auto kern = decode_q8_kernel<T, D, NSRC>;
  static KernelReady ready;   // (for the largest batch and group)
  static_assert(Q8Cfg<D, NSRC>::STAGE_BYTES * Q8Shape<D, NSRC>::W * Q8Shape<D, NSRC>::NS +
                        (int)q8_aux_bytes(Q8Shape<D, NSRC>::W, Q8Shape<D, NSRC>::NS, 1024) +
                        Q8Shape<D, NSRC>::W * 4 * partial_stride(D) * 4 <= 232448,
                "shared memory of the largest batch and group");
  const cudaError_t e = ready.check(kern, a.device, (int)q8_smem_bytes<D, NSRC>(1024, 4), 0, 0);
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
