// Causal prefill attention over 8-bit caches (e4m3 codes, one scale per 32
// rows of a KV head; q8_device.cuh) on the tcgen05 tensor cores of sm_103a:
// one source (vanilla, Lite, scaled) or two (fused: FusedKV slides,
// Eqs.(4)-(5)), rebuilt tile by tile in shared memory.
//
// What one call computes: for every sequence b, query head h (KV head
// kh = h / G) and query position m of the chunk
//     o_{h,m} = sum_{t <= m, t > m - W} softmax_t(scale * q_{h,m} . K_t) V_t.
//
// The operands are fp16, which holds every e4m3 code exactly, and the scales
// stay outside the products.  With K_t = s_t k_t and V_t = r_t v_t (k, v the
// tile's fp16 elements; s, r the same for a block of 32 keys),
//     o = sum_t p_t r_t v_t / sum_t p_t,
//     p_t r_t = 2^(c s_t (q . k_t) + log2 r_t),   c = scale * log2 e,
// so a key scale multiplies the score and a value scale's logarithm is added
// to it (down to kQ8MinValue; the rest of a smaller one goes into the tile):
// the running maximum is that of the sum, and P' = p r, at most
// 2^(kBias + kSlack) in its frame, is rounded to fp16 (2^-12) whatever the
// scales are.  The softmax's sum takes p = P' / r.  A row of Q (times its key
// weights in the scaled mode) is brought to fp16 with a power of two that
// places its largest element below 2^15.  Two sources are combined as
//     w0 (c0 r0) + w1 (c1 r1),  r_i = s_i W_i / s,  s = max(s0 W0, s1 W1) or the power of two above,
// in packed fp16 arithmetic (four instructions for two channels), with each
// source's weights divided by the power of two above the head's largest, W_i.
// So a source counts by its scales times its weights, whichever make it large
// (weights that share one power of two, and ratios of the scales alone, lost a
// source whose scales were 2^25 times smaller although its weights made up for
// it).  The weights come times 2^4 and the ratios times 2^2, which keeps the sum
// below 2^16 and leaves the weights 11 bits down to 2^-18 of their head's largest,
// the ratios down to 2^-16 (powers of two: to 2^-26, which is what appended rows
// have), and a source's codes 2^-12 of their largest down to ratios of 2^-26.
//
// Structure (as prefill_wide.cu): a CTA owns two groups of 128 query rows over
// the same keys (two heads of a KV head, or two row tiles of one head), each
// with a softmax warpgroup and an MMA-issuing warp that takes turns with the
// other's; S / P and O live in tensor memory, Q in shared memory.  Two warps
// bring tiles of codes by cp.async.bulk (a tile's rows are contiguous, in two
// pieces where a ring wraps, so no ring size is excluded), the issuers bring
// their group's query rows the same way (read row by row by their threads,
// they took 10,000 to 20,000 cycles a CTA), and a conversion warpgroup writes
// the fp16 tiles in the swizzled layout that the MMAs read.
// Its step k makes V_{k-1} and K_k, what MMA step k reads.  Tiles start at
// multiples of 32 keys, so that a block of one scale is whole in its tile.
//
// Key rows that a query may not see do not reach it, whatever they hold:
// scores are masked by position, and a value that is not a number is 0 in the
// tile and makes NaN of the rows that see it at the end.
//
// Where a call has few query tiles over many keys (a short chunk behind a long
// prefix), the key tiles of a CTA's rows are split over a cluster of 2, 4 or 8
// CTAs, which join their O, maxima and sums through distributed shared memory,
// each for its share of the rows.
//
// What bounds it: each group's chain of softmax (about 1550 cycles for 128 keys
// of 96 channels), hand-offs (400) and products (1450, in turns with the other
// group's), at 39% of the tensor pipe's cycles, half of the issue slots and 44%
// of shared memory's; and about 8 us a CTA before its first scores and after
// its last products.  The same chain over bf16 tiles takes 707 us of 650M Lite's
// 892: the rest is the conversion beside it.  650M calls of 8192 rows, 824.7 GFLOP: Lite 892 us (925
// TFLOP/s), fused 1153 (715); 1.5B: Lite 991 (1110), fused 1484 (741).
//
// Every wait is bounded; a wait that runs out sets an abort flag that each
// role checks, flags the device status, and the CTA frees its tensor memory.
#pragma once

#include <cfloat>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "fkv_kernels.h"
#include "q8_device.cuh"
#include "tc_device.cuh"

namespace fkv {
namespace q8p {

constexpr int BM = 128;            // query rows per group
constexpr int NG = 2;              // groups per CTA
constexpr int GROUP_COLS = 256;    // TMEM columns per group: S/P, O
constexpr int SMEM_LIMIT = 232448; // opt-in dynamic shared memory per CTA (227 KB)
constexpr float kSlack = 8.f;      // log2 growth of the running max tolerated before O is rescaled
constexpr float kBias = 7.f;       // P' <= 2^(7 + 8) < 65504, and is not flushed above 2^-31
constexpr int NSR = 8;             // conversion-step barriers and scale records
constexpr float kWeightFrame = 16.f, kRatioFrame = 4.f;   // of two sources' weights and ratios
constexpr float kFrame = 64.f, kLogFrame = 6.f;          // and of their elements
static_assert(kWeightFrame * kRatioFrame == kFrame, "");

constexpr int cap(int x, int most) { return x > most ? most : x; }

template <int D, int NSRC>
struct Cfg {
  // keys per tile; at D = 128 two sources' codes leave room for 96
  static constexpr int BN = D == 128 && NSRC == 2 ? 96 : 128;
  static constexpr int NGRP = BN / kQ8Block;            // blocks of a tile
  static constexpr int CB = (D + kSWE - 1) / kSWE;      // 32-element column blocks
  static constexpr int Q_BYTES = CB * BM * kSW;         // one group's Q tile
  static constexpr int KV_BYTES = CB * BN * kSW;        // one fp16 tile
  static constexpr int RAW_BYTES = BN * D;              // one tile of codes of one source
  static constexpr int O_COL = BN;
  static_assert(O_COL + D <= GROUP_COLS, "S and O do not fit a group's columns");
  // fp16 weights [4][D], scale records [NSR][NGRP] float4, [NSR][2][NGRP] ratios, barriers and words
  static constexpr int FIXED =
      (NSRC == 2 ? 4 * D * 2 + NSR * 2 * NGRP * 8 : 0) + NSR * NGRP * 16 + 512;
  static constexpr int ROOM = SMEM_LIMIT - 512 - FIXED - NG * Q_BYTES;
  static constexpr int NS = 2;   // K and V slots: a K slot is freed by its only product, a step before its V's
  static constexpr int NR = cap((ROOM - 2 * NS * KV_BYTES) / (2 * NSRC * RAW_BYTES), 2);   // slots of codes
  static_assert(NR >= 1, "shared memory too small for the tiles");
  static_assert(NSR > NS + 2, "step barriers must outnumber the tile slots");
  static constexpr size_t SMEM =
      512 + (size_t)FIXED + NG * Q_BYTES + (size_t)2 * NR * NSRC * RAW_BYTES + (size_t)2 * NS * KV_BYTES;
  static_assert(SMEM <= SMEM_LIMIT, "shared memory above the opt-in limit");
  static constexpr int SOFTMAX_WARPS = 4 * NG;
  static constexpr int K_PRODUCER_WARP = SOFTMAX_WARPS;
  static constexpr int MMA_WARP = K_PRODUCER_WARP + 1;   // + g for group g
  static constexpr int V_PRODUCER_WARP = MMA_WARP + NG;
  static constexpr int CONV_WARP = SOFTMAX_WARPS + 4;
  static constexpr int THREADS = 32 * (SOFTMAX_WARPS + 8);
  // registers: 128 per thread at launch (65536 / 512); a warpgroup may only give
  // some up (conversion, control) or take some (softmax).  Two sources
  // (650M fused): 104 and 184 take 0.7% more than 120 and 176, 88 and 192 4%
  // more; one source (650M Lite): 72 and 200 1.2% more than 104 and 184.
  static constexpr int REGS_CONTROL = 40, REGS_CONV = NSRC == 2 ? 120 : 104, REGS_SOFTMAX = NSRC == 2 ? 176 : 184;
  static constexpr long long REGS_SPLIT =
      (long long)NG * 128 * REGS_SOFTMAX + 128LL * REGS_CONTROL + 128LL * REGS_CONV;
  static_assert(REGS_SPLIT <= (long long)THREADS * 128, "register split above the launch allocation");
  static_assert(REGS_CONTROL <= 128 && REGS_CONV <= 128 && REGS_SOFTMAX >= 128, "each moves its own way");
};

struct Params {
  const uint8_t* k[2];
  const uint8_t* v[2];
  const float* ks[2];
  const float* vs[2];
  const float* a[2];   // key weights [H_kv, D] of the sources (null: none)
  const float* b[2];
  const void* q;       // [B, H_q, S, D] bf16
  void* out;           // [B, H_q, S, D] bf16
  int* status;
  const unsigned long long* wait_limit;
  int H_kv, G;
  int S;               // query rows of this call (the chunk length C)
  int q_start;         // cache position of query row 0
  int S_kv;            // key positions: q_start + C
  int window;
  int rows;            // rows of a (sequence, KV head) in the caches
  int ring;            // > 0: position t at row t % ring
  float scale_log2;
  int splits;          // CTAs of a cluster, which share the key tiles
};

// All of the warpgroup's 128 threads arrive; true where all were ok.
__device__ __forceinline__ bool group_and(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

// The same for the 256 softmax threads.
__device__ __forceinline__ bool softmax_and(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 2, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

// The 128 threads of softmax warpgroup g meet.
__device__ __forceinline__ void group_sync(int g) {
  if (g == 0)
    asm volatile("barrier.cta.sync 3, 128;" ::: "memory");
  else
    asm volatile("barrier.cta.sync 4, 128;" ::: "memory");
}

// All threads of the cluster's CTAs meet (every one of them gets here, since
// every wait before is bounded).
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// A word of another CTA's shared memory, at this CTA's address `addr`.
__device__ __forceinline__ float ld_cluster(uint32_t addr, int rank) {
  float v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
      : "=f"(v)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

__device__ __forceinline__ uint32_t hmul2u(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hfma2u(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b),
                            *reinterpret_cast<__half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Packed fp32 pairs as 64-bit operands (made once where a pair is used often:
// the compiler copies both halves for every use of a pair made in place).
__device__ __forceinline__ unsigned long long pair_of(float x, float y) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(unsigned long long p, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
}
__device__ __forceinline__ unsigned long long ffma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long fadd2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Whether one of four codes is not a number.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// 2^e with 2^e <= x < 2^(e+1) for a normal x > 0 (0 for what is smaller).
__device__ __forceinline__ int exponent_of(float x) { return (int)((__float_as_uint(x) >> 23) & 255u) - 127; }
__device__ __forceinline__ float reciprocal_of_power(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }
__device__ __forceinline__ float power_of_two(int e) {   // e clamped to the normal range
  e = e < -126 ? -126 : (e > 127 ? 127 : e);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// SPLIT: a cluster of p.splits CTAs shares the key tiles.
template <int D, int NSRC, bool SPLIT>
__global__ void __launch_bounds__(Cfg<D, NSRC>::THREADS, 1) prefill_q8_kernel(const Params p) {
  using C = Cfg<D, NSRC>;
  constexpr int BN = C::BN, NS = C::NS, NGRP = C::NGRP, NR = C::NR;
  extern __shared__ uint8_t smem_raw[];
  // 512-byte alignment: the period of the 64-byte swizzle pattern
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 511) & ~uintptr_t(511));
  uint8_t* sQ = smem;                                   // fp16 queries of the two groups
  uint8_t* sK = sQ + NG * C::Q_BYTES;                   // fp16 tiles
  uint8_t* sV = sK + NS * C::KV_BYTES;
  uint8_t* sRawK = sV + NS * C::KV_BYTES;               // codes, the sources of a slot side by side
  uint8_t* sRawV = sRawK + NR * NSRC * C::RAW_BYTES;
  float4* sScale = reinterpret_cast<float4*>(sRawV + NR * NSRC * C::RAW_BYTES);   // {s (times what the weights were divided by), log2 r, 1 / r, rest of r}
  // of K and V: 2^2 (r0, r1), each as two equal halves
  uint2* sRatio = reinterpret_cast<uint2*>(sScale + NSR * NGRP);
  uint16_t* sW = reinterpret_cast<uint16_t*>(sRatio + (NSRC == 2 ? NSR * 2 * NGRP : 0));   // fp16 2^4 (a0 / W0, a1 / W1), of b0 and b1 alike
  uint64_t* bars = reinterpret_cast<uint64_t*>(sW + (NSRC == 2 ? 4 * D : 0));
  uint64_t* q_ready = bars;
  uint64_t* q_raw = q_ready + 1;          // [NG]
  uint64_t* k_empty = q_raw + NG;         // [NS]
  uint64_t* v_empty = k_empty + NS;       // [NS]
  uint64_t* rk_full = v_empty + NS;       // [NR]
  uint64_t* rk_empty = rk_full + NR;
  uint64_t* rv_full = rk_empty + NR;
  uint64_t* rv_empty = rv_full + NR;
  uint64_t* step_ready = rv_empty + NR;   // [NSR]
  uint64_t* s_full = step_ready + NSR;    // [NG]
  uint64_t* p_full = s_full + NG;         // [NG]
  uint64_t* mma_drain = p_full + NG;      // [NG]
  uint32_t* words = reinterpret_cast<uint32_t*>(mma_drain + NG);
  uint32_t* tmem_slot = words;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(words + 1);
  int* sm_issued = reinterpret_cast<int*>(words + 2);   // [2] tiles each producer issued
  uint32_t* w_top = words + 4;     // [4] largest weight of a0, a1, b0, b1 (bits)
  uint32_t* bad = words + 8;       // [1 + 8 + 8] values that are not numbers: 1: seen by all, 2: some near
                                   // the diagonal or the window's start; which (bits of positions)

  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  int ux, mt;
  const int splits = SPLIT ? p.splits : 1;
  const int rank = SPLIT ? (int)blockIdx.x % splits : 0;   // in the cluster
  if constexpr (SPLIT) {
    ux = (int)blockIdx.x / splits;
    mt = (int)(gridDim.y - 1 - blockIdx.y);
  } else {
    prefill_cta_tile(ux, mt);   // longest query tiles first
  }
  const bool two_heads = p.G % 2 == 0;
  const int pairs = two_heads ? p.G / 2 : p.G;   // CTAs of a unit's heads
  const int unit = ux / pairs, pair = ux % pairs;
  const int H_q = p.H_kv * p.G;
  const int b = unit / p.H_kv, kh = unit % p.H_kv;
  // group g: query head and first query row (within the chunk)
  auto g_head = [&](int g) { return kh * p.G + (two_heads ? pair * 2 + g : pair); };
  auto g_row0 = [&](int g) { return two_heads ? mt * BM : mt * (NG * BM) + g * BM; };
  const int S_kv = p.S_kv;
  const int W = p.window;
  // key tiles of positions start + j * BN: from the first group's window start
  // (down to the start of its block) to each group's last position
  const int pos_first = p.q_start + g_row0(0);
  const int start = W > 0 ? max(0, pos_first - W + 1) / kQ8Block * kQ8Block : 0;
  // (positions end at 2^31 - 1: no sum below goes past the chunk's last)
  auto g_end = [&](int g) { return p.q_start + min(g_row0(g) + BM, p.S); };   // behind its last position
  auto all_tiles = [&](int g) { return (int)(((unsigned)(g_end(g) - start) + BN - 1) / BN); };
  // of which the CTA takes [jb, je) (all of them but in a cluster), group 1 all
  // and group 0 those up to its own last position, one at least (a tile that is
  // masked for all its rows, if need be); a CTA with none (idle: the first query
  // rows have few keys) takes its neighbour's, masked
  const int n_all = all_tiles(1);
  const int jb = rank * n_all / splits, je = max((rank + 1) * n_all / splits, jb + 1);
  const bool idle = SPLIT && (rank + 1) * n_all / splits == jb;
  const int pos0 = start + jb * BN;
  auto n_tiles = [&](int g) { return max(1, min(all_tiles(g), je) - jb); };
  const int n_max = je - jb;

  auto tile_k = [&](int j) { return sK + (size_t)(j % NS) * C::KV_BYTES; };
  auto tile_v = [&](int j) { return sV + (size_t)(j % NS) * C::KV_BYTES; };

  if (tid == 0) {
    mbar_init(q_ready, 128 * NG);
    for (int g = 0; g < NG; ++g) mbar_init(&q_raw[g], 1);
    for (int s = 0; s < NSR; ++s) mbar_init(&step_ready[s], 128);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&k_empty[s], NG);    // one commit per group that reads the tile
      mbar_init(&v_empty[s], NG);
    }
    for (int s = 0; s < NR; ++s) {
      mbar_init(&rk_full[s], 1);
      mbar_init(&rk_empty[s], 128);  // the conversion threads, once they have read it
      mbar_init(&rv_full[s], 1);
      mbar_init(&rv_empty[s], 128);
    }
    for (int g = 0; g < NG; ++g) {
      mbar_init(&s_full[g], 1);
      // the group's 128 softmax threads, plus the other group's issuer once
      // its previous step's PV products are queued (the turn)
      mbar_init(&p_full[g], 129);
      mbar_init(&mma_drain[g], 1);
    }
    *abort_flag = 0;
    sm_issued[0] = sm_issued[1] = 0;
    for (int i = 0; i < 17; ++i) bad[i] = 0;
    fence_mbar_init();
  }
  if (warp == C::MMA_WARP) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const unsigned long long wlim = wait_limit_ns(p.wait_limit);
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (*abort_flag) return false;
    if (mbar_wait_bounded(bar, parity, wlim)) return true;
    *abort_flag = 1;
    flag_status(p.status, kDevTimeout);
    return false;
  };

  if (warp >= C::CONV_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_CONV));
    // ---------------- conversion warpgroup ----------------
    const int ft = tid - 32 * C::CONV_WARP;   // 0..127
    const size_t scols = (size_t)q8_scale_cols(p.rows);
    // Scale records of tile j, one thread per block.
    float ns[2 * NSRC];
    float k_power = 1.f;   // what the key weights were divided by
    [[maybe_unused]] float by_top[4];   // W_i over the larger one's, of keys and of values
    auto load_scales = [&](int j) {
#pragma unroll
      for (int i = 0; i < 2 * NSRC; ++i) ns[i] = 1.f;   // (blocks behind the last key: any finite one)
      if (ft < NGRP && j < n_max && ft * kQ8Block < S_kv - (pos0 + j * BN)) {
        const int pos = pos0 + j * BN + ft * kQ8Block;
        const size_t at = (size_t)unit * scols + (p.ring > 0 ? pos % p.ring : pos) / kQ8Block;
#pragma unroll
        for (int i = 0; i < NSRC; ++i) {
          ns[i] = __ldg(p.ks[i] + at);
          ns[NSRC + i] = __ldg(p.vs[i] + at);
        }
      }
    };
    auto store_scales = [&](int j) {
      if (ft >= NGRP) return;
      float4& rec = sScale[(j % NSR) * NGRP + ft];
      if constexpr (NSRC == 1) {
        const float r = fmaxf(ns[1], kQ8MinValue);
        rec = make_float4(ns[0], log2f(r), 1.f / r, ns[1] / r);
      } else {
        // the larger scale's power of two goes into the record, the rest into the
        // ratios (two divisions and a logarithm here, in the chain from a step's
        // tiles to its barrier, were 3 to 6% of a call)
#pragma unroll
        for (int i = 0; i < 4; ++i) ns[i] *= by_top[i];
        float es, is, er, ir;
        ceil_log2(fmaxf(fmaxf(ns[0], ns[1]), FLT_MIN), es, is);
        ceil_log2(fmaxf(fmaxf(ns[2], ns[3]), kQ8MinValue), er, ir);
        auto twice = [](float x) { return f16x2_of(x * kRatioFrame, x * kRatioFrame); };
        uint2* ratio = sRatio + (size_t)(j % NSR) * 2 * NGRP;
        ratio[ft] = make_uint2(twice(ns[0] * is), twice(ns[1] * is));
        ratio[NGRP + ft] = make_uint2(twice(ns[2] * ir), twice(ns[3] * ir));
        rec = make_float4(k_power * reciprocal_of_power(is), er - kLogFrame, ir * kFrame, 1.f);
      }
    };
    // A value that is not a number: noted for the rows that see it, 0 in the tile.
    auto note_bad = [&](int n0, int row) {
      const int q0 = pos_first, q1 = g_end(NG - 1) - 1;   // the CTA's query positions
      if (row >= S_kv - n0) return;
      const int pos = n0 + row, hi = pos - q0, lo = hi <= 0 ? hi + (W - 1) : 0;
      if (hi <= 0 && (W == 0 || pos > q1 - W))
        atomicOr(&bad[0], 1u);
      else {
        atomicOr(&bad[0], 2u);
        if (hi > 0 && hi < NG * BM) atomicOr(&bad[1 + (hi >> 5)], 1u << (hi & 31));
        if (W > 0 && hi <= 0 && lo >= 0 && lo < NG * BM) atomicOr(&bad[9 + (lo >> 5)], 1u << (lo & 31));
      }
    };
    // A tile is runs of 16 codes, D / 16 a row, which become two 16-byte chunks
    // of the swizzled tile each.  The 8 threads that a shared-memory pass
    // serves take 4 rows times 2 runs of a 32-channel block: their chunks lie
    // in 8 different bank groups.  Where the blocks are even in number, rows
    // of the other row pair take the neighbouring block, so that the reads of
    // 64- and 128-byte rows spread over the banks too (2 passes at most).
    constexpr int CPR = D / 16, CP = CPR / 2;
    constexpr bool TWO = CP % 2 == 0;                // threads over 32 rows and 2 blocks, or 64 rows and 1
    constexpr int RI = TWO ? 32 : 64;                // rows of an item of 128 runs
    constexpr int KI = BN / RI;
    constexpr int PAIRED = (TWO ? CP / 2 : CP) * KI; // items; a D = 80 row's fifth run adds one (row = thread)
    constexpr int ITEMS = PAIRED + CPR % 2;
    static_assert(BN % RI == 0 && (CPR % 2 == 0 || BN == 128), "items of 128 runs");
    const int rr = (ft >> 1) & 3;
    const int row0 = (TWO ? ft >> 4 : ft >> 3) * 4 + rr;
    const int blk0 = TWO ? ((ft >> 3) ^ (rr >> 1)) & 1 : 0;
    const uint32_t raw0 = (uint32_t)(row0 * D + blk0 * 32 + (ft & 1) * 16);
    const uint32_t place0 = (uint32_t)(blk0 * BN * kSW) + swz64(row0, (ft & 1) * 2);
    const uint32_t place80 = (uint32_t)(CP * BN * kSW) + swz64(ft, 0);
    // item it + i, of the same channels as item `it` -> row, run in the row,
    // offsets of the codes and of the first chunk (the other: ^ 16)
    auto item_row = [&](int it, int i) { return it < PAIRED ? row0 + (it % KI + i) * RI : ft; };
    auto item_run = [&](int it) {
      return it < PAIRED ? 2 * (blk0 + it / KI * (TWO ? 2 : 1)) + (ft & 1) : CPR - 1;
    };
    auto item_raw = [&](int it, int i) {
      return it < PAIRED ? raw0 + (uint32_t)((it % KI + i) * RI * D + it / KI * (TWO ? 64 : 32))
                         : (uint32_t)(ft * D + (CPR - 1) * 16);
    };
    auto item_place = [&](int it, int i) {
      return it < PAIRED ? place0 + (uint32_t)((it % KI + i) * RI * kSW + it / KI * (TWO ? 2 : 1) * BN * kSW) : place80;
    };
    // The head's fp16 weights of both sources for 16 channels.
    struct Weights {
      uint32_t w[2][8];
    };
    auto load_weights = [&](int it, bool value, Weights& w) {
      if constexpr (NSRC == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4* src = reinterpret_cast<const uint4*>(sW + (value ? 2 * D : 0) + i * D + item_run(it) * 16);
          const uint4 x = src[0], y = src[1];
          w.w[i][0] = x.x, w.w[i][1] = x.y, w.w[i][2] = x.z, w.w[i][3] = x.w;
          w.w[i][4] = y.x, w.w[i][5] = y.y, w.w[i][6] = y.z, w.w[i][7] = y.w;
        }
      }
    };
    // 16 codes of one source or two -> 8 fp16 pairs; r: the sources' ratios
    auto combine = [&](const uint4& x, const uint4& y, const uint2& r, const Weights& w, uint32_t* o) {
      const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
      if constexpr (NSRC == 2) {
        const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t cx[2], cy[2];
          e4m3x4_to_f16(xw[e], cx[0], cx[1]);
          e4m3x4_to_f16(yw[e], cy[0], cy[1]);
#pragma unroll
          for (int f = 0; f < 2; ++f)
            o[2 * e + f] = hfma2u(hmul2u(cx[f], r.x), w.w[0][2 * e + f], hmul2u(hmul2u(cy[f], r.y), w.w[1][2 * e + f]));
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) e4m3x4_to_f16(xw[e], o[2 * e], o[2 * e + 1]);
      }
    };
    auto load_item = [&](const uint8_t* raw, int it, int i, int j, int left, bool value, uint4& x, uint4& y, uint2& r) {
      const int row = item_row(it, i);
      x = *reinterpret_cast<const uint4*>(raw + item_raw(it, i));
      y = x;
      if constexpr (NSRC == 2) {
        y = *reinterpret_cast<const uint4*>(raw + C::RAW_BYTES + item_raw(it, i));
        r = sRatio[((j % NSR) * 2 + (value ? 1 : 0)) * NGRP + row / kQ8Block];
      }
      if (row >= left) x = y = make_uint4(0, 0, 0, 0);   // behind the last key
    };
    auto put = [&](uint8_t* dst, int it, int i, const uint32_t* o) {
      *reinterpret_cast<uint4*>(dst + item_place(it, i)) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(dst + (item_place(it, i) ^ 16u)) = make_uint4(o[4], o[5], o[6], o[7]);
    };
    // Tile j of codes -> fp16 in the swizzled layout; then `empty` is told.
    // One copy of a short loop for K and V: the softmax warps' code, unrolled
    // over a tile, and this one share the instruction caches (650M fused: 10% more
    // with the tile's items unrolled for K and for V).
    auto convert = [&](uint8_t* dst, const uint8_t* raw, int j, bool value, uint64_t* empty) {
      const int left = S_kv - (pos0 + j * BN);   // keys from the tile's first on
      uint32_t nan[4] = {0, 0, 0, 0};   // 0, or not a number once a value was none
      Weights w;
      // N items from `it` on, of the same channels
      auto items = [&](int it, auto count) {
        constexpr int N = decltype(count)::value;
        uint4 x[N], y[N];
        uint2 r[N];
        load_weights(it, value, w);
#pragma unroll
        for (int i = 0; i < N; ++i) load_item(raw, it, i, j, left, value, x[i], y[i], r[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          uint32_t o[8];
          combine(x[i], y[i], r[i], w, o);
          if (value) {   // 0 x + nan: no code is infinite
#pragma unroll
            for (int e = 0; e < 8; ++e) nan[e & 3] = hfma2u(o[e], 0u, nan[e & 3]);
          }
          put(dst, it, i, o);
        }
      };
#pragma unroll 1
      for (int it = 0; it < PAIRED; it += KI) items(it, std::integral_constant<int, KI>{});
      if constexpr (ITEMS > PAIRED) items(PAIRED, std::integral_constant<int, 1>{});
      if (value) {
        // the rest of one source's scale, where the exponents do not take it whole
        [[maybe_unused]] const float4* rec = sScale + (j % NSR) * NGRP;
        bool whole = true;
        if constexpr (NSRC == 1) {
#pragma unroll
          for (int gr = 0; gr < NGRP; ++gr) whole = whole && rec[gr].w == 1.f;
        }
        if (((nan[0] | nan[1] | nan[2] | nan[3]) & 0x7fff7fffu) != 0 || !whole) {
          // values that are no numbers: noted, and zeros put in their places
#pragma unroll 1
          for (int it = 0; it < ITEMS; ++it) {
            uint4 x, y;
            uint2 r;
            uint32_t any = 0, o[8];
            load_item(raw, it, 0, j, left, true, x, y, r);
            uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              any |= nan_codes(xw[e]) | nan_codes(yw[e]);
              xw[e] &= ~((nan_codes(xw[e]) >> 7) * 255u);
              yw[e] &= ~((nan_codes(yw[e]) >> 7) * 255u);
            }
            if (any) note_bad(pos0 + j * BN, item_row(it, 0));
            if (!any && whole) continue;
            load_weights(it, true, w);
            combine(make_uint4(xw[0], xw[1], xw[2], xw[3]), make_uint4(yw[0], yw[1], yw[2], yw[3]), r, w, o);
            if constexpr (NSRC == 1) {
              const float rest = rec[item_row(it, 0) / kQ8Block].w;
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = hmul2u(o[e], f16x2_of(rest, rest));
            }
            put(dst, it, 0, o);
          }
        }
      }
      // (only now: the arrival does not wait for loads whose values nothing has
      // used yet, and the slot's next copy would overtake them)
      mbar_arrive(empty);
    };
    if constexpr (NSRC == 2) {
      // the head's weights below 2^4, by a power of two for each vector
      const int v = ft / 32;   // a warp's vector
      const float* src = (v == 0 ? p.a[0] : v == 1 ? p.a[1] : v == 2 ? p.b[0] : p.b[1]) + kh * D;
      float x[(D + 31) / 32];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < (D + 31) / 32; ++i) {
        x[i] = lane + 32 * i < D ? src[lane + 32 * i] : 0.f;
        const uint32_t u = __float_as_uint(fabsf(x[i]));
        if (u < 0x7f800000u) top = max(top, u);
      }
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) w_top[v] = top;
      (void)group_and(true);
      int e[4];   // W_i = 2^e
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = exponent_of(__uint_as_float(w_top[i])) + 1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int below = max(e[i & 2], e[i | 1]) - e[i];
        by_top[i] = below > 126 ? 0.f : power_of_two(-below);
      }
      k_power = power_of_two(max(e[0], e[1])) * (1.f / kFrame);
      // (two factors, since 2^-e alone may lie outside the normal range)
      const int ev = v == 0 ? e[0] : v == 1 ? e[1] : v == 2 ? e[2] : e[3];
      const float f0 = power_of_two(-(ev / 2)), f1 = power_of_two(ev / 2 - ev) * kWeightFrame;
#pragma unroll
      for (int i = 0; i < (D + 31) / 32; ++i)
        if (lane + 32 * i < D) {
          const __half h = __float2half_rn(x[i] * f0 * f1);
          sW[v * D + lane + 32 * i] = *reinterpret_cast<const uint16_t*>(&h);
        }
    }
    load_scales(0);
    store_scales(0);
    (void)group_and(true);
    // step 0 makes K_0; step k > 0 makes V_{k-1}, then K_k (k < n_max)
    for (int k = 0; k <= n_max; ++k) {
      const int t = k - 1;
      load_scales(k + 1);
      // Each warp waits for itself: one look where the phases are over, else
      // one lane waits (32 that spin take issue slots from the softmax).  K's
      // operands are awaited after V is made, so that with one slot of codes
      // K's copy has had the time of V's conversion, and the next V's that of
      // K's.
      auto ready = [&](uint64_t* full, uint32_t full_parity, uint64_t* empty, uint32_t empty_parity, bool reused) {
        auto look = [&]() { return mbar_try_wait(full, full_parity) && (!reused || mbar_try_wait(empty, empty_parity)); };
        if (__all_sync(0xffffffffu, look())) return true;
        bool ok = true;
        if (lane == 0) ok = wait(full, full_parity) && (!reused || wait(empty, empty_parity));
        return __all_sync(0xffffffffu, ok) && __all_sync(0xffffffffu, look());
      };
      bool ok = true;
#pragma unroll 1
      for (int which = k > 0 ? 0 : 1; ok && which < (k < n_max ? 2 : 1); ++which) {
        const bool value = which == 0;
        const int c = value ? t : k;   // the tile
        uint64_t *full = value ? rv_full : rk_full, *empty = value ? rv_empty : rk_empty;
        ok = ready(&full[c % NR], (uint32_t)(c / NR) & 1u, &(value ? v_empty : k_empty)[c % NS],
                   (uint32_t)(c / NS - 1) & 1u, c >= NS);
        if (ok)
          convert(value ? tile_v(c) : tile_k(c), (value ? sRawV : sRawK) + (size_t)(c % NR) * NSRC * C::RAW_BYTES, c, value,
                  &empty[c % NR]);
      }
      if (ok) {
        store_scales(k + 1);
        // the tiles are read by the tensor cores (async proxy)
        fence_proxy_async_smem();
        mbar_arrive(&step_ready[k % NSR]);
      }
      // one decision for all; and the next step's scale records are in place
      if (!group_and(ok)) break;
    }
    if constexpr (SPLIT) {   // the partials are there; the partials are read
      cluster_sync();
      cluster_sync();
    }
  } else if (warp >= C::SOFTMAX_WARPS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_CONTROL));
    if ((warp == C::K_PRODUCER_WARP || warp == C::V_PRODUCER_WARP) && lane == 0) {
      // ---------------- producers: K codes, V codes ----------------
      const bool is_k = warp == C::K_PRODUCER_WARP;
      uint64_t* empty = is_k ? rk_empty : rv_empty;
      uint64_t* full = is_k ? rk_full : rv_full;
      uint8_t* ring = is_k ? sRawK : sRawV;
      uint64_t policy;   // the CTAs of a unit read the same tiles
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
      int issued = 0;
      for (int j = 0; j < n_max; ++j) {
        if (j >= NR && !wait(&empty[j % NR], (uint32_t)(j / NR - 1) & 1u)) break;
        const int n0 = pos0 + j * BN;
        const int nv = min(BN, S_kv - n0);
        const int row0 = p.ring > 0 ? n0 % p.ring : n0;
        const int n1 = p.ring > 0 ? min(nv, p.ring - row0) : nv;
        const uint32_t b1 = (uint32_t)n1 * D, b2 = (uint32_t)(nv - n1) * D;
        mbar_arrive_expect_tx(&full[j % NR], (b1 + b2) * NSRC);
#pragma unroll
        for (int i = 0; i < NSRC; ++i) {
          uint8_t* dst = ring + ((size_t)(j % NR) * NSRC + i) * C::RAW_BYTES;
          const uint8_t* src = (is_k ? p.k[i] : p.v[i]) + (size_t)unit * p.rows * D;
          bulk_g2s(dst, src + (size_t)row0 * D, b1, &full[j % NR], policy);
          if (b2) bulk_g2s(dst + b1, src, b2, &full[j % NR], policy);
        }
        issued = j + 1;
      }
      sm_issued[is_k ? 0 : 1] = issued;
    } else if (warp >= C::MMA_WARP && warp < C::MMA_WARP + NG && lane == 0) {
      // ---------------- MMA issuer of group g ----------------
      const int g = warp - C::MMA_WARP;
      constexpr uint32_t IDESC_QK = idesc_with_f16(idesc_bf16(BM, BN, false));
      constexpr uint32_t IDESC_PV = idesc_with_f16(idesc_bf16(BM, D, true));
      const uint32_t t_g = tmem + g * GROUP_COLS;
      const uint32_t qbase = smem_u32(sQ + g * C::Q_BYTES);
      {
        // the group's query rows, as they are, where they will be as fp16
        const int rows = max(0, min(BM, p.S - g_row0(g)));
        mbar_arrive_expect_tx(&q_raw[g], (uint32_t)rows * D * 2);
        if (rows > 0)
          bulk_g2s(sQ + g * C::Q_BYTES,
                   static_cast<const __nv_bfloat16*>(p.q) + (((size_t)b * H_q + g_head(g)) * p.S + g_row0(g)) * D,
                   (uint32_t)rows * D * 2, &q_raw[g], l2_policy_evict_first());
      }
      // S_g = Q_g K_j^T: M = 128 rows, N = BN keys, K = D in steps of 16
      auto issue_qk = [&](int j) {
        const uint32_t kbase = smem_u32(tile_k(j));
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (uint32_t)(k & 1) * 32;
          const uint64_t ad = sdesc(qbase + (k >> 1) * BM * kSW + off, 16, 8 * kSW);
          const uint64_t bd = sdesc(kbase + (k >> 1) * BN * kSW + off, 16, 8 * kSW);
          mma_bf16(t_g, ad, bd, IDESC_QK, k > 0);
        }
      };
      // O_g += P_g V_j: A = P_g (two per column, in the first BN/2 columns of
      // S_g), B = V_j as an MN-major operand, K = BN keys
      auto issue_pv = [&](int j) {
        const uint32_t vbase = smem_u32(tile_v(j));
#pragma unroll
        for (int k = 0; k < BN / 16; ++k) {
          const uint64_t bd = sdesc(vbase + k * 16 * kSW, BN * kSW, 8 * kSW);
          mma_bf16_ts(t_g + C::O_COL, t_g + k * 8, bd, IDESC_PV, (j > 0 || k > 0) ? 1u : 0u);
        }
      };
      // Step k of group g issues PV_g(k-1) (k > 0) and QK_g(k) (k < n_g), once
      // conversion step k has put V_{k-1} and K_k in place.  The two issuers
      // take turns, group 0's step k before group 1's: the turn is one more
      // arrival on the other group's p_full, passed once a step's PV products
      // are issued, so that each group's softmax overlaps the other group's
      // products.  Group 1 of a one-head CTA may read up to two tiles more
      // than group 0: group 0 then passes the turn for them, and their slots
      // are never refilled (NS >= 2), so their empty phases are never awaited.
      const int ng = n_tiles(g);
      auto pass_turn = [&]() { mbar_arrive(&p_full[1 - g]); };
      auto step_operands = [&](int k) {
        return wait(&step_ready[k % NSR], (uint32_t)(k / NSR) & 1u);
      };
      bool ok = wait(q_ready, 0) && step_operands(0);
      if (ok) {
        tc_fence_after();
        issue_qk(0);
        mma_commit(&s_full[g]);
        mma_commit(&k_empty[0]);
        if (g == 1) pass_turn();   // group 0's step 1 follows group 1's step 0
      }
      for (int j = 0; ok && j < ng; ++j) {
        const bool more = j + 1 < ng;
        // every wait comes before the step's first product
        if (!wait(&p_full[g], (uint32_t)j & 1u) || !step_operands(j + 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        issue_pv(j);
        pass_turn();
        if (more) issue_qk(j + 1);
        mma_commit(&s_full[g]);
        mma_commit(&v_empty[j % NS]);
        if (more) mma_commit(&k_empty[(j + 1) % NS]);
      }
      // pass group 1's extra turns once the phase before has completed (an
      // early arrival would count towards that phase)
      if (g == 0)
        for (int j = ng; ok && j < n_tiles(1); ++j) {
          ok = wait(&p_full[1], (uint32_t)(j - 1) & 1u);
          if (ok) pass_turn();
        }
    }
    __syncwarp();
    if constexpr (SPLIT) {
      cluster_sync();
      cluster_sync();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
    // ---------------- softmax warpgroup of group g ----------------
    const int g = warp >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const int m_row = g_row0(g) + row;       // query row within the chunk
    const int qpos = p.q_start + min(m_row, p.S - 1);   // its cache position (behind the chunk: the last one)
    // tiles that start in [full_from, full_to] are seen whole by all of the group's rows
    const int pos_g = p.q_start + min(g_row0(g), p.S - 1);
    const int full_to = pos_g - BN, full_from = W == 0 ? 0 : W <= BM ? INT_MAX : pos_g - (W - BM);
    const int ng = n_tiles(g);
    const bool row_valid = m_row < p.S;
    const uint32_t t_s = tmem + ((uint32_t)(quarter * 32) << 16) + g * GROUP_COLS;
    const uint32_t t_o = t_s + C::O_COL;
    float c_row = 0.f;   // what a raw score times its key scale is multiplied by
    bool ok = __all_sync(0xffffffffu, wait(&q_raw[g], 0));
    {
      // this thread's Q row (times its key weights where one source has some)
      // to fp16, its largest element in [2^14, 2^15), in the place of the
      // group's rows as they came; rows beyond the chunk are zero.  Neighbours
      // read from chunks of 8 channels next to each other, whatever a row's
      // length, so that they meet in few banks.
      constexpr int N = D / 8;
      uint8_t* qg = sQ + g * C::Q_BYTES;
      auto place = [&](int i) {   // the i-th chunk that this thread takes
        const int c = row % N + i;
        return c < N ? c : c - N;
      };
      uint4 raw[N];
#pragma unroll
      for (int i = 0; i < N; ++i)
        raw[i] = ok && row_valid ? *reinterpret_cast<const uint4*>(qg + row * D * 2 + place(i) * 16) : make_uint4(0, 0, 0, 0);
      auto fill = [&](auto weighted) {
        auto chunk = [&](int i, float* f) {
          unpack16<__nv_bfloat16>(raw[i], f);
          if constexpr (decltype(weighted)::value) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= p.a[0][(size_t)kh * D + place(i) * 8 + e];
          }
        };
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float f[8];
          chunk(i, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
        }
        const int eq = top > 0.f && top < INFINITY ? 14 - exponent_of(top) : 0;
        // two factors, since 2^eq alone may lie outside the normal range
        const float f0 = power_of_two(eq / 2), f1 = power_of_two(eq - eq / 2);
        c_row = p.scale_log2 / f0 / f1;
        group_sync(g);   // all rows are read
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float f[8];
          chunk(i, f);
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = f16x2_of(f[2 * e] * f0 * f1, f[2 * e + 1] * f0 * f1);
          const int c = place(i);
          *reinterpret_cast<uint4*>(qg + (c >> 2) * BM * kSW + swz64(row, c & 3)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      };
      if (NSRC == 1 && p.a[0])
        fill(std::true_type{});
      else
        fill(std::false_type{});
      fence_proxy_async_smem();
      mbar_arrive(q_ready);
    }
    float m_run = -FLT_MAX, l_run = 0.f;
    for (int j = 0; ok && j < ng; ++j) {
      const int n0 = pos0 + j * BN;
      // waits are made warp-uniform: tcgen05.ld/st below are warp-collective
      if (!__all_sync(0xffffffffu, wait(&step_ready[j % NSR], (uint32_t)(j / NSR) & 1u))) {
        ok = false;
        break;
      }
      // the blocks' factors, before the scores are there: a load between two
      // blocks' stores of P would stop the pipeline of their exponentials
      const float4* rec = sScale + (j % NSR) * NGRP;
      float f[NGRP], lv[NGRP], rv[NGRP];
#pragma unroll
      for (int gr = 0; gr < NGRP; ++gr) {
        const float4 sc = rec[gr];
        f[gr] = fminf(fmaxf(c_row * sc.x, FLT_MIN), FLT_MAX);
        lv[gr] = sc.y;
        rv[gr] = sc.z;
      }
      if (!__all_sync(0xffffffffu, wait(&s_full[g], (uint32_t)j & 1u))) {
        ok = false;
        break;
      }
      tc_fence_after();
      // masking needed: the causal diagonal, the key extent, or (window) the
      // lowest row-window start of the tile (warp-uniform).  It is done where
      // the scores lie, so that the usual tile's registers are not merged with
      // a masked tile's (128 moves a thread).
      if (n0 > full_to || n0 < full_from || idle) {
        // visible keys of this row, as tile columns: lo <= c < hi
        const int hi = idle ? 0 : qpos - n0 + 1;
        const int lo = W > 0 ? max(qpos - n0, -1) - W + 1 : INT_MIN;
#pragma unroll 1
        for (int c = 0; c < BN; c += 32) {
          float x[32];
          tmem_ld32(t_s + c, x);
          tmem_wait_ld();
          uint32_t y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(c + e >= hi || c + e < lo ? -INFINITY : x[e]);
          tmem_st32(t_s + c, y);
        }
        tmem_wait_st();
      }
      float sv[BN];
#pragma unroll
      for (int c = 0; c + 32 <= BN; c += 32) tmem_ld32(t_s + c, sv + c);
      tmem_wait_ld();
      // row max of score + log2 value scale: per block the raw scores' (the
      // factors are positive, so it commutes)
      float mt_row = -INFINITY;
#pragma unroll
      for (int gr = 0; gr < NGRP; ++gr) {
        const float* x = sv + gr * 32;
        float mx[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) mx[r] = fmaxf(x[2 * r], x[2 * r + 1]);
#pragma unroll
        for (int c = 8; c < 32; c += 8)
#pragma unroll
          for (int r = 0; r < 4; ++r) mx[r] = fmax3f(mx[r], x[c + 2 * r], x[c + 2 * r + 1]);
        mt_row = fmaxf(mt_row, fmaf(fmaxf(fmax3f(mx[0], mx[1], mx[2]), mx[3]), f[gr], lv[gr]));
      }
      // Keep a stale max until it is exceeded by more than 2^8: P' stays below
      // 2^15 and O needs no rescaling.
      const float m_new = mt_row > m_run + kSlack ? mt_row : m_run;
      const float alpha = fast_exp2(m_run - m_new);
      const float neg_m = kBias - m_new;
      unsigned long long lsum = 0ull;   // (0, 0)
      // P' over the S tile just read: BN / 2 packed columns, 16 a block
#pragma unroll
      for (int gr = 0; gr < NGRP; ++gr) {
        const float add = lv[gr] + neg_m;
        const unsigned long long f2 = pair_of(f[gr], f[gr]), add2 = pair_of(add, add);
        float pk[16];
        unsigned long long ps[4];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const int cc = gr * 32 + 2 * c;
          // s * f + log2 r - m for two scores with one packed FMA; exp2(-inf) = 0
          float x0, x1;
          unpair(ffma2(pair_of(sv[cc], sv[cc + 1]), f2, add2), x0, x1);
          const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
          const unsigned long long e2 = pair_of(e0, e1);
          ps[c & 3] = c < 4 ? e2 : fadd2(ps[c & 3], e2);
          pk[c] = __uint_as_float(f16x2_of(e0, e1));
        }
        tmem_st16(t_s + gr * 16, pk);
        lsum = ffma2(fadd2(fadd2(ps[0], ps[1]), fadd2(ps[2], ps[3])), pair_of(rv[gr], rv[gr]), lsum);
      }
      if (j > 0 && __any_sync(0xffffffffu, alpha < 1.f)) {
        // O_g holds every PV product up to tile j-1 (s_full of tile j); the
        // next one is issued only after p_full below
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          float ov[16];
          tmem_ld16(t_o + c, ov);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) ov[e] *= alpha;
          tmem_st16(t_o + c, ov);
        }
      }
      float l0, l1;
      unpair(lsum, l0, l1);
      l_run = l_run * alpha + (l0 + l1);
      m_run = m_new;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[g]);
    }
    // the commit after the last PV product is phase ng of s_full[g]
    ok = ok && __all_sync(0xffffffffu, wait(&s_full[g], (uint32_t)ng & 1u) &&
                                           wait(&step_ready[ng % NSR], (uint32_t)(ng / NSR) & 1u));
    if (ok) {
      tc_fence_after();
      // values that are not numbers among the keys that this row sees
      const uint32_t noted = *const_cast<volatile uint32_t*>(&bad[0]);
      bool nan = (noted & 1u) != 0;
      const int q0 = pos_first, lo0 = q0 - W + 1;
      for (int i = 0; i < 8 && (noted & 2u); ++i) {
        uint32_t x = *const_cast<volatile uint32_t*>(&bad[1 + i]);
        while (x) {
          const int pos = q0 + i * 32 + __ffs((int)x) - 1;
          x &= x - 1;
          nan = nan || (pos <= qpos && (W == 0 || pos > qpos - W));
        }
        x = *const_cast<volatile uint32_t*>(&bad[9 + i]);
        while (x) {
          const int pos = lo0 + i * 32 + __ffs((int)x) - 1;
          x &= x - 1;
          nan = nan || (pos <= qpos && pos > qpos - W);
        }
      }
      if (nan) l_run = __uint_as_float(0x7fffffffu);
    }
    const float out_scale = NSRC == 2 ? power_of_two(exponent_of(__uint_as_float(max(w_top[2], w_top[3]))) + 1) : 1.f;
    const float* wb = NSRC == 1 && p.b[0] && p.a[0] ? p.b[0] + (size_t)kh * D : nullptr;
    if (!SPLIT && ok) {
      const float inv = out_scale / l_run;
      __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) +
                            (((size_t)b * H_q + g_head(g)) * p.S + m_row) * D;
#pragma unroll
      for (int c = 0; c < D; c += 16) {
        float ov[16];
        tmem_ld16(t_o + c, ov);
        tmem_wait_ld();
        if (wb) {
#pragma unroll
          for (int e = 0; e < 16; ++e) ov[e] *= wb[c + e];
        }
        uint32_t o8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          __nv_bfloat162 v2 = __floats2bfloat162_rn(ov[2 * e] * inv, ov[2 * e + 1] * inv);
          o8[e] = *reinterpret_cast<uint32_t*>(&v2);
        }
        if (row_valid) {
          uint4* dst = reinterpret_cast<uint4*>(orow + c);
          dst[0] = make_uint4(o8[0], o8[1], o8[2], o8[3]);
          dst[1] = make_uint4(o8[4], o8[5], o8[6], o8[7]);
        }
      }
    }
    if constexpr (SPLIT) {
      // The partials go where Q and the tiles were: O [D][256 rows], the
      // maxima, the sums.  (Both groups' products are done once all are here.)
      constexpr int ROWS = NG * BM;
      static_assert((size_t)(D + 2) * ROWS * 4 <= (size_t)NG * C::Q_BYTES + 2 * NS * C::KV_BYTES, "partials fit");
      float* part = reinterpret_cast<float*>(sQ);
      const int r = g * BM + row;
      if (softmax_and(ok)) {
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          float ov[16];
          tmem_ld16(t_o + c, ov);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) part[(c + e) * ROWS + r] = ov[e];
        }
        part[D * ROWS + r] = m_run;
        part[(D + 1) * ROWS + r] = l_run;
      }
      cluster_sync();
      bool stop = false;   // a CTA of the cluster gave up
      for (int k = 0; k < splits; ++k)
        stop = stop || __float_as_int(ld_cluster(smem_u32(const_cast<int*>(abort_flag)), k)) != 0;
      // this CTA's share of the rows, SP threads a row: the channels of several
      // loads at once, since each is a trip to another SM
      auto join = [&](auto parts) {
        constexpr int SP = decltype(parts)::value, WIDTH = D / SP;
        constexpr int CH = WIDTH % 16 == 0 && SP == 2 ? 16 : WIDTH % 8 == 0 && SP <= 4 ? 8 : WIDTH % 4 == 0 ? 4 : 2;
        static_assert(WIDTH % CH == 0, "whole batches of channels");
        constexpr int SHARE = ROWS / SP;
        const int mine = rank * SHARE + r % SHARE, piece = r / SHARE;
        const int og = mine / BM, orow = g_row0(og) + mine % BM;
        if (orow >= p.S) return;
        const uint32_t at = smem_u32(part) + mine * 4;
        float top = -FLT_MAX, sum = 0.f, w[SP], l[SP];
#pragma unroll
        for (int k = 0; k < SP; ++k) {
          w[k] = ld_cluster(at + D * ROWS * 4, k);
          l[k] = ld_cluster(at + (D + 1) * ROWS * 4, k);
        }
#pragma unroll
        for (int k = 0; k < SP; ++k) top = fmaxf(top, w[k]);
#pragma unroll
        for (int k = 0; k < SP; ++k) {
          w[k] = fast_exp2(w[k] - top);
          sum = fmaf(w[k], l[k], sum);
        }
        const float inv = out_scale / sum;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + (((size_t)b * H_q + g_head(og)) * p.S + orow) * D;
#pragma unroll 1
        for (int d = piece * WIDTH; d < (piece + 1) * WIDTH; d += CH) {
          float x[CH][SP];
#pragma unroll
          for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int k = 0; k < SP; ++k) x[c][k] = ld_cluster(at + (d + c) * ROWS * 4, k);
          uint32_t o[CH / 2];
#pragma unroll
          for (int c = 0; c < CH; c += 2) {
            float y[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < SP; ++k) {
              y[0] = fmaf(w[k], x[c][k], y[0]);
              y[1] = fmaf(w[k], x[c + 1][k], y[1]);
            }
            if (wb) y[0] *= wb[d + c], y[1] *= wb[d + c + 1];
            const __nv_bfloat162 v2 = __floats2bfloat162_rn(y[0] * inv, y[1] * inv);
            o[c / 2] = *reinterpret_cast<const uint32_t*>(&v2);
          }
          if constexpr (CH >= 8) {
#pragma unroll
            for (int c = 0; c < CH / 8; ++c)
              reinterpret_cast<uint4*>(dst + d)[c] = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          } else {
#pragma unroll
            for (int c = 0; c < CH / 2; ++c) reinterpret_cast<uint32_t*>(dst + d)[c] = o[c];
          }
        }
      };
      if (!stop) {
        if (splits == 2) join(std::integral_constant<int, 2>{});
        else if (splits == 4) join(std::integral_constant<int, 4>{});
        else join(std::integral_constant<int, 8>{});
      }
      cluster_sync();
    }
  }

  // (a producer that stopped early has let its copies in flight land)
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // A wait ran out somewhere, so no role may have awaited the last copies
    // and products: each producer lets its copies in flight land (the last NR
    // tiles; an older one was consumed before its slot was refilled) and each
    // issuer lets its own products finish, before the CTA frees tensor memory
    // and exits.
    if ((warp == C::K_PRODUCER_WARP || warp == C::V_PRODUCER_WARP) && lane == 0) {
      const bool is_k = warp == C::K_PRODUCER_WARP;
      const int issued = sm_issued[is_k ? 0 : 1];
      for (int j = max(0, issued - NR); j < issued; ++j)
        (void)mbar_wait_bounded(&(is_k ? rk_full : rv_full)[j % NR], (uint32_t)(j / NR) & 1u, kDrainLimitNs);
    }
    if (warp >= C::MMA_WARP && warp < C::MMA_WARP + NG && lane == 0) {
      (void)mbar_wait_bounded(&q_raw[warp - C::MMA_WARP], 0, kDrainLimitNs);
      mma_commit(&mma_drain[warp - C::MMA_WARP]);
      (void)mbar_wait_bounded(&mma_drain[warp - C::MMA_WARP], 0, kDrainLimitNs);
    }
    tc_fence_before();
    __syncthreads();
  }
  if (warp == C::MMA_WARP) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int NSRC>
cudaError_t launch(const PrefillArgs& a, cudaStream_t stream) {
  using C = Cfg<D, NSRC>;
  Params p;
  for (int i = 0; i < 2; ++i) {
    p.k[i] = static_cast<const uint8_t*>(a.k[i]);
    p.v[i] = static_cast<const uint8_t*>(a.v[i]);
    p.ks[i] = a.k_scale[i];
    p.vs[i] = a.v_scale[i];
    p.a[i] = a.a[i];
    p.b[i] = a.b[i];
  }
  p.q = a.q;
  p.out = a.out;
  p.status = a.status;
  p.wait_limit = a.wait_limit;
  p.H_kv = a.kv_heads;
  p.G = a.group;
  p.S = a.S;
  p.q_start = a.q_start;
  p.S_kv = a.q_start + a.S;
  p.window = a.window;
  p.rows = a.plane_rows;
  p.ring = a.ring;
  p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  // one CTA per (unit, 128 query rows of two heads, or 256 of one)
  const bool two_heads = a.group % 2 == 0;
  const int rows_per_cta = two_heads ? BM : NG * BM;
  const long long units = (long long)a.batch * a.kv_heads * (two_heads ? a.group / 2 : a.group);
  const long long tiles = ((long long)a.S + rows_per_cta - 1) / rows_per_cta;
  if (tiles > 65535 || units * tiles > INT_MAX / 8) return cudaErrorNotSupported;
  // Few CTAs with many key tiles each: clusters that share them, of as many
  // CTAs as still find an SM each, with two tiles a CTA at least (a join costs
  // about a tile).  8 units of 16 rows behind 16368 keys (D = 96): 232 us with
  // one CTA a unit, 42 with 8.
  long long keys = p.S_kv;
  if (a.window > 0 && (long long)a.window + rows_per_cta < keys) keys = (long long)a.window + rows_per_cta;
  const long long key_tiles = (keys + C::BN - 1) / C::BN;
  p.splits = 1;
  while (p.splits < 8 && units * tiles * p.splits * 2 <= a.num_sms && key_tiles >= 4 * p.splits) p.splits *= 2;
  auto kern = p.splits > 1 ? prefill_q8_kernel<D, NSRC, true> : prefill_q8_kernel<D, NSRC, false>;
  // The register split inside the kernel must fit the launch allocation, or
  // the softmax warpgroups' increase would never be granted: refused then.
  static KernelReady ready[2];
  const cudaError_t e = ready[p.splits > 1].check(kern, a.device, (int)C::SMEM, C::THREADS, (int)C::REGS_SPLIT);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * p.splits), (unsigned)tiles);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.splits;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace q8p
}  // namespace fkv
