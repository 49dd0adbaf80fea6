// Decode attention over 8-bit caches (e4m3 codes, one scale per 32 rows of a
// KV head; q8_device.cuh): dequantised, fused and reduced in registers.
//
// The structure is decode_split_kernel's (per-warp cp.async.bulk rings,
// stream-K row partition, merge by the last warp of a unit).  A lane owns E
// channels of a row, one or half a 16-byte chunk of codes.  The scales stay
// outside the products,
//     q . (s c) = s (q . c),      sum_t p_t (s_t c_t) = sum_t (p_t s_t) c_t,
// so an element costs half a conversion e4m3 -> fp16 (two at a time, exact),
// one fp16 -> fp32 and half a packed FMA per query head of the group.  A
// tile's scales come with its codes, in 16-byte pieces of the unit's scales
// that cover the tile's rows, under the same barrier.
//
// Bound: HBM, nsrc * 2 * (D + 1/8) bytes a row; the conversions and FMAs take
// about half the issue slots at that rate.
#pragma once

#include "decode_impl.cuh"
#include "q8_device.cuh"

namespace fkv {

// Warps per CTA, ring stages per warp and bytes per stage.  Two sources, and
// four heads a group, need more registers than the 168 that 12 warps leave.
template <int NSRC, int G, bool F32>
struct Q8Shape {
  static constexpr int W = NSRC == 1 && G <= 2 && !F32 ? 12 : 8;
  static constexpr int NS = 2;
  static constexpr int SB = W == 12 ? 8832 : 12288;
  // channels a lane: four heads and two sources at 16 would need 256 registers for q and o
  static constexpr int E = NSRC == 2 && G == 4 ? 8 : 16;
};

template <int D, int NSRC, int G, bool F32>
struct Q8Cfg {
  using S = Q8Shape<NSRC, G, F32>;
  static constexpr int E = S::E;
  static constexpr int C = D / E;                     // lanes per row
  static constexpr int R = 32 / C;                    // rows per warp step
  static constexpr int STEPS_RAW = S::SB / (2 * NSRC * R * D);
  static constexpr int STEPS = STEPS_RAW < 1 ? 1 : STEPS_RAW;
  static constexpr int TR = R * STEPS;
  static constexpr int TILE_BYTES = TR * D;           // codes of one plane's tile
  // scales of one plane's tile: TR rows reach TR / 32 + 2 blocks at most, in
  // whole 16-byte pieces; a tile that wraps in a ring has two such runs
  static constexpr int SCW = (TR / kQ8Block + 2 + 6) / 4 * 4;
  static constexpr int CODE_BYTES = 2 * NSRC * TILE_BYTES;
  static constexpr int STAGE_BYTES = CODE_BYTES + 2 * NSRC * 2 * SCW * 4;
  static_assert(TILE_BYTES % 16 == 0 && STAGE_BYTES % 16 == 0, "stages are read in 16-byte pieces");
};

struct Q8Params {
  SplitParams p;
  const float* ks[2];
  const float* vs[2];
};

// E codes of shared memory -> fp32.
template <int E>
__device__ __forceinline__ void load_codes(const uint8_t* src, float* f) {
  if constexpr (E == 16) {
    const uint4 q = *reinterpret_cast<const uint4*>(src);
    e4m3x4_to_f32(q.x, f);
    e4m3x4_to_f32(q.y, f + 4);
    e4m3x4_to_f32(q.z, f + 8);
    e4m3x4_to_f32(q.w, f + 12);
  } else {
    const uint2 q = *reinterpret_cast<const uint2*>(src);
    e4m3x4_to_f32(q.x, f);
    e4m3x4_to_f32(q.y, f + 4);
  }
}

template <typename T, int D, int NSRC, bool WGT, int G>
__global__ void __launch_bounds__(Q8Shape<NSRC, G, sizeof(T) == 4>::W * 32, 1)
    decode_q8_kernel(const Q8Params prm) {
  const SplitParams& p = prm.p;
  using Cfg = Q8Cfg<D, NSRC, G, sizeof(T) == 4>;
  using S = typename Cfg::S;
  constexpr int C = Cfg::C, R = Cfg::R, E = Cfg::E, TR = Cfg::TR, STEPS = Cfg::STEPS, SCW = Cfg::SCW;
  constexpr int TILE = Cfg::TILE_BYTES, STAGE = Cfg::STAGE_BYTES;
  constexpr int NS = S::NS, W = S::W;
  constexpr int PS = partial_stride(D);

  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (size_t)W * NS * STAGE);
  int* lens = reinterpret_cast<int*>(bars + W * NS);
  int* pre = lens + p.B;
  int* first = pre + p.B + 1;

  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < NS; ++s) mbar_init(&bars[warp * NS + s], 1);
    fence_mbar_init();
  }
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
    lens[i] = Le;
    // cache row of the first attended position (in a ring: its row)
    first[i] = p.ring > 0 ? (L - Le) % p.ring : L - Le;
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
  const long long total = (long long)H * pre[p.B];
  const long long N = (long long)gridDim.x * W;
  const long long w = (long long)blockIdx.x * W + warp;
  const long long r0 = w * total / N, r1 = (w + 1) * total / N;
  if (r0 >= r1) return;

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

  // Row of the tile's row 0, and how many of its n rows come before a ring's
  // end (the others follow from the ring's start).
  auto tile_rows = [&](int b, int t, int n, int& row0, int& n1) {
    row0 = first[b] + t;
    if (p.ring > 0 && row0 >= p.ring) row0 -= p.ring;
    n1 = p.ring > 0 && row0 + n > p.ring ? p.ring - row0 : n;
  };

  auto issue = [&](int stage, int b, int h, int t, int n) {
    if (lane == 0) {
      uint8_t* dst = wring + (size_t)stage * STAGE;
      float* dsc = reinterpret_cast<float*>(dst + Cfg::CODE_BYTES);
      uint64_t* bar = &wbars[stage];
      const size_t u = (size_t)b * H + h;
      int row0, n1;
      tile_rows(b, t, n, row0, n1);
      const int n2 = n - n1;
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
    if (!prod.next(lens, H, p.B, TR, tb, th, tt, tn, tl)) break;
    issue(s, tb, th, tt, tn);
    ++issued;
  }

  const int g = lane / C, c = lane % C;   // row in step, channel run
  const bool active = g < R;

  float qa[NSRC][G][E];    // q (.) a_src * scale * log2 e, per source
  float oc[NSRC][G][E];    // sum_t (p_t s_t) c_t per source
  float m[G], l[G];
  bool fresh = true;
  int consumed = 0;

#pragma unroll 1
  for (;;) {
    int b, h, t0, n;
    bool last;
    if (!walk.next(lens, H, p.B, TR, b, h, t0, n, last)) break;
    const int stage = consumed % NS;
    const uint32_t parity = (uint32_t)(consumed / NS) & 1u;

    if (fresh) {
      const T* qp = static_cast<const T*>(p.q) + ((size_t)b * H * G + (size_t)h * G) * D + c * E;
      constexpr int EC = 16 / (int)sizeof(T);
#pragma unroll
      for (int sidx = 0; sidx < NSRC; ++sidx) {
        float wa[E];
#pragma unroll
        for (int e = 0; e < E; ++e) wa[e] = 1.f;
        if (NSRC == 2 || WGT) {
          const float* ap = (sidx == 0 ? p.a0 : p.a1) + (size_t)h * D + c * E;
#pragma unroll
          for (int e = 0; e < E; ++e) wa[e] = ap[e];
        }
#pragma unroll
        for (int hq = 0; hq < G; ++hq) {
          float qf[E];
#pragma unroll
          for (int v = 0; v < E / EC; ++v)
            unpack16<T>(*reinterpret_cast<const uint4*>(qp + (size_t)hq * D + v * EC), qf + v * EC);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            qa[sidx][hq][e] = qf[e] * p.qscale * wa[e];
            oc[sidx][hq][e] = 0.f;
          }
        }
      }
#pragma unroll
      for (int hq = 0; hq < G; ++hq) {
        m[hq] = -FLT_MAX;
        l[hq] = 0.f;
      }
      fresh = false;
    }

    // warp-uniform: every lane leaves, or none does (shuffles follow)
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&wbars[stage], parity, wlim))) {
      flag_status(p.status, kDevTimeout);
      // let every stage issued and not yet consumed land, this one included
      for (int k = consumed; k < issued; ++k)
        (void)mbar_wait_bounded(&wbars[k % NS], (uint32_t)(k / NS) & 1u, kDrainLimitNs);
      return;
    }

    const uint8_t* st = wring + (size_t)stage * STAGE;
    const float* scales = reinterpret_cast<const float*>(st + Cfg::CODE_BYTES);
    int row0, n1;
    tile_rows(b, t0, n, row0, n1);
    const int sc0 = row0 / (4 * kQ8Block) * 4;
    // where the scale of the tile's row `row` lies in a plane's run of scales
    // (a row behind the tile's last reads some scale of the run, and is not used)
    auto scale_at = [&](int row) {
      return row < n1 || row >= n ? min((row0 + row) / kQ8Block - sc0, SCW - 1)
                                  : SCW + (row - n1) / kQ8Block;
    };

    // scores
    float s[STEPS][G];
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      const int row = j * R + g;
      float acc[G];
#pragma unroll
      for (int hq = 0; hq < G; ++hq) acc[hq] = 0.f;
      if (active) {
        const int at = scale_at(row);
#pragma unroll
        for (int sidx = 0; sidx < NSRC; ++sidx) {
          float cf[E];
          load_codes<E>(st + sidx * TILE + row * D + c * E, cf);
          const float sc = scales[sidx * 2 * SCW + at];
#pragma unroll
          for (int hq = 0; hq < G; ++hq) {
            float d0 = 0.f, d1 = 0.f;
#pragma unroll
            for (int e = 0; e < E; e += 2)
              fma2(d0, d1, qa[sidx][hq][e], qa[sidx][hq][e + 1], cf[e], cf[e + 1]);
            acc[hq] = fmaf(sc, d0 + d1, acc[hq]);
          }
        }
      }
#pragma unroll
      for (int hq = 0; hq < G; ++hq) s[j][hq] = acc[hq];
    }
    // the rows' sums, all steps at once: independent shuffle chains overlap
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      const bool ok = active && j * R + g < n;
#pragma unroll
      for (int hq = 0; hq < G; ++hq) {
        const float v = group_sum<C>(s[j][hq], lane);
        s[j][hq] = ok ? v : -FLT_MAX;
      }
    }

#pragma unroll
    for (int hq = 0; hq < G; ++hq) {
      float mt = s[0][hq];
#pragma unroll
      for (int j = 1; j < STEPS; ++j) mt = fmaxf(mt, s[j][hq]);
      mt = warp_max(mt);
      if (mt > m[hq]) {
        const float alpha = fast_exp2(m[hq] - mt);
        l[hq] *= alpha;
#pragma unroll
        for (int sidx = 0; sidx < NSRC; ++sidx)
#pragma unroll
          for (int e = 0; e < E; ++e) oc[sidx][hq][e] *= alpha;
        m[hq] = mt;
      }
    }

    // values
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      const int row = j * R + g;
      if (active && row < n) {
        const int at = scale_at(row);
        float pj[G];
#pragma unroll
        for (int hq = 0; hq < G; ++hq) {
          pj[hq] = fast_exp2(s[j][hq] - m[hq]);
          l[hq] += pj[hq];
        }
#pragma unroll
        for (int sidx = 0; sidx < NSRC; ++sidx) {
          float cf[E];
          load_codes<E>(st + (NSRC + sidx) * TILE + row * D + c * E, cf);
          const float sc = scales[(NSRC + sidx) * 2 * SCW + at];
#pragma unroll
          for (int hq = 0; hq < G; ++hq) {
            const float ps = pj[hq] * sc;
#pragma unroll
            for (int e = 0; e < E; e += 2)
              fma2(oc[sidx][hq][e], oc[sidx][hq][e + 1], ps, ps, cf[e], cf[e + 1]);
          }
        }
      }
    }

    ++consumed;
    __syncwarp();
    // refill the stage just read with the warp's next tile
    {
      int tb, th, tt, tn;
      bool tl;
      if (prod.next(lens, H, p.B, TR, tb, th, tt, tn, tl)) {
        issue(stage, tb, th, tt, tn);
        ++issued;
      }
    }

    if (last) {
      // combine the R row groups, apply the value weights, write the partial
      const long long u = (long long)b * H + h;
      float* rec = p.ws + ((size_t)(w + u) * G) * PS;
      float wb[NSRC][E];
#pragma unroll
      for (int sidx = 0; sidx < NSRC; ++sidx) {
#pragma unroll
        for (int e = 0; e < E; ++e) wb[sidx][e] = 1.f;
        if (NSRC == 2 || WGT) {
          const float* bp = (sidx == 0 ? p.b0 : p.b1) + (size_t)h * D + c * E;
#pragma unroll
          for (int e = 0; e < E; ++e) wb[sidx][e] = bp[e];
        }
      }
#pragma unroll
      for (int hq = 0; hq < G; ++hq) {
        float lt = 0.f;
#pragma unroll
        for (int k = 0; k < R; ++k) lt += __shfl_sync(0xffffffffu, l[hq], k * C);
        float ov[E];
#pragma unroll
        for (int e = 0; e < E; ++e) ov[e] = 0.f;
#pragma unroll
        for (int sidx = 0; sidx < NSRC; ++sidx) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            float x = 0.f;
#pragma unroll
            for (int k = 0; k < R; ++k) x += __shfl_sync(0xffffffffu, oc[sidx][hq][e], k * C + c);
            ov[e] += wb[sidx][e] * x;
          }
        }
        if (g == 0) {
          float4* dst = reinterpret_cast<float4*>(rec + (size_t)hq * PS + c * E);
#pragma unroll
          for (int e = 0; e < E; e += 4) dst[e / 4] = make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
        }
        if (lane == 0) {
          rec[(size_t)hq * PS + D] = m[hq];
          rec[(size_t)hq * PS + D + 1] = lt;
        }
      }
      fresh = true;

      const long long su = (long long)H * pre[b] + (long long)h * lens[b];
      const long long eu = su + lens[b];
      const long long wf = ((su + 1) * N - 1) / total, wl = (eu * N - 1) / total;
      int need = 0;
      for (long long w0 = wf; w0 <= wl; w0 += 32) {
        const long long ww = w0 + lane;
        need += __popc(__ballot_sync(0xffffffffu,
                                     ww <= wl && ww * total / N < (ww + 1) * total / N));
      }
      __threadfence();
      __syncwarp();
      unsigned arrived = 0;
      if (lane == 0) arrived = unit_arrive(p.counters + u, p.epoch);
      arrived = __shfl_sync(0xffffffffu, arrived, 0);
      if (arrived == 0) flag_status(p.status, lane == 0 ? kDevTimeout : 0);
      if (arrived == (unsigned)need) {
        // No arrival of this call can follow: clear the word, so that a call
        // with the same epoch (a CUDA graph replaying this launch) starts at 1.
        if (lane == 0) p.counters[u] = 0ull;
        __threadfence();
        merge_unit<T, D, G>(p.ws, static_cast<T*>(p.out), u, wf, wl, N, total, b, h, H, lane);
      }
    }
  }
}

template <int D, int NSRC, int G, bool F32>
size_t q8_smem_bytes(int B) {
  using S = Q8Shape<NSRC, G, F32>;
  return (size_t)S::W * S::NS * Q8Cfg<D, NSRC, G, F32>::STAGE_BYTES + decode_aux_bytes(S::W, S::NS, B);
}

template <typename T, int D, int NSRC, bool WGT, int G>
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
  auto kern = decode_q8_kernel<T, D, NSRC, WGT || NSRC == 2, G>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan.smem_bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(plan.ctas), dim3(plan.warps_per_cta * 32), plan.smem_bytes, stream, prm);
}

template <typename T, int D, int NSRC, bool WGT>
cudaError_t q8_by_group(const DecodeArgs& a, const DecodePlan& pl, cudaStream_t s) {
  switch (a.group) {
    case 1: return launch_q8<T, D, NSRC, WGT, 1>(a, pl, s);
    case 2: return launch_q8<T, D, NSRC, WGT, 2>(a, pl, s);
    case 4: return launch_q8<T, D, NSRC, WGT, 4>(a, pl, s);
    default: return cudaErrorNotSupported;
  }
}

template <typename T, int D>
cudaError_t q8_by_src(const DecodeArgs& a, const DecodePlan& pl, cudaStream_t s) {
  if (a.nsrc == 2) return q8_by_group<T, D, 2, true>(a, pl, s);
  return a.a[0] ? q8_by_group<T, D, 1, true>(a, pl, s) : q8_by_group<T, D, 1, false>(a, pl, s);
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
