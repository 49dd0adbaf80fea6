// fkv_tree_attn over fp32 caches, on the CUDA cores: fp32 products keep the
// accuracy that an fp32 context is chosen for (the tensor cores would round
// operands to 11 bits).  Bound by fp32 FMAs from about 16 query rows on, by
// latency below.
//
// A CTA of 16 x 16 threads takes one range of key tiles (tree_common.cuh) and
// RT = 16 or 64 query rows (row r of a unit is query head r / T of the group,
// node r % T).  Keys and values of a tile of 64 are rebuilt in shared memory
// (the fused sum of two sources, or the scaled one).  Thread (ty, tx) owns
// rows ty * RT / 16 .. and, in turn, keys tx, tx + 16, tx + 32, tx + 48 of the
// score tile and channels 4 tx .. 4 tx + 3 (+ 64) of the value product, so a
// row's maximum and sum are shuffles over 16 lanes and stay in registers.
// Packed FMAs (two channels an instruction) in both products.  A call of one
// sequence over 256 rows (4 query heads, 7 nodes, fused) takes 12.5 us on the
// device: eight CTAs of one tile each, a chain of dependent reads (lengths,
// queries and masks, keys and values), then a merge of four partials through L2.
// 2 x 4 KV heads of 8192 rows, 4 query heads each: 16 nodes of 64 channels 68 us,
// 40 nodes 119 us, 40 nodes of 128 channels 272 us (16, 23 and 20 TFLOP/s of the
// products asked for, of 78 that the CUDA cores have).
#include <type_traits>

#include "decode_impl.cuh"   // fma2
#include "tree_common.cuh"

namespace fkv {
namespace {

constexpr int KT = 64;        // keys per tile
constexpr int NT = 256;       // threads

template <int D, int NSRC, bool WGT, int RT>
__global__ void __launch_bounds__(NT) tree_f32_kernel(const TreeParams p) {
  constexpr int LD = D + 4;          // padded rows: conflict-free column reads
  constexpr int C4 = D / 4;
  constexpr int RPT = RT / 16;       // rows a thread
  constexpr int KPT = KT / 16;       // keys a thread
  constexpr int NCG = (C4 + 15) / 16;   // groups of four channels a thread
  extern __shared__ __align__(16) uint8_t smem[];
  float* sQ = reinterpret_cast<float*>(smem);   // [RT][LD], times scale * log2(e)
  float* sK = sQ + RT * LD;                     // [KT][LD]
  float* sV = sK + KT * LD;                     // [KT][LD]
  float* sP = sV + KT * LD;                     // [KT][RT]
  float* sScratch = sP + KT * RT;               // [2 RT] merge
  unsigned long long* sMask = reinterpret_cast<unsigned long long*>(sScratch + 2 * RT);   // [RT][2]
  int* sDepth = reinterpret_cast<int*>(sMask + RT * 2);                                    // [nodes]
  int* sBad = sDepth + kTreeMaxNodes;                                                      // [KT]
  int* flag = sBad + KT;
  const TreeSeqs sq = tree_seqs(flag + 1, p.B);

  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  grid_dep_trigger();
  grid_dep_wait();
  const TreeCut cut = tree_cut<float, D>(p, sq, KT, gridDim.x, 0);
  if ((int)blockIdx.x >= cut.ranges) return;
  const int rt = blockIdx.y;
  const size_t plane = p.ring > 0 ? p.ring : p.S_max;
  TreeWalk walk;
  walk.begin(cut, sq.pre, p.B, p.H, blockIdx.x);
  TreePiece pc;
  while (walk.next(sq.pre, p.B, p.H, pc)) {
    const TreeSeq s = tree_seq(p, sq.P[pc.b], sq.N[pc.b]);
    const size_t unit = (size_t)pc.b * p.H + pc.h;
    const int rows = min(RT, p.G * p.T - rt * RT);
    __syncthreads();
    for (int it = tid; it < RT * C4; it += NT) {
      const int r = it / C4, d = (it - r * C4) * 4;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (r < rows) {
        const float4 q = *reinterpret_cast<const float4*>(
            static_cast<const float*>(p.q) + (unit * p.G * p.T + rt * RT + r) * D + d);
        x[0] = q.x * p.scale_log2;
        x[1] = q.y * p.scale_log2;
        x[2] = q.z * p.scale_log2;
        x[3] = q.w * p.scale_log2;
      }
      tree_store4(sQ + r * LD + d, x);
    }
    for (int i = tid; i < s.N; i += NT) sDepth[i] = tree_depth(p, pc.b, i, s.N);
    if (tid < RT) {
      const int i = (rt * RT + tid) % p.T;
      for (int w = 0; w < 2; ++w)
        sMask[tid * 2 + w] = tid < rows && i < s.N && w < p.words ? tree_mask_word(p, pc.b, i, w, s.N) : 0ull;
    }
    float m[RPT], l[RPT], acc[RPT][NCG][4];
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      m[r] = -FLT_MAX;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < NCG; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][c][e] = 0.f;
    }

    for (int kt = pc.k0; kt < pc.k1; ++kt) {
      const TreeTile t = tree_tile(p, s, kt, KT);
      const bool masked = t.cnt < KT || t.pos + t.cnt > s.P || p.window > 0;
      __syncthreads();   // the tile before is read
      if (masked && tid < KT) sBad[tid] = 0;
      if (masked) __syncthreads();
#pragma unroll 2
      for (int it = tid; it < KT * C4; it += NT) {
        const int r = it / C4, d = (it - r * C4) * 4;
        float4 k0 = make_float4(0.f, 0.f, 0.f, 0.f), v0 = k0;
        if (r < t.cnt) {
          const size_t at = (unit * plane + t.row + r) * D + d;
          k0 = *reinterpret_cast<const float4*>(static_cast<const float*>(p.k[0]) + at);
          v0 = *reinterpret_cast<const float4*>(static_cast<const float*>(p.v[0]) + at);
          if constexpr (WGT) {
            const size_t w = (size_t)pc.h * D + d;
            const float4 a0 = *reinterpret_cast<const float4*>(p.a[0] + w);
            const float4 b0 = *reinterpret_cast<const float4*>(p.b[0] + w);
            k0 = make_float4(k0.x * a0.x, k0.y * a0.y, k0.z * a0.z, k0.w * a0.w);
            v0 = make_float4(v0.x * b0.x, v0.y * b0.y, v0.z * b0.z, v0.w * b0.w);
            if constexpr (NSRC == 2) {
              const float4 k1 = *reinterpret_cast<const float4*>(static_cast<const float*>(p.k[1]) + at);
              const float4 v1 = *reinterpret_cast<const float4*>(static_cast<const float*>(p.v[1]) + at);
              const float4 a1 = *reinterpret_cast<const float4*>(p.a[1] + w);
              const float4 b1 = *reinterpret_cast<const float4*>(p.b[1] + w);
              k0 = make_float4(fmaf(a1.x, k1.x, k0.x), fmaf(a1.y, k1.y, k0.y), fmaf(a1.z, k1.z, k0.z),
                               fmaf(a1.w, k1.w, k0.w));
              v0 = make_float4(fmaf(b1.x, v1.x, v0.x), fmaf(b1.y, v1.y, v0.y), fmaf(b1.z, v1.z, v0.z),
                               fmaf(b1.w, v1.w, v0.w));
            }
          }
          if (masked) {
            // 0 * NaN is no 0: a value that is not finite becomes 0 here, and
            // the probabilities of the rows that see its key NaN
            const bool f0 = isfinite(v0.x), f1 = isfinite(v0.y), f2 = isfinite(v0.z), f3 = isfinite(v0.w);
            if (!(f0 && f1 && f2 && f3)) {
              sBad[r] = 1;
              v0 = make_float4(f0 ? v0.x : 0.f, f1 ? v0.y : 0.f, f2 ? v0.z : 0.f, f3 ? v0.w : 0.f);
            }
          }
        }
        *reinterpret_cast<float4*>(sK + r * LD + d) = k0;
        *reinterpret_cast<float4*>(sV + r * LD + d) = v0;
      }
      __syncthreads();

      float sc[RPT][KPT];
      {
        float s0[RPT][KPT], s1[RPT][KPT];   // even and odd channels
#pragma unroll
        for (int r = 0; r < RPT; ++r)
#pragma unroll
          for (int k = 0; k < KPT; ++k) s0[r][k] = s1[r][k] = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
          float4 q[RPT], k[KPT];
#pragma unroll
          for (int r = 0; r < RPT; ++r) q[r] = *reinterpret_cast<const float4*>(sQ + (ty * RPT + r) * LD + d);
#pragma unroll
          for (int j = 0; j < KPT; ++j) k[j] = *reinterpret_cast<const float4*>(sK + (tx + 16 * j) * LD + d);
#pragma unroll
          for (int r = 0; r < RPT; ++r)
#pragma unroll
            for (int j = 0; j < KPT; ++j) {
              fma2(s0[r][j], s1[r][j], q[r].x, q[r].y, k[j].x, k[j].y);
              fma2(s0[r][j], s1[r][j], q[r].z, q[r].w, k[j].z, k[j].w);
            }
        }
#pragma unroll
        for (int r = 0; r < RPT; ++r)
#pragma unroll
          for (int j = 0; j < KPT; ++j) sc[r][j] = s0[r][j] + s1[r][j];
      }
      if (masked) {
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
          const int row = ty * RPT + r, i = (rt * RT + row) % p.T;
          const bool live = row < rows && i < s.N;
          const int floor = live && p.window > 0 ? sDepth[i] - p.window : -kTreeMaxNodes - p.S_max;
#pragma unroll
          for (int j = 0; j < KPT; ++j) {
            const int key = tx + 16 * j, q = t.pos + key - s.P;   // >= 0: drafted node q
            bool see = live && key < t.cnt;
            if (see) see = q < 0 ? q > floor
                                 : (sMask[row * 2 + (q >> 6)] >> (q & 63) & 1) && sDepth[q] > floor;
            sc[r][j] = !see ? -INFINITY : sBad[key] ? NAN : sc[r][j];
          }
        }
      }
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        float top = m[r];
#pragma unroll
        for (int j = 0; j < KPT; ++j) top = fmaxf(top, sc[r][j]);
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float f = exp2f(m[r] - top);
        m[r] = top;
        l[r] *= f;
#pragma unroll
        for (int c = 0; c < NCG; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[r][c][e] *= f;
#pragma unroll
        for (int j = 0; j < KPT; ++j) {
          const float e = exp2f(sc[r][j] - top);
          l[r] += e;
          sP[(tx + 16 * j) * RT + ty * RPT + r] = e;
        }
      }
      __syncwarp();   // a row's probabilities are written and read by one warp
#pragma unroll 4
      for (int key = 0; key < KT; ++key) {
        float pr[RPT];
        if constexpr (RPT == 4) {
          const float4 w = *reinterpret_cast<const float4*>(sP + key * RT + ty * 4);
          pr[0] = w.x; pr[1] = w.y; pr[2] = w.z; pr[3] = w.w;
        } else {
          pr[0] = sP[key * RT + ty];
        }
#pragma unroll
        for (int c = 0; c < NCG; ++c) {
          if (C4 % 16 != 0 && tx + 16 * c >= C4) break;
          const float4 v = *reinterpret_cast<const float4*>(sV + key * LD + (tx + 16 * c) * 4);
#pragma unroll
          for (int r = 0; r < RPT; ++r) {
            fma2(acc[r][c][0], acc[r][c][1], pr[r], pr[r], v.x, v.y);
            fma2(acc[r][c][2], acc[r][c][3], pr[r], pr[r], v.z, v.w);
          }
        }
      }
    }
    const bool whole = pc.k1 - pc.k0 == pc.tiles;
    float* rec = p.ws + ((size_t)(2 * blockIdx.x + (pc.first ? 0 : 1)) * p.row_tiles + rt) *
                            tree_record_floats(RT, D);
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
      const int row = ty * RPT + r, out = rt * RT + row;
      const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
#pragma unroll
      for (int c = 0; c < NCG; ++c) {
        if (C4 % 16 != 0 && tx + 16 * c >= C4) break;
        const int d = (tx + 16 * c) * 4;
        if (whole) {
          if (row < rows && out % p.T < s.N) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[r][c][e] *= inv;
            tree_store4(static_cast<float*>(p.out) + (unit * p.G * p.T + out) * D + d, acc[r][c]);
          }
        } else {
          tree_store4(rec + row * D + d, acc[r][c]);
        }
      }
      if (!whole && tx == 0) {
        rec[RT * D + row] = m[r];
        rec[RT * D + RT + row] = l[r];
      }
    }
    if (!whole)
      tree_publish<float, D, RT, NT>(p, cut, sq.pre, pc.b, pc.h, s.N, tid, flag, sScratch, [] { __syncthreads(); });
  }
}

template <int D, int NSRC, bool WGT, int RT>
cudaError_t launch_f32(const TreeParams& p, const TreeArgs& a, const TreePlan& plan, cudaStream_t stream) {
  auto kern = tree_f32_kernel<D, NSRC, WGT, RT>;
  static KernelReady ready;
  const cudaError_t e = ready.check(kern, a.device, 232448, NT, 0);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(plan.ranges, plan.row_tiles), dim3(NT), plan.smem_bytes, stream, p);
}

// Registers a thread of an instance, asked for once; 255 where that fails.
template <int D, int NSRC, bool WGT, int RT>
int f32_registers() {
  static const int regs = [] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, tree_f32_kernel<D, NSRC, WGT, RT>) == cudaSuccess ? fa.numRegs : 255;
  }();
  return regs;
}

// Call f with the call's head dimension, sources, weights and rows a CTA as
// integral constants.
template <typename F>
auto dispatch_f32(const TreeArgs& a, int rows, F f) {
  auto src = [&](auto d, auto rt) {
    if (a.k[1]) return f(d, std::integral_constant<int, 2>(), std::true_type(), rt);
    if (a.a[0]) return f(d, std::integral_constant<int, 1>(), std::true_type(), rt);
    return f(d, std::integral_constant<int, 1>(), std::false_type(), rt);
  };
  auto row = [&](auto d) {
    return rows == 64 ? src(d, std::integral_constant<int, 64>()) : src(d, std::integral_constant<int, 16>());
  };
  switch (a.head_dim) {
    case 64: return row(std::integral_constant<int, 64>());
    case 80: return row(std::integral_constant<int, 80>());
    case 96: return row(std::integral_constant<int, 96>());
    default: return row(std::integral_constant<int, 128>());
  }
}

// What an SM holds: registers, and shared memory with 1 KB of it taken by each
// CTA beside its own.
constexpr int SM_REGS = 65536;
constexpr size_t SM_SMEM = 233472, CTA_SMEM = 1024;

}  // namespace

void tree_f32_plan(const TreeArgs& a, int num_sms, TreePlan* plan) {
  const int rows = a.group * a.T;
  plan->tensor = false;
  plan->rows = rows <= 16 ? 16 : 64;
  plan->row_tiles = (rows + plan->rows - 1) / plan->rows;
  const int RT = plan->rows, LD = a.head_dim + 4;
  plan->smem_bytes = (size_t)(RT * LD + 2 * KT * LD + KT * RT + 2 * RT) * 4 + RT * 16 +
                     (kTreeMaxNodes + KT + 1) * 4 + tree_seqs_bytes(a.batch);
  // One wave: ranges times row tiles are at most the CTAs that the device holds
  // at once, two an SM or one (64 rows of 80 or 96 channels take too many
  // registers for two, of 128 too much shared memory).  The device takes fewer
  // ranges where there are fewer key tiles.
  const int regs = dispatch_f32(a, plan->rows, [](auto d, auto ns, auto wt, auto rt) {
    return f32_registers<decltype(d)::value, decltype(ns)::value, decltype(wt)::value, decltype(rt)::value>();
  });
  const bool two = 2 * NT * ((regs + 7) / 8 * 8) <= SM_REGS && 2 * (plan->smem_bytes + CTA_SMEM) <= SM_SMEM;
  const int ranges = (two ? 2 : 1) * num_sms / plan->row_tiles;
  plan->ranges = a.num_ctas > 0 ? a.num_ctas : ranges > 0 ? ranges : 1;
}

cudaError_t tree_f32_launch(const TreeParams& p, const TreeArgs& a, const TreePlan& plan, cudaStream_t stream) {
  return dispatch_f32(a, plan.rows, [&](auto d, auto ns, auto wt, auto rt) {
    return launch_f32<decltype(d)::value, decltype(ns)::value, decltype(wt)::value, decltype(rt)::value>(p, a, plan,
                                                                                                        stream);
  });
}

}  // namespace fkv
