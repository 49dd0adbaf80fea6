// fkv_tree_attn on the CUDA cores: every cache format (fp32, bf16, 4-bit
// records), every mode, head_dim and group size.
//
// A CTA takes one range of key tiles (tree_common.cuh) and one tile of 16
// query rows (row r of a unit is query head r / T of the group, node r % T).
// The tile's keys and values are rebuilt in fp32 in shared memory (the fused
// sum of two sources, the scaled or dequantised one), so one code path serves
// every mode; scores, probabilities and sums are fp32.
#include <type_traits>

#include "tree_common.cuh"

namespace fkv {
namespace {

constexpr int KT = 64;        // keys per tile
constexpr int RT = 16;        // query rows per CTA
constexpr int NT = 256;       // threads

enum TreeFormat { kTreeBf16, kTreeF32, kTreeQ4 };

// Four consecutive channels of a cache row -> fp32.
template <int FMT, int D>
__device__ __forceinline__ void load4(const void* base, size_t row, int d, float* x) {
  if constexpr (FMT == kTreeF32) {
    const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + row * D + d);
    x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
  } else if constexpr (FMT == kTreeBf16) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(base) + row * D + d);
    x[0] = bf16lo(w.x); x[1] = bf16hi(w.x); x[2] = bf16lo(w.y); x[3] = bf16hi(w.y);
  } else {
    const uint8_t* rec = static_cast<const uint8_t*>(base) + row * q4_row_bytes(D);
    const uint32_t c = *reinterpret_cast<const uint16_t*>(rec + d / 2);
    const uint32_t prm = *reinterpret_cast<const uint32_t*>(rec + D / 2 + d / kQ4Group * 4);
    const float sc = bf16lo(prm), lo = bf16hi(prm);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = fmaf((float)((c >> (4 * e)) & 15u), sc, lo);
  }
}

template <int FMT, int D, int NSRC, bool WGT>
__global__ void __launch_bounds__(NT) tree_simt_kernel(const TreeParams p) {
  using E = typename std::conditional<FMT == kTreeF32, float, __nv_bfloat16>::type;
  constexpr int LD = D + 4;          // padded rows: conflict-free column reads
  constexpr int C4 = D / 4;
  constexpr int ITEMS = (RT * C4 + NT - 1) / NT;
  extern __shared__ __align__(16) uint8_t smem[];
  float* sQ = reinterpret_cast<float*>(smem);   // [RT][LD]
  float* sK = sQ + RT * LD;                     // [KT][LD]
  float* sV = sK + KT * LD;                     // [KT][LD]
  float* sP = sV + KT * LD;                     // [RT][KT]
  float* sM = sP + RT * KT;                     // [RT] running max
  float* sL = sM + RT;                          // [RT] running sum
  float* sA = sL + RT;                          // [RT] rescale of this tile
  unsigned long long* sMask = reinterpret_cast<unsigned long long*>(sA + RT);   // [RT][2]
  int* sDepth = reinterpret_cast<int*>(sMask + RT * 2);                          // [kTreeMaxNodes]
  int* flag = sDepth + kTreeMaxNodes;
  const TreeSeqs sq = tree_seqs(flag + 1, p.B);
  const int* pre = sq.pre;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_trigger();
  grid_dep_wait();
  const TreeCut cut = tree_cut<E, D>(p, sq, KT, gridDim.x);
  if ((int)blockIdx.x >= cut.ranges) return;
  const int rt = blockIdx.y;
  const size_t plane = p.ring > 0 ? p.ring : p.S_max;
  TreeWalk walk;
  walk.begin(cut, pre, p.B, p.H, blockIdx.x);
  TreePiece pc;
  while (walk.next(pre, p.B, p.H, pc)) {
    const TreeSeq s = tree_seq(p, sq.P[pc.b], sq.N[pc.b]);
    const size_t unit = (size_t)pc.b * p.H + pc.h;
    const int rows = min(RT, p.G * p.T - rt * RT);
    __syncthreads();
    for (int it = tid; it < RT * C4; it += NT) {
      const int r = it / C4, d = (it - r * C4) * 4;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (r < rows) {
        const E* q = static_cast<const E*>(p.q) + (unit * p.G * p.T + rt * RT + r) * D + d;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = (float)q[e] * p.scale_log2;
      }
      tree_store4(sQ + r * LD + d, x);
    }
    for (int i = tid; i < s.N; i += NT) sDepth[i] = tree_depth(p, pc.b, i, s.N);
    if (tid < RT) {
      sM[tid] = -FLT_MAX;
      sL[tid] = 0.f;
      const int i = (rt * RT + tid) % p.T;
      for (int w = 0; w < 2; ++w)
        sMask[tid * 2 + w] = tid < rows && i < s.N && w < p.words ? tree_mask_word(p, pc.b, i, w, s.N) : 0ull;
    }
    float acc[ITEMS][4];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[k][e] = 0.f;

    for (int kt = pc.k0; kt < pc.k1; ++kt) {
      const TreeTile t = tree_tile(p, s, kt, KT);
      __syncthreads();
      for (int it = tid; it < KT * C4; it += NT) {
        const int r = it / C4, d = (it - r * C4) * 4;
        float k0[4] = {0.f, 0.f, 0.f, 0.f}, v0[4] = {0.f, 0.f, 0.f, 0.f};
        if (r < t.cnt) {
          const size_t row = unit * plane + t.row + r;
          load4<FMT, D>(p.k[0], row, d, k0);
          load4<FMT, D>(p.v[0], row, d, v0);
          if constexpr (WGT) {
            const size_t w = (size_t)pc.h * D + d;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              k0[e] *= p.a[0][w + e];
              v0[e] *= p.b[0][w + e];
            }
            if constexpr (NSRC == 2) {
              float k1[4], v1[4];
              load4<FMT, D>(p.k[1], row, d, k1);
              load4<FMT, D>(p.v[1], row, d, v1);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                k0[e] = fmaf(p.a[1][w + e], k1[e], k0[e]);
                v0[e] = fmaf(p.b[1][w + e], v1[e], v0[e]);
              }
            }
          }
        }
        tree_store4(sK + r * LD + d, k0);
        tree_store4(sV + r * LD + d, v0);
      }
      __syncthreads();
      // scores: warp w takes rows 2w and 2w + 1, a lane keys lane and lane + 32
#pragma unroll
      for (int rr = 0; rr < RT / 8; ++rr) {
        const int r = warp * (RT / 8) + rr;
        float sc[KT / 32];
#pragma unroll
        for (int kk = 0; kk < KT / 32; ++kk) {
          const int key = lane + 32 * kk;
          float x = 0.f, y = 0.f;
#pragma unroll 8
          for (int d = 0; d < D; d += 4) {
            const float4 q = *reinterpret_cast<const float4*>(sQ + r * LD + d);
            const float4 k = *reinterpret_cast<const float4*>(sK + key * LD + d);
            x = fmaf(q.x, k.x, x);
            y = fmaf(q.y, k.y, y);
            x = fmaf(q.z, k.z, x);
            y = fmaf(q.w, k.w, y);
          }
          const int pos = t.pos + key, j = pos - s.P;
          const int i = (rt * RT + r) % p.T;
          bool see = key < t.cnt && r < rows && i < s.N;
          if (see) {
            const int di = sDepth[i];
            if (j < 0) see = p.window == 0 || j > di - p.window;
            else see = (sMask[r * 2 + (j >> 6)] >> (j & 63) & 1) &&
                       (p.window == 0 || sDepth[j] > di - p.window);
          }
          sc[kk] = see ? x + y : -INFINITY;
        }
        float m = sc[0];
#pragma unroll
        for (int kk = 1; kk < KT / 32; ++kk) m = fmaxf(m, sc[kk]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float old = sM[r], top = fmaxf(old, m);
        float l = 0.f;
#pragma unroll
        for (int kk = 0; kk < KT / 32; ++kk) {
          const float e = exp2f(sc[kk] - top);
          sP[r * KT + lane + 32 * kk] = e;
          l += e;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        __syncwarp();
        if (lane == 0) {
          const float f = exp2f(old - top);
          sA[r] = f;
          sM[r] = top;
          sL[r] = fmaf(sL[r], f, l);
        }
      }
      __syncthreads();
      // values: a thread's items are four channels of a row
#pragma unroll
      for (int k = 0; k < ITEMS; ++k) {
        const int it = tid + k * NT;
        if (it >= RT * C4) break;
        const int r = it / C4, d = (it - r * C4) * 4;
        const float f = sA[r];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[k][e] *= f;
#pragma unroll 4
        for (int key = 0; key < KT; ++key) {
          const float pr = sP[r * KT + key];
          if (pr == 0.f) continue;   // a masked row's value is not used, whatever it holds
          const float4 v = *reinterpret_cast<const float4*>(sV + key * LD + d);
          acc[k][0] = fmaf(pr, v.x, acc[k][0]);
          acc[k][1] = fmaf(pr, v.y, acc[k][1]);
          acc[k][2] = fmaf(pr, v.z, acc[k][2]);
          acc[k][3] = fmaf(pr, v.w, acc[k][3]);
        }
      }
    }
    __syncthreads();
    const bool whole = pc.k1 - pc.k0 == pc.tiles;
    float* rec = p.ws + ((size_t)(2 * blockIdx.x + (pc.first ? 0 : 1)) * p.row_tiles + rt) *
                            tree_record_floats(RT, D);
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int it = tid + k * NT;
      if (it >= RT * C4) break;
      const int r = it / C4, d = (it - r * C4) * 4;
      if (whole) {
        const int row = rt * RT + r;
        if (r < rows && row % p.T < s.N) {
          const float inv = sL[r] == 0.f ? 0.f : 1.f / sL[r];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[k][e] *= inv;
          tree_store4(static_cast<E*>(p.out) + (unit * p.G * p.T + row) * D + d, acc[k]);
        }
      } else {
        tree_store4(rec + r * D + d, acc[k]);
      }
    }
    if (!whole) {
      if (tid < RT) {
        rec[RT * D + tid] = sM[tid];
        rec[RT * D + RT + tid] = sL[tid];
      }
      tree_publish<E, D, RT, NT>(p, cut, pre, pc.b, pc.h, s.N, tid, flag, sM, [] { __syncthreads(); });
    }
  }
}

template <int FMT, int D, int NSRC, bool WGT>
cudaError_t launch_simt(const TreeParams& p, const TreeArgs& a, const TreePlan& plan, cudaStream_t stream) {
  auto kern = tree_simt_kernel<FMT, D, NSRC, WGT>;
  static KernelReady ready;
  const cudaError_t e = ready.check(kern, a.device, 232448, NT, 0);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(plan.ranges, plan.row_tiles), dim3(NT), plan.smem_bytes, stream, p);
}

template <int FMT, int D>
cudaError_t launch_simt_src(const TreeParams& p, const TreeArgs& a, const TreePlan& plan,
                            cudaStream_t stream) {
  if (p.k[1]) return launch_simt<FMT, D, 2, true>(p, a, plan, stream);
  if (p.a[0]) return launch_simt<FMT, D, 1, true>(p, a, plan, stream);
  return launch_simt<FMT, D, 1, false>(p, a, plan, stream);
}

template <int FMT>
cudaError_t launch_simt_dim(const TreeParams& p, const TreeArgs& a, const TreePlan& plan,
                            cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return launch_simt_src<FMT, 64>(p, a, plan, stream);
    case 80: return launch_simt_src<FMT, 80>(p, a, plan, stream);
    case 96: return launch_simt_src<FMT, 96>(p, a, plan, stream);
    default: return launch_simt_src<FMT, 128>(p, a, plan, stream);
  }
}

}  // namespace

void tree_simt_plan(const TreeArgs& a, int num_sms, TreePlan* plan) {
  const int rows = a.group * a.T;
  plan->rows = RT;
  plan->row_tiles = (rows + RT - 1) / RT;
  // two CTAs an SM over ranges and row tiles; the device takes fewer ranges
  // where there are fewer key tiles
  plan->ranges = a.num_ctas > 0 ? a.num_ctas : (2 * num_sms + plan->row_tiles - 1) / plan->row_tiles;
  plan->smem_bytes = (size_t)(RT * (a.head_dim + 4) + 2 * KT * (a.head_dim + 4) + RT * KT + 3 * RT) * 4 +
                     RT * 16 + kTreeMaxNodes * 4 + 4 + tree_seqs_bytes(a.batch);
}

cudaError_t tree_simt_launch(const TreeParams& p, const TreeArgs& a, const TreePlan& plan,
                             cudaStream_t stream) {
  if (a.is_f32) return launch_simt_dim<kTreeF32>(p, a, plan, stream);
  if (a.q4) return launch_simt_dim<kTreeQ4>(p, a, plan, stream);
  return launch_simt_dim<kTreeBf16>(p, a, plan, stream);
}

}  // namespace fkv
