// fkv_append_kv on an 8-bit layer: quantise the new rows as they are written.
//
// A block is kQ8Block rows of one (sequence, KV head) of K or V, with one
// scale.  With amax the largest finite magnitude of the block's new rows and
//     need = 2^e, e = min { e : amax <= 448 * 2^e }, clamped to [-100, 119],
// the block's scale becomes s = need where its first row is new, and
// max(s, need) where rows before the new ones keep their places in it.  New
// rows store e4m3(x / s), not finite elements the NaN code; where s grew, the
// rows before the new ones store e4m3(code * s_old / s) (zeros, where s_old is
// 0).  Rows of the block behind the new ones are free.
//
// One warp per block; a lane holds up to D/8 runs of 8 channels in registers
// between the maximum and the codes, so the new rows are read once; a load of
// the warp is 512 contiguous bytes (bf16) and a store of codes 256.  A block
// belongs to one warp (the host refuses calls whose rows would come round to
// their first block of a ring), so nothing is atomic.  Bound: HBM, 3 bytes an
// element (bf16) for prompts (16 sequences of 8 heads, 2001 rows of 128
// channels: 39.6 us, 4.97 TB/s, the ALU pipe at 68%), latency for single tokens
// (32 sequences of 8 heads: 2.4 us).
#include <type_traits>

#include "fkv_kernels.h"
#include "q8_device.cuh"

namespace fkv {
namespace {

constexpr int kWarps = 8;   // of a CTA, at most

// 8 elements of the context's type, as they are, and their bits as fp32.
template <typename T>
struct Run8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* src) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = __ldcs(reinterpret_cast<const uint4*>(src) + i);
  }
  __device__ __forceinline__ void values(float* f) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) unpack16<T>(v[i], f + i * (16 / (int)sizeof(T)));
  }
};

// The smallest power of two whose 448-fold (1.75 * 2^8) reaches amax.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < kQ8MinExp ? kQ8MinExp : (e > kQ8MaxExp ? kQ8MaxExp : e);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) append_q8_kernel(AppendArgs a, int blocks) {
  constexpr int PER = D / 8;   // runs of 8 channels per row, and per lane and block
  static_assert(kQ8Block == 32, "a lane's runs of a block are one row's");
  grid_dep_trigger();
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int units = a.batch * a.kv_heads;
  const int warps = (int)blockDim.x >> 5;
  for (int i = (int)blockIdx.y * warps + (threadIdx.x >> 5); i < blocks; i += (int)gridDim.y * warps) {   // block of the call
    const bool value = (int)blockIdx.x >= units;
    const int u = (int)blockIdx.x - (value ? units : 0);
    const int b = u / a.kv_heads;
    const int p = a.pos[b];
    if (p < 0 || (long long)p + a.T > a.max_seq) {
      if (lane == 0 && i == 0 && !value && u % a.kv_heads == 0) flag_status(a.status, kDevBadArg);
      return;
    }
    // rows [r0, r1) of block g are new; the first of them is row t0 of the call
    const int g = p / kQ8Block + i;
    if (g > (p + a.T - 1) / kQ8Block) continue;
    const int base = g * kQ8Block;
    const int r0 = p > base ? p - base : 0;
    const int r1 = p + a.T - base < kQ8Block ? p + a.T - base : kQ8Block;
    const int t0 = base + r0 - p;
    const int rows = a.ring > 0 ? a.ring : a.max_seq;
    const int slot = a.ring > 0 ? g % (a.ring / kQ8Block) : g;
    uint8_t* codes = static_cast<uint8_t*>(value ? a.v_cache : a.k_cache) +
                     ((size_t)u * rows + (size_t)slot * kQ8Block) * D;
    float* sp = (value ? a.v_scale : a.k_scale) + (size_t)u * q8_scale_cols(rows) + slot;
    const T* src = static_cast<const T*>(value ? a.v_new : a.k_new) + ((size_t)u * a.T + t0) * D;
    const int runs = (r1 - r0) * PER;

    const float s_old = r0 > 0 ? *sp : 0.f;
    Run8<T> x[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k)
      if (lane + 32 * k < runs) x[k].load(src + (size_t)(lane + 32 * k) * 8);
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      if (lane + 32 * k < runs) {
        float f[8];
        x[k].values(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t m = __float_as_uint(f[e]) & 0x7fffffffu;
          if (m < 0x7f800000u) top = m > top ? m : top;
        }
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const float need = scale_for(__uint_as_float(top));
    const bool had = s_old >= 0.f && s_old < INFINITY;   // (0: the rows before are zeros, whatever their codes)
    const float s = had && s_old > need ? s_old : need;
    // dividing by a power of two is multiplying by its reciprocal
    const bool power = (__float_as_uint(s) & 0x7fffffu) == 0 && s > 0x1p-120f && s < 0x1p+120f;
    auto encode = [&](auto divide) {
      const float inv = 1.f / s;
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int c = lane + 32 * k;
        if (c < runs) {
          float f[8];
          x[k].values(f);
          uint32_t o[2];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const bool finite = (__float_as_uint(f[e]) & 0x7fffffffu) < 0x7f800000u;
            if constexpr (decltype(divide)::value) f[e] = __fdiv_rn(f[e], s);
            else f[e] *= inv;
            if (!finite) f[e] = __uint_as_float(0x7fffffffu);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
            o[e] = e4m3x2_of(f[4 * e], f[4 * e + 1]) | (e4m3x2_of(f[4 * e + 2], f[4 * e + 3]) << 16);
          *reinterpret_cast<uint2*>(codes + (size_t)r0 * D + c * 8) = make_uint2(o[0], o[1]);
        }
      }
    };
    if (power)
      encode(std::false_type{});
    else
      encode(std::true_type{});
    if (had && s != s_old) {
      const float ratio = __fdiv_rn(s_old, s);
      for (int c = lane; c < r0 * (D / 16); c += 32) {
        uint4* pc = reinterpret_cast<uint4*>(codes + c * 16);
        const uint4 q = *pc;
        const uint32_t in[4] = {q.x, q.y, q.z, q.w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float f[4];
          e4m3x4_to_f32(in[e], f);
          o[e] = e4m3x2_of(f[0] * ratio, f[1] * ratio) | (e4m3x2_of(f[2] * ratio, f[3] * ratio) << 16);
        }
        *pc = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    __syncwarp();   // all lanes have read the scale
    if (lane == 0) *sp = s;
  }
}

template <typename T>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
  // blocks that T rows can touch, wherever they start
  const int blocks = (a.T + kQ8Block - 2) / kQ8Block + 1;
  const int warps = blocks < kWarps ? blocks : kWarps;
  const int rows = (blocks + warps - 1) / warps;   // of the grid: a unit's K or V is a column
  const dim3 grid((unsigned)(2LL * a.batch * a.kv_heads), (unsigned)(rows < 65535 ? rows : 65535)), block(warps * 32);
  switch (a.head_dim) {
    case 64: return launch_pdl(append_q8_kernel<T, 64>, grid, block, 0, stream, a, blocks);
    case 80: return launch_pdl(append_q8_kernel<T, 80>, grid, block, 0, stream, a, blocks);
    case 96: return launch_pdl(append_q8_kernel<T, 96>, grid, block, 0, stream, a, blocks);
    case 128: return launch_pdl(append_q8_kernel<T, 128>, grid, block, 0, stream, a, blocks);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace

cudaError_t append_q8_launch(const AppendArgs& a, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  return a.elem_bytes == 4 ? launch<float>(a, stream) : launch<__nv_bfloat16>(a, stream);
}

}  // namespace fkv
