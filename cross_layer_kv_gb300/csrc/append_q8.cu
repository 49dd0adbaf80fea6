// fkv_append_kv on an 8-bit layer: quantise the new rows as they are written.
//
// A block is kQ8Block rows of one (sequence, KV head) of K or V, with one
// scale.  With amax the largest finite magnitude of the block's new rows and
//     need = 2^e, e = min { e : amax <= 448 * 2^e }, clamped to [-100, 119],
// the block's scale becomes s = need where its first row is new, and
// max(s, need) where rows before the new ones keep their places in it.  New
// rows store e4m3(x / s), not finite elements the NaN code; where s grew, the
// rows before the new ones store e4m3(code * s_old / s).  Rows of the block
// behind the new ones are free.
//
// One warp per block; a lane holds up to D/16 runs of 16 channels in
// registers between the maximum and the codes, so the new rows are read once,
// in 32 (bf16) or 64 (fp32) contiguous bytes a lane, and the codes are written
// 16 bytes a lane.  A block belongs to one warp (the host refuses calls whose
// rows would come round to their first block of a ring), so nothing is atomic.
#include "fkv_kernels.h"
#include "q8_device.cuh"

namespace fkv {
namespace {

constexpr int kWarps = 8;

// 16 elements of the context's type -> fp32.
__device__ __forceinline__ void load16(const __nv_bfloat16* src, float* f) {
  unpack16<__nv_bfloat16>(reinterpret_cast<const uint4*>(src)[0], f);
  unpack16<__nv_bfloat16>(reinterpret_cast<const uint4*>(src)[1], f + 8);
}
__device__ __forceinline__ void load16(const float* src, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack16<float>(reinterpret_cast<const uint4*>(src)[i], f + 4 * i);
}

// The smallest power of two whose 448-fold (1.75 * 2^8) reaches amax.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < kQ8MinExp ? kQ8MinExp : (e > kQ8MaxExp ? kQ8MaxExp : e);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) append_q8_kernel(AppendArgs a, int blocks) {
  constexpr int PER = D / 16;   // runs of 16 channels per row, and per lane and block
  static_assert(kQ8Block == 32, "a lane's runs of a block are one row's");
  grid_dep_trigger();
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const long long units = (long long)a.batch * a.kv_heads;
  const long long total = 2 * units * blocks;
  for (long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); w < total;
       w += (long long)gridDim.x * kWarps) {
    const int i = (int)(w % blocks);           // block of the call
    const long long u2 = w / blocks;
    const bool value = u2 >= units;
    const long long u = value ? u2 - units : u2;
    const int b = (int)(u / a.kv_heads);
    const int p = a.pos[b];
    if (p < 0 || (long long)p + a.T > a.max_seq) {
      if (lane == 0 && i == 0 && !value && u % a.kv_heads == 0) flag_status(a.status, kDevBadArg);
      continue;
    }
    // rows [r0, r1) of block g are new; the first of them is row t0 of the call
    const int g = p / kQ8Block + i;
    const int base = g * kQ8Block;
    if (base >= p + a.T) continue;
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
    float x[PER][16];
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int c = lane + 32 * k;
      if (c < runs) {
        load16(src + (size_t)c * 16, x[k]);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t m = __float_as_uint(x[k][e]) & 0x7fffffffu;
          if (m < 0x7f800000u) top = m > top ? m : top;
        }
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const float need = scale_for(__uint_as_float(top));
    const bool had = s_old > 0.f && s_old < INFINITY;
    const float s = had && s_old > need ? s_old : need;
    // dividing by a power of two is multiplying by its reciprocal
    const bool power = (__float_as_uint(s) & 0x7fffffu) == 0 && s > 0x1p-120f && s < 0x1p+120f;
    const float inv = power ? 1.f / s : 0.f;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int c = lane + 32 * k;
      if (c < runs) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const float v = x[k][4 * e + f];
            y[f] = power ? v * inv : __fdiv_rn(v, s);
            if ((__float_as_uint(v) & 0x7fffffffu) >= 0x7f800000u) y[f] = __uint_as_float(0x7fffffffu);
          }
          o[e] = e4m3x2_of(y[0], y[1]) | (e4m3x2_of(y[2], y[3]) << 16);
        }
        *reinterpret_cast<uint4*>(codes + (size_t)r0 * D + c * 16) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    if (had && s != s_old) {
      const float ratio = __fdiv_rn(s_old, s);
      for (int c = lane; c < r0 * PER; c += 32) {
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
    if (lane == 0) *sp = s;
  }
}

template <typename T>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
  // blocks that T rows can touch, wherever they start
  const int blocks = (a.T + kQ8Block - 2) / kQ8Block + 1;
  const long long total = 2LL * a.batch * a.kv_heads * blocks;
  long long ctas = (total + kWarps - 1) / kWarps;
  if (ctas > 65535LL * 8) ctas = 65535LL * 8;
  const dim3 grid((unsigned)ctas), block(kWarps * 32);
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
