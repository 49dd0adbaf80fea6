// fkv_read_kv: rows of a layer as its attention sees them, in the context's
// type (FusedKV slides, Eqs.(4)-(6)): its own rows (vanilla), K^s and V^t
// (Lite), those times channel weights (scaled), or
//     K^i = a_1 (.) K^s1 + a_2 (.) K^s2,  V^i = b_1 (.) V^t1 + b_2 (.) V^t2
// (fused), from plain, 4-bit or 8-bit caches.  fp32 arithmetic, one rounding.
//
// A thread takes 16 channels of a row of K or V: 16 bytes of 8-bit codes (8 of
// 4-bit codes with their group's two parameters, 32 or 64 of plain rows), and
// writes 32 or 64 bytes; consecutive threads take consecutive runs, so every
// warp reads and writes contiguous bytes.
#include "fkv_kernels.h"
#include "q8_device.cuh"

namespace fkv {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load_plain(const void* plane, size_t elem, float* f) {
  constexpr int N = 16 / (int)sizeof(T);
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(plane) + elem);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) unpack16<T>(src[i], f + i * N);
}

// Channels [16 c, 16 c + 16) of row `row` of unit u.
template <typename T, int D, int FMT>
__device__ __forceinline__ void load_run(const void* plane, const float* scale, size_t u, int rows, int row,
                                         int c, float* f) {
  const size_t r = u * rows + row;
  if constexpr (FMT == kCacheQ8) {
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(plane) + r * D + c * 16);
    const float s = scale[u * q8_scale_cols(rows) + row / kQ8Block];
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) e4m3x4_to_f32(w[i], f + 4 * i);
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] *= s;
  } else if constexpr (FMT == kCacheQ4) {
    const uint8_t* rec = static_cast<const uint8_t*>(plane) + r * q4_row_bytes(D);
    const uint2 q = *reinterpret_cast<const uint2*>(rec + c * 8);
    const uint32_t prm = *reinterpret_cast<const uint32_t*>(rec + D / 2 + c * 4);
    const float s = bf16lo(prm), lo = bf16hi(prm);
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] = fmaf((float)(((e < 8 ? q.x : q.y) >> (4 * (e & 7))) & 15u), s, lo);
  } else {
    load_plain<T>(plane, r * D + c * 16, f);
  }
}

__device__ __forceinline__ void store16(float* dst, const float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(dst)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* dst, const float* f) {
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    o[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// grid (rows of runs, K and V of every unit); WGT: the sources have weights.
template <typename T, int D, int FMT, int NSRC, bool WGT>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadArgs a) {
  constexpr int C = D / 16;
  grid_dep_trigger();
  grid_dep_wait();
  const long long units = (long long)a.batch * a.kv_heads;
  const bool value = (long long)blockIdx.x >= units;
  const size_t u = blockIdx.x - (value ? units : 0);
  const int b = (int)(u / a.kv_heads), h = (int)(u - (size_t)b * a.kv_heads);
  const int p = a.pos[b];
  if (p < 0 || (long long)p + a.T > a.max_seq) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && !value && h == 0) flag_status(a.status, kDevBadArg);
    return;
  }
  const int rows = a.ring > 0 ? a.ring : a.max_seq;
  const long long runs = (long long)a.T * C;
  T* out = static_cast<T*>(value ? a.v_out : a.k_out) + u * a.T * D;
  for (long long i = (long long)blockIdx.y * kThreads + threadIdx.x; i < runs;
       i += (long long)gridDim.y * kThreads) {
    const int t = (int)(i / C), c = (int)(i - (long long)t * C);
    const int row = a.ring > 0 ? (p + t) % a.ring : p + t;
    float x[16];
    load_run<T, D, FMT>(value ? a.v[0] : a.k[0], value ? a.v_scale[0] : a.k_scale[0], u, rows, row, c, x);
    if constexpr (WGT) {
      float w[16];
      load_plain<float>(value ? a.b[0] : a.a[0], (size_t)h * D + c * 16, w);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] *= w[e];
      if constexpr (NSRC == 2) {
        float y[16];
        load_run<T, D, FMT>(value ? a.v[1] : a.k[1], value ? a.v_scale[1] : a.k_scale[1], u, rows, row, c, y);
        load_plain<float>(value ? a.b[1] : a.a[1], (size_t)h * D + c * 16, w);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = fmaf(w[e], y[e], x[e]);
      }
    }
    store16(out + (size_t)t * D + c * 16, x);
  }
}

template <typename T, int D, int FMT>
cudaError_t by_src(const ReadArgs& a, dim3 grid, cudaStream_t s) {
  if (a.nsrc == 2) return launch_pdl(read_kernel<T, D, FMT, 2, true>, grid, dim3(kThreads), 0, s, a);
  if (a.a[0]) return launch_pdl(read_kernel<T, D, FMT, 1, true>, grid, dim3(kThreads), 0, s, a);
  return launch_pdl(read_kernel<T, D, FMT, 1, false>, grid, dim3(kThreads), 0, s, a);
}

template <int D>
cudaError_t by_format(const ReadArgs& a, cudaStream_t s) {
  const long long runs = (long long)a.T * (D / 16);
  const long long need = (runs + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)(2LL * a.batch * a.kv_heads), (unsigned)(need < 65535 ? need : 65535));
  if (a.format == kCacheQ8)
    return a.is_f32 ? by_src<float, D, kCacheQ8>(a, grid, s) : by_src<__nv_bfloat16, D, kCacheQ8>(a, grid, s);
  if (a.format == kCacheQ4) return by_src<__nv_bfloat16, D, kCacheQ4>(a, grid, s);
  return a.is_f32 ? by_src<float, D, kCachePlain>(a, grid, s) : by_src<__nv_bfloat16, D, kCachePlain>(a, grid, s);
}

}  // namespace

cudaError_t read_launch(const ReadArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return by_format<64>(a, stream);
    case 80: return by_format<80>(a, stream);
    case 96: return by_format<96>(a, stream);
    case 128: return by_format<128>(a, stream);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace fkv
