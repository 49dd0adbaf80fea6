// fkv_read_kv: rows of a layer as its attention sees them, in the context's
// type (FusedKV slides, Eqs.(4)-(6)): its own rows (vanilla), K^s and V^t
// (Lite), those times channel weights (scaled), or
//     K^i = a_1 (.) K^s1 + a_2 (.) K^s2,  V^i = b_1 (.) V^t1 + b_2 (.) V^t2
// (fused), from plain, 4-bit or 8-bit caches.  fp32 arithmetic, one rounding.
//
// A thread takes runs of 8 channels of a row of K or V: 8 bytes of 8-bit codes
// (4 of 4-bit codes with their group's two parameters, 16 or 32 of plain
// rows), and writes 16 or 32 bytes; consecutive threads take consecutive runs,
// so that a store of a bf16 warp is 512 contiguous bytes, and each has several of
// them in flight.  Bound: HBM, 3 bytes an element (bf16 from one 8-bit source).
#include "fkv_kernels.h"
#include "q8_device.cuh"

namespace fkv {
namespace {

constexpr int kThreads = 256;   // of a CTA, at most
// Runs in flight per thread: 8 carry 98% of the measured copy rate where there
// are CTAs enough (4 x 16 heads x 16384 rows of 80 channels: 77 us, against 101
// with 2), and short calls spread over more CTAs with 2 (32 x 8 heads x 77 rows,
// two sources: 4.5 us, against 5.7 with 8).
constexpr int kRunsLong = 8, kRunsShort = 2;
constexpr long long kLongCtas = 8 * 152;   // 8 an SM of a GB300

// 8 elements of a plain row.
template <typename T>
__device__ __forceinline__ void load_plain(const void* plane, size_t elem, float* f) {
  constexpr int N = 16 / (int)sizeof(T);
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(plane) + elem);
#pragma unroll
  for (int i = 0; i < 8 / N; ++i) unpack16<T>(src[i], f + i * N);
}

// Channels [8 c, 8 c + 8) of row `row` of unit u: as they lie, then as fp32.
template <typename T, int D, int FMT>
struct Run {
  uint4 v[sizeof(T) / 2];   // plain
  uint2 q;                  // codes (4-bit: x only)
  uint32_t prm;             // scale (4-bit: scale and minimum)
  __device__ __forceinline__ void load(const void* plane, const float* scale, size_t u, int rows, int row, int c) {
    const size_t r = u * rows + row;
    if constexpr (FMT == kCacheQ8) {
      q = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(plane) + r * D + c * 8));
      prm = __float_as_uint(scale[u * q8_scale_cols(rows) + row / kQ8Block]);
    } else if constexpr (FMT == kCacheQ4) {
      const uint8_t* rec = static_cast<const uint8_t*>(plane) + r * q4_row_bytes(D);
      q.x = *reinterpret_cast<const uint32_t*>(rec + c * 4);
      prm = *reinterpret_cast<const uint32_t*>(rec + D / 2 + c / 2 * 4);
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(plane) + r * D + c * 8);
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = __ldcs(src + i);
    }
  }
  __device__ __forceinline__ void values(float* f) const {
    if constexpr (FMT == kCacheQ8) {
      e4m3x4_to_f32(q.x, f);
      e4m3x4_to_f32(q.y, f + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= __uint_as_float(prm);
    } else if constexpr (FMT == kCacheQ4) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = fmaf((float)((q.x >> (4 * e)) & 15u), bf16lo(prm), bf16hi(prm));
    } else {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) unpack16<T>(v[i], f + i * (16 / (int)sizeof(T)));
    }
  }
};

__device__ __forceinline__ void store8(float* dst, const float* f) {
  __stcs(reinterpret_cast<float4*>(dst), make_float4(f[0], f[1], f[2], f[3]));
  __stcs(reinterpret_cast<float4*>(dst) + 1, make_float4(f[4], f[5], f[6], f[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float* f) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    o[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  __stcs(reinterpret_cast<uint4*>(dst), make_uint4(o[0], o[1], o[2], o[3]));
}

// grid (rows of runs, K and V of every unit); WGT: the sources have weights.
template <typename T, int D, int FMT, int NSRC, bool WGT, int kRuns>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadArgs a) {
  constexpr int C = D / 8;
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
  T* out = static_cast<T*>(value ? a.v_out : a.k_out) + u * a.T * D;
  // the thread's channels, and the rows of the CTA that its threads take at once
  const int c = (int)threadIdx.x % C, tr = (int)threadIdx.x / C, step = (int)blockDim.x / C;
  if (tr >= step) return;
  float w[NSRC][8];
  if constexpr (WGT) {
#pragma unroll
    for (int i = 0; i < NSRC; ++i) load_plain<float>(value ? a.b[i] : a.a[i], (size_t)h * D + c * 8, w[i]);
  }
  for (long long t0 = (long long)blockIdx.y * step * kRuns + tr; t0 < a.T; t0 += (long long)gridDim.y * step * kRuns) {
    // all loads first, without branches (a row behind the last is the last again)
    Run<T, D, FMT> x[NSRC][kRuns];
#pragma unroll
    for (int k = 0; k < kRuns; ++k) {
      const int t = (int)(t0 + k * step < a.T ? t0 + k * step : a.T - 1);
      const int row = a.ring > 0 ? (int)(((long long)p + t) % a.ring) : p + t;
#pragma unroll
      for (int i = 0; i < NSRC; ++i)
        x[i][k].load(value ? a.v[i] : a.k[i], value ? a.v_scale[i] : a.k_scale[i], u, rows, row, c);
    }
#pragma unroll
    for (int k = 0; k < kRuns; ++k) {
      float f[8];
      x[0][k].values(f);
      if constexpr (WGT) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= w[0][e];
      }
      if constexpr (NSRC == 2) {
        float y[8];
        x[NSRC - 1][k].values(y);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = fmaf(w[NSRC - 1][e], y[e], f[e]);
      }
      if (t0 + k * step < a.T) store8(out + (size_t)(t0 + k * step) * D + c * 8, f);
    }
  }
}

template <typename T, int D, int FMT, int RUNS>
cudaError_t by_src(const ReadArgs& a, cudaStream_t s) {
  // whole rows of threads; few rows take fewer threads
  const long long runs = (long long)a.T * (D / 8);
  const int threads = runs < kThreads ? (int)(runs + 31) / 32 * 32 : kThreads;
  const long long rows = (long long)(threads / (D / 8)) * RUNS, need = (a.T + rows - 1) / rows;
  const long long columns = 2LL * a.batch * a.kv_heads;
  if constexpr (RUNS == kRunsLong)
    if (columns * need < kLongCtas) return by_src<T, D, FMT, kRunsShort>(a, s);
  const dim3 grid((unsigned)columns, (unsigned)(need < 65535 ? need : 65535)), block(threads);
  if (a.nsrc == 2) return launch_pdl(read_kernel<T, D, FMT, 2, true, RUNS>, grid, block, 0, s, a);
  if (a.a[0]) return launch_pdl(read_kernel<T, D, FMT, 1, true, RUNS>, grid, block, 0, s, a);
  return launch_pdl(read_kernel<T, D, FMT, 1, false, RUNS>, grid, block, 0, s, a);
}

template <int D>
cudaError_t by_format(const ReadArgs& a, cudaStream_t s) {
  if (a.format == kCacheQ8)
    return a.is_f32 ? by_src<float, D, kCacheQ8, kRunsLong>(a, s) : by_src<__nv_bfloat16, D, kCacheQ8, kRunsLong>(a, s);
  if (a.format == kCacheQ4) return by_src<__nv_bfloat16, D, kCacheQ4, kRunsLong>(a, s);
  return a.is_f32 ? by_src<float, D, kCachePlain, kRunsLong>(a, s) : by_src<__nv_bfloat16, D, kCachePlain, kRunsLong>(a, s);
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
