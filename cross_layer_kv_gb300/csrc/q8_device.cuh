// 8-bit caches: the format and its conversions.
//
// A plane (the K or V cache of a layer) is e4m3 codes [B, H_kv, rows, D] and
// fp32 scales [B, H_kv, q8_scale_cols(rows)], one per kQ8Block consecutive
// rows of a (sequence, KV head); an element's value is code * scale.  e4m3 has
// 4 significant bits at every exponent from 2^-6 on (below it, steps of 2^-9),
// so a block's scale only has to place the block's largest value below 448:
// the append takes the power of two that does.  A later, larger row of the
// same block then moves the codes before it by whole exponents, which rounds
// nothing but what falls below 2^-6: by at most 2^-10 new scales each time that
// the scale grows, below 2^-9 of the last one in all (a scale at least doubles),
// 2^-16.8 of the block's largest value, which is above 224 scales.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fkv_device.cuh"

namespace fkv {

// Attention keeps a block's value scale in the exponents of its softmax
// weights, down to this one.  Below it (a block of zeros has 2^-100, one never
// written 0) the rest of the scale goes into the product, so that such a block
// still takes its part of the softmax's sum beside blocks of far larger scales.
constexpr float kQ8MinValue = 0x1p-64f;

// Four e4m3 codes -> two fp16 pairs (the lower codes first), exactly.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

__device__ __forceinline__ uint32_t f16x2_of(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two fp32 -> e4m3 codes (x in the low byte): nearest even, above 448 to 448,
// NaN to NaN.
__device__ __forceinline__ uint32_t e4m3x2_of(float x, float y) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %2, %1;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(r)
      : "f"(x), "f"(y));
  return r;
}

// Four codes in a word -> fp32, exactly.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float* f) {
  uint32_t h0, h1;
  e4m3x4_to_f16(w, h0, h1);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
}

// The smallest e with x <= 2^e, for a normal x > 0 (126 at most); and 2^-e.
__device__ __forceinline__ void ceil_log2(float x, float& e, float& inverse) {
  const uint32_t biased = min((__float_as_uint(x) + 0x7fffffu) >> 23, 253u);
  e = __uint_as_float(0x4b000000u | biased) - (8388608.f + 127.f);   // (2^23 + biased, as it lies)
  inverse = __uint_as_float((254u - biased) << 23);
}

}  // namespace fkv
