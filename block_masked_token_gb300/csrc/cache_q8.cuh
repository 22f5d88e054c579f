// The 8-bit paged cache: a page holds e4m3 codes, and for each KV head a scale byte x that stands
// for 2^(x - 127). Scales are powers of two, so that a page whose scale grows under an append
// changes its codes' exponents only, and no product with a scale rounds.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace mars {
namespace q8 {

constexpr int kBias = 127;
constexpr int kLeast = 87, kMost = 167;      // scale bytes in use: 2^-40 .. 2^40

// A scale byte as every kernel reads it.
MARS_DEV int scale_byte(uint8_t x) { return min(max((int)x, kLeast), kMost); }
// 2^(x - 127) and its inverse, for 0 < x < 254.
MARS_DEV float power(int x) { return __int_as_float(x << 23); }
MARS_DEV float inverse_power(int x) { return __int_as_float((2 * kBias - x) << 23); }

// The smallest scale byte under which a largest magnitude of `amax` (bf16 bits, finite) needs no
// code beyond 448 = 1.75 * 2^8.
MARS_DEV int scale_for(uint32_t amax) {
  const int x = (int)(amax >> 7) - 8 + ((amax & 0x7fu) > 0x60u ? 1 : 0);
  return min(max(x, kLeast), kMost);
}

// Two floats as halves.
MARS_DEV uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Codes of two floats; beyond the range they end at its border, NaN stays.
MARS_DEV uint32_t encode2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
// The two pairs of codes of a word as halves, exactly. (The header's conversion of a pair takes 6
// cycles of a warp where this takes 2: it moves the halves about one by one.)
MARS_DEV void decode4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
MARS_DEV float2 halves(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }

}  // namespace q8
}  // namespace mars
