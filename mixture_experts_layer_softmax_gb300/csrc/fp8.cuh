// FP8 tensors with a scale for each block of 128: E4M3 codes (uint8, row-major)
// and fp32 scales, one for each 128 columns of a row (activations) or each
// 128 x 128 block (weights).
//
// A block with largest magnitude m gets a = max(m, 448 2^-125), the scale
// a / 448 and the codes E4M3(448 x / a), to nearest even.  The quotient is taken
// as (0.875 x) / (2^-9 a): neither product overflows, the first is exact for
// bf16 x (11 bits) and the second always, so the one division's rounding is the
// only one before the code's own: a bf16 x on the border of two codes is seen to
// lie there, which x times a rounded 448 / a misses for 0.5% of values.
// An infinity or a NaN makes the block's scale and codes NaN.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {
namespace fp8 {

constexpr int BLOCK = 128;

// The bits of |v|: ordered like the magnitudes, infinities and NaNs above all.
MOE_D uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The block's a from the largest magnitude's bits.
MOE_D float block_top(uint32_t bits) {
  if (bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  return fmaxf(__uint_as_float(bits), 448.f * 0x1p-125f);
}
MOE_D float block_scale(float a) { return a / 448.f; }

// 448 v / a before its rounding to E4M3 (d = 2^-9 a).
MOE_D float ratio(float v, float d) { return (v * 0.875f) / d; }

MOE_D uint32_t codes2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
// Eight values of a block with top a -> eight codes.
MOE_D uint2 codes8(const float* v, float a) {
  const float d = a * 0x1p-9f;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = codes2(ratio(v[2 * i], d), ratio(v[2 * i + 1], d));
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

MOE_D float decode(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(__half(h));
}

}  // namespace fp8
}  // namespace moe
