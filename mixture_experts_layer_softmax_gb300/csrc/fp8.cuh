// FP8 tensors with a scale for each block of 128: E4M3 codes (uint8, row-major)
// and fp32 scales, one for each 128 columns of a row (activations) or each
// 128 x 128 block (weights).
//
// A block with largest magnitude m gets a = max(m, 448 2^-125), the scale
// a / 448 and the codes E4M3(448 x / a), to nearest even; an infinity or a NaN
// makes the block's scale and codes NaN.  The quotient is x times the rounded
// 448 / a, within 2^-23 of itself.  For bf16 x that is made exact: with integers
// 7 m and A for the mantissas of 448 x and a, and T (at most five bits) for a
// border between two codes, 7 m 2^p and T A 2^r either agree or differ by 1 of at
// most 31 x 255, so no quotient but one on a border is within 2^-13 of it, and
// rounding the product to 20 bits puts those there (without it, 0.5% of normally
// distributed values fall to the wrong side).  A division gives the same codes;
// it took the weights' quantiser 1013 us for 8 x 28672 x 4096 values.
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
MOE_D float block_inverse(float a) { return 448.f / a; }

// 448 x / a of a bf16 x, on a border where the exact quotient is (see above).
MOE_D float snap(float t) { return __uint_as_float((__float_as_uint(t) + 8u) & ~15u); }

MOE_D uint32_t codes2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
// Four quotients -> four codes.
MOE_D uint32_t codes4(float a, float b, float c, float d) {
  return codes2(a, b) | (codes2(c, d) << 16);
}
// Eight fp32 values of a block -> eight codes, by x times the rounded 448 / a: a quotient
// within 2^-23 of a border of two codes may fall to either.  (The values are rounded sums;
// what they are off themselves is as much.)
MOE_D uint2 codes8(const float* v, float inv) {
  return make_uint2(codes4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    codes4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

// The two bf16 numbers of a word.
MOE_D float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
MOE_D float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// Four bf16 values of a block -> four codes, exact (snap() has no NaN of a NaN).
MOE_D uint32_t codes4(uint32_t x, uint32_t y, float inv) {
  const uint32_t c = codes4(snap(bf16_lo(x) * inv), snap(bf16_hi(x) * inv), snap(bf16_lo(y) * inv),
                            snap(bf16_hi(y) * inv));
  return inv == inv ? c : 0x7f7f7f7fu;
}
MOE_D uint2 codes8(const uint4& x, float inv) {
  return make_uint2(codes4(x.x, x.y, inv), codes4(x.z, x.w, inv));
}
// The larger magnitudes of two words' low and high bf16 numbers, as 15-bit integers.
MOE_D uint32_t mag_max2(uint32_t a, uint32_t b) { return __vmaxu2(a & 0x7fff7fffu, b & 0x7fff7fffu); }
MOE_D uint32_t mag_max2(const uint4& x) {
  return __vmaxu2(mag_max2(x.x, x.y), mag_max2(x.z, x.w));
}
// The fp32 bits of the larger of a word's two magnitudes.
MOE_D uint32_t mag_bits2(uint32_t m) { return max(m << 16, m & 0xffff0000u); }

}  // namespace fp8
}  // namespace moe
