// ckpt8.cuh - the 8-bit checkpoint format: groups of 64 channels of one row,
// one power-of-two step per group, int8 codes (see ckpt8_pack in sdm.h).
#pragma once

#include "common.cuh"

namespace sdm {
namespace ckpt8 {

constexpr int kGroup = 64;

inline __host__ __device__ int groups(int D) { return (D + kGroup - 1) / kGroup; }

// The biased exponent byte of a group whose largest magnitude has the fp32
// bits `top`: the smallest e with |x| <= 127 * 2^e.  127 is 1.984375 * 2^6, so
// e is top's own exponent less 6, and one more where top's fraction is above
// 0.984375 * 2^23 = 0x7e0000: adding 0x1ffff carries into the exponent exactly
// then.  255 for NaN, infinities and what is above 127 * 2^121 (bits
// 0x7f7e0000): one exponent more, and a code's value could leave fp32's range.
__device__ __forceinline__ uint32_t exp_byte(uint32_t top) {
  const int e = static_cast<int>((top + 0x1ffffu) >> 23) - 6;
  return top > 0x7f7e0000u ? 255u : static_cast<uint32_t>(e < 1 ? 1 : e);
}

// 1 / step and step of an exponent byte.  byte 255: 1 / step is NaN (the codes
// are then forced to 0) and the step is infinite, so that 0 * step is NaN.
__device__ __forceinline__ float inv_step(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
__device__ __forceinline__ float step(uint32_t byte) { return __uint_as_float(byte << 23); }

// x / step rounded to nearest even, in the low byte: adding 1.5 * 2^23 leaves
// the whole number in the low bits of the sum, and x * inv is exact, so the
// one rounding of the FMA is the rounding of the format.
__device__ __forceinline__ uint32_t code_bits(float x, float inv) {
  return __float_as_uint(fmaf(x, inv, 12582912.f));
}

}  // namespace ckpt8
}  // namespace sdm
