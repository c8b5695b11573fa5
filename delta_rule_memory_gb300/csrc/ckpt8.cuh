// ckpt8.cuh - the 8-bit checkpoint format: groups of 64 channels of one row,
// one power-of-two step per group, int8 codes (see ckpt8_pack in sdm.h).
#pragma once

#include "common.cuh"

namespace sdm {
namespace ckpt8 {

constexpr int kGroup = 64;

inline __host__ __device__ int groups(int D) { return (D + kGroup - 1) / kGroup; }

constexpr uint32_t kTop = 0x7f7e0000u;  // bits of 127 * 2^121, the largest magnitude that has a code
constexpr uint32_t kLast = 248;         // its exponent byte

// The step (its bits: the exponent byte << 23) of a group whose largest
// magnitude has the fp32 bits `top`: the smallest 2^e with |x| <= 127 * 2^e.
// 127 is 1.984375 * 2^6, so e is top's own exponent less 6, and one more where
// top's fraction is above 0.984375 * 2^23 = 0x7e0000: adding 0x1ffff carries into
// the exponent exactly then.  A top above kTop gives a byte above kLast.
__device__ __forceinline__ uint32_t step_bits(uint32_t top) {
  return max(static_cast<int32_t>(((top + 0x1ffffu) & 0xff800000u) - (6u << 23)), 1 << 23);
}
// The exponent byte as it is kept: 255 for NaN, infinities and what is above kTop
// (one exponent more, and a code's value could leave fp32's range).
__device__ __forceinline__ uint32_t exp_byte(uint32_t top) { return top > kTop ? 255u : step_bits(top) >> 23; }

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

// Two codes to their values: code + 128 in the low bits of 2^23 is a float, and
// less 2^23 + 128 it is the code.
__device__ __forceinline__ float2 decode2(uint32_t codes, float step) {
  codes ^= 0x8080u;
  const float2 v = make_float2(__uint_as_float(__byte_perm(codes, 0x4b000000u, 0x7440)),
                               __uint_as_float(__byte_perm(codes, 0x4b000000u, 0x7441)));
  return __fmul2_rn(__fadd2_rn(v, make_float2(-8388736.f, -8388736.f)), make_float2(step, step));
}

}  // namespace ckpt8
}  // namespace sdm
