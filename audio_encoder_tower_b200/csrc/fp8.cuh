// Device helpers of the 8-bit format: e4m3 values with one power-of-two scale
// (e8m0) for each block of 128 columns of a row.
#pragma once

#include "common.cuh"

namespace enc {

constexpr int kFp8Block = 128;

__host__ __device__ inline int fp8_blocks(int cols) { return (cols + kFp8Block - 1) / kFp8Block; }
__host__ __device__ inline int fp8_pitch(int cols) { return (fp8_blocks(cols) + 3) & ~3; }

// e8m0 byte (exponent + 127) of the least 2^e, e >= -126, with amax <= 448 * 2^e,
// from the bits of a finite amax >= 0. 448 = 1.75 * 2^8: the exponent is amax's own
// less 8, and one more where amax's fraction is above 0.75 (0x600000 of 0x800000).
__device__ __forceinline__ uint32_t e8m0_of_amax(uint32_t amax_bits) {
  const int b = static_cast<int>((amax_bits + 0x1FFFFFu) >> 23) - 8;
  return static_cast<uint32_t>(b > 1 ? b : 1);
}

// 2^-e of an e8m0 byte in 1 .. 247 (all that e8m0_of_amax gives): exact in fp32.
__device__ __forceinline__ float e8m0_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Magnitude bits that count for a block's amax: a NaN or an infinity counts as 0.
__device__ __forceinline__ uint32_t finite_abs_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}

// Four values, already divided by their scale, as e4m3 (low byte first). Finite values are at
// most 448 in magnitude; e4m3 keeps NaN, and an infinity has been turned into NaN before.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

}  // namespace enc
