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

// Two values / 2^e as e4m3 (low byte: a). |value / 2^e| <= 448 where it is finite; an
// infinity turns into NaN by the product with zero, and e4m3 keeps NaN.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b, float inv) {
  a = fmaf(a, 0.f, a * inv);
  b = fmaf(b, 0.f, b * inv);
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float inv) {
  return e4m3x2(a, b, inv) | (e4m3x2(c, d, inv) << 16);
}

}  // namespace enc
