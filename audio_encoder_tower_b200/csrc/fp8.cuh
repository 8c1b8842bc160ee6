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

// --------------------------------------------------- overlap of consecutive launches
// These kernels may start while the kernel before them in the stream is still running (they are
// launched with programmatic stream serialisation), so that its tail hides their set-up. Every
// thread calls grid_dependency() before it touches global memory: it returns once the kernel
// before has completed and its writes are visible. The second instruction lets the next kernel
// do the same as soon as all blocks of this one have got here.
__device__ __forceinline__ void grid_dependency() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, unsigned cluster,
                              cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// ------------------------------------------------- block-scaled tensor-core products
constexpr int kBK = 128;                    // K elements (and bytes) per ring stage: one scale block
constexpr uint32_t kUnitScale = 0x7F7F7F7Fu;   // scales of rows outside the matrix: 2^0

// Instruction descriptor, kind::mxf8f6f4: fp32 accumulator, e4m3 A and B, both
// K-major, e8m0 scales; `id` is the byte (0..3) of the scale words to use.
__host__ __device__ constexpr uint32_t idesc_mxf8(int m, int n) {
  return (static_cast<uint32_t>(n >> 3) << 17)     // N / 8
         | (1u << 23)                              // scale type: e8m0
         | (static_cast<uint32_t>(m >> 7) << 27);  // M / 128
}
__device__ __forceinline__ uint32_t idesc_scale_id(uint32_t id) { return (id << 4) | (id << 29); }   // B, A

// Shared-memory descriptor of 32 rows of 16 bytes of scales (512 contiguous bytes): no swizzle, 8-row core matrices of
// 16-byte rows, 128 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 16) |
         (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

// Word of scales (blocks 4 g .. 4 g + 3) of a row; rows outside the matrix scale by 1.
__device__ __forceinline__ uint32_t scale_word(const uint8_t* s, int pitch, int row, int rows, int g) {
  return row < rows ? __ldg(reinterpret_cast<const uint32_t*>(s + (int64_t)row * pitch) + g) : kUnitScale;
}

// GELU for a bf16 result, on packed pairs: gelu_fast2 with the clamped magnitude as the tail's
// factor too, so that an infinite sum gives infinity (or the tail's last value, 2.6e-10 below 0).
__device__ __forceinline__ void gelu_bf16_2(float& x0, float& x1) {
  using namespace gelu_tail;
  const float a0 = fminf(fabsf(x0), kA), a1 = fminf(fabsf(x1), kA);
  float g0, g1;
  fma2(g0, g1, c7, c7, a0, a1, c6, c6);
  fma2(g0, g1, g0, g1, a0, a1, c5, c5);
  fma2(g0, g1, g0, g1, a0, a1, c4, c4);
  fma2(g0, g1, g0, g1, a0, a1, c3, c3);
  fma2(g0, g1, g0, g1, a0, a1, c2, c2);
  fma2(g0, g1, g0, g1, a0, a1, c1, c1);
  fma2(g0, g1, g0, g1, a0, a1, c0, c0);
  x0 = fmaf(-a0, ex2(g0), x0 < 0.f ? 0.f : x0);   // not fmaxf: NaN stays NaN
  x1 = fmaf(-a1, ex2(g1), x1 < 0.f ? 0.f : x1);
}

// GELU for an fp32 result, on packed pairs: the same form with G of degree 10 from a minimax fit
// over [0, 6]. With fp32's roundings it is within 1.7 * 2^-24 (|x| + |GELU|) of GELU there, and
// ex2 adds 2^-22 of the tail's at most 0.17; beyond 6 both are within 6e-9 of max(x, 0). erff
// takes three times the instructions (23456 x 2384 x 256: 91 us).
__device__ __forceinline__ void gelu_fp32_2(float& x0, float& x1) {
  constexpr float c[11] = {-0.9999997019767761f,     -1.1511183977127075f,    -0.45912185311317444f,
                           -0.052702922374010086f,   0.007291511632502079f,   -0.00025596003979444504f,
                           -0.00016587991558481008f, 4.562117828754708e-05f,  -5.9832109400304034e-06f,
                           4.178519361630606e-07f,   -1.2412963101837704e-08f};
  const float a0 = fminf(fabsf(x0), 16.f), a1 = fminf(fabsf(x1), 16.f);   // G keeps falling up to there
  float g0 = c[10], g1 = c[10];
#pragma unroll
  for (int k = 9; k >= 0; --k) fma2(g0, g1, g0, g1, a0, a1, c[k], c[k]);
  x0 = fmaf(-a0, ex2(g0), x0 < 0.f ? 0.f : x0);
  x1 = fmaf(-a1, ex2(g1), x1 < 0.f ? 0.f : x1);
}

// GELU for an e4m3 result, on packed pairs: max(x, 0) - |x| 2^G(|x|) as gelu_fast2, with
// G = log2 Phi(-a) from a minimax polynomial of degree 5 over [0, 5.5] (relative error of the
// result there at most 2.5e-4, a 250th of half an e4m3 step: of 24000 x 5120 values 0.08% round to
// the neighbour of erff's; degree 7 makes that 0.006% and 137.5 us 140.4). Beyond, the polynomial keeps
// falling, so no clamp is needed: the result is within 1.9e-8 |x| of max(x, 0), as GELU is.
__device__ __forceinline__ void gelu_e4m3_2(float& x0, float& x1) {
  constexpr float c0 = -1.000359058380127f, c1 = -1.1462607383728027f, c2 = -0.4696812331676483f,
                  c3 = -0.04459895193576813f, c4 = 0.004869762342423201f, c5 = -0.00023325053916778415f;
  const float a0 = fabsf(x0), a1 = fabsf(x1);
  float g0, g1;
  fma2(g0, g1, c5, c5, a0, a1, c4, c4);
  fma2(g0, g1, g0, g1, a0, a1, c3, c3);
  fma2(g0, g1, g0, g1, a0, a1, c2, c2);
  fma2(g0, g1, g0, g1, a0, a1, c1, c1);
  fma2(g0, g1, g0, g1, a0, a1, c0, c0);
  x0 = fmaf(-a0, ex2(g0), fmaxf(x0, 0.f));   // NaN stays NaN by its magnitude; an infinity becomes NaN
  x1 = fmaf(-a1, ex2(g1), fmaxf(x1, 0.f));
}

}  // namespace enc
