// Row kernels of the 8-bit format: quantisation, and the norm with the residual's
// addition. Both read each input once and write each output once; HBM bounds them.
#include "fp8.cuh"
#include "internal.h"

namespace enc {

namespace {

constexpr int kWarps = 8;

// Four consecutive values of a row.
template <typename T>
__device__ __forceinline__ float4 load4(const T* p) {
  if constexpr (sizeof(T) == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
  } else {
    return *reinterpret_cast<const float4*>(p);
  }
}

// A warp's block of 128 columns (four per lane): scale byte, and the lane's four e4m3.
__device__ __forceinline__ uint32_t quantize_block(const float4& v, uint32_t& byte) {
  const uint32_t m = max(max(finite_abs_bits(v.x), finite_abs_bits(v.y)),
                         max(finite_abs_bits(v.z), finite_abs_bits(v.w)));
  byte = e8m0_of_amax(__reduce_max_sync(0xffffffffu, m));
  return e4m3x4(v.x, v.y, v.z, v.w, e8m0_inverse(byte));
}

// One warp per run of up to kRun blocks of one row: kRun loads in flight per lane.
constexpr int kRun = 8;

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
quantize_fp8_kernel(const T* __restrict__ x, int64_t ldx, int rows, int cols, int runs, uint8_t* __restrict__ q,
                    uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t row = item / runs;
  const int run = static_cast<int>(item - row * runs);
  if (row >= rows) return;
  const int c0 = run * kRun * kFp8Block + 4 * lane;
  const T* xr = x + row * ldx + c0;
  uint8_t* qr = q + row * cols + c0;
  float4 v[kRun];
#pragma unroll
  for (int i = 0; i < kRun; ++i)
    v[i] = c0 + i * kFp8Block < cols ? load4(xr + i * kFp8Block) : make_float4(0.f, 0.f, 0.f, 0.f);
  uint32_t mine = 127;
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    uint32_t byte;
    const uint32_t p = quantize_block(v[i], byte);
    if (c0 + i * kFp8Block < cols) *reinterpret_cast<uint32_t*>(qr + i * kFp8Block) = p;
    if (lane == i && run * kRun + i < fp8_blocks(cols)) mine = byte;
  }
  // kRun is a multiple of four, so the runs cover the padded row of scales exactly
  const int g = run * kRun + lane;
  if (lane < kRun && g < fp8_pitch(cols)) scales[row * fp8_pitch(cols) + g] = static_cast<uint8_t>(mine);
}

// Sum over the WPR warps of a row (each warp's total in, the row's total out).
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* shared, int warp) {
  v = warp_sum(v);
  if constexpr (WPR == 1) return v;
  __syncthreads();   // the previous sum has been read
  if ((threadIdx.x & 31) == 0) shared[warp] = v;
  __syncthreads();
  const int w0 = warp / WPR * WPR;
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < WPR; ++w) s += shared[w0 + w];
  return s;
}

struct NormParams {
  int kind;
  int64_t ldx, ldd, ldxo;
  const void* delta;
  int delta_bf16;
  const float *gamma, *beta;
  float eps;
  int rows, d;
  uint8_t *q, *scales;
};

// WPR warps per row, NV blocks of 128 columns per warp, the row in registers.
template <typename T, int NV, int WPR>
__global__ void __launch_bounds__(kWarps * 32)
norm_fp8_kernel(const T* x, T* x_out, const NormParams p) {
  __shared__ float shared[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row0 = (int64_t)blockIdx.x * (kWarps / WPR) + warp / WPR;
  const bool live = row0 < p.rows;           // all warps stay for the block's barriers
  const int64_t row = live ? row0 : 0;
  const int part = warp % WPR;
  const int c0 = part * NV * kFp8Block + 4 * lane;
  const int d = p.d;
  float4 v[NV];
  const T* xr = x + row * p.ldx + c0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    v[i] = c0 + i * kFp8Block < d ? load4(xr + i * kFp8Block) : make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.delta) {
    float4 t[NV];
    if (p.delta_bf16) {
      const bf16* dr = reinterpret_cast<const bf16*>(p.delta) + row * p.ldd + c0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        t[i] = c0 + i * kFp8Block < d ? load4(dr + i * kFp8Block) : make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
      const float* dr = reinterpret_cast<const float*>(p.delta) + row * p.ldd + c0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        t[i] = c0 + i * kFp8Block < d ? load4(dr + i * kFp8Block) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {   // the stream as it is stored: rounded to its type
      v[i].x = to_float(from_float<T>(v[i].x + t[i].x));
      v[i].y = to_float(from_float<T>(v[i].y + t[i].y));
      v[i].z = to_float(from_float<T>(v[i].z + t[i].z));
      v[i].w = to_float(from_float<T>(v[i].w + t[i].w));
    }
  }
  if (x_out && live) {
    T* xo = x_out + row * p.ldxo + c0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (c0 + i * kFp8Block < d) {
        if constexpr (sizeof(T) == 2)
          *reinterpret_cast<uint2*>(xo + i * kFp8Block) =
              make_uint2(pack_bf16x2(v[i].x, v[i].y), pack_bf16x2(v[i].z, v[i].w));
        else
          *reinterpret_cast<float4*>(xo + i * kFp8Block) = v[i];
      }
  }
  float mean = 0.f;
  if (p.kind == ENC_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) s += (v[i].x + v[i].y) + (v[i].z + v[i].w);
    mean = row_sum<WPR>(s, shared, warp) / d;
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (c0 + i * kFp8Block < d) {
      const float a = v[i].x - mean, b = v[i].y - mean, c = v[i].z - mean, e = v[i].w - mean;
      ss += (a * a + b * b) + (c * c + e * e);
    }
  }
  const float rstd = 1.0f / sqrtf(row_sum<WPR>(ss, shared, warp) / d + p.eps);
  if (!live) return;
  uint8_t* qr = p.q + row * d + c0;
  uint32_t mine = 127;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * kFp8Block;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < d) {
      const float4 g = *reinterpret_cast<const float4*>(p.gamma + c);
      float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p.beta) b = *reinterpret_cast<const float4*>(p.beta + c);
      y = make_float4((v[i].x - mean) * rstd * g.x + b.x, (v[i].y - mean) * rstd * g.y + b.y,
                      (v[i].z - mean) * rstd * g.z + b.z, (v[i].w - mean) * rstd * g.w + b.w);
    }
    uint32_t byte;
    const uint32_t packed = quantize_block(y, byte);
    if (c < d) *reinterpret_cast<uint32_t*>(qr + i * kFp8Block) = packed;
    if (lane == i && part * NV + i < fp8_blocks(d)) mine = byte;
  }
  // the row's last warp also writes the padding of its scales
  const int g = part * NV + lane;
  if ((lane < NV || part == WPR - 1) && g < fp8_pitch(d))
    p.scales[row * fp8_pitch(d) + g] = static_cast<uint8_t>(mine);
}

template <typename T, int NV, int WPR>
cudaError_t launch_norm(const void* x, void* x_out, const NormParams& p, cudaStream_t s) {
  constexpr int rpb = kWarps / WPR;
  norm_fp8_kernel<T, NV, WPR><<<(p.rows + rpb - 1) / rpb, kWarps * 32, 0, s>>>(
      reinterpret_cast<const T*>(x), reinterpret_cast<T*>(x_out), p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_norm_t(const void* x, void* x_out, const NormParams& p, cudaStream_t s) {
  const int g = fp8_blocks(p.d);
  if (g <= 1) return launch_norm<T, 1, 1>(x, x_out, p, s);
  if (g <= 2) return launch_norm<T, 2, 1>(x, x_out, p, s);
  if (g <= 4) return launch_norm<T, 4, 1>(x, x_out, p, s);
  if (g <= 6) return launch_norm<T, 6, 1>(x, x_out, p, s);
  if (g <= 8) return launch_norm<T, 8, 1>(x, x_out, p, s);
  if (g <= 10) return launch_norm<T, 10, 1>(x, x_out, p, s);
  if (g <= 12) return launch_norm<T, 12, 1>(x, x_out, p, s);
  if (g <= 16) return launch_norm<T, 16, 1>(x, x_out, p, s);
  if (g <= 32) return launch_norm<T, 8, 4>(x, x_out, p, s);
  return launch_norm<T, 16, 4>(x, x_out, p, s);
}

}  // namespace

cudaError_t launch_quantize_fp8(const void* x, bool x_bf16, int64_t ldx, int rows, int cols, uint8_t* q,
                                uint8_t* scales, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  const int runs = (fp8_blocks(cols) + kRun - 1) / kRun;
  const int64_t blocks = ((int64_t)rows * runs + kWarps - 1) / kWarps;
  if (x_bf16)
    quantize_fp8_kernel<bf16><<<(unsigned)blocks, kWarps * 32, 0, s>>>(reinterpret_cast<const bf16*>(x), ldx, rows,
                                                                       cols, runs, q, scales);
  else
    quantize_fp8_kernel<float><<<(unsigned)blocks, kWarps * 32, 0, s>>>(reinterpret_cast<const float*>(x), ldx, rows,
                                                                        cols, runs, q, scales);
  return cudaGetLastError();
}

cudaError_t launch_norm_fp8(int kind, const void* x, bool x_bf16, int64_t ldx, const void* delta, bool delta_bf16,
                            int64_t ldd, const float* gamma, const float* beta, float eps, int rows, int d,
                            void* x_out, int64_t ldxo, uint8_t* q, uint8_t* scales, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  const NormParams p{kind, ldx, ldd, ldxo, delta, delta_bf16 ? 1 : 0, gamma, beta, eps, rows, d, q, scales};
  return x_bf16 ? launch_norm_t<bf16>(x, x_out, p, s) : launch_norm_t<float>(x, x_out, p, s);
}

}  // namespace enc
