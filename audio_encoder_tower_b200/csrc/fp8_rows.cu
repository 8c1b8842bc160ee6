// Row kernels of the 8-bit format: quantisation, and the norm with the residual's
// addition. Both read each input once and write each output once; HBM bounds them.
#include "fp8.cuh"
#include "internal.h"

namespace enc {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// e8m0 of a block and 2^-e of it, from the bits of its amax (see e8m0_of_amax): t carries the
// exponent plus 8 in the place of an fp32 exponent, so that both take one operation more.
__device__ __forceinline__ uint32_t scale_bits(uint32_t amax_bits) {
  return (max(amax_bits, 9u << 23) + 0x1FFFFFu) & 0xFF800000u;
}
__device__ __forceinline__ float inverse_of(uint32_t t) { return __uint_as_float(0x83000000u - t); }
__device__ __forceinline__ uint32_t byte_of(uint32_t t) { return (t >> 23) - 8; }

__device__ __forceinline__ void mul2(float& a, float& b, float s) { enc::mul2(a, b, a, b, s, s); }

constexpr uint32_t kInf = 0x7F800000u;

// ------------------------------------------------------------------ quantisation
// 16 columns per lane, eight lanes per block of 128. The kernel's instructions bound it before
// memory does, so it spends few on each value: 32-byte loads, 16-byte stores, bf16 magnitudes
// compared in pairs, three shuffles and one exponent for 16 values. 48000 x 1280 bf16: four
// columns per lane and a warp per block took 39 us at 85% of the issue slots, this 28.1 (6.6 TB/s).
template <typename T> struct Chunk;
template <> struct Chunk<bf16> {
  uint32_t w[8];
  __device__ __forceinline__ uint32_t amax_bits() const {   // of fp32; NaN and infinity count as what they are
    uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    return max(m << 16, m & 0xFFFF0000u);
  }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
};
template <> struct Chunk<float> {
  uint32_t w[16];
  __device__ __forceinline__ uint32_t amax_bits() const {
    uint32_t m = w[0] & 0x7FFFFFFFu;
#pragma unroll
    for (int i = 1; i < 16; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ float at(int i) const { return __uint_as_float(w[i]); }
};

// kWide: rows are 32-byte aligned; otherwise 8 bytes at a time
template <typename T, bool kWide>
__device__ __forceinline__ void load_chunk(Chunk<T>& c, const T* p) {
  constexpr int n = sizeof(c.w) / 4;
  const uint32_t* s = reinterpret_cast<const uint32_t*>(p);
  if constexpr (kWide) {
#pragma unroll
    for (int i = 0; i < n; i += 8)
      asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(c.w[i]), "=r"(c.w[i + 1]), "=r"(c.w[i + 2]), "=r"(c.w[i + 3]), "=r"(c.w[i + 4]),
                     "=r"(c.w[i + 5]), "=r"(c.w[i + 6]), "=r"(c.w[i + 7])
                   : "l"(s + i)
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < n; i += 2) {
      const uint2 u = *reinterpret_cast<const uint2*>(s + i);
      c.w[i] = u.x;
      c.w[i + 1] = u.y;
    }
  }
}

// Division of numbers below 2^31 by a divisor known at launch.
struct Divider {
  uint32_t magic, shift;
  explicit Divider(uint32_t d) {   // shift = ceil(log2 d), magic = floor(2^32 (2^shift - d) / d) + 1
    shift = 0;
    while ((1ull << shift) < d) ++shift;
    magic = (uint32_t)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(n, magic) + n) >> shift; }
};

constexpr int kUnroll = 2;   // chunks per thread, loaded before the work on either

template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads)
quantize_fp8_kernel(const T* __restrict__ x, int64_t ldx, int rows, int cols, int blocks, const Divider by_blocks,
                    uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  grid_dependency();
  const int sub = threadIdx.x & 7;
  Chunk<T> c[kUnroll] = {};
  uint32_t row[kUnroll];
  int g[kUnroll];
  bool ok[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t b = (blockIdx.x * kUnroll + u) * (kThreads / 8) + (threadIdx.x >> 3);   // block of the matrix
    row[u] = by_blocks(b);
    g[u] = static_cast<int>(b - row[u] * blocks);
    ok[u] = row[u] < static_cast<uint32_t>(rows) && g[u] * kFp8Block + 16 * sub < cols;
    if (ok[u]) load_chunk<T, kWide>(c[u], x + row[u] * ldx + g[u] * kFp8Block + 16 * sub);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    uint32_t m = c[u].amax_bits();
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = c[u].at(i);
    if (__any_sync(0xffffffffu, m >= kInf)) {   // NaN or infinity in the warp: the largest finite magnitude
      m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        m = max(m, finite_abs_bits(y[i]));
        y[i] = fmaf(y[i], 0.f, y[i]);           // an infinity turns into NaN
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    const uint32_t t = scale_bits(m);
    const float inv = inverse_of(t);
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mul2(y[4 * i], y[4 * i + 1], inv);
      mul2(y[4 * i + 2], y[4 * i + 3], inv);
      p[i] = e4m3x4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
    }
    if (ok[u]) {
      *reinterpret_cast<uint4*>(q + (int64_t)row[u] * cols + g[u] * kFp8Block + 16 * sub) =
          make_uint4(p[0], p[1], p[2], p[3]);
    }
    // one byte per block; the row's last block also has the padding written (at most three bytes)
    const int pitch = fp8_pitch(cols);
    if (row[u] < static_cast<uint32_t>(rows) && (sub == 0 || (g[u] + 1 == blocks && g[u] + sub < pitch)))
      scales[(int64_t)row[u] * pitch + g[u] + sub] = static_cast<uint8_t>(sub == 0 ? byte_of(t) : 127u);
  }
}

// -------------------------------------------------------------------------- norm
// Four consecutive values of a row as they are stored (8 bytes of bf16, 16 of fp32), loaded
// past L1. volatile keeps a run of loads together, in front of the work on them.
template <typename T> struct Raw4;
template <> struct Raw4<bf16> { uint2 u; };
template <> struct Raw4<float> { float4 u; };

__device__ __forceinline__ Raw4<bf16> load4(const bf16* p) {
  Raw4<bf16> r;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.u.x), "=r"(r.u.y) : "l"(p) : "memory");
  return r;
}
__device__ __forceinline__ Raw4<float> load4(const float* p) {
  Raw4<float> r;
  asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(r.u.x), "=f"(r.u.y), "=f"(r.u.z), "=f"(r.u.w)
               : "l"(p)
               : "memory");
  return r;
}
__device__ __forceinline__ float4 widen(const Raw4<bf16>& r) {
  return make_float4(__uint_as_float(r.u.x << 16), __uint_as_float(r.u.x & 0xFFFF0000u), __uint_as_float(r.u.y << 16),
                     __uint_as_float(r.u.y & 0xFFFF0000u));
}
__device__ __forceinline__ float4 widen(const Raw4<float>& r) { return r.u; }

// Sum over the WPR warps of a row (each warp's total in, the row's total out).
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* shared, int warp) {
  v = warp_sum(v);
  if constexpr (WPR == 1) return v;
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
  const float *gamma, *beta;
  float eps;
  int rows, d, sm_count;
  uint8_t *q, *scales;
};

template <int kDelta> struct DeltaType { using type = bf16; };
template <> struct DeltaType<2> { using type = float; };

// Blocks per SM that the compiler's own choice of registers allows (126 for NV = 10, 198 for 16):
// it keeps a row's loads together in front, and is the faster form where all rows run at once.
constexpr int own_blocks(int nv) { return 512 / (12 * nv + 10); }
// And with many rows: a row is a chain of latencies (loads, two sums over the warp, a block's maximum
// before its scale), which other rows have to fill. Up to four bytes of input per column as many rows
// as fit without spills, more still where the warps of a row wait for each other. Own choice against
// this (us): 12000 x 1648 bf16 23.9 / 15.9, bf16 + bf16 31.2 / 22.8; 7118 x 4096 fp32 31.0 / 26.1;
// 24000 x 1024 bf16 22.7 / 17.5; 8191 x 4016 bf16 + bf16 40.6 / 41.3; but 1500 x 1280 bf16 3.4 / 3.8.
template <typename T, int kDelta, int NV, int WPR>
constexpr int kManyBlocks = sizeof(T) + (kDelta == 0 ? 0 : kDelta == 1 ? 2 : 4) > 4 ? 512 / (6 * NV + 56)
                            : NV > 12                                                  ? 512 / (4 * NV + 50)
                            : WPR == 4                                                 ? 512 / (4 * NV + 38)
                            : sizeof(T) == 2 && kDelta == 0                            ? 512 / (4 * NV + 32)
                                                                                       : 512 / (4 * NV + 50);

// WPR warps per row, the row in registers: block i * WPR + part of 128 columns is the i-th of
// warp `part`, four columns per lane. One read of each input and one write of each output. With
// six or eight bytes of input and output per column and more memory bounds it (24000 x 1280 fp32 +
// bf16 53 us, 6.4 TB/s; 8191 x 4016 bf16 + bf16 41 us, 5.6), below that the row's latencies (24000 x
// 1280 bf16 22.7 us, 4.1). Only the last kRagged of the NV blocks may lie past the row's end.
// kDelta: 0 none, 1 bf16, 2 fp32.
// kMany: for more rows than run at once with the compiler's choice. (The bound of one block is what
// keeps the loads together: without it 24000 x 1280 fp32 + bf16 took 58 us against 53.6.)
template <typename T, int kDelta, int NV, int WPR, bool kMany>
__global__ void __launch_bounds__(kThreads, kMany ? kManyBlocks<T, kDelta, NV, WPR> : 1)
norm_fp8_kernel(const T* x, T* x_out, const NormParams p) {
  __shared__ float shared[2][kWarps];   // of the two sums
  grid_dependency();
  constexpr int kRagged = 2;
  constexpr int kStep = WPR * kFp8Block;     // columns from one of a warp's blocks to its next
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Without a delta, rows from the last to the first: a product that updated x just before, tiles
  // in ascending order, has left the last rows in L2, and the next product reads the first rows
  // first (the encoder's norms 35.3 -> 33.8 us at 24000 x 1280). With one, upwards.
  const int64_t block = kDelta == 0 ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
  const int64_t row0 = block * (kWarps / WPR) + warp / WPR;
  const bool live = row0 < p.rows;           // all warps stay for the block's barriers
  const int64_t row = live ? row0 : 0;
  const int part = warp % WPR;
  const int c0 = part * kFp8Block + 4 * lane;
  const int d = p.d;
  auto inside = [&](int i) { return i < NV - kRagged || c0 + i * kStep < d; };
  Raw4<T> raw[NV] = {};
  // A warp past the last row reads gamma in the place of its row: all of x may be being written, in place
  const T* xr = (live ? x + row * p.ldx : reinterpret_cast<const T*>(p.gamma)) + c0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (inside(i)) raw[i] = load4(xr + i * kStep);
  float4 v[NV];
  if constexpr (kDelta != 0) {
    using D = typename DeltaType<kDelta>::type;
    Raw4<D> t[NV] = {};
    const D* dr = reinterpret_cast<const D*>(p.delta) + row * p.ldd + c0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (inside(i)) t[i] = load4(dr + i * kStep);
#pragma unroll
    for (int i = 0; i < NV; ++i) {   // the stream as it is stored: rounded to its type
      const float4 a = widen(raw[i]), b = widen(t[i]);
      add2(v[i].x, v[i].y, a.x, a.y, b.x, b.y);
      add2(v[i].z, v[i].w, a.z, a.w, b.z, b.w);
      if constexpr (sizeof(T) == 2) {
        raw[i].u = make_uint2(pack_bf16x2(v[i].x, v[i].y), pack_bf16x2(v[i].z, v[i].w));
        v[i] = widen(raw[i]);
      } else {
        raw[i].u = v[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = widen(raw[i]);
  }
  if (x_out && live) {
    T* xo = x_out + row * p.ldxo + c0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (inside(i)) *reinterpret_cast<decltype(raw[i].u)*>(xo + i * kStep) = raw[i].u;
  }
  if (p.kind == ENC_NORM_LAYER) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      add2(s0, s1, s0, s1, v[i].x, v[i].y);
      add2(s0, s1, s0, s1, v[i].z, v[i].w);
    }
    const float mean = row_sum<WPR>(s0 + s1, shared[0], warp) / d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float m = inside(i) ? -mean : 0.f;   // columns past the end stay zero
      add2(v[i].x, v[i].y, v[i].x, v[i].y, m, m);
      add2(v[i].z, v[i].w, v[i].z, v[i].w, m, m);
    }
  }
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    fma2(s0, s1, v[i].x, v[i].y, v[i].x, v[i].y, s0, s1);
    fma2(s0, s1, v[i].z, v[i].w, v[i].z, v[i].w, s0, s1);
  }
  const float rstd = 1.0f / sqrtf(row_sum<WPR>(s0 + s1, shared[1], warp) / d + p.eps);
  if (!live) return;
  uint8_t* qr = p.q + row * d + c0;
  const float* gr = p.gamma + c0;
  const float* br = p.beta + c0;
  uint32_t mine = 135u << 23, worst = 0;   // 135 << 23: scale byte 127
  // y of block i, and the bits of its amax (fmaxf passes over NaN, which e4m3 keeps by itself)
  auto norm_of = [&](int i) {
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (inside(i)) {
      const float4 g = __ldg(reinterpret_cast<const float4*>(gr + i * kStep));
      y = v[i];
      mul2(y.x, y.y, rstd);
      mul2(y.z, y.w, rstd);
      float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p.beta) b = __ldg(reinterpret_cast<const float4*>(br + i * kStep));
      fma2(y.x, y.y, y.x, y.y, g.x, g.y, b.x, b.y);
      fma2(y.z, y.w, y.z, y.w, g.z, g.w, b.z, b.w);
    }
    return y;
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float4 y = norm_of(i);
    const float top = fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w)));
    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    worst = max(worst, m);
    const uint32_t t = scale_bits(m);
    const float inv = inverse_of(t);
    mul2(y.x, y.y, inv);
    mul2(y.z, y.w, inv);
    if (inside(i)) *reinterpret_cast<uint32_t*>(qr + i * kStep) = e4m3x4(y.x, y.y, y.z, y.w);
    if (lane == i && i * WPR + part < fp8_blocks(d)) mine = t;
  }
  if (worst >= kInf) {   // an infinity somewhere in the row: over again with finite magnitudes
#pragma unroll 1
    for (int i = 0; i < NV; ++i) {
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (k == i) y = norm_of(k);
      const uint32_t t = scale_bits(__reduce_max_sync(
          0xffffffffu, max(max(finite_abs_bits(y.x), finite_abs_bits(y.y)),
                           max(finite_abs_bits(y.z), finite_abs_bits(y.w)))));
      const float inv = inverse_of(t);
      y = make_float4(fmaf(y.x, 0.f, y.x * inv), fmaf(y.y, 0.f, y.y * inv), fmaf(y.z, 0.f, y.z * inv),
                      fmaf(y.w, 0.f, y.w * inv));
      if (c0 + i * kStep < d) *reinterpret_cast<uint32_t*>(qr + i * kStep) = e4m3x4(y.x, y.y, y.z, y.w);
      if (lane == i && i * WPR + part < fp8_blocks(d)) mine = t;
    }
  }
  // scales, and the padding: bytes i * WPR + part below the pitch
  const int g = lane * WPR + part;
  if (g < fp8_pitch(d)) p.scales[row * fp8_pitch(d) + g] = static_cast<uint8_t>(byte_of(mine));
}

template <typename T, int kDelta, int NV, int WPR>
cudaError_t launch_norm(const void* x, void* x_out, const NormParams& p, cudaStream_t s) {
  constexpr int rpb = kWarps / WPR;
  const unsigned grid = (unsigned)(((int64_t)p.rows + rpb - 1) / rpb);
  if constexpr (kManyBlocks<T, kDelta, NV, WPR> > own_blocks(NV)) {
    if (grid > (unsigned)(p.sm_count * own_blocks(NV)))
      return launch_overlapped(norm_fp8_kernel<T, kDelta, NV, WPR, true>, grid, kThreads, 0, 1, s,
                               reinterpret_cast<const T*>(x), reinterpret_cast<T*>(x_out), p);
  }
  return launch_overlapped(norm_fp8_kernel<T, kDelta, NV, WPR, false>, grid, kThreads, 0, 1, s,
                           reinterpret_cast<const T*>(x), reinterpret_cast<T*>(x_out), p);
}

// A warp per row up to 16 blocks of 128 columns, four from there on (the registers hold 16
// blocks per warp); NV is at most one block per warp above what the row needs.
template <typename T, int kDelta>
cudaError_t launch_norm_d(const void* x, void* x_out, const NormParams& p, cudaStream_t s) {
  const int g = fp8_blocks(p.d);
#define ENC_NORM_CASE(NV, WPR) if (g <= NV * WPR) return launch_norm<T, kDelta, NV, WPR>(x, x_out, p, s)
  ENC_NORM_CASE(1, 1); ENC_NORM_CASE(2, 1); ENC_NORM_CASE(4, 1); ENC_NORM_CASE(6, 1); ENC_NORM_CASE(8, 1);
  ENC_NORM_CASE(10, 1); ENC_NORM_CASE(12, 1); ENC_NORM_CASE(14, 1); ENC_NORM_CASE(16, 1);
  ENC_NORM_CASE(6, 4); ENC_NORM_CASE(8, 4); ENC_NORM_CASE(10, 4); ENC_NORM_CASE(12, 4); ENC_NORM_CASE(14, 4);
  ENC_NORM_CASE(16, 4);
#undef ENC_NORM_CASE
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_norm_t(const void* x, void* x_out, const NormParams& p, bool delta_bf16, cudaStream_t s) {
  if (!p.delta) return launch_norm_d<T, 0>(x, x_out, p, s);
  return delta_bf16 ? launch_norm_d<T, 1>(x, x_out, p, s) : launch_norm_d<T, 2>(x, x_out, p, s);
}

template <typename T>
cudaError_t launch_quantize_t(const void* x, int64_t ldx, int rows, int cols, uint8_t* q, uint8_t* scales,
                              cudaStream_t s) {
  const int blocks = fp8_blocks(cols);
  const int64_t per = kUnroll * (kThreads / 8), grid = ((int64_t)rows * blocks + per - 1) / per;
  if (grid * per >= 1ll << 31) return cudaErrorInvalidValue;   // Divider's range; the caller checks
  const T* p = reinterpret_cast<const T*>(x);
  const bool wide = reinterpret_cast<uintptr_t>(x) % 32 == 0 && ldx * sizeof(T) % 32 == 0;
  const auto kernel = wide ? quantize_fp8_kernel<T, true> : quantize_fp8_kernel<T, false>;
  return launch_overlapped(kernel, (unsigned)grid, kThreads, 0, 1, s, p, ldx, rows, cols, blocks, Divider(blocks), q, scales);
}

}  // namespace

cudaError_t launch_quantize_fp8(const void* x, bool x_bf16, int64_t ldx, int rows, int cols, uint8_t* q,
                                uint8_t* scales, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  return x_bf16 ? launch_quantize_t<bf16>(x, ldx, rows, cols, q, scales, s)
                : launch_quantize_t<float>(x, ldx, rows, cols, q, scales, s);
}

cudaError_t launch_norm_fp8(int kind, const void* x, bool x_bf16, int64_t ldx, const void* delta, bool delta_bf16,
                            int64_t ldd, const float* gamma, const float* beta, float eps, int rows, int d,
                            void* x_out, int64_t ldxo, uint8_t* q, uint8_t* scales, int sm_count, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  const NormParams p{kind, ldx, ldd, ldxo, delta, gamma, beta, eps, rows, d, sm_count, q, scales};
  return x_bf16 ? launch_norm_t<bf16>(x, x_out, p, delta_bf16, s) : launch_norm_t<float>(x, x_out, p, delta_bf16, s);
}

}  // namespace enc
