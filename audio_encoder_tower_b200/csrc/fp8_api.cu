// C entry points of the 8-bit operators (include/enc_fp8.h): checks, tensor maps, launches.
#include <string.h>

#include "../../include/enc_fp8.h"
#include "fp8.cuh"
#include "internal.h"

using namespace enc;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(int32_t t) { return t == ENC_DTYPE_BF16 || t == ENC_DTYPE_FP32; }
// a row-strided [rows, cols] matrix that is read or written four values at a time
bool rows_ok(const void* p, int64_t ld, int32_t cols) {
  return aligned(p, 16) && ld >= cols && ld % 4 == 0;
}

// SMs of the current device; 0: a CUDA error, -1: not an sm_100
int sm_count_current() {
  static DeviceOnce once;
  static int sms[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const bool ready = once.run(dev, [&] {
    int major = 0, minor = 0, n = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return false;
    sms[dev & 63] = major == 10 && minor == 0 ? n : -1;
    return true;
  });
  if (!ready) {
    cudaGetLastError();
    return 0;
  }
  return sms[dev & 63];
}

enc_status device_status(int sms) { return sms > 0 ? ENC_OK : sms < 0 ? ENC_ERR_UNSUPPORTED : ENC_ERR_CUDA; }
enc_status launched(cudaError_t e) {
  if (e == cudaSuccess) return ENC_OK;
  cudaGetLastError();   // the error is the return value, not the next CUDA call's
  return ENC_ERR_CUDA;
}

}  // namespace

extern "C" {

int32_t enc_fp8_scale_pitch(int32_t cols) { return cols < 1 ? 0 : (int32_t)(((int64_t)cols + 511) / 512 * 4); }

enc_status enc_quantize_fp8(const void* x, int32_t x_dtype, int64_t ldx, int32_t rows, int32_t cols, void* q,
                            void* scales, cudaStream_t stream) {
  if (!dtype_ok(x_dtype) || rows < 0 || cols <= 0) return ENC_ERR_INVALID_ARG;
  if (cols % 16 || cols > 65536 || (int64_t)rows * fp8_blocks(cols) >= (1ll << 31) - 4096) return ENC_ERR_UNSUPPORTED;
  if (rows == 0) return ENC_OK;
  if (!x || !q || !scales || !rows_ok(x, ldx, cols) || !aligned(q, 16) || !aligned(scales, 4))
    return ENC_ERR_INVALID_ARG;
  const int sms = sm_count_current();
  if (sms <= 0) return device_status(sms);
  return launched(launch_quantize_fp8(x, x_dtype == ENC_DTYPE_BF16, ldx, rows, cols, reinterpret_cast<uint8_t*>(q),
                                      reinterpret_cast<uint8_t*>(scales), stream));
}

enc_status enc_norm_fp8(int32_t kind, const void* x, int32_t x_dtype, int64_t ldx, const void* delta,
                        int32_t delta_dtype, int64_t ldd, const float* gamma, const float* beta, float eps,
                        int32_t rows, int32_t d, void* x_out, int64_t ldxo, void* q, void* scales,
                        cudaStream_t stream) {
  if ((kind != ENC_NORM_RMS && kind != ENC_NORM_LAYER) || !dtype_ok(x_dtype) || rows < 0 || d <= 0 || !(eps > 0.f))
    return ENC_ERR_INVALID_ARG;
  if (d % 16 || d > 8192) return ENC_ERR_UNSUPPORTED;
  if (rows == 0) return ENC_OK;
  if (!x || !gamma || !q || !scales || !rows_ok(x, ldx, d) || !aligned(q, 16) || !aligned(scales, 4) ||
      !aligned(gamma, 16) || !aligned(beta, 16))
    return ENC_ERR_INVALID_ARG;
  if (delta && (!dtype_ok(delta_dtype) || !rows_ok(delta, ldd, d))) return ENC_ERR_INVALID_ARG;
  if (x_out && (!rows_ok(x_out, ldxo, d) || (x_out == x && ldxo != ldx) || x_out == delta))
    return ENC_ERR_INVALID_ARG;
  const int sms = sm_count_current();
  if (sms <= 0) return device_status(sms);
  return launched(launch_norm_fp8(kind, x, x_dtype == ENC_DTYPE_BF16, ldx, delta, delta_dtype == ENC_DTYPE_BF16, ldd,
                                  gamma, beta, eps, rows, d, x_out, ldxo, reinterpret_cast<uint8_t*>(q),
                                  reinterpret_cast<uint8_t*>(scales), sms, stream));
}

enc_status enc_linear_fp8(const void* A, const void* a_scales, const void* W, const void* w_scales, const float* bias,
                          void* out, void* out_scales, int32_t out_kind, int32_t M, int32_t N, int32_t K,
                          int32_t gelu, int* status, cudaStream_t stream) {
  if (out_kind < ENC_FP8_OUT_BF16 || out_kind > ENC_FP8_OUT_RESID || M < 0 || N <= 0 || K <= 0)
    return ENC_ERR_INVALID_ARG;
  if (gelu && out_kind == ENC_FP8_OUT_RESID) return ENC_ERR_INVALID_ARG;
  // tiles reach past the last row and column by up to 255, and blocks past K by 127: their indexes stay in 32 bits
  if (K % 16 || N % 16 || K > INT32_MAX - 512 || M > INT32_MAX - 512 || N > INT32_MAX - 512 ||
      (int64_t)(M / 256 + 1) * (N / 256 + 1) > INT32_MAX / 2)
    return ENC_ERR_UNSUPPORTED;
  if (M == 0) return ENC_OK;
  if (!A || !a_scales || !W || !w_scales || !out || (out_kind == ENC_FP8_OUT_FP8 && !out_scales))
    return ENC_ERR_INVALID_ARG;
  if (!aligned(A, 16) || !aligned(W, 16) || !aligned(out, 16) || !aligned(bias, 16) || !aligned(a_scales, 4) ||
      !aligned(w_scales, 4))
    return ENC_ERR_INVALID_ARG;
  const int sms = sm_count_current();
  if (sms <= 0) return device_status(sms);
  const GemmFp8SmallPlan small = plan_gemm_fp8_small(M, N, K, sms);
  GemmFp8Maps m;
  if (!make_fp8_operand_map(&m.a, A, M, K, small.tile_m ? small.tile_m : 128) ||
      !make_fp8_operand_map(&m.w, W, N, K, small.tile_m ? 128 : 64) ||
      (!small.tile_m && !make_fp8_out_map(&m.c, out, out_kind, M, N)))
    return ENC_ERR_CUDA;
  GemmFp8Params p;
  memset(&p, 0, sizeof(p));
  p.M = M; p.N = N; p.num_kb = fp8_blocks(K);
  p.a_scales = reinterpret_cast<const uint8_t*>(a_scales);
  p.w_scales = reinterpret_cast<const uint8_t*>(w_scales);
  p.k_pitch = fp8_pitch(K);
  p.bias = bias;
  p.gelu = gelu ? 1 : 0;
  p.out_scales = reinterpret_cast<uint8_t*>(out_scales);
  p.out_pitch = fp8_pitch(N);
  p.status = status;
  if (small.tile_m) return launched(launch_gemm_fp8_small(m.a, m.w, small, p, out, out_kind, stream));
  return launched(launch_gemm_fp8(m, p, out_kind, sms, stream));
}

}  // extern "C"
