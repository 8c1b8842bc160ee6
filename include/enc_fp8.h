/*
 * enc_fp8.h -- 8-bit (e4m3) operators of the encoder library: rows of values to
 * e4m3 with a power-of-two scale for each block of 128, a norm with the
 * residual's addition that writes them, and the matrix product that takes them.
 *
 * Same conventions as enc.h and enc_kernels.h: device pointers, row-major,
 * asynchronous on `stream`, nothing traps; host-detectable errors return before
 * any launch. These calls allocate nothing and keep nothing: the caller owns
 * every buffer, and calls on different streams are independent of each other.
 * They can be captured into a graph. A kernel's set-up may overlap the end of the
 * kernel before it in the stream; it touches memory only after that one is done.
 * Every buffer is on the current device, which must be an sm_100.
 * A call with no rows is ENC_OK and launches nothing.
 *
 * The 8-bit format ("e4m3 rows with block scales") of a [rows, cols] matrix:
 *   q       e4m3, [rows, cols], cols a multiple of 16, 16-byte aligned
 *   scales  e8m0 bytes, [rows, enc_fp8_scale_pitch(cols)], 4-byte aligned: byte g of a
 *           row is the scale of columns 128 g .. 128 g + 127 (the last block may be
 *           shorter); the value 2^(byte - 127), and byte 255 is NaN. The bytes past
 *           the last block are written as 127 and never used.
 *   element (r, c) stands for q[r, c] * scales[r, c / 128].
 * The calls below that write the format choose for each block the least scale
 * 2^e, e >= -126, with amax <= 448 * 2^e, amax the largest finite magnitude of the
 * block, and round value / 2^e to e4m3 (nearest, ties to even). A NaN or an
 * infinity becomes e4m3's NaN; the rest of its block is not affected.
 *
 * A power of two as the scale loses at most one bit of the block's range against
 * amax / 448 and no precision inside it (e4m3 is a floating-point format), and it
 * is the form that the tensor cores of sm_100 apply to the operands themselves.
 */
#ifndef AUDIO_ENCODER_TOWER_ENC_FP8_H
#define AUDIO_ENCODER_TOWER_ENC_FP8_H

#include "enc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of one row of a scale matrix: ceil(cols / 128) rounded up to a multiple
 * of four. 0 for cols < 1. Host only. */
ENC_API int32_t enc_fp8_scale_pitch(int32_t cols);

/*
 * Rows to e4m3 with block scales.
 *   x       [rows, cols] of x_dtype (enc_dtype), row stride ldx elements (>= cols);
 *           16-byte aligned, ldx a multiple of 4
 *   cols    a multiple of 16, <= 65536; rows * ceil(cols / 128) below 2^31 - 4096
 * q and scales overlap neither x nor each other.
 */
ENC_API enc_status enc_quantize_fp8(const void *x, int32_t x_dtype, int64_t ldx, int32_t rows, int32_t cols,
                                    void *q, void *scales, cudaStream_t stream);

typedef enum enc_norm_kind {
  ENC_NORM_RMS = 0,   /* y = x / sqrt(mean(x^2) + eps) * gamma + beta */
  ENC_NORM_LAYER = 1  /* y = (x - mean(x)) / sqrt(var(x) + eps) * gamma + beta, biased variance */
} enc_norm_kind;

/*
 * Norm of a residual stream, with the addition of a sub-layer's output, to e4m3
 * with block scales:
 *   x' = x + delta (rounded to x_dtype);  x_out = x';  (q, scales) = norm(x')
 * The norm is that of the stored stream, so one call gives what an addition and
 * a norm of its result give. Statistics and the norm itself are in fp32: the sum of
 * squares must stay within fp32's range (|x'| up to 2e17 at any d). A NaN in a row
 * makes that row NaN, and no other.
 *   x       [rows, d] of x_dtype, row stride ldx
 *   delta   [rows, d] of delta_dtype, row stride ldd, or NULL (x' = x)
 *   gamma   fp32 [d], 16-byte aligned;  beta  fp32 [d] or NULL (zeros)
 *   x_out   [rows, d] of x_dtype, row stride ldxo; may be x itself (with ldxo ==
 *           ldx) and may otherwise not overlap x or delta. NULL: not written.
 *   d       a multiple of 16, <= 8192;  eps > 0
 * Alignment of x, delta and x_out as x of enc_quantize_fp8; q and scales overlap
 * none of the others.
 */
ENC_API enc_status enc_norm_fp8(int32_t kind, const void *x, int32_t x_dtype, int64_t ldx, const void *delta,
                                int32_t delta_dtype, int64_t ldd, const float *gamma, const float *beta, float eps,
                                int32_t rows, int32_t d, void *x_out, int64_t ldxo, void *q, void *scales,
                                cudaStream_t stream);

typedef enum enc_fp8_out {
  ENC_FP8_OUT_BF16 = 0,   /* out: bf16 [M, N] */
  ENC_FP8_OUT_FP32 = 1,   /* out: fp32 [M, N] */
  ENC_FP8_OUT_FP8 = 2,    /* out: e4m3 [M, N] with out_scales */
  ENC_FP8_OUT_RESID = 3   /* out: fp32 [M, N], added to: out += A W^T + bias (no act) */
} enc_fp8_out;

/*
 * Linear layer on e4m3 operands with block scales, fp32 accumulation on the
 * tensor cores:
 *   out[M, N] = act(A[M, K] * W[N, K]^T + bias[N])      (act = GELU when gelu != 0)
 *   A, a_scales   e4m3 rows with block scales, [M, K]
 *   W, w_scales   the same, [N, K]
 *   bias          fp32 [N], 16-byte aligned, or NULL
 *   out           as out_kind says, 16-byte aligned, overlapping none of the others
 *   out_scales    ENC_FP8_OUT_FP8 only, [M, enc_fp8_scale_pitch(N)]
 *   K, N          multiples of 16; at least 16. M, N and K at most 2^31 - 513, at most
 *                 2^30 tiles of 256 x 256
 *   status        device int (may be NULL) set to ENC_ERR_TIMEOUT if a bounded
 *                 wait inside the kernel runs out
 * The order in which an element's products are summed depends on M, N, K and the
 * device's number of SMs alone: on a device the same call gives the same bits every time
 * (ENC_FP8_OUT_RESID as well: every element is added to once). NaN in a row of A or W (an element or a scale) makes that
 * row or column of the output NaN; sums past fp32's range are not finite, and NaN in
 * e4m3, with GELU too. (In bf16 and fp32 GELU takes a sum of minus infinity to its limit,
 * zero.)
 *   GELU is x Phi(x) from a polynomial in |x| and one exponential, before the rounding to
 * the output's type: with fp32 output within 2^-22 (|x| + |GELU|), with bf16 output within 1.1e-5
 * of its value and 2.7e-10, with e4m3 output within 2.5e-4 of its value where |x| <= 5.5 and
 * within 1.9e-8 |x| beyond.
 */
ENC_API enc_status enc_linear_fp8(const void *A, const void *a_scales, const void *W, const void *w_scales,
                                  const float *bias, void *out, void *out_scales, int32_t out_kind, int32_t M,
                                  int32_t N, int32_t K, int32_t gelu, int *status, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* AUDIO_ENCODER_TOWER_ENC_FP8_H */
