/*
 * rms_norm.h -- C ABI of the root-mean-square norm with the residual's addition
 * on AMD MI355X (gfx950), into 16 bits or into the 8-bit operands of the FP8
 * products.  For each of T rows of H elements:
 *
 *   s = x + r                                 (s = x without a residual)
 *   y = s / sqrt(mean(s^2) + eps) * w         (w = 1 without weights)
 *
 * s, the sum of its squares and y are held in fp32; y goes by the s that has
 * not been rounded.  Storage types, ownership, streams, errors and thread safety
 * are those of gemm_nt_f16.h; the calls need no workspace.
 */
#ifndef RMS_NORM_H
#define RMS_NORM_H

#include "gemm_nt_w4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * X, R, Y, S: rows of H elements of the 16-bit type `dtype` (GEMM_T_F16 or
 * GEMM_T_BF16), row t at X + t * ldx elements and so on, each stride at least H.
 * W: H elements of that type, or NULL.  R: the residual, or NULL; S: where s goes,
 * rounded (NULL: nowhere; needs R).  An S that fp16 does not hold becomes
 * infinite, without harm to Y.
 *
 * Y or S may be X or R itself (same address, same stride): a row is read before
 * it is written.  Other overlaps of an output with an input or with the other
 * output are refused.  Rows with an infinite or NaN element come out as the
 * formulas say in fp32.  H in [1, GEMM_MAX_K], eps >= 0 and finite.  T == 0 is a
 * no-op.  Returns GEMM_OK, GEMM_EINVAL or GEMM_ELAUNCH.
 */
int rms_norm(const void *X, const void *R, const void *W, void *Y, void *S, int64_t T, int64_t H,
             int64_t ldx, int64_t ldr, int64_t ldy, int64_t lds, float eps, int dtype,
             hipStream_t stream);

/*
 * The same into OCP E4M3 or E5M2 bytes Q (format GEMM_FP8_E4M3 or GEMM_FP8_E5M2;
 * row t at Q + t * ldq bytes): q = y / scale, rounded to the nearest, ties to even,
 * past the largest number (448 or 57344) to that.
 *
 * scales != NULL: each row's own, scale = max|y| / largest, goes into scales[t]
 * (fp32).  A row of zeros has the scale 0 and q = 0; one with an infinite or NaN
 * y has the scale NaN and q = 0.  `scale` is not used.
 * scales == NULL: `scale` (> 0, finite) for every row, as gemm_nt_fp8 takes it;
 * a NaN y becomes a NaN.
 *
 * Q overlaps nothing else; S as above.
 */
int rms_norm_fp8(const void *X, const void *R, const void *W, void *Q, float *scales, void *S,
                 int64_t T, int64_t H, int64_t ldx, int64_t ldr, int64_t ldq, int64_t lds,
                 float eps, float scale, int format, int dtype, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RMS_NORM_H */
