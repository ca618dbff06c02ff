/*
 * gemm_nt_w4.h -- C ABI of the 4-bit weight operators for AMD MI355X
 * (gfx950): quantisation of a weight matrix to 4 bits with one scale (and
 * zero point) per group along K, its reversal, and the "NT" product with such
 * a weight,
 *
 *     D[m,n] = sum_{k<K} A[m,k] * w[n,k],
 *     w[n,k] = (q[n,k] - z[n,g]) * s[n,g],    g = k / group,
 *
 * with q and z in 0 .. 15.  Storage types, row-major NT layout, ownership,
 * streams, errors and thread safety are those of gemm_nt_f16.h; what differs
 * is said here.
 *
 * Packed weight.  Q: N rows of ceil(K / 128) blocks of 64 bytes, one block
 * for 128 consecutive k.  Element k sits in block k / 128; with
 * j = k % 128 / 32, c = k % 32 / 8 and e = k % 8 it is in the block's 32-bit
 * little-endian word 4 * c + j, in the four bits from bit
 * 4 * (e / 2) + 16 * (e % 2) up.  So 16 consecutive bytes hold what one lane
 * feeds to four consecutive matrix instructions, and the even and odd
 * elements of a pair land in the two halves of a register.  The bits for
 * k >= K are written as 0 and never read for a result.
 * S: N x G scales, G = ceil(K / group), row-major, in the 16-bit type.
 * Z: N x G bytes, row-major, or NULL: every zero point is 8.  Only the low
 * four bits of a byte count.
 * group: 32, 64 or 128; K need not be a multiple of it.
 * dtype: the 16-bit type of A, D, S and W, GEMM_T_F16 or GEMM_T_BF16.
 * Q is 16-byte aligned, A, D, S and W 2-byte aligned.
 */
#ifndef GEMM_NT_W4_H
#define GEMM_NT_W4_H

#include "gemm_nt_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_T_F16 0   /* IEEE binary16 */
#define GEMM_T_BF16 1  /* bfloat16 */

/* Host-only: bytes of Q for an N x K weight (0 for sizes out of range). */
int64_t gemm_w4_packed_bytes(int64_t N, int64_t K);

/*
 * Quantises W (N x K, row n at W + n * ldw elements, ldw >= K) into Q, S
 * and, where Z is not NULL, Z.  Per group, in fp32 with IEEE division:
 *   Z == NULL: s = round16(max|w| / 7), q = clamp(rint(w / s), -8, 7) + 8;
 *   else lo = min(w, 0), hi = max(w, 0) over the group,
 *        s = round16((hi - lo) / 15), z = clamp(rint(-lo / s), 0, 15),
 *        q = clamp(rint(w / s) + z, 0, 15).
 * round16 rounds to the 16-bit type, rint to the nearest even; the divisions
 * by s use the rounded s.  A group whose s rounds to 0 gets q = z = 8.  Where
 * hi - lo passes fp32 (bfloat16 of both signs near its largest), s is
 * infinite, q = z = 0 and the values are NaN: only symmetric groups take all
 * of that type's range.  A group that holds an infinity or a NaN gets s = NaN
 * and q = z = 8, so its products are NaN rather than wrong numbers.
 *
 * Returns GEMM_OK, GEMM_EINVAL (sizes out of range, ldw < K, an unknown group
 * or type, a NULL or misaligned pointer to data with at least one element, or
 * an output that overlaps W or another output) or GEMM_ELAUNCH.
 */
int gemm_w4_quantize(const void *W, void *Q, void *S, void *Z, int64_t N, int64_t K, int64_t ldw,
                     int group, int dtype, hipStream_t stream);

/*
 * W[n,k] = w[n,k] rounded to the 16-bit type (formed in fp32: one rounding),
 * for k < K only; the elements between K and ldw stay as they are.
 * Arguments and errors as gemm_w4_quantize.
 */
int gemm_w4_dequantize(const void *Q, const void *S, const void *Z, void *W, int64_t N, int64_t K,
                       int64_t ldw, int group, int dtype, hipStream_t stream);

/*
 * The product above.  A: M x K, row m at A + m * lda elements (lda >= K);
 * D: M x N, row m at D + m * ldd (ldd >= N), the elements between N and ldd
 * stay as they are.  Sizes as gemm_nt_f16, lda up to GEMM_W4_MAX_LDA, ldd up
 * to 2^40; K == 0 sets D to +0.
 *
 * The sums are held in fp32 and rounded once.  A call with M up to
 * GEMM_W4_DIRECT_M rows, and any call without a workspace, unpacks the
 * weight on its way into the matrix units: there q - z is exact and s
 * multiplies each group's fp32 sum.  Above that, where A and D are dense
 * (lda == K, ldd == N) and the workspace is large enough, the weight is
 * unpacked once into the workspace, rounded to the 16-bit type as
 * gemm_w4_dequantize does, and the 16-bit product reads it there.
 *
 * workspace: device memory of gemm_nt_w4_ws_size(M, N, K) bytes or more,
 * 256-byte aligned, overlapping no operand, or NULL with ws_bytes 0.  Its
 * contents mean nothing between calls; calls that may run at the same time
 * need one each.  Several host threads may share one on a stream: each call's
 * launches are enqueued side by side.
 *
 * Returns GEMM_OK, GEMM_EINVAL (as gemm_nt_f16 and gemm_w4_quantize, lda < K,
 * ldd < N, D overlapping an operand, or a negative ws_bytes, a NULL or
 * misaligned workspace with ws_bytes > 0, or one that overlaps an operand)
 * or GEMM_ELAUNCH.
 */
int gemm_nt_w4(const void *A, const void *Q, const void *S, const void *Z, void *D, int64_t M,
               int64_t N, int64_t K, int64_t lda, int64_t ldd, int group, int dtype,
               void *workspace, int64_t ws_bytes, hipStream_t stream);

#define GEMM_W4_MAX_LDA 16777215

/* Rows up to which gemm_nt_w4 never uses a workspace.  In us, K = 8192 in
 * groups of 128 (32), unpacking on the way and unpacking first, by columns:
 *                16384               8192               4096
 *   256 fp16  112 (133) 179 (176)   57 (67)  77 (77)   30 (40) 41 (44)
 *       bf16  123 (151) 178 (178)   63 (76)  74 (76)   33 (39) 40 (41)
 *   384 fp16  166 (199) 207 (202)   84 (100) 77 (81)   57 (67) 59 (61)
 *       bf16  184 (224) 207 (202)   93 (113) 76 (79)   62 (75) 60 (59)
 *   512 fp16  221 (263) 209 (213)  111 (132) 89 (92)   57 (67) 62 (61)
 *       bf16  244 (298) 209 (206)  123 (150) 83 (89)   63 (76) 61 (61)
 * The rows alone decide, as they decide the rounding above: with 8192 columns
 * unpacking first would win from 320 on, with 4096 and fp16 from about 600. */
#define GEMM_W4_DIRECT_M 384

/* Host-only: bytes of workspace gemm_nt_w4 can use for these sizes with
 * dense A and D (0: none, or sizes out of range). */
int64_t gemm_nt_w4_ws_size(int64_t M, int64_t N, int64_t K);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_NT_W4_H */
