/*
 * lora_nt.h -- C ABI of low-rank adapters beside a shared projection on AMD MI355X
 * (gfx950), many requests at once: row m of X has an adapter a = ids[m] of its
 * own, or none,
 *
 *     D[m,n] = sum_k X[m,k] * W[n,k] + s[a] * sum_j u[m,j] * B[a][n,j]
 *     u[m,j] = sum_k X[m,k] * A[a][j,k]
 *
 * (without an adapter the first sum alone).  W is dense in 16 bits or packed as
 * gemm_nt_w4.h lays out.  Storage types, ownership, streams, errors and thread
 * safety are those of gemm_nt_f16.h.
 */
#ifndef LORA_NT_H
#define LORA_NT_H

#include "gemm_nt_w4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_MAX_RANK 256
#define LORA_MAX_LDX 16777215

/*
 * The adapters, all in device memory, read only: A is count x rank x K, B is
 * count x N x rank, both in the 16-bit type of the call and without padding; s
 * holds count fp32 scales, or is NULL: 1 for all.  rank in [1, LORA_MAX_RANK],
 * count >= 0; an adapter of a smaller rank is one whose last rows of A and
 * columns of B are 0.
 */
typedef struct lora_nt_adapters {
    const void *A, *B;
    const float *s;
    int64_t count, rank;
} lora_nt_adapters;

/*
 * X: M rows of K elements, row m at X + m * ldx elements (K <= ldx <= LORA_MAX_LDX);
 * D: M rows of N, row m at D + m * ldd (N <= ldd); ids: M int32, any order, an id
 * outside [0, count) means no adapter.  The same adapter may serve any of the rows.
 * group == 0: W is N x K of the type `dtype` and S and Z are NULL.  group 32, 64 or 128:
 * W, S and Z are a packed weight's Q, S and Z.
 *
 * Sums are held in fp32, u too, and D is rounded once, where the tiles for few rows
 * serve the call.  Where the large ones do, u and the adapters' part of D are rounded to
 * the 16-bit type (u times a power of two, so that it is in range) before the weight's
 * sum is added in fp32 and D is rounded, and a packed weight is unpacked to 16 bits
 * first.  They serve dense rows (ldx == K and ldd == N) of packed weights past
 * GEMM_W4_DIRECT_M rows, and of 16-bit ones
 *   up to 16 rows   with N > 4096 and M * (K rounded up to 128, + 8) * 2 > 66 KB,
 *   from 17 on      with N > 2048 or ceil(M / 32) * ceil(N / 32) > 256, but not up to 32
 *                   rows with K <= 2048.
 * An infinite or NaN value of one adapter, or of a row, changes no other's rows.
 *
 * workspace: device memory of gemm_nt_lora_ws_size bytes or more, 256-byte aligned, any
 * contents; calls that share it must not run at the same time: they go on one stream,
 * or are ordered by events.  Several host threads may make them on that stream, each
 * call's launches are enqueued side by side.
 *
 * Returns GEMM_OK, GEMM_EINVAL (sizes, strides, group or type out of range, a NULL or
 * misaligned pointer to data with at least one element (2 bytes; packed weights 16, ids and
 * s 4), a workspace too small, or D or the workspace overlapping an input or each other)
 * or GEMM_ELAUNCH.  M == 0 or N == 0 is a no-op; K == 0 sets D to +0.
 */
int gemm_nt_lora(const void *X, const void *W, const void *S, const void *Z,
                 const lora_nt_adapters *a, const int32_t *ids, void *D, int64_t M, int64_t N,
                 int64_t K, int64_t ldx, int64_t ldd, int group, int dtype, void *workspace,
                 int64_t ws_bytes, hipStream_t stream);

/* Host-only: bytes of workspace that call needs (0: sizes out of range). */
int64_t gemm_nt_lora_ws_size(int64_t M, int64_t N, int64_t K, int64_t rank, int group);

#ifdef __cplusplus
}
#endif

#endif /* LORA_NT_H */
