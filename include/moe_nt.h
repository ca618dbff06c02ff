/*
 * moe_nt.h -- C ABI of a mixture-of-experts layer for a few tokens on AMD
 * MI355X (gfx950).  For each token x (a row of X, hidden elements):
 *
 *   logits[e] = sum_h x[h] * router[e,h]
 *   p = softmax(logits) over all experts
 *   the topk experts e_0, e_1, ... with the largest logits, in falling order,
 *   equal ones by rising index; w_j = p[e_j], divided by their sum if
 *   MOE_RENORMALIZE is set
 *   h_j = silu(W13[e_j][0:inner] x) * (W13[e_j][inner:2*inner] x)
 *   y = sum_j w_j * W2[e_j] h_j             silu(g) = g / (1 + exp(-g))
 *
 * Every product is an "NT" product with the weight stored output row by
 * output row.  Storage types, ownership, streams, errors and thread safety
 * are those of gemm_nt_f16.h.
 */
#ifndef MOE_NT_H
#define MOE_NT_H

#include "gemm_nt_w4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_TOPK 16
#define MOE_MAX_INNER 1048576
#define MOE_MAX_LDX 16777215
#define MOE_RENORMALIZE 1  /* flag: the chosen weights sum to 1 */

/*
 * The layer's weights, all in device memory, read only:
 *   router: experts x hidden, dense, in the 16-bit type `dtype`;
 *   w13: experts x 2*inner x hidden (gate rows, then up rows);
 *   w2: experts x hidden x inner.
 * group == 0: w13 and w2 are dense in the 16-bit type and the scale and zero
 * pointers are NULL.  group 32, 64 or 128: they are packed weights of
 * experts * 2 * inner and experts * hidden rows as gemm_nt_w4.h lays out, with
 * their scales, and zeros or NULL.
 * experts in [1, MOE_MAX_EXPERTS], hidden in [1, GEMM_MAX_K], inner in
 * [1, MOE_MAX_INNER].
 */
typedef struct moe_nt_weights {
    const void *router;
    const void *w13, *w13_scales, *w13_zeros;
    const void *w2, *w2_scales, *w2_zeros;
    int64_t experts, hidden, inner;
    int32_t group, dtype;
} moe_nt_weights;

/*
 * Router: ids[t*topk + j] (int32) and weights[t*topk + j] (fp32) of the T
 * rows of X, row t at X + t * ldx elements (hidden <= ldx <= MOE_MAX_LDX).
 * The logits are summed in fp32.  A row with a NaN logit, or whose largest is
 * infinite, gets NaN weights and topk distinct valid ids.  topk in
 * [1, min(experts, MOE_MAX_TOPK)].  Of *w the sizes, group, dtype and router
 * have to be valid; w13, w2 and their scales and zeros are not used.
 *
 * workspace: device memory of moe_nt_ws_size(T, w, topk) bytes or more,
 * 256-byte aligned, zero-filled before its first use; every call leaves it
 * ready for the next, whatever its sizes.  Calls that share a workspace must
 * not run at the same time: they go on one stream, or are ordered by events.
 * Several host threads may make them on that stream, each call's launches are
 * enqueued side by side.
 *
 * Returns GEMM_OK, GEMM_EINVAL (a NULL w, sizes, topk, flags or types out of
 * range, ldx or ldd too, a NULL or misaligned pointer to data with at least
 * one element, a workspace too small, or an output that overlaps an input,
 * the workspace or another output) or GEMM_ELAUNCH.  T == 0 is a no-op.
 */
int moe_nt_route(const moe_nt_weights *w, const void *X, int32_t *ids, float *weights, int64_t T,
                 int64_t ldx, int topk, int flags, void *workspace, int64_t ws_bytes,
                 hipStream_t stream);

/*
 * Experts: y of the T rows of X for given ids and weights, into D (row t at
 * D + t * ldd, ldd >= hidden), 16-bit.  An id outside [0, experts) marks a
 * slot that is left out, whatever its weight: a row all of whose slots are
 * left out becomes +0, so a shard of the experts can run with the ids of the
 * others.  An expert may appear more than once in a row.
 *
 * All sums are held in fp32.  h_j is rounded to the 16-bit type (as a layer
 * that stores it between two products does; past the type's range it becomes
 * infinite); y is rounded once, after the weighted sum.  That sum's order is
 * fixed, so results do not depend on timing: over j where a chunk has two or
 * more tokens; for one token over pieces of the products, each times its
 * weight.  Tokens run in chunks of 64, or of 512 / topk where that is less:
 * within a chunk an expert's weights are read once for each 16 of its rows
 * where there are 8 or fewer for each expert on average, else once for each
 * 32.
 *
 * topk in [1, MOE_MAX_TOPK]; router may be NULL.  Workspace and errors as
 * moe_nt_route.
 */
int moe_nt_experts(const moe_nt_weights *w, const void *X, const int32_t *ids,
                   const float *weights, void *D, int64_t T, int64_t ldx, int64_t ldd, int topk,
                   void *workspace, int64_t ws_bytes, hipStream_t stream);

/* moe_nt_route into ids and weights, then moe_nt_experts with them. */
int moe_nt_layer(const moe_nt_weights *w, const void *X, void *D, int32_t *ids, float *weights,
                 int64_t T, int64_t ldx, int64_t ldd, int topk, int flags, void *workspace,
                 int64_t ws_bytes, hipStream_t stream);

/* Host-only: bytes of workspace the calls above need (0: sizes out of range). */
int64_t moe_nt_ws_size(int64_t T, const moe_nt_weights *w, int topk);

#ifdef __cplusplus
}
#endif

#endif /* MOE_NT_H */
