// gemm_nt_bf16_add.hip -- the bfloat16 GEMM added to what D holds, for the low-rank adapters'
// entry point.  Kernels, tile choice and launch helpers are in gemm_kernels.h.
//
// The 256 x 256 tiles spill 15 registers of a lane (59 with three B stages) while D's values
// and the first steps are on their way, none in the K-loop: against the plain product, 7 us at
// 2048 x 8192 x 8192 and 10 at K = 8200, of which reading D is 6.
#include "gemm_add.h"
#include "gemm_kernels.h"

void gemm18_add_bf16(const void *A, const void *B, void *D, int M, int N, int K, hipStream_t s)
{
    launch_plain<false, true, true>(choose_tile(M, N, K), A, B, D, M, N, K, s);
}
