// gemm_nt_bf16_ex.hip -- the bfloat16 GEMM added to what D holds, for the low-rank
// adapters' entry point.  Kernels, tile choice and launch helpers are in gemm_kernels.h.
#include "gemm_add.h"
#include "gemm_kernels.h"

void gemm18_add_bf16(const void *A, const void *B, void *D, int M, int N, int K, hipStream_t s)
{
    const Epi epi{(const _Float16 *)D, nullptr, 1.0f, 1.0f};
    launch_plain<true, true>(choose_tile(M, N, K), A, B, D, M, N, K, s, epi);
}
