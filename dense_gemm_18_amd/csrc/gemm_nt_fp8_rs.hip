// gemm_nt_fp8_rs.hip -- launches of the FP8 GEMM with row scales and B in E4M3 (A in
// either format).  Kernels and helpers: gemm_kernels.h, gemm_fp8.h.
#include "gemm_fp8.h"

void gemm18_fp8_launch_rs(int f8, const void *A, const void *B, void *D, int64_t M, int64_t N,
                          int64_t K, const Fp8Scales &scales, hipStream_t s)
{
    if (f8 == 5)
        launch_fp8<5>(A, B, D, M, N, K, scales, s);
    else
        launch_fp8<6>(A, B, D, M, N, K, scales, s);
}
