// gemm_add.h -- D += A * B^T with one rounding: sizes of at least 1, operands as
// gemm_nt_f16's and gemm_nt_bf16's.
#pragma once

#include <hip/hip_runtime.h>

// Not exported from the library.
__attribute__((visibility("hidden"))) void gemm18_add_f16(const void *A, const void *B, void *D,
                                                          int M, int N, int K, hipStream_t s);
__attribute__((visibility("hidden"))) void gemm18_add_bf16(const void *A, const void *B, void *D,
                                                           int M, int N, int K, hipStream_t s);
