// gemm_fp8_few.h -- what the FP8 entry points hand to the kernels for few rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

struct Fp8Call {
    const void *A, *B;
    void *D;
    int64_t M, N, K;
    float scale;
    const float *col, *row;    // may be null
    bool bf;                   // D's type
    int f8;                    // 1 + fa + 2 * fb, the operands' formats
};

// Launches the product if a tile for few rows is its best; false if not.  Not exported
// from the library.
__attribute__((visibility("hidden"))) bool gemm18_fp8_few(const Fp8Call &x, hipStream_t stream);
