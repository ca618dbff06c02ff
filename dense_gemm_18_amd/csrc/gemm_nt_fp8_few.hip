// gemm_nt_fp8_few.hip -- launches of the FP8 product with row scales for few rows.
#include "fp8_few.h"
#include "gemm_fp8_few.h"

bool gemm18_fp8_few(const Fp8Call &x, hipStream_t stream)
{
    const FewTile t = few_tile(x.A, x.B, x.M, x.N, x.K);
    if (!t.rows)
        return false;
    Fp8FewArgs a{};
    a.A = (const uint16_t *)x.A;
    a.B = (const uint16_t *)x.B;
    a.D = (uint16_t *)x.D;
    a.row = x.row;
    a.col = x.col;
    a.scale = x.scale;
    a.M = (int)x.M;
    a.N = (int)x.N;
    a.K = (int)(x.K / 2);
    a.bf = x.bf;
    switch (x.f8) {
    case 1: launch_few<1>(a, t, stream); break;
    case 2: launch_few<2>(a, t, stream); break;
    case 3: launch_few<3>(a, t, stream); break;
    default: launch_few<4>(a, t, stream); break;
    }
    return true;
}
