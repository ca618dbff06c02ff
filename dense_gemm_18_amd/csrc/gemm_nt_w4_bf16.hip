// gemm_nt_w4_bf16.hip -- the 4-bit weight product's launches with bfloat16 A
// and D.
#include "w4_product.h"

void gemm18_w4_bf16(const W4Args &a, int group, hipStream_t stream)
{
    launch_w4<true>(a, group, stream);
}
