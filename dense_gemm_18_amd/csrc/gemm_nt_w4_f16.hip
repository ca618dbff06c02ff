// gemm_nt_w4_f16.hip -- the 4-bit weight product's launches with fp16 A and D.
#include "w4_product.h"

void gemm18_w4_f16(const W4Args &a, int group, hipStream_t stream)
{
    launch_w4<false>(a, group, stream);
}
