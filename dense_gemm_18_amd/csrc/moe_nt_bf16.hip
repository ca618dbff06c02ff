// moe_nt_bf16.hip -- the mixture-of-experts layer's launches with bfloat16
// activations.
#include "moe_product.h"

MoeLaunch gemm18_moe_bf16()
{
    return {launch_route<true>, launch_experts<true>};
}
