// moe_nt_f16.hip -- the mixture-of-experts layer's launches with fp16
// activations.
#include "moe_product.h"

MoeLaunch gemm18_moe_f16()
{
    return {launch_route<false>, launch_experts<false>};
}
