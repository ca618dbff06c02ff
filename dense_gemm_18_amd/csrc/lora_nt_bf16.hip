// lora_nt_bf16.hip -- the low-rank adapters' launches in bfloat16.
#include "lora.h"

LoraLaunch gemm18_lora_bf16()
{
    return {lora_shrink<true>, lora_fused<true>, lora_expand<true>};
}
