// lora_nt_f16.hip -- the low-rank adapters' launches in fp16.
#include "lora.h"

LoraLaunch gemm18_lora_f16()
{
    return {lora_shrink<false>, lora_fused<false>, lora_expand<false>};
}
