// moe_gate.h -- the choice of experts from logits: the kernel's arguments and its
// launch, which the layer's entry points share.
#pragma once

#include "skinny.h"

struct GateArgs {
    const void *logits;            // T rows of E, ldl apart; `parts` of them, summed in order
    const float *bias;
    int32_t *ids;                  // T x topk
    float *weights;                // T x topk
    int64_t T, ldl, part_stride;
    int E, topk, parts, dtype, renorm;
    int sigmoid, groups, kept, group_top;
    float scale;
};

// Not exported from the library.
__attribute__((visibility("hidden"))) void gemm18_moe_gate(const GateArgs &a, hipStream_t stream);
// Whether *g is in range for E experts.
__attribute__((visibility("hidden"))) bool gemm18_moe_gate_ok(const moe_nt_gate *g, int64_t E,
                                                              int topk);
__attribute__((visibility("hidden"))) GateArgs gemm18_moe_gate_args(const moe_nt_gate *g,
                                                                    int flags);
