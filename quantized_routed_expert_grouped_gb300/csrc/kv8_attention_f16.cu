// kv8_attention_f16.cu - the attention kernel for fp16 queries, weights in two parts.
#include "kv8_attention.cuh"

namespace moe {

cudaError_t launch_attn_f16(const AttnPlan& p, cudaStream_t st) {
    if (p.prec == kAttnPlain) return launch_attn_bf16(p, st);  // (one kernel for both types)
    switch (p.a.c.D) {
    case 32: return launch_attn<32, 1, kAttnWeights>(p, st);
    case 64: return launch_attn<64, 1, kAttnWeights>(p, st);
    case 96: return launch_attn<96, 1, kAttnWeights>(p, st);
    case 128: return launch_attn<128, 1, kAttnWeights>(p, st);
    case 160: return launch_attn<160, 1, kAttnWeights>(p, st);
    case 192: return launch_attn<192, 1, kAttnWeights>(p, st);
    case 224: return launch_attn<224, 1, kAttnWeights>(p, st);
    default: return launch_attn<256, 1, kAttnWeights>(p, st);
    }
}

}  // namespace moe
