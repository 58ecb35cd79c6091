// kv8_attention_f32.cu - the attention kernel for fp32 queries.
#include "kv8_attention.cuh"

namespace moe {

cudaError_t launch_attn_f32(const AttnPlan& p, cudaStream_t st) {
    switch (p.a.c.D) {
    case 32: return launch_attn<32, 1, kAttnSplit>(p, st);
    case 64: return launch_attn<64, 1, kAttnSplit>(p, st);
    case 96: return launch_attn<96, 1, kAttnSplit>(p, st);
    case 128: return launch_attn<128, 1, kAttnSplit>(p, st);
    case 160: return launch_attn<160, 1, kAttnSplit>(p, st);
    case 192: return launch_attn<192, 1, kAttnSplit>(p, st);
    case 224: return launch_attn<224, 1, kAttnSplit>(p, st);
    default: return launch_attn<256, 1, kAttnSplit>(p, st);
    }
}

}  // namespace moe
