// kv8_attention_bf16.cu - the attention kernel for bf16 queries, and fp16 ones with weights in one part.
#include "kv8_attention.cuh"

namespace moe {

cudaError_t launch_attn_bf16(const AttnPlan& p, cudaStream_t st) {
    const bool two = p.g.MT == 2;
    switch (p.a.c.D) {
    case 32: return two ? launch_attn<32, 2, kAttnPlain>(p, st) : launch_attn<32, 1, kAttnPlain>(p, st);
    case 64: return two ? launch_attn<64, 2, kAttnPlain>(p, st) : launch_attn<64, 1, kAttnPlain>(p, st);
    case 96: return two ? launch_attn<96, 2, kAttnPlain>(p, st) : launch_attn<96, 1, kAttnPlain>(p, st);
    case 128: return two ? launch_attn<128, 2, kAttnPlain>(p, st) : launch_attn<128, 1, kAttnPlain>(p, st);
    case 160: return launch_attn<160, 1, kAttnPlain>(p, st);
    case 192: return launch_attn<192, 1, kAttnPlain>(p, st);
    case 224: return launch_attn<224, 1, kAttnPlain>(p, st);
    default: return launch_attn<256, 1, kAttnPlain>(p, st);
    }
}

}  // namespace moe
