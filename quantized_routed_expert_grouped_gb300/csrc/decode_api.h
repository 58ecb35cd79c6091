// decode_api.h - launchers of the kernels of moe_decode.h. Internal header.
#pragma once

#include "head_rope.cuh"

namespace moe {

struct HeadRopeArgs {
    HeadSet q, k;
    RopeArgs r;
    const int32_t* positions;
    int64_t n;
    int D, w_type;
    float eps;
    int tokens, warps, splits;  // of a CTA; of a token in a CTA; CTAs of a token
};
cudaError_t launch_head_norm_rope(HeadRopeArgs a, int type, cudaStream_t st);

struct AppendArgs {
    KvCache c;
    const void *k, *v;
    int64_t kt, kh, vt, vh;  // strides in elements: token, head
    bool kvec, vvec;
    const void* k_weight;
    HeadSet q;
    RopeArgs r;
    const int32_t *cu, *start, *positions;
    int64_t n_tokens;
    int w_type;
    float eps;
    int32_t* err;
    // of a block: CTAs for keys, for values and for queries, heads of each; its queries' tokens are split over 1 << qshift
    int kparts, kheads, vparts, vheads, qparts, qheads, qshift;
};
cudaError_t launch_kv8_append(AppendArgs a, int type, cudaStream_t st);

struct LogprobArgs {
    const void* x;
    int64_t stride;
    int rows, V, n_ids, top;
    float scale, c;  // c: scale * log2 e
    const int32_t* ids;
    float *logprobs, *top_logprobs;
    int32_t* top_ids;
    float *entropy, *lse;
    int cluster;  // CTAs of a row
};
bool logprobs_short(const LogprobArgs& a, int type);  // whether rows are short enough for the next
cudaError_t launch_token_logprobs_short(const LogprobArgs& a, int type, cudaStream_t st);
cudaError_t launch_token_logprobs(const LogprobArgs& a, int type, cudaStream_t st);

}  // namespace moe
