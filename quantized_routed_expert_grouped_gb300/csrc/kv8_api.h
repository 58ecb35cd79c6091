// kv8_api.h - launchers of the cache, attention and norm kernels. Internal header.
#pragma once

#include "kv8.cuh"

namespace moe {

cudaError_t launch_kv8_write(const KvCache& c, const moe_kv8_rows& r, const int32_t* cu, const int32_t* start,
                             int32_t* err, bool kvec, bool vvec, cudaStream_t st);
cudaError_t launch_kv8_read(const KvCache& c, const moe_kv8_rows& r, const int32_t* cu, const int32_t* start,
                            int32_t* err, bool kvec, bool vvec, cudaStream_t st);

struct AttnArgs {
    KvCache c;
    const void* q;
    int64_t qs, qt, qh;  // strides in elements: sequence, token, head
    bool qvec;           // 16-byte vectors of queries
    int T, n_heads, G;
    const int32_t* lens;
    const int32_t* tree;
    const int32_t* depth;  // nullptr where it has no effect
    int window;
    float scale;
    void* out;
    float* lse;
    void* workspace;
    int32_t* err;
    int test_expire;  // test hook: 1: each stage waits for an arrival that never comes
};
bool attn_list_fits(const AttnArgs& a);
int64_t attn_workspace_bytes(int n_seqs, int T, int n_heads, int n_kv, int D);
cudaError_t launch_kv8_attention(const AttnArgs& a, int type, cudaStream_t st);

cudaError_t launch_add_rms_norm_q8_1(const moe_norm_call& c, cudaStream_t st);
cudaError_t launch_dequantize_q8_1(const moe_q8_1* xq, int64_t n_blocks, void* out, int type, cudaStream_t st);

}  // namespace moe
