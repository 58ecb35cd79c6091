// api_kv8.cu - the C ABI of moe_kv8.h: host-side argument checks and launches. Nothing here reads
// device memory or allocates.
#include "api_checks.h"

using namespace moe;

extern "C" {

int64_t moe_kv8_block_bytes(int head_dim) {
    return head_dim > 0 && head_dim <= 256 && head_dim % 32 == 0 ? kv8_record_bytes(head_dim) : 0;
}

int moe_kv8_write(const moe_kv8_cache* cache, const moe_kv8_rows* rows, const int32_t* cu_tokens, const int32_t* start,
                  int32_t* err, cudaStream_t stream) {
    KvCache k;
    bool kvec, vvec;
    const int rc = cache_rows(cache, rows, cu_tokens, start, err, k, kvec, vvec);
    if (rc || rows->n_tokens == 0) return rc;
    return status(launch_kv8_write(k, *rows, cu_tokens, start, err, kvec, vvec, stream));
}

int moe_kv8_read(const moe_kv8_cache* cache, const moe_kv8_rows* rows, const int32_t* cu_tokens, const int32_t* start,
                 int32_t* err, cudaStream_t stream) {
    KvCache k;
    bool kvec, vvec;
    const int rc = cache_rows(cache, rows, cu_tokens, start, err, k, kvec, vvec);
    if (rc || rows->n_tokens == 0) return rc;
    return status(launch_kv8_read(k, *rows, cu_tokens, start, err, kvec, vvec, stream));
}

int64_t moe_kv8_attention_workspace_bytes(int n_seqs, int T, int n_heads, int n_kv_heads, int head_dim) {
    if (n_seqs <= 0 || T < 1 || T > 32 || n_kv_heads <= 0 || n_heads <= 0 || n_heads % n_kv_heads ||
        moe_kv8_block_bytes(head_dim) == 0)
        return 0;
    return attn_workspace_bytes(n_seqs, T, n_heads, n_kv_heads, head_dim);
}

int moe_kv8_attention(const moe_kv8_attention_call* call, cudaStream_t stream) {
    if (!call) return MOE_E_NULL;
    AttnArgs a{};
    const int rc = check_cache(call->cache, a.c);
    if (rc) return rc;
    if (!call->q || !call->lens || !call->out || !call->workspace) return MOE_E_NULL;
    if (!valid_elem(call->type)) return MOE_E_TYPE;
    if (call->T < 1 || call->T > 32 || call->n_heads <= 0 || call->n_heads % a.c.n_kv || call->window < 0 ||
        (call->depth && !call->tree))
        return MOE_E_SHAPE;
    if (static_cast<int64_t>(a.c.n_seqs) * call->T * call->n_heads > 0x7fffffff) return MOE_E_CAP;
    const int eb = elem_bytes(call->type);
    if (reinterpret_cast<uintptr_t>(call->q) % eb || off16(call->out) || off16(call->workspace) ||
        off4(call->lens, call->tree, call->depth, call->lse, call->err))
        return MOE_E_ALIGN;
    if (call->workspace_bytes < moe_kv8_attention_workspace_bytes(a.c.n_seqs, call->T, call->n_heads, a.c.n_kv, a.c.D))
        return MOE_E_SCRATCH;
    a.q = call->q;
    a.qs = call->q_seq_stride;
    a.qt = call->q_token_stride;
    a.qh = call->q_head_stride;
    a.qvec = !off16(call->q) && a.qs * eb % 16 == 0 && a.qt * eb % 16 == 0 && a.qh * eb % 16 == 0;
    a.T = call->T;
    a.n_heads = call->n_heads;
    a.G = call->n_heads / a.c.n_kv;
    a.lens = call->lens;
    a.tree = call->tree;
    a.window = call->window < kKvNoWindow ? call->window : 0;
    a.depth = a.window > 0 ? call->depth : nullptr;
    a.scale = call->scale;
    a.out = call->out;
    a.lse = call->lse;
    a.workspace = call->workspace;
    a.err = call->err;
    a.test_expire = (call->flags & MOE_F_TEST_EXPIRE) != 0;
    if (!attn_list_fits(a)) return MOE_E_CAP;
    return status(launch_kv8_attention(a, call->type, stream));
}

int moe_add_rms_norm_q8_1(const moe_norm_call* c, cudaStream_t stream) {
    if (!c || !c->x || !c->weight || (!c->sum && !c->y && !c->xq)) return MOE_E_NULL;
    if (!valid_elem(c->type) || !valid_elem(c->w_type)) return MOE_E_TYPE;
    if (c->rows < 0 || c->rows > 0x7fffffff || c->cols <= 0 || c->cols % 32 || c->cols > 32768 ||
        (c->rows > 1 && (c->x_stride < c->cols || (c->residual && c->residual_stride < c->cols))))
        return MOE_E_SHAPE;
    const int eb = elem_bytes(c->type);
    if (off16(c->x) || off16(c->residual) || off16(c->weight) || off16(c->sum) || off16(c->y) ||
        off4(c->xq) || c->x_stride * eb % 16 ||
        (c->residual && c->residual_stride * eb % 16))
        return MOE_E_ALIGN;
    return status(launch_add_rms_norm_q8_1(*c, stream));
}

int moe_dequantize_q8_1(const moe_q8_1* xq, int64_t rows, int64_t cols, void* out, int type, cudaStream_t stream) {
    if (!xq || !out) return MOE_E_NULL;
    if (!valid_elem(type)) return MOE_E_TYPE;
    if (rows < 0 || cols <= 0 || cols % 32 || rows > 0x7fffffff || cols > 0x7fffffff || rows * (cols / 32) > 0x7fffffff)
        return MOE_E_SHAPE;
    if (off4(xq) || off16(out)) return MOE_E_ALIGN;
    return status(launch_dequantize_q8_1(xq, rows * (cols / 32), out, type, stream));
}

}  // extern "C"
