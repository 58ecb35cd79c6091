// api_decode.cu - the C ABI of moe_decode.h: host-side argument checks and launches. Nothing here reads device memory or
// allocates.
#include "api_checks.h"
#include "decode_api.h"

using namespace moe;

namespace {

int check_rope(const moe_rope& r, int D, RopeArgs& to) {
    to = RopeArgs{};
    if (!r.turns) return MOE_OK;
    if (r.rot <= 0 || r.rot > D || r.rot % 16 || r.start < 0 || r.start % 8 || r.start > D - r.rot) return MOE_E_SHAPE;
    if (reinterpret_cast<uintptr_t>(r.turns) & 7u) return MOE_E_ALIGN;
    to = RopeArgs{r.turns, r.rot, r.start, r.interleaved != 0, r.factor};
    return MOE_OK;
}

int check_heads(const moe_heads& h, int eb, int64_t n, HeadSet& to) {
    to = HeadSet{};
    if (h.n_heads < 0) return MOE_E_SHAPE;
    if (h.n_heads == 0) return MOE_OK;
    if (h.n_heads > 65535) return MOE_E_CAP;
    if (n > 0 && (!h.x || !h.out)) return MOE_E_NULL;
    to = HeadSet{h.x, h.out, h.weight, h.x_token_stride, h.x_head_stride, h.out_token_stride, h.out_head_stride, h.n_heads, false, false};
    if (off16(h.weight)) return MOE_E_ALIGN;
    const int rc = check_rows(h.x, h.x_token_stride, h.x_head_stride, eb, to.xvec);
    return rc ? rc : check_rows(h.out, h.out_token_stride, h.out_head_stride, eb, to.ovec);
}

}  // namespace

extern "C" {

int moe_head_norm_rope(const moe_head_norm_call* c, cudaStream_t stream) {
    if (!c) return MOE_E_NULL;
    if (!valid_elem(c->type)) return MOE_E_TYPE;
    if (c->n_tokens < 0 || c->n_tokens > 0x7fffffff || c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16) return MOE_E_SHAPE;
    HeadRopeArgs a{};
    const int eb = elem_bytes(c->type);
    int rc = check_heads(c->q, eb, c->n_tokens, a.q);
    if (!rc) rc = check_heads(c->k, eb, c->n_tokens, a.k);
    if (!rc) rc = check_rope(c->rope, c->head_dim, a.r);
    if (rc) return rc;
    if ((a.q.weight || a.k.weight) && !valid_elem(c->w_type)) return MOE_E_TYPE;
    if (c->n_tokens * (static_cast<int64_t>(a.q.n) + a.k.n) > 0x7fffffff) return MOE_E_CAP;
    if (c->n_tokens > 0 && a.r.rot && !c->positions) return MOE_E_NULL;
    if (off4(c->positions)) return MOE_E_ALIGN;
    if (c->n_tokens == 0 || a.q.n + a.k.n == 0) return MOE_OK;
    a.positions = c->positions;
    a.n = c->n_tokens;
    a.D = c->head_dim;
    a.w_type = c->w_type;
    a.eps = c->eps;
    return status(launch_head_norm_rope(a, c->type, stream));
}

int moe_kv8_append(const moe_kv8_append_call* c, cudaStream_t stream) {
    if (!c) return MOE_E_NULL;
    AppendArgs a{};
    int rc = cache_rows(&c->cache, &c->rows, c->cu_tokens, c->start, c->err, a.c, a.kvec, a.vvec);
    if (!rc) rc = check_heads(c->q, elem_bytes(c->rows.type), c->rows.n_tokens, a.q);
    if (!rc) rc = check_rope(c->rope, a.c.D, a.r);
    if (rc) return rc;
    if ((a.q.weight || c->k_weight) && !valid_elem(c->w_type)) return MOE_E_TYPE;
    if (kv8_slots(c->rows.n_tokens, a.c.n_seqs) * (static_cast<int64_t>(a.c.n_kv) + a.q.n) > 0x3fffffff) return MOE_E_CAP;
    if (off16(c->k_weight) || off4(c->positions)) return MOE_E_ALIGN;
    if (c->rows.n_tokens == 0) return MOE_OK;
    a.k = c->rows.k;
    a.v = c->rows.v;
    a.kt = c->rows.k_token_stride;
    a.kh = c->rows.k_head_stride;
    a.vt = c->rows.v_token_stride;
    a.vh = c->rows.v_head_stride;
    a.k_weight = c->k_weight;
    a.cu = c->cu_tokens;
    a.start = c->start;
    a.positions = c->positions;
    a.n_tokens = c->rows.n_tokens;
    a.w_type = c->w_type;
    a.eps = c->eps;
    a.err = c->err;
    return status(launch_kv8_append(a, c->rows.type, stream));
}

int moe_token_logprobs(const moe_logprobs_call* c, cudaStream_t stream) {
    if (!c) return MOE_E_NULL;
    if (!valid_elem(c->type)) return MOE_E_TYPE;
    if (c->rows < 0 || c->vocab <= 0 || c->n_ids < 0 || c->top < 0 || c->top > 32 || c->top > c->vocab || !(c->scale >= 0x1p-100f && c->scale <= 0x1p100f) ||
        (c->rows > 1 && c->row_stride < c->vocab))
        return MOE_E_SHAPE;
    if (static_cast<int64_t>(c->rows) * (c->n_ids > 8 ? c->n_ids : 8) > 0x7fffffff) return MOE_E_CAP;
    if (c->rows == 0) return MOE_OK;
    if (!c->logits || (c->n_ids && (!c->ids || !c->logprobs)) || (c->top && (!c->top_logprobs || !c->top_ids))) return MOE_E_NULL;
    if (reinterpret_cast<uintptr_t>(c->logits) % elem_bytes(c->type) || off4(c->ids, c->logprobs, c->top_logprobs, c->top_ids, c->entropy, c->lse)) return MOE_E_ALIGN;
    LogprobArgs a{};
    a.x = c->logits;
    a.stride = c->row_stride;
    a.rows = c->rows;
    a.V = c->vocab;
    a.n_ids = c->n_ids;
    a.top = c->top;
    a.scale = c->scale;
    a.ids = c->ids;
    a.logprobs = c->logprobs;
    a.top_logprobs = c->top_logprobs;
    a.top_ids = c->top_ids;
    a.entropy = c->entropy;
    a.lse = c->lse;
    return status(launch_token_logprobs(a, c->type, stream));
}

}  // extern "C"
