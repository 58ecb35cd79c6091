// api_checks.h - checks of arguments that the C ABIs of moe_kv8.h and moe_decode.h share. Internal header.
#pragma once

#include "internal.h"
#include "kv8_api.h"

namespace moe {

inline bool valid_elem(int t) { return t == MOE_F32 || t == MOE_F16 || t == MOE_BF16; }
inline int elem_bytes(int t) { return t == MOE_F32 ? 4 : 2; }
inline bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
// int32 and fp32 arrays (a null one is aligned)
template <typename... P>
bool off4(const P*... p) { return ((reinterpret_cast<uintptr_t>(p) | ...) & 3u) != 0; }
inline int status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_E_CUDA; }

inline int check_cache(const moe_kv8_cache& c, KvCache& k) {
    if (!c.pool || !c.page_table) return MOE_E_NULL;
    if (moe_kv8_block_bytes(c.head_dim) == 0 || c.page_tokens <= 0 || c.page_tokens % kKvBlock) return MOE_E_SHAPE;
    if (c.n_pages <= 0 || c.n_pages > 0x7fffffff || c.n_kv_heads <= 0 || c.n_kv_heads > 65535 || c.max_pages <= 0 ||
        c.n_seqs <= 0 || c.n_seqs > (1 << 20) || c.table_stride < c.max_pages)
        return MOE_E_CAP;
    // positions are 32-bit: no table past 2^31 - 1 of them is addressable
    if (off16(c.pool) || off4(c.page_table)) return MOE_E_ALIGN;
    k = KvCache{static_cast<uint8_t*>(c.pool), c.page_table, c.table_stride, c.n_pages, c.n_kv_heads, c.head_dim,
                c.page_tokens / kKvBlock, c.max_pages, c.n_seqs, kv8_record_bytes(c.head_dim)};
    return MOE_OK;
}

// dense rows: element alignment is required, 16-byte vectors are used where everything keeps them
inline int check_rows(const void* p, int64_t ts, int64_t hs, int eb, bool& vec) {
    if (reinterpret_cast<uintptr_t>(p) % eb) return MOE_E_ALIGN;
    vec = !off16(p) && ts * eb % 16 == 0 && hs * eb % 16 == 0;
    return MOE_OK;
}

inline int cache_rows(const moe_kv8_cache* cache, const moe_kv8_rows* rows, const int32_t* cu, const int32_t* start,
               const int32_t* err, KvCache& k, bool& kvec, bool& vvec) {
    if (!cache || !rows || !cu || !start) return MOE_E_NULL;
    int rc = check_cache(*cache, k);
    if (rc) return rc;
    if (!valid_elem(rows->type)) return MOE_E_TYPE;
    if (rows->n_tokens < 0 || rows->n_tokens > 0x7fffffff) return MOE_E_SHAPE;
    // one CTA per (block, head)
    if (kv8_slots(rows->n_tokens, cache->n_seqs) * cache->n_kv_heads > 0x3fffffff) return MOE_E_CAP;
    if (rows->n_tokens > 0 && (!rows->k || !rows->v)) return MOE_E_NULL;
    if (off4(cu, start, err)) return MOE_E_ALIGN;
    const int eb = elem_bytes(rows->type);
    rc = check_rows(rows->k, rows->k_token_stride, rows->k_head_stride, eb, kvec);
    return rc ? rc : check_rows(rows->v, rows->v_token_stride, rows->v_head_stride, eb, vvec);
}

}  // namespace moe
