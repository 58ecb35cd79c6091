/* moe_kv8.h - C ABI of the attention side of a decode layer next to the grouped experts (GB300,
 * sm_103a): a paged key/value cache held in 8 bits, attention of a verify window over it, and the
 * residual + norm + q8_1 step that hands the result to the experts. The conventions of
 * moe_grouped.h hold (device pointers, caller-owned buffers, asynchronous on `stream`, negative
 * status codes for what the host can see, MOE_ERR_* bits in *err for bad device-resident data).
 *
 * Element types of dense rows: MOE_F32, MOE_F16, MOE_BF16.
 *
 * The cache. Positions 32j .. 32j+31 of a sequence form a block; a block of one key/value head is
 * one record of moe_kv8_block_bytes(D) = 16 + 64 D bytes (D = head_dim, a multiple of 32, at most
 * 256):
 *   f32 k_scale, f32 v_scale, 8 bytes unused, u8 k[32 D], u8 v[32 D]
 * A code c stands for (c - 128) * scale, 1 <= c <= 255. Keys lie as [4 groups][D/32][8 rows][32
 * dims], token t of the block at group (t >> 1) & 3, row 2 (t >> 3) + (t & 1); values as
 * [D dims][32 tokens]. (A group's rows and the values' tokens are what the lanes of one matrix
 * instruction take, eight contiguous bytes each.) The pool is [n_pages][n_kv_heads]
 * [page_tokens/32] records; page_tokens is a multiple of 32. page_table[b][i] names the page that
 * holds positions i * page_tokens .. of sequence b; entries that no call's range reaches are not
 * read. A page may be shared by sequences that only read it.
 *
 * Numbers. A block's scale is max |x| / 127 over its tokens and dims (fp32, IEEE divide); codes
 * are x * (1 / scale) (fp32) rounded to nearest, ties to even. A block whose max |x| is below
 * 2^-100 is stored with scale 0, as zeros. A block that was given an infinity or a NaN has scale
 * NaN: it reads back as NaN throughout. */
#ifndef MOE_KV8_H
#define MOE_KV8_H

#include "moe_grouped.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- element types */
#define MOE_F32 0
#define MOE_F16 1
#define MOE_BF16 2

/* ---- device-side error bits, OR-ed into *err (next to those of moe_grouped.h) */
#define MOE_ERR_PAGE 256 /* a page id outside [0, n_pages), or a position past the page table (block skipped) */
#define MOE_ERR_LEN 512  /* a negative length or start, or cu_tokens not monotone within [0, n_tokens] (sequence skipped) */

typedef struct moe_kv8_cache {
    void* pool;                /* records, 16-byte aligned */
    int64_t n_pages;
    int32_t n_kv_heads, head_dim, page_tokens;
    const int32_t* page_table; /* [n_seqs][max_pages], rows table_stride apart */
    int64_t table_stride;
    int32_t max_pages, n_seqs;
} moe_kv8_cache;

/* Dense rows of keys and values: element (token i, head h, dim d) of k at
 * i * k_token_stride + h * k_head_stride + d (strides in elements); v likewise. */
typedef struct moe_kv8_rows {
    void *k, *v;
    int32_t type;
    int64_t n_tokens;
    int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride;
} moe_kv8_rows;

/* Bytes of one record (0 if head_dim is not valid). Host only. */
int64_t moe_kv8_block_bytes(int head_dim);

/* Quantise rows into the cache. Rows cu_tokens[b] .. cu_tokens[b+1] (cu_tokens: int32 [n_seqs+1],
 * ascending from 0 to n_tokens) become positions start[b], start[b]+1, .. of sequence b, and the
 * sequence ends with them: what the last block held after them is not kept. Tokens that a first
 * block holds before start[b] are kept; where the new tokens need a larger scale, the block's
 * scale grows and the kept codes are requantised, c' - 128 = rint((c - 128) * (old / new)).
 * (A window whose drafts were rejected is written over from the first rejected position; the
 * block keeps the grown scale, and so its tokens the coarser step, until it is written from its first
 * token on.) Each growth rounds the kept codes once more: a value is off by at most half a step of
 * each scale that its block has had since it was written, 16 steps of the last one at most. (Normal
 * values written a token at a time end 0.37 steps off, rms, windows of four 0.36; quantised at once
 * 0.29.) Writing the same rows again leaves the same bytes. Sequences of one call must
 * not share a block that is written. Alignment: rows 16-byte aligned with strides that keep it are
 * read in vectors, others by element. Errors: MOE_E_NULL, MOE_E_TYPE, MOE_E_SHAPE (head_dim,
 * page_tokens, negative n_tokens), MOE_E_CAP (n_pages, n_seqs, max_pages, n_kv_heads),
 * MOE_E_ALIGN (the pool, rows off their element's boundary, or page_table, cu_tokens, start or err
 * off 4 bytes), MOE_E_CUDA. */
int moe_kv8_write(const moe_kv8_cache* cache, const moe_kv8_rows* rows, const int32_t* cu_tokens,
                  const int32_t* start, int32_t* err, cudaStream_t stream);

/* Read positions start[b] .. of each sequence back into rows cu_tokens[b] .. cu_tokens[b+1] of the
 * dense k and v (rounded to their type). Rows of a skipped sequence or block are not written. */
int moe_kv8_read(const moe_kv8_cache* cache, const moe_kv8_rows* rows, const int32_t* cu_tokens,
                 const int32_t* start, int32_t* err, cudaStream_t stream);

/* Attention of T query tokens per sequence over the cache (which holds the T tokens' own keys and
 * values already). Sequence b holds lens[b] positions; query t sits at position p = lens[b] - T + t
 * and sees position j when 0 <= j < lens[b], p >= 0 and
 *   - without tree: j <= p;  with tree: j < lens[b] - T, or bit j - (lens[b] - T) of tree[b][t] is set;
 *   - window == 0 or j > p - window (a window of 2^31 - 64 or more counts as 0, no limit).
 * In a tree, positions in a path are not those in the window: with depth, the distance that `window`
 * limits is counted from lens[b] - T + depth[b][t] to j, or to lens[b] - T + depth[b][i] for window
 * token i = j - (lens[b] - T). (depth: a token's number of ancestors in the window, at most its index t;
 * one outside [0, t] counts as the nearer end. Each query then sees what it would if its path were
 * decoded token by token.)
 * out[b][t][h] = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), s_j = scale * q[b][t][h] . k_j, over the
 * positions seen, with the key/value head h / (n_heads / n_kv_heads); a query that sees nothing
 * gives zeros. lse[b][t][h] = log sum_j e^(s_j) (-inf where nothing is seen).
 * q, out have type `type`. Products of 16-bit queries with the codes are exact; weights are held in
 * fp16, the largest near 2^10, so that weights down to 2^-34 of it count; sums are fp32 (the matrix
 * instructions' truncate: an output over a long context comes out short by up to 6e-6 of itself). A weight is
 * one fp16 number for bf16, two (its rounding and the rest) for fp32, and for fp16 two where a
 * key/value head has up to 16 rows (T * n_heads / n_kv_heads) or the page tables up to 4096 blocks in
 * all, one otherwise. fp32 queries are two fp16 numbers each. Scores are products of a factor per row with a
 * block's key scale, in fp32: |scale| * max |q| of a row, and that times the key scale, are 0 or from 2^-110
 * to 2^115 (and max |q| itself 0 or 2^-120 at least); smaller ones lose bits, larger ones may give infinities
 * or NaN. A page that cannot be read
 * (MOE_ERR_PAGE) counts as not seen.
 * Limits: 1 <= T <= 32, n_heads a multiple of n_kv_heads; n_seqs * T * n_heads, and n_seqs *
 * n_kv_heads * max_pages * page_tokens / 32 (times the passes over the rows of a key/value head, 32
 * rows each), below 2^31 (MOE_E_CAP). lens may be 0 (nothing seen) and is clamped to the page table
 * (MOE_ERR_PAGE).
 * workspace: moe_kv8_attention_workspace_bytes(...) bytes, 16-byte aligned, of any contents; calls
 * that may run at the same time need one each. out is 16-byte aligned, q on its element's boundary,
 * lens, tree, depth, lse and err on 4 bytes (MOE_E_ALIGN). */
typedef struct moe_kv8_attention_call {
    moe_kv8_cache cache;
    const void* q; /* element (b, t, h, d) at b * q_seq_stride + t * q_token_stride + h * q_head_stride + d */
    int32_t type, T, n_heads;
    int64_t q_seq_stride, q_token_stride, q_head_stride;
    const int32_t* lens; /* [n_seqs] */
    const int32_t* tree; /* [n_seqs][T] bit masks, or NULL */
    int32_t window;      /* 0: no limit */
    float scale;
    void* out;  /* [n_seqs][T][n_heads][head_dim], contiguous */
    float* lse; /* [n_seqs][T][n_heads], or NULL */
    void* workspace;
    int64_t workspace_bytes;
    int32_t* err; /* optional */
    const int32_t* depth; /* [n_seqs][T], or NULL; only with tree (MOE_E_SHAPE) */
    int32_t flags;        /* 0, or MOE_F_TEST_EXPIRE: a test hook, the copies' barriers never complete (MOE_ERR_TIMEOUT
                           * after about a second per ring stage, at most 13; out and lse then hold anything) */
} moe_kv8_attention_call;

int64_t moe_kv8_attention_workspace_bytes(int n_seqs, int T, int n_heads, int n_kv_heads, int head_dim);
int moe_kv8_attention(const moe_kv8_attention_call* call, cudaStream_t stream);

/* Residual addition, root-mean-square norm and q8_1 rows in one pass:
 *   h = x + residual (x where residual is NULL), sum = h rounded to `type`,
 *   y = h * (1 / sqrt(mean(h^2) + eps)) * weight (fp32), y rounded to `type`, xq = q8_1 of the fp32 y.
 * x, residual: [rows][cols], rows x_stride / residual_stride elements apart; weight: [cols] of
 * w_type; sum, y: [rows][cols] contiguous, or NULL; xq: [rows][cols/32], or NULL (one of the three
 * at least). sum may be the residual or x itself, and y may be x, where those are contiguous.
 * cols: a multiple of 32, at most 32768. All pointers 16-byte aligned and strides multiples of 16
 * bytes (MOE_E_ALIGN); xq 4-byte aligned. */
typedef struct moe_norm_call {
    const void *x, *residual, *weight;
    void *sum, *y;
    moe_q8_1* xq;
    int32_t type, w_type;
    int64_t rows, x_stride, residual_stride;
    int32_t cols;
    float eps;
} moe_norm_call;

int moe_add_rms_norm_q8_1(const moe_norm_call* call, cudaStream_t stream);

/* The values that q8_1 rows stand for: out[i] = d * q[i], rounded to `type`. xq: [rows][cols/32],
 * 4-byte aligned; out: [rows][cols] contiguous, 16-byte aligned. */
int moe_dequantize_q8_1(const moe_q8_1* xq, int64_t rows, int64_t cols, void* out, int type,
                        cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_KV8_H */
