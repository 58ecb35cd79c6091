/* moe_decode.h - C ABI of the steps that a decode loop takes around the cache, the attention and the
 * experts (GB300, sm_103a): norm and rotation of query and key heads, the same on the way into the 8-bit
 * cache, and the log probabilities that a window's logits give. The conventions of moe_grouped.h hold
 * (device pointers, caller-owned buffers, asynchronous on `stream`, negative status codes for what the host can
 * see, MOE_ERR_* bits in *err for bad device-resident data). */
#ifndef MOE_DECODE_H
#define MOE_DECODE_H

#include "moe_kv8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rotation by position. Dims start .. start + rot of a head are rot / 2 pairs: dims (start + i, start + i + rot / 2),
 * or with interleaved (start + 2 i, start + 2 i + 1). At position p pair i = (a, b) becomes
 *   factor * (a cos t - b sin t, a sin t + b cos t),  t = p * f_i;
 * the other dims stay. turns[i] = round(f_i / (2 pi) * 2^64) mod 2^64, f_i the pair's angle per position (radians): p *
 * turns[i] mod 2^64 is the place on the circle, to 2^-34 of a turn at any 32-bit position, negative
 * ones too (which turn back). rot and the head's dims are multiples of 16, start of 8. */
typedef struct moe_rope {
    const uint64_t* turns; /* [rot / 2], 8-byte aligned; NULL: no rotation (the other fields are not read) */
    int32_t rot, start, interleaved;
    float factor;
} moe_rope;

/* Heads of dense rows, in and out: element (token i, head h, dim d) of x at i * x_token_stride + h * x_head_stride + d
 * (strides in elements), of out likewise. out may be x with the same strides; it must not overlap any row that is read
 * otherwise. Rows 16-byte aligned with strides that keep it are moved in vectors, others by element. */
typedef struct moe_heads {
    const void* x;
    void* out;
    const void* weight; /* [head_dim] of w_type, 16-byte aligned, or NULL: no norm */
    int64_t x_token_stride, x_head_stride, out_token_stride, out_head_stride;
    int32_t n_heads; /* at most 65535; 0: none (the other fields are not read) */
} moe_heads;

/* y = x * (1 / sqrt(mean(x^2) + eps)) * weight over a head's dims (where there is a weight), then the rotation, in
 * fp32 (squares too: they overflow above 1.8e19), rounded once to `type`. Row i is at positions[i], any 32-bit number. Errors:
 * MOE_E_NULL, MOE_E_TYPE, MOE_E_SHAPE (head_dim: a multiple of 16 from 16 to 256; rot, start; negative counts), MOE_E_CAP
 * (more than 65535 heads of a set, n_tokens * heads of 2^31 or more), MOE_E_ALIGN (x and out off their element's boundary, weights off 16 bytes,
 * positions off 4, turns off 8), MOE_E_CUDA. */
typedef struct moe_head_norm_call {
    moe_heads q, k;
    moe_rope rope;
    const int32_t* positions; /* [n_tokens]; may be NULL without rotation */
    int64_t n_tokens;
    int32_t type, w_type, head_dim;
    float eps;
} moe_head_norm_call;

int moe_head_norm_rope(const moe_head_norm_call* call, cudaStream_t stream);

/* moe_kv8_write with keys that are normed (k_weight; NULL: not) and rotated on the way, and the queries of the same tokens
 * beside them. A key's fp32 result is quantised as it is, without a rounding to the rows' type; without norm and
 * rotation the records are moe_kv8_write's. Rotation positions: positions[i] of row i (a draft token may turn by its depth in a
 * tree), or NULL: the row's position in the cache. q: rows of n_tokens tokens like k and v, with q.out as moe_head_norm_rope
 * gives it (q.n_heads 0: none; rows of a sequence that is skipped are not written, those of a block without a page are; q.out must not overlap k or v). The cache, the rows and the lists are as moe_kv8_write
 * takes them, with its errors; MOE_E_CAP also counts the query heads. */
typedef struct moe_kv8_append_call {
    moe_kv8_cache cache;
    moe_kv8_rows rows;
    moe_heads q;
    moe_rope rope;
    const void* k_weight; /* [head_dim] of w_type, 16-byte aligned, or NULL */
    const int32_t *cu_tokens, *start;
    const int32_t* positions; /* [n_tokens], or NULL */
    int32_t w_type;
    float eps;
    int32_t* err; /* optional */
} moe_kv8_append_call;

int moe_kv8_append(const moe_kv8_append_call* call, cudaStream_t stream);

/* Of each row of logits x[0 .. vocab), with p = softmax(scale * x):
 *   logprobs[row][i] = log p[ids[row][i]] (-inf for an id outside [0, vocab)),
 *   top_ids[row][0 .. top): the largest logits' indices in descending order, among equal ones the lower first (-0 equals
 *     0), and top_logprobs[row][..] their log p,
 *   entropy[row] = -sum p log p, lse[row] = log sum e^(scale * x); log p is at most 0 and the entropy at least 0, rounded too.
 * Logits of -inf have p = 0; a row of nothing else gives -inf, entropy 0, and the first indices. A row with a NaN or +inf
 * gives NaN for all but top_ids, in which NaN logits have no place (-1 behind the last). Sums are fp32. logits: rows row_stride
 * elements apart, on their element's boundary; 0 < vocab < 2^31, 0 <= top <= min(32, vocab), scale from 2^-100 to 2^100.
 * entropy and lse may be NULL; logprobs and ids where n_ids is 0, top_* where top is 0. Errors: MOE_E_NULL,
 * MOE_E_TYPE, MOE_E_SHAPE, MOE_E_CAP (rows * max(n_ids, 8) of 2^31 or more), MOE_E_ALIGN, MOE_E_CUDA. */
typedef struct moe_logprobs_call {
    const void* logits;
    int64_t row_stride;
    int32_t type, rows, vocab, n_ids, top;
    float scale;
    const int32_t* ids; /* [rows][n_ids] */
    float* logprobs;    /* [rows][n_ids] */
    float* top_logprobs;
    int32_t* top_ids; /* [rows][top] */
    float *entropy, *lse;
} moe_logprobs_call;

int moe_token_logprobs(const moe_logprobs_call* call, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DECODE_H */
