/*
 * spec_attn: the paged key-value cache and the attention that make a
 * verification step's target rows, for one NVIDIA GB300 (sm_103a).
 *
 * "The target verifies the whole chain in one forward pass" ("Optimizing
 * speculative decoding", section "The draft model moved inside"): per layer,
 * the keys and values of the k+1 new tokens are written to the cache
 * (spec_attn_append) and the new tokens attend over it (spec_attn_chunk).
 * After the verification the rejected tokens are dropped by lowering the
 * sequence's length; nothing in the cache moves.  Prompts run through
 * spec_attn_prompt, and spec_attn_read copies a cached range out.
 *
 * Sequences and positions.  A batch holds n_seqs sequences.  Sequence b has
 * n_b = cu[b+1] - cu[b] new tokens (0 allowed), packed at rows cu[b] ..
 * cu[b+1]-1 of the token tensors, and kv_len[b] tokens in all, the new ones
 * last.  New token i is at position kv_len[b] - n_b + i; position p lives in
 * slot p % page_size of page page_table[b, p / page_size].  A token whose
 * position is negative (kv_len[b] < n_b) has no slot: append skips it, read
 * gives zeros, and its attention row sees nothing.  Slots at or past
 * kv_len[b] are never used, whatever they hold.
 *
 * Pools.  k and v are [num_pages, kv_heads, page_size, head_dim], contiguous,
 * 16-byte aligned; SV_BF16, or SV_E4M3 with k_scale and v_scale
 * [num_pages, kv_heads, page_size] of one byte for each cached vector: the
 * vector is code * 2^(byte - 127).  The exponent is the least e >= -120 with
 * max|x| <= 448 * 2^e, so codes use the format's whole range and the scaling
 * itself rounds nothing; a vector that holds an infinity or NaN is stored as
 * NaN (byte 255) and reads back as NaN; so does any vector of byte 255,
 * whatever its codes.
 *
 * Precision of the attention calls.  Sums, maxima and the products' accumulators
 * are 32 bits wide; the output is rounded once, to bf16.  Inputs of the matrix
 * products are 16 bits wide, so these are rounded before:
 *   - the softmax weights: to bf16 over bf16 keys and values (relative 2^-8; the
 *     sum they are divided by is corrected for the largest weight of every 64
 *     keys), or to a sum of two bf16 (2^-16) for rows of up to 1152 keys, 128
 *     where two row tiles share a CTA; to f16 over an e4m3 pool (2^-11, and
 *     2^-25 of the row's largest contribution, or of its largest weight where
 *     the vectors share a scale: a zero vector that takes nearly all the weight
 *     leaves the others 2^-25 of their size);
 *   - over an e4m3 pool query rows to f16 (2^-11, and 2^-25 of the row's largest
 *     element).  Codes and scales are used as they are, but vectors of scale
 *     2^-112 or less may count as zero.
 * A weight below 2^-126 of its row's largest is 0 (times an infinite value: NaN).
 * Scores scale * q.k reach 2^25 in magnitude over an e4m3 pool and 2^30
 * otherwise; past that weights may leave the range of their type.
 *
 * Conventions are those of spec_verify.h: device pointers, caller's buffers,
 * asynchronous on `cuda_stream`, status codes, argument errors found on the
 * host before any launch, no exception crosses the interface, one handle per
 * stream.  Calls need the device that was current at spec_attn_init to be
 * current (SV_ERR_ARG otherwise; spec_attn_destroy does not).  Token tensors are
 * bf16 with a contiguous last dimension, 16-byte aligned, token and head strides
 * (in elements) multiples of 8; the attention calls refuse (SV_ERR_ARG) strides
 * their copies cannot express, such as 0 over several heads.  n_tokens * q_heads
 * stays below 2^31, n_tokens and every kv_len below 2^31 - 511.  Metadata (cu,
 * kv_len, page_table) is int32 on the device and is checked there: a sequence
 * with a decreasing or out-of-range cu, a kv_len outside [0, max_pages *
 * page_size] or past that limit, or a page outside [0, num_pages) makes no
 * access out of bounds; spec_attn_get_error reports SV_ERR_DATA, append skips
 * the token, and rows of read and of attention that cannot be computed are NaN.
 * Rows outside every sequence's range are not written.
 */
#ifndef SPEC_ATTN_H
#define SPEC_ATTN_H

#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct spec_attn_ctx* spec_attn_t;

/* Element type of a quantised pool (bf16 pools are SV_BF16). */
enum { SV_E4M3 = 2 };

/* A pool of cache pages (see above). */
typedef struct spec_attn_pool {
  void* k;
  void* v;
  uint8_t* k_scale;   /* NULL for SV_BF16 */
  uint8_t* v_scale;
  int32_t dtype;      /* SV_BF16 or SV_E4M3 */
  int32_t num_pages;
  int32_t page_size;  /* 16, 32, 64 or 128 */
} spec_attn_pool;

/* The sequences of one call. */
typedef struct spec_attn_batch {
  const int32_t* cu;          /* [n_seqs + 1] */
  const int32_t* kv_len;      /* [n_seqs] */
  const int32_t* page_table;  /* [n_seqs, max_pages] */
  int32_t n_seqs;
  int32_t n_tokens;           /* rows of the token tensors; cu[n_seqs] <= n_tokens */
  int32_t max_pages;
  int32_t max_kv;             /* no kv_len is above this, as far as the caller knows; 0: max_pages * page_size
                               * stands for it.  Decides only which kernel spec_attn_chunk launches: give it
                               * where page_table is wider than the batch needs.  >= 0 */
} spec_attn_batch;

/* A token tensor [n_tokens, heads, head_dim] of bf16. */
typedef struct spec_attn_rows {
  const void* ptr;
  int64_t token_stride;       /* elements */
  int64_t head_stride;
} spec_attn_rows;

/* Create a handle for q_heads query heads in groups of q_heads / kv_heads per
 * key-value head, head_dim 64 or 128, and batches of up to max_seqs
 * sequences.  Allocates the workspace of the split attention (fixed size,
 * independent of the lengths).  SV_ERR_SIZE for sizes outside the limits:
 * q_heads a multiple of kv_heads, group <= 64, q_heads <= 1024, 1 <= max_seqs
 * <= 65536.  Uses the current CUDA device. */
int spec_attn_init(spec_attn_t* h, int q_heads, int kv_heads, int head_dim, int max_seqs);

/* Write the new tokens' keys and values into the pool, quantising to e4m3
 * where the pool holds that.  One kernel launch. */
int spec_attn_append(spec_attn_t h, const spec_attn_pool* pool, const spec_attn_batch* batch,
                     const spec_attn_rows* k, const spec_attn_rows* v, void* cuda_stream);

/* Copy the batch's tokens (positions kv_len[b] - n_b .. kv_len[b] - 1) out of
 * the pool into k_out and v_out, [n_tokens, kv_heads, head_dim] contiguous
 * bf16, 32-byte aligned (e4m3 values times their power of two, rounded to nearest even where
 * bf16 is not exact: only below its normal range).  One kernel launch. */
int spec_attn_read(spec_attn_t h, const spec_attn_pool* pool, const spec_attn_batch* batch,
                   void* k_out, void* v_out, void* cuda_stream);

/* Attention of the new tokens over the cache, which already holds them (append
 * comes first).  Query head g attends with key-value head g / (q_heads /
 * kv_heads).  Token i of sequence b sees positions 0 .. kv_len[b] - n_b + i
 * (causal != 0) or 0 .. kv_len[b] - 1 (causal == 0: draft steps that attend
 * only to target-written entries pass the length of those; "Optimizing
 * speculative decoding", section "IndexShare and KVShare").
 *   out [n_tokens, q_heads, head_dim] contiguous bf16, 32-byte aligned: sum_j softmax(scale * q.k_j) v_j
 *   lse [n_tokens, q_heads] fp32 or NULL: ln sum_j exp(scale * q.k_j)
 * A row that sees nothing gets out = 0 and lse = -inf.  scale > 0, finite.
 * One kernel launch; single tokens and chunks of any length. */
int spec_attn_chunk(spec_attn_t h, const spec_attn_pool* pool, const spec_attn_batch* batch,
                    const spec_attn_rows* q, int causal, float scale, void* out, float* lse, void* cuda_stream);

/* Causal attention over whole prompts: sequence b's tokens are rows cu[b] ..
 * cu[b+1]-1 of q, k and v, and row i sees rows 0 .. i of its sequence.  No
 * pool is involved; outputs as above.  One kernel launch. */
int spec_attn_prompt(spec_attn_t h, int n_seqs, int n_tokens, const int32_t* cu,
                     const spec_attn_rows* q, const spec_attn_rows* k, const spec_attn_rows* v,
                     float scale, void* out, float* lse, void* cuda_stream);

/* Synchronise the device and report what the kernels flagged since the last
 * call: SV_OK, SV_ERR_DATA, SV_ERR_TIMEOUT or SV_ERR_CUDA.  Clears the flags. */
int spec_attn_get_error(spec_attn_t h);

/* Free the handle and its device memory (NULL is a no-op). */
void spec_attn_destroy(spec_attn_t h);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_ATTN_H */
