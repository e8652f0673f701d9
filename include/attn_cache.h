/*
 * attn_cache.h - C ABI of the serving operators that stand next to the masked
 * attention of attn_block_mask.h: rotary positions, a paged key / value cache
 * in 8 bits, attention over it, the attention weight its tokens receive, and
 * eviction by that weight.  Used in this order:
 *   attn_rope -> attn_cache_append -> attn_cache_fwd -> attn_cache_weights
 *   -> attn_cache_evict
 * attn_rope also serves training: its inverse is its gradient.
 *
 * The cache
 *   Keys and values are e4m3 numbers (one byte: sign, four exponent bits, three
 *   mantissa bits, largest 448) in pages of page_size tokens.  Every page has
 *   one power-of-two scale for its keys and one for its values per key / value
 *   head: the number a code stands for is code * scale.  With powers of
 *   two a change of a page's scale moves exponents only: re-scaled codes are
 *   rounded only where they fall below the smallest normal e4m3 number.
 *   Sequence b's token j lives in slot j % page_size of page
 *   page_table[b][j / page_size].  The caller owns the lengths and the page
 *   table (a scheduler's state); the library keeps neither.  Sequences may
 *   share pages that are only read; a page that attn_cache_append or
 *   attn_cache_evict writes must belong to one sequence.
 *
 * New tokens
 *   The calls take a packed batch of new tokens, rows cu_seqlens[b] ..
 *   cu_seqlens[b + 1] - 1 for sequence b, and seq_lens[b], the tokens that the
 *   sequence holds with the new ones counted in.  New token i of n stands at
 *   position seq_lens[b] - n + i.  Rows behind cu_seqlens[batch] are neither
 *   read nor written.
 *
 * Heads
 *   num_heads is a multiple of num_kv_heads; query heads [h G, (h + 1) G) read
 *   key / value head h, with G = num_heads / num_kv_heads.
 *
 * Conventions are those of attn_block_mask.h: device pointers owned by the
 * caller, no allocation, asynchronous calls, status codes; what the device
 * finds wrong (malformed cu_seqlens or seq_lens, a page number outside the
 * pool) is recorded in the cache's status word.  The sequence concerned is then
 * left out: its outputs keep what they held.  (A bad page alone leaves out the
 * tokens of that page.)  Nothing traps.
 */
#ifndef ATTN_CACHE_H
#define ATTN_CACHE_H

#include "attn_block_mask.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ rotary positions */

#define ATTN_ROPE_MAX_PAIRS 64

/* How the angles theta_i = base^(-2 i / rotary_dim) are changed for contexts
 * longer than the trained one, s = factor:
 *   NONE    theta_i
 *   LINEAR  theta_i / s                                (interpolated positions)
 *   NTK     the base becomes base * s^(r / (r - 2)), r = rotary_dim
 *   RAMP    theta_i (g + (1 - g) / s), g = clamp((r_i - alpha) / (beta - alpha), 0, 1),
 *           r_i = original_context theta_i / (2 pi) the turns that pair i makes
 *           in the trained context: fast pairs keep their angle, slow ones are
 *           interpolated */
typedef enum attn_rope_scaling {
  ATTN_ROPE_NONE = 0,
  ATTN_ROPE_LINEAR = 1,
  ATTN_ROPE_NTK = 2,
  ATTN_ROPE_RAMP = 3
} attn_rope_scaling;

/* Filled by attn_rope_plan_init(); plain host data. */
typedef struct attn_rope_plan {
  uint32_t magic;
  int32_t rotary_dim;
  int32_t interleaved;
  float result_factor;
  uint64_t turn[ATTN_ROPE_MAX_PAIRS]; /* 2^64 theta_i / (2 pi): the turn one position makes */
} attn_rope_plan;

/*
 * Prepare a rotation (host only, no CUDA call).
 *   rotary_dim     even, 2 .. 128: the leading dimensions of each head that are
 *                  rotated; the others are copied
 *   interleaved    0: pairs (i, i + rotary_dim / 2); 1: pairs (2 i, 2 i + 1)
 *   base           > 1
 *   factor         >= 1; scaling, original_context (> 0), alpha < beta: above
 *                  (read only by the scalings that name them; NTK needs rotary_dim > 2)
 *   result_factor  multiplies the rotated dimensions; 0 means 1, and for RAMP
 *                  0.1 ln(factor) + 1
 */
ATTN_API attn_status attn_rope_plan_init(attn_rope_plan* plan, int32_t rotary_dim,
                                         int32_t interleaved, double base,
                                         attn_rope_scaling scaling, double factor,
                                         double original_context, double alpha, double beta,
                                         double result_factor);

/*
 * Rotate q and k by their positions: each pair (x, y) of the rotated
 * dimensions becomes result_factor (x cos a - y sin a, y cos a + x sin a),
 * a = position * theta_i.  With inverse != 0 the angle is negated, which is the
 * transposed matrix: the gradient of the rotation's input from that of its
 * output.
 *   q, q_out     [total_tokens, num_heads, head_dim]; heads are dense, tokens
 *                q_stride / q_out_stride elements apart.  q_out == q rotates in
 *                place and needs the same stride; no other overlaps.
 *   k, k_out     the same with num_kv_heads; NULL with num_kv_heads = 0
 *   dtype        of all four
 *   head_dim     32, 64 or 128, at least the plan's rotary_dim
 *   positions    device int32[total_tokens], any value; or NULL, and then
 *   cu_seqlens   device int32[batch + 1]: row cu_seqlens[b] + i stands at
 *                position i, or, where seq_lens (device int32[batch]) is given,
 *                at seq_lens[b] - n + i (not for a sequence that an eviction
 *                has shortened).  Rows outside every sequence keep what they
 *                held.
 * The angle is reduced exactly: position times the 64-bit turn fraction of the
 * plan, modulo 2^64, in integers; so far positions lose nothing.  Arithmetic
 * is fp32, rounded once.
 */
ATTN_API attn_status attn_rope(const void* q, void* q_out, int64_t q_stride, int64_t q_out_stride,
                               int32_t num_heads, const void* k, void* k_out, int64_t k_stride,
                               int64_t k_out_stride, int32_t num_kv_heads, attn_dtype dtype,
                               int32_t total_tokens, int32_t head_dim, const int32_t* positions,
                               const int32_t* cu_seqlens, const int32_t* seq_lens, int32_t batch,
                               const attn_rope_plan* plan, int32_t inverse, attn_stream_t stream);

/* ------------------------------------------------------------------ the cache */

typedef struct attn_kv_cache {
  uint8_t* k_pages;          /* e4m3 [num_pages, num_kv_heads, page_size, head_dim], 16-byte aligned */
  uint8_t* v_pages;
  float* k_scale;            /* [num_pages, num_kv_heads], powers of two */
  float* v_scale;
  const int32_t* page_table; /* [batch, max_pages]; entries past a sequence's tokens are not read */
  int32_t* status;           /* one word, zeroed by the caller before the first use */
  int32_t num_pages;
  int32_t num_kv_heads;
  int32_t page_size;         /* 16, 32, 64 or 128 */
  int32_t head_dim;          /* 32, 64 or 128 */
  int32_t batch;
  int32_t max_pages;
} attn_kv_cache;

/*
 * Write a packed batch of new keys and values into the cache.
 *   k, v         device [total_tokens, num_kv_heads, head_dim], heads dense,
 *                tokens k_stride / v_stride elements apart (multiples of 16
 *                bytes); bf16 or fp32
 *   max_new      at least every sequence's number of new tokens
 *   seq_lens     device int32[batch], each at least the sequence's new tokens
 * The scale of a page and head is 2^e with the least e, -80 <= e <= 120, for
 * which the largest finite new value is at most 448 * 2^e.  A page that holds
 * earlier tokens of the sequence keeps its scale if that is larger; otherwise
 * the earlier codes are re-scaled.  Rounding is to nearest even; infinities are
 * stored as +-448 * scale, NaN as NaN.  Slots behind the last token are left
 * as they were.  Appending the same tokens to the same place again stores the
 * same codes.
 */
ATTN_API attn_status attn_cache_append(const void* k, const void* v, int64_t k_stride,
                                       int64_t v_stride, attn_dtype dtype, int32_t total_tokens,
                                       const int32_t* cu_seqlens, const int32_t* seq_lens,
                                       int32_t max_new, const attn_kv_cache* cache,
                                       attn_stream_t stream);

/* Bytes of device workspace attn_cache_fwd() needs (0 is possible).  Host only. */
ATTN_API attn_status attn_cache_fwd_workspace_size(const attn_kv_cache* cache, int32_t total_tokens,
                                                   int32_t num_heads, int32_t max_new,
                                                   int32_t max_seqlen, size_t* bytes);

/*
 * Attention of the new tokens' queries over the cache, which holds their keys
 * and values already:
 *   O[i,h,:] = sum_j softmax_j(scale * q_i . k_j) v_j,  LSE[h,i] as in attn_fwd()
 * over the visible tokens j of the sequence: with ATTN_MASK_CAUSAL those at or
 * before the query's position, with ATTN_MASK_NONE all seq_lens[b].  Other kinds
 * are not supported.  A row that sees no token gets O = 0 and LSE = -inf.
 *   q, o         device bf16 [total_tokens, num_heads, head_dim]
 *   lse          device fp32 [num_heads, total_tokens]
 *   scale        0 means 1/sqrt(head_dim)
 *   max_new      at least every sequence's number of new tokens
 *   max_seqlen   at least every sequence length; at most max_pages * page_size
 *   workspace    256-byte aligned scratch of attn_cache_fwd_workspace_size()
 *                bytes, for this call alone while it runs; NULL if that is 0
 * Cached numbers inside a sequence must be finite, as for attn_bwd(); what
 * lies behind its end may hold anything.  Cached numbers enter the products
 * exactly.  q is scaled by a power of two per row.  Up to 16 rows (max_new * G)
 * it is then fp16: elements down to 2^-17 of their row's largest are exact,
 * smaller ones within 2^-25 of that largest.  With more rows it is the sum of
 * two e4m3 numbers: exact down to 2^-9 of the largest, within 2^-17 of it below.  The weights (times their page's value scale) are
 * rounded to fp16: by 2^-11 of themselves, and below 2^-21 of the row's largest
 * by 2^-32 of that.  Sums are fp32, and LSE does not depend on the values.
 * Repeated calls are bit-identical.  o may be q.
 */
ATTN_API attn_status attn_cache_fwd(const void* q, void* o, float* lse, attn_dtype dtype,
                                    int32_t total_tokens, int32_t num_heads, float scale,
                                    const int32_t* cu_seqlens, int32_t max_new,
                                    const int32_t* seq_lens, int32_t max_seqlen,
                                    attn_mask_kind kind, const attn_kv_cache* cache,
                                    void* workspace, size_t workspace_bytes, attn_stream_t stream);

/*
 * The attention weight that each cached token receives from these queries:
 *   weights[b,h,j] = prev[b,h,j] + sum over the queries i of sequence b and
 *                    the query heads g of key / value head h of
 *                    exp(scale * q_ig . k_j - LSE[g,i])      (visible j only)
 *   q, lse       attn_cache_fwd()'s q and its LSE; kind and scale the same
 *   prev         device fp32 [batch, num_kv_heads, weight_stride] or NULL (0);
 *                prev == weights adds in place
 *   weights      the same shape; weight_stride >= max_seqlen.  Entries at and
 *                behind seq_lens[b] keep what they held.
 * q enters as in attn_cache_fwd(), its second form from more than 24 rows on.
 * Sums are fp32 in a fixed order: repeated calls are bit-identical.
 */
ATTN_API attn_status attn_cache_weights(const void* q, const float* lse, attn_dtype dtype,
                                        int32_t total_tokens, int32_t num_heads, float scale,
                                        const int32_t* cu_seqlens, int32_t max_new,
                                        const int32_t* seq_lens, int32_t max_seqlen,
                                        attn_mask_kind kind, const attn_kv_cache* cache,
                                        const float* prev, float* weights, int64_t weight_stride,
                                        attn_stream_t stream);

/*
 * Shorten sequences to the tokens that received most attention.  Sequence b
 * keeps n_b = min(seq_lens[b], budgets[b]) tokens, chosen for each key / value
 * head by itself: its last min(recent, n_b) tokens and, of the others, those
 * of the largest weights; equal weights go to the lower index, NaN counts as
 * -inf.  (Weights set to -inf name the tokens to drop first.)  The kept tokens
 * are copied in order to slots 0 .. n_b - 1 of dst's pages; a dst page's scale
 * is the largest of its tokens' scales, and codes from pages with smaller ones
 * are re-scaled.
 * Keys stay as they were rotated: n_b is the number of tokens held, no longer a
 * position, so that later tokens are rotated by attn_rope's positions and not by
 * its seq_lens (attn_cache_fwd's causal order is that of the slots, as before).
 *   weights      device fp32 [batch, num_kv_heads, weight_stride], weight_stride >= max_seqlen
 *   budgets      device int32[batch], 0 <= budgets[b]
 *   max_keep     at least every n_b
 *   kept         device int32 [batch, num_kv_heads, max_keep]: the kept
 *                tokens' indices, ascending, then -1
 *   new_weights  device fp32 [batch, num_kv_heads, new_stride], new_stride >=
 *                max_keep: the kept tokens' weights, then 0; not weights itself
 *   new_lens     device int32[batch]: n_b; not seq_lens itself
 *   cache, dst   the same heads, head_dim, page_size and batch; dst's pages of
 *                these sequences are none of the pages that they are read from
 *                (the pools may be one; one table over one pool is refused)
 */
ATTN_API attn_status attn_cache_evict(const float* weights, int64_t weight_stride,
                                      const int32_t* seq_lens, const int32_t* budgets,
                                      int32_t recent, int32_t max_seqlen, int32_t max_keep,
                                      const attn_kv_cache* cache, const attn_kv_cache* dst,
                                      int32_t* kept, float* new_weights, int64_t new_stride,
                                      int32_t* new_lens, attn_stream_t stream);

/*
 * Synchronise `stream`, then report and clear the cache's status word (and any
 * pending CUDA error): ATTN_OK, ATTN_ERR_DEVICE_INVALID_INPUT,
 * ATTN_ERR_DEVICE_TIMEOUT or ATTN_ERR_CUDA.
 */
ATTN_API attn_status attn_cache_get_status(const attn_kv_cache* cache, attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_CACHE_H */
