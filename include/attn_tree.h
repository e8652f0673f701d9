/*
 * attn_tree.h - C ABI of the operators that serve trees of drafted tokens over
 * the cache of attn_cache.h: a step of speculative decoding puts several
 * continuations of a sequence into its cache at once, attends with all of them,
 * and keeps the one path that the model accepts.  Used in this order:
 *   attn_cache_tree_build      masks and positions of the trees, once per step
 *   attn_cache_append_rope     per layer: rotate q and k, keys and values into the cache
 *   attn_cache_tree_fwd        per layer: attention
 *   attn_cache_tree_keep       per layer, once the path is known
 * attn_cache_append_rope serves plain decode steps and prompts too.
 *
 * A tree
 *   The new tokens of a sequence (attn_cache.h) are the nodes of its tree, new
 *   token i in the slot of token seq_lens[b] - n + i.  A node's parent comes
 *   before it; several nodes may have no parent (they follow the last token of
 *   the text).  What node i sees is the text, tokens 0 .. seq_lens[b] - n - 1, and
 *   the nodes that its bits name: bit j % 32 of word j / 32 of its row of
 *   tree_bits stands for node j.  attn_cache_tree_build sets those of the node
 *   and of its ancestors; any other masks serve as well.
 *
 * attn_cache_weights has no tree masks: tokens are weighed for an eviction by
 * queries that see a chain, such as those of plain steps.
 *
 * Conventions are those of attn_cache.h: device pointers owned by the caller,
 * packed batches, no allocation, asynchronous calls, status codes, and what the
 * device finds wrong in the cache's status word, with the sequence left out.
 */
#ifndef ATTN_TREE_H
#define ATTN_TREE_H

#include "attn_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Masks and positions of the trees.
 *   parents      device int32[total_tokens]: the parent's number in its own
 *                sequence, or -1; below the node's own number.  A sequence with
 *                another one is left out and noted in the cache's status word.
 *   tree_bits    device uint32 [total_tokens, tree_words], all words written;
 *                32 * tree_words >= max_new
 *   positions    device int32[total_tokens] or NULL: seq_lens[b] - n + the number
 *                of the node's ancestors, for attn_cache_append_rope and attn_rope.
 *                Where an eviction has shortened the sequence, that is not where it
 *                stands in its text: the caller adds the number of tokens dropped
 *   cu_seqlens, seq_lens, max_new   as for attn_cache_append(); of the cache only
 *                its sizes and status word are used
 * The results overlap neither each other nor the inputs (refused).
 */
ATTN_API attn_status attn_cache_tree_build(const int32_t* parents, int32_t total_tokens,
                                           const int32_t* cu_seqlens, const int32_t* seq_lens,
                                           int32_t max_new, uint32_t* tree_bits,
                                           int32_t tree_words, int32_t* positions,
                                           const attn_kv_cache* cache, attn_stream_t stream);

/*
 * attn_rope() and attn_cache_append() in one: rotate q, and write the rotated
 * keys and the values into the cache.  A rotated key is not rounded on its way: it
 * goes from fp32 to its code at once (attn_rope would round it to bf16 before).
 * Everything else is as those two describe.
 *   q, q_out     [total_tokens, num_heads, head_dim] as for attn_rope(), q_out == q
 *                allowed; NULL with num_heads = 0 (keys and values alone)
 *   k, v, cu_seqlens, seq_lens, max_new   as for attn_cache_append()
 *   dtype        of q, k, v and q_out: bf16 or fp32
 *   positions    device int32[total_tokens], any value; or NULL: new token i of n
 *                stands at seq_lens[b] - n + i (not behind an eviction)
 *   plan         rotary_dim at most the cache's head_dim
 * Rows behind the last sequence and those of a sequence that is left out keep what
 * q_out held.
 */
ATTN_API attn_status attn_cache_append_rope(const void* q, void* q_out, int64_t q_stride,
                                            int64_t q_out_stride, int32_t num_heads,
                                            const void* k, const void* v, int64_t k_stride,
                                            int64_t v_stride, attn_dtype dtype,
                                            int32_t total_tokens, const int32_t* positions,
                                            const int32_t* cu_seqlens, const int32_t* seq_lens,
                                            int32_t max_new, const attn_rope_plan* plan,
                                            const attn_kv_cache* cache, attn_stream_t stream);

/* Bytes of device workspace attn_cache_tree_fwd() needs (0 is possible).  Host only. */
ATTN_API attn_status attn_cache_tree_fwd_workspace_size(const attn_kv_cache* cache,
                                                        int32_t total_tokens, int32_t num_heads,
                                                        int32_t max_new, int32_t max_seqlen,
                                                        size_t* bytes);

/*
 * Attention of the trees' queries over the cache, which holds their keys and values
 * already: attn_cache_fwd() with the visible tokens of each node as above.  A
 * sequence with more new tokens than seq_lens[b] is left out.
 *   tree_bits    device uint32 [total_tokens, tree_words], 32 * tree_words >=
 *                max_new; bits of nodes that the sequence does not have are ignored
 * q, o, lse, scale, bounds and workspace are attn_cache_fwd()'s, and so is what is
 * said there of finite numbers, of empty rows, of repeats and of o being q.  A query
 * enters as the sum of two e4m3 numbers whatever the number of rows: with m the
 * largest magnitude of a row, its elements down to 2^-9 m are exact, and smaller ones
 * are off by 2^-17 m at most.
 * max_new settles which kernel runs and how its rows are padded, for the lengths are
 * the device's alone: a bound near the largest tree is faster than a wide one (64 trees of 4
 * to 8 nodes with 4 query heads a group: 137 us with a bound of 8, 191 with 16, 198 with 64).
 * Above 64 rows (max_new * G) the workspace is 40 MB at a head_dim of 128, whatever the batch.
 */
ATTN_API attn_status attn_cache_tree_fwd(const void* q, void* o, float* lse, attn_dtype dtype,
                                         int32_t total_tokens, int32_t num_heads, float scale,
                                         const uint32_t* tree_bits, int32_t tree_words,
                                         const int32_t* cu_seqlens, int32_t max_new,
                                         const int32_t* seq_lens, int32_t max_seqlen,
                                         const attn_kv_cache* cache, void* workspace,
                                         size_t workspace_bytes, attn_stream_t stream);

/*
 * Keep the accepted path of each tree: node path[b][j] moves to the slot of token
 * seq_lens[b] - n + j, for j < counts[b], and the sequence then holds
 * new_lens[b] = seq_lens[b] - n + counts[b] tokens.  Slots behind them keep their
 * tokens where they are not written.
 *   path         device int32 [batch, path_stride]: ascending numbers of nodes;
 *                entries from counts[b] on are not read.  A sequence whose path is
 *                not ascending or names nodes it does not have is left out.
 *   counts       device int32[batch], 0 <= counts[b] <= n and path_stride
 *   new_lens     device int32[batch]; overlaps none of the inputs (refused)
 *   max_new      at least every sequence's number of new tokens
 * A page that receives tokens from pages with a larger scale takes the largest of
 * them, and all its codes of tokens are re-scaled (rounded only where they fall below
 * the smallest normal number).  Keys stay as they were rotated: a path's nodes stand
 * at the positions that their slots then have.  The pages from the first new token on
 * must belong to the sequence alone.
 */
ATTN_API attn_status attn_cache_tree_keep(const int32_t* path, int32_t path_stride,
                                          const int32_t* counts, const int32_t* cu_seqlens,
                                          const int32_t* seq_lens, int32_t max_new,
                                          int32_t* new_lens,
                                          const attn_kv_cache* cache, attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_TREE_H */
