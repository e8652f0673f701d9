// C ABI of the rotary and cache operators (include/attn_cache.h, include/attn_tree.h):
// argument checks and dispatch.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <utility>

#include "cache.cuh"

namespace attnmask {
namespace {

constexpr double kPi = 3.14159265358979323846;
// Launches put the batch on a grid's y or z axis, heads on y (two per head).
constexpr int kMaxBatch = 65535, kMaxHeads = 32767;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Arrays of m and n 32-bit numbers that share some.
bool overlap(const void* a, int64_t m, const void* b, int64_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && m > 0 && n > 0 && x < y + uintptr_t(n) * 4 && y < x + uintptr_t(m) * 4;
}

// The cache's own fields, and the view the kernels take.
attn_status check_cache(const attn_kv_cache* c, CacheView* v) {
  if (c == nullptr || !c->k_pages || !c->v_pages || !c->k_scale || !c->v_scale || !c->page_table || !c->status)
    return ATTN_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->num_kv_heads < 1 || c->batch < 1 || c->max_pages < 1) return ATTN_ERR_INVALID_ARG;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return ATTN_ERR_UNSUPPORTED;
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128) return ATTN_ERR_UNSUPPORTED;
  if (c->batch > kMaxBatch || c->num_kv_heads > kMaxHeads) return ATTN_ERR_UNSUPPORTED;
  if (int64_t(c->max_pages) * c->page_size > (int64_t(1) << 30)) return ATTN_ERR_UNSUPPORTED;
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(c->page_table, 4) || !aligned(c->status, 4))
    return ATTN_ERR_INVALID_ARG;
  v->k_pages = c->k_pages;
  v->v_pages = c->v_pages;
  v->k_scale = c->k_scale;
  v->v_scale = c->v_scale;
  v->table = c->page_table;
  v->status = c->status;
  v->num_pages = c->num_pages;
  v->heads = c->num_kv_heads;
  v->page_log2 = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  v->head_dim = c->head_dim;
  v->batch = c->batch;
  v->max_pages = c->max_pages;
  return ATTN_OK;
}

// Sizes that the attention, its workspace and the weights share.
attn_status check_sizes(const attn_kv_cache* c, int32_t total_tokens, int32_t num_heads, int32_t max_new,
                        int32_t max_seqlen) {
  if (total_tokens < 0 || num_heads < 1 || max_new < 0 || max_seqlen < 0) return ATTN_ERR_INVALID_ARG;
  if (num_heads % c->num_kv_heads != 0) return ATTN_ERR_INVALID_ARG;
  if (int64_t(max_seqlen) > int64_t(c->max_pages) * c->page_size) return ATTN_ERR_INVALID_ARG;
  // rows of one sequence and of the call, units of 64 tokens and a launch's blocks fit 31 bits
  if (int64_t(total_tokens) * num_heads > (int64_t(1) << 30) || int64_t(max_new) * num_heads > (int64_t(1) << 30))
    return ATTN_ERR_UNSUPPORTED;
  if (int64_t(c->batch) * c->num_kv_heads * (int64_t(max_seqlen) / 64 + 1) > INT_MAX) return ATTN_ERR_UNSUPPORTED;
  const int64_t tiles = (int64_t(max_new) * (num_heads / c->num_kv_heads) + 15) / 16;
  if (tiles * ((int64_t(max_seqlen) + 255) / 256) > (int64_t(1) << 30)) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// What the appends check alike; fills `a`.
attn_status check_append(const void* k, const void* v, int64_t k_stride, int64_t v_stride, attn_dtype dtype,
                         int32_t total_tokens, const int32_t* cu_seqlens, const int32_t* seq_lens, int32_t max_new,
                         const attn_kv_cache* cache, AppendArgs* a) {
  if (!cu_seqlens || !seq_lens || total_tokens < 0 || max_new < 0) return ATTN_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!k || !v)) return ATTN_ERR_INVALID_ARG;
  const attn_status st = check_cache(cache, &a->cache);
  if (st != ATTN_OK) return st;
  if (dtype != ATTN_DTYPE_BF16 && dtype != ATTN_DTYPE_FP32) return ATTN_ERR_INVALID_ARG;
  const int64_t size = dtype == ATTN_DTYPE_BF16 ? 2 : 4;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cu_seqlens, 4) || !aligned(seq_lens, 4)) return ATTN_ERR_INVALID_ARG;
  if (total_tokens > 1) {
    const int64_t need = int64_t(cache->num_kv_heads) * cache->head_dim;
    if (k_stride < need || v_stride < need || (k_stride * size) % 16 != 0 || (v_stride * size) % 16 != 0)
      return ATTN_ERR_INVALID_ARG;
  }
  a->k = k;
  a->v = v;
  a->k_stride = k_stride;
  a->v_stride = v_stride;
  a->total_tokens = total_tokens;
  a->max_new = max_new < total_tokens ? max_new : total_tokens;
  a->cu = cu_seqlens;
  a->lens = seq_lens;
  a->bf16 = dtype == ATTN_DTYPE_BF16;
  return ATTN_OK;
}

// What the attention and the weights check alike; fills `a`.
attn_status check_queries(const void* q, const float* lse, attn_dtype dtype, int32_t total_tokens, int32_t num_heads,
                          float scale, const int32_t* cu_seqlens, int32_t max_new, const int32_t* seq_lens,
                          int32_t max_seqlen, attn_mask_kind kind, const attn_kv_cache* cache, CacheQueryArgs* a) {
  if (!cu_seqlens || !seq_lens || (total_tokens > 0 && (!q || !lse))) return ATTN_ERR_INVALID_ARG;
  attn_status st = check_cache(cache, &a->cache);
  if (st != ATTN_OK) return st;
  if (!std::isfinite(scale) || scale < 0.f) return ATTN_ERR_INVALID_ARG;
  if (dtype != ATTN_DTYPE_BF16 && dtype != ATTN_DTYPE_FP32) return ATTN_ERR_INVALID_ARG;
  if (dtype != ATTN_DTYPE_BF16) return ATTN_ERR_UNSUPPORTED;
  if (kind < ATTN_MASK_CAUSAL || kind > ATTN_MASK_DENSE) return ATTN_ERR_INVALID_ARG;
  if (kind != ATTN_MASK_CAUSAL && kind != ATTN_MASK_NONE) return ATTN_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(lse, 4) || !aligned(cu_seqlens, 4) || !aligned(seq_lens, 4))
    return ATTN_ERR_INVALID_ARG;
  st = check_sizes(cache, total_tokens, num_heads, max_new, max_seqlen);
  if (st != ATTN_OK) return st;
  a->q = q;
  a->total_tokens = total_tokens;
  a->num_heads = num_heads;
  a->max_new = max_new < total_tokens ? max_new : total_tokens;
  a->max_seqlen = max_seqlen;
  a->scale = scale > 0.f ? scale : 1.0f / std::sqrt(float(cache->head_dim));
  a->causal = kind == ATTN_MASK_CAUSAL;
  a->cu = cu_seqlens;
  a->lens = seq_lens;
  return ATTN_OK;
}

}  // namespace
}  // namespace attnmask

using namespace attnmask;

extern "C" {

attn_status attn_rope_plan_init(attn_rope_plan* plan, int32_t rotary_dim, int32_t interleaved, double base,
                                attn_rope_scaling scaling, double factor, double original_context, double alpha,
                                double beta, double result_factor) {
  if (plan == nullptr) return ATTN_ERR_INVALID_ARG;
  if (rotary_dim < 2 || rotary_dim % 2 != 0) return ATTN_ERR_INVALID_ARG;
  if (rotary_dim > 2 * ATTN_ROPE_MAX_PAIRS) return ATTN_ERR_UNSUPPORTED;
  if (!(base > 1.0) || !std::isfinite(base)) return ATTN_ERR_INVALID_ARG;
  if (scaling < ATTN_ROPE_NONE || scaling > ATTN_ROPE_RAMP) return ATTN_ERR_INVALID_ARG;
  if (scaling != ATTN_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return ATTN_ERR_INVALID_ARG;
  if (scaling == ATTN_ROPE_NTK && rotary_dim == 2) return ATTN_ERR_INVALID_ARG;
  if (scaling == ATTN_ROPE_RAMP &&
      (!(original_context > 0.0) || !std::isfinite(original_context) || !(alpha < beta) || !std::isfinite(alpha) ||
       !std::isfinite(beta)))
    return ATTN_ERR_INVALID_ARG;
  if (!(result_factor >= 0.0) || !std::isfinite(result_factor)) return ATTN_ERR_INVALID_ARG;

  attn_rope_plan p;
  std::memset(&p, 0, sizeof(p));
  p.magic = kRopeMagic;
  p.rotary_dim = rotary_dim;
  p.interleaved = interleaved != 0;
  if (result_factor == 0.0) result_factor = scaling == ATTN_ROPE_RAMP ? 0.1 * std::log(factor) + 1.0 : 1.0;
  p.result_factor = float(result_factor);
  const double r = rotary_dim;
  if (scaling == ATTN_ROPE_NTK) base *= std::pow(factor, r / (r - 2.0));
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double theta = std::pow(base, -2.0 * i / r);
    if (scaling == ATTN_ROPE_LINEAR) theta /= factor;
    if (scaling == ATTN_ROPE_RAMP) {
      double g = (original_context * theta / (2.0 * kPi) - alpha) / (beta - alpha);
      g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
      theta *= g + (1.0 - g) / factor;
    }
    // theta <= 1, so the turn is below 2^62
    p.turn[i] = uint64_t(std::ldexp(theta / (2.0 * kPi), 64));
  }
  *plan = p;
  return ATTN_OK;
}

attn_status attn_rope(const void* q, void* q_out, int64_t q_stride, int64_t q_out_stride, int32_t num_heads,
                      const void* k, void* k_out, int64_t k_stride, int64_t k_out_stride, int32_t num_kv_heads,
                      attn_dtype dtype, int32_t total_tokens, int32_t head_dim, const int32_t* positions,
                      const int32_t* cu_seqlens, const int32_t* seq_lens, int32_t batch, const attn_rope_plan* plan,
                      int32_t inverse, attn_stream_t stream) {
  if (!plan || num_heads < 1 || num_kv_heads < 0 || total_tokens < 0) return ATTN_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!q || !q_out || (num_kv_heads > 0 && (!k || !k_out)))) return ATTN_ERR_INVALID_ARG;
  if (plan->magic != kRopeMagic) return ATTN_ERR_INVALID_ARG;
  if (dtype != ATTN_DTYPE_BF16 && dtype != ATTN_DTYPE_FP32) return ATTN_ERR_INVALID_ARG;
  if (head_dim != 32 && head_dim != 64 && head_dim != 128) return ATTN_ERR_UNSUPPORTED;
  if (plan->rotary_dim > head_dim) return ATTN_ERR_INVALID_ARG;
  if (num_heads > kMaxHeads || num_kv_heads > kMaxHeads) return ATTN_ERR_UNSUPPORTED;
  if (total_tokens > 0 && positions == nullptr && (cu_seqlens == nullptr || batch < 1)) return ATTN_ERR_INVALID_ARG;
  const uintptr_t size = dtype == ATTN_DTYPE_BF16 ? 2 : 4;
  for (const void* p : {q, static_cast<const void*>(q_out), num_kv_heads ? k : nullptr,
                        static_cast<const void*>(num_kv_heads ? k_out : nullptr)})
    if (!aligned(p, size)) return ATTN_ERR_INVALID_ARG;
  for (const int32_t* p : {positions, cu_seqlens, seq_lens})
    if (!aligned(p, 4)) return ATTN_ERR_INVALID_ARG;
  // tokens must not overlap; one token alone needs no stride
  const int64_t need_q = int64_t(num_heads) * head_dim, need_k = int64_t(num_kv_heads) * head_dim;
  if (total_tokens > 1 && (q_stride < need_q || q_out_stride < need_q)) return ATTN_ERR_INVALID_ARG;
  if (total_tokens > 1 && num_kv_heads > 0 && (k_stride < need_k || k_out_stride < need_k)) return ATTN_ERR_INVALID_ARG;
  // in place, a token's row must be its own
  if (total_tokens > 1 && ((q == q_out && q_stride != q_out_stride) ||
                           (num_kv_heads > 0 && k == k_out && k_stride != k_out_stride)))
    return ATTN_ERR_INVALID_ARG;
  if (total_tokens == 0) return ATTN_OK;
  RopeArgs a;
  a.q = q;
  a.q_out = q_out;
  a.k = k;
  a.k_out = k_out;
  a.q_stride = q_stride;
  a.q_out_stride = q_out_stride;
  a.k_stride = k_stride;
  a.k_out_stride = k_out_stride;
  a.num_heads = num_heads;
  a.num_kv_heads = num_kv_heads;
  a.total_tokens = total_tokens;
  a.head_dim = head_dim;
  a.batch = batch;
  a.positions = positions;
  a.cu = cu_seqlens;
  a.lens = seq_lens;
  a.inverse = inverse != 0;
  a.bf16 = dtype == ATTN_DTYPE_BF16;
  return launch_rope(a, *plan, reinterpret_cast<cudaStream_t>(stream));
}

attn_status attn_cache_append(const void* k, const void* v, int64_t k_stride, int64_t v_stride, attn_dtype dtype,
                              int32_t total_tokens, const int32_t* cu_seqlens, const int32_t* seq_lens,
                              int32_t max_new, const attn_kv_cache* cache, attn_stream_t stream) {
  AppendArgs a;
  const attn_status st =
      check_append(k, v, k_stride, v_stride, dtype, total_tokens, cu_seqlens, seq_lens, max_new, cache, &a);
  if (st != ATTN_OK) return st;
  if (total_tokens == 0 || max_new == 0) return ATTN_OK;
  return launch_cache_append(a, reinterpret_cast<cudaStream_t>(stream));
}

attn_status attn_cache_fwd_workspace_size(const attn_kv_cache* cache, int32_t total_tokens, int32_t num_heads,
                                          int32_t max_new, int32_t max_seqlen, size_t* bytes) {
  if (bytes == nullptr) return ATTN_ERR_INVALID_ARG;
  CacheView v;
  attn_status st = check_cache(cache, &v);
  if (st == ATTN_OK) st = check_sizes(cache, total_tokens, num_heads, max_new, max_seqlen);
  if (st != ATTN_OK) return st;
  *bytes = size_t(cache_fwd_workspace(v, total_tokens, num_heads, max_new < total_tokens ? max_new : total_tokens,
                                      max_seqlen));
  return ATTN_OK;
}

attn_status attn_cache_fwd(const void* q, void* o, float* lse, attn_dtype dtype, int32_t total_tokens,
                           int32_t num_heads, float scale, const int32_t* cu_seqlens, int32_t max_new,
                           const int32_t* seq_lens, int32_t max_seqlen, attn_mask_kind kind,
                           const attn_kv_cache* cache, void* workspace, size_t workspace_bytes,
                           attn_stream_t stream) {
  CacheQueryArgs a;
  std::memset(&a, 0, sizeof(a));
  const attn_status st = check_queries(q, lse, dtype, total_tokens, num_heads, scale, cu_seqlens, max_new, seq_lens,
                                       max_seqlen, kind, cache, &a);
  if (st != ATTN_OK) return st;
  if ((total_tokens > 0 && !o) || !aligned(o, 16)) return ATTN_ERR_INVALID_ARG;
  const uint64_t need = cache_fwd_workspace(a.cache, total_tokens, num_heads, a.max_new, max_seqlen);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 256))) return ATTN_ERR_INVALID_ARG;
  if (uint64_t(workspace_bytes) < need) return ATTN_ERR_WORKSPACE_TOO_SMALL;
  if (total_tokens == 0 || max_new == 0) return ATTN_OK;
  a.o = o;
  a.lse = lse;
  a.workspace = static_cast<float*>(workspace);
  return launch_cache_fwd(a, reinterpret_cast<cudaStream_t>(stream));
}

attn_status attn_cache_weights(const void* q, const float* lse, attn_dtype dtype, int32_t total_tokens,
                               int32_t num_heads, float scale, const int32_t* cu_seqlens, int32_t max_new,
                               const int32_t* seq_lens, int32_t max_seqlen, attn_mask_kind kind,
                               const attn_kv_cache* cache, const float* prev, float* weights, int64_t weight_stride,
                               attn_stream_t stream) {
  CacheQueryArgs a;
  std::memset(&a, 0, sizeof(a));
  const attn_status st = check_queries(q, lse, dtype, total_tokens, num_heads, scale, cu_seqlens, max_new, seq_lens,
                                       max_seqlen, kind, cache, &a);
  if (st != ATTN_OK) return st;
  if ((max_seqlen > 0 && !weights) || !aligned(weights, 4) || !aligned(prev, 4) || weight_stride < max_seqlen)
    return ATTN_ERR_INVALID_ARG;
  if (max_seqlen == 0) return ATTN_OK;
  a.lse = const_cast<float*>(lse);
  a.prev = prev;
  a.weights = weights;
  a.weight_stride = weight_stride;
  return launch_cache_weights(a, reinterpret_cast<cudaStream_t>(stream));
}

attn_status attn_cache_evict(const float* weights, int64_t weight_stride, const int32_t* seq_lens,
                             const int32_t* budgets, int32_t recent, int32_t max_seqlen, int32_t max_keep,
                             const attn_kv_cache* cache, const attn_kv_cache* dst, int32_t* kept, float* new_weights,
                             int64_t new_stride, int32_t* new_lens, attn_stream_t stream) {
  if (!seq_lens || !budgets || !new_lens || (max_seqlen > 0 && !weights)) return ATTN_ERR_INVALID_ARG;
  if ((max_keep > 0 && !kept) || (new_stride > 0 && !new_weights)) return ATTN_ERR_INVALID_ARG;
  EvictArgs a;
  std::memset(&a, 0, sizeof(a));
  attn_status st = check_cache(cache, &a.src);
  if (st == ATTN_OK) st = check_cache(dst, &a.dst);
  if (st != ATTN_OK) return st;
  if (recent < 0 || max_seqlen < 0 || max_keep < 0 || weight_stride < max_seqlen || new_stride < max_keep)
    return ATTN_ERR_INVALID_ARG;
  if (cache->num_kv_heads != dst->num_kv_heads || cache->head_dim != dst->head_dim ||
      cache->page_size != dst->page_size || cache->batch != dst->batch)
    return ATTN_ERR_INVALID_ARG;
  if (int64_t(max_seqlen) > int64_t(cache->max_pages) * cache->page_size ||
      int64_t(max_keep) > int64_t(dst->max_pages) * dst->page_size)
    return ATTN_ERR_INVALID_ARG;
  if ((weights && new_weights == weights) || new_lens == seq_lens) return ATTN_ERR_INVALID_ARG;
  // one table over one pool: every page would be read and written in no order
  if (max_keep > 0 && cache->page_table == dst->page_table &&
      (cache->k_pages == dst->k_pages || cache->v_pages == dst->v_pages))
    return ATTN_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(weights), static_cast<const void*>(seq_lens),
                        static_cast<const void*>(budgets), static_cast<const void*>(kept),
                        static_cast<const void*>(new_weights), static_cast<const void*>(new_lens)})
    if (!aligned(p, 4)) return ATTN_ERR_INVALID_ARG;
  a.weights = weights;
  a.weight_stride = weight_stride;
  a.new_stride = new_stride;
  a.lens = seq_lens;
  a.budgets = budgets;
  a.recent = recent;
  a.max_seqlen = max_seqlen;
  a.max_keep = max_keep;
  a.kept = kept;
  a.new_weights = new_weights;
  a.new_lens = new_lens;
  return launch_cache_evict(a, reinterpret_cast<cudaStream_t>(stream));
}

attn_status attn_cache_tree_build(const int32_t* parents, int32_t total_tokens, const int32_t* cu_seqlens,
                                  const int32_t* seq_lens, int32_t max_new, uint32_t* tree_bits, int32_t tree_words,
                                  int32_t* positions, const attn_kv_cache* cache, attn_stream_t stream) {
  if (!cu_seqlens || !seq_lens || total_tokens < 0 || max_new < 0) return ATTN_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!parents || (tree_words > 0 && !tree_bits))) return ATTN_ERR_INVALID_ARG;
  TreeBuildArgs a;
  const attn_status st = check_cache(cache, &a.cache);
  if (st != ATTN_OK) return st;
  if (tree_words < 0 || int64_t(tree_words) * 32 < max_new) return ATTN_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(parents), static_cast<const void*>(cu_seqlens),
                        static_cast<const void*>(seq_lens), static_cast<const void*>(tree_bits),
                        static_cast<const void*>(positions)})
    if (!aligned(p, 4)) return ATTN_ERR_INVALID_ARG;
  if (total_tokens == 0 || max_new == 0) return ATTN_OK;
  // results over what other CTAs still read: a walk would go by them
  const int64_t words = int64_t(total_tokens) * tree_words, batch = cache->batch;
  if (overlap(tree_bits, words, positions, total_tokens)) return ATTN_ERR_INVALID_ARG;
  for (const auto& in : {std::pair<const void*, int64_t>(parents, total_tokens), {cu_seqlens, batch + 1}, {seq_lens, batch}})
    if (overlap(tree_bits, words, in.first, in.second) || overlap(positions, total_tokens, in.first, in.second))
      return ATTN_ERR_INVALID_ARG;
  a.parents = parents;
  a.bits = tree_bits;
  a.positions = positions;
  a.words = tree_words;
  a.total_tokens = total_tokens;
  a.max_new = max_new < total_tokens ? max_new : total_tokens;
  a.cu = cu_seqlens;
  a.lens = seq_lens;
  return launch_tree_build(a, reinterpret_cast<cudaStream_t>(stream));
}

attn_status attn_cache_append_rope(const void* q, void* q_out, int64_t q_stride, int64_t q_out_stride,
                                   int32_t num_heads, const void* k, const void* v, int64_t k_stride,
                                   int64_t v_stride, attn_dtype dtype, int32_t total_tokens, const int32_t* positions,
                                   const int32_t* cu_seqlens, const int32_t* seq_lens, int32_t max_new,
                                   const attn_rope_plan* plan, const attn_kv_cache* cache, attn_stream_t stream) {
  if (!plan || plan->magic != kRopeMagic || num_heads < 0) return ATTN_ERR_INVALID_ARG;
  AppendArgs a;
  attn_status st = check_append(k, v, k_stride, v_stride, dtype, total_tokens, cu_seqlens, seq_lens, max_new, cache, &a);
  if (st != ATTN_OK) return st;
  if (plan->rotary_dim > cache->head_dim || !aligned(positions, 4)) return ATTN_ERR_INVALID_ARG;
  if (num_heads > kMaxHeads) return ATTN_ERR_UNSUPPORTED;
  // a launch's blocks fit 31 bits
  if ((int64_t(total_tokens) / cache->page_size + 2ll * cache->batch) * 2 * cache->num_kv_heads +
          int64_t(total_tokens) * (num_heads + 1) / 8 > INT_MAX)
    return ATTN_ERR_UNSUPPORTED;
  const uintptr_t size = dtype == ATTN_DTYPE_BF16 ? 2 : 4;
  if (num_heads > 0 && total_tokens > 0) {
    if (!q || !q_out || !aligned(q, size) || !aligned(q_out, size)) return ATTN_ERR_INVALID_ARG;
    // tokens must not overlap; in place, a token's row must be its own
    const int64_t need = int64_t(num_heads) * cache->head_dim;
    if (total_tokens > 1 && (q_stride < need || q_out_stride < need || (q == q_out && q_stride != q_out_stride)))
      return ATTN_ERR_INVALID_ARG;
  }
  if (total_tokens == 0 || max_new == 0) return ATTN_OK;
  RopeArgs r;
  std::memset(&r, 0, sizeof(r));
  r.q = q;
  r.q_out = q_out;
  r.q_stride = q_stride;
  r.q_out_stride = q_out_stride;
  r.num_heads = num_heads;
  r.total_tokens = total_tokens;
  r.head_dim = cache->head_dim;
  r.batch = cache->batch;
  r.positions = positions;
  r.cu = cu_seqlens;
  r.lens = seq_lens;
  r.bf16 = a.bf16;
  return launch_cache_append_rope(a, r, *plan, reinterpret_cast<cudaStream_t>(stream));
}

attn_status attn_cache_tree_fwd_workspace_size(const attn_kv_cache* cache, int32_t total_tokens, int32_t num_heads,
                                               int32_t max_new, int32_t max_seqlen, size_t* bytes) {
  if (bytes == nullptr) return ATTN_ERR_INVALID_ARG;
  CacheView v;
  attn_status st = check_cache(cache, &v);
  if (st == ATTN_OK) st = check_sizes(cache, total_tokens, num_heads, max_new, max_seqlen);
  if (st != ATTN_OK) return st;
  *bytes = size_t(cache_tree_workspace(v, total_tokens, num_heads, max_new < total_tokens ? max_new : total_tokens,
                                       max_seqlen));
  return ATTN_OK;
}

attn_status attn_cache_tree_fwd(const void* q, void* o, float* lse, attn_dtype dtype, int32_t total_tokens,
                                int32_t num_heads, float scale, const uint32_t* tree_bits, int32_t tree_words,
                                const int32_t* cu_seqlens, int32_t max_new, const int32_t* seq_lens,
                                int32_t max_seqlen, const attn_kv_cache* cache, void* workspace,
                                size_t workspace_bytes, attn_stream_t stream) {
  CacheQueryArgs a;
  std::memset(&a, 0, sizeof(a));
  const attn_status st = check_queries(q, lse, dtype, total_tokens, num_heads, scale, cu_seqlens, max_new, seq_lens,
                                       max_seqlen, ATTN_MASK_NONE, cache, &a);
  if (st != ATTN_OK) return st;
  if ((total_tokens > 0 && !o) || !aligned(o, 16)) return ATTN_ERR_INVALID_ARG;
  if (tree_words < 0 || int64_t(tree_words) * 32 < max_new || !aligned(tree_bits, 4)) return ATTN_ERR_INVALID_ARG;
  if (total_tokens > 0 && max_new > 0 && !tree_bits) return ATTN_ERR_INVALID_ARG;
  const uint64_t need = cache_tree_workspace(a.cache, total_tokens, num_heads, a.max_new, max_seqlen);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 256))) return ATTN_ERR_INVALID_ARG;
  if (uint64_t(workspace_bytes) < need) return ATTN_ERR_WORKSPACE_TOO_SMALL;
  if (total_tokens == 0 || max_new == 0) return ATTN_OK;
  a.o = o;
  a.lse = lse;
  a.workspace = static_cast<float*>(workspace);
  return launch_cache_tree(a, TreeMasks{tree_bits, tree_words}, reinterpret_cast<cudaStream_t>(stream));
}

attn_status attn_cache_tree_keep(const int32_t* path, int32_t path_stride, const int32_t* counts,
                                 const int32_t* cu_seqlens, const int32_t* seq_lens, int32_t max_new,
                                 int32_t* new_lens, const attn_kv_cache* cache, attn_stream_t stream) {
  if (!counts || !cu_seqlens || !seq_lens || !new_lens || max_new < 0 || path_stride < 0 || (path_stride > 0 && !path))
    return ATTN_ERR_INVALID_ARG;
  TreeKeepArgs a;
  const attn_status st = check_cache(cache, &a.cache);
  if (st != ATTN_OK) return st;
  for (const void* p : {static_cast<const void*>(path), static_cast<const void*>(counts),
                        static_cast<const void*>(cu_seqlens), static_cast<const void*>(seq_lens),
                        static_cast<const void*>(new_lens)})
    if (!aligned(p, 4)) return ATTN_ERR_INVALID_ARG;
  // written while others still read the old ones
  const int64_t batch = cache->batch;
  for (const auto& in : {std::pair<const void*, int64_t>(path, batch * path_stride), {counts, batch},
                         {cu_seqlens, batch + 1}, {seq_lens, batch}})
    if (overlap(new_lens, batch, in.first, in.second)) return ATTN_ERR_INVALID_ARG;
  a.path = path;
  a.counts = counts;
  a.new_lens = new_lens;
  a.path_stride = path_stride;
  a.max_new = max_new;
  a.cu = cu_seqlens;
  a.lens = seq_lens;
  return launch_tree_keep(a, reinterpret_cast<cudaStream_t>(stream));
}

attn_status attn_cache_get_status(const attn_kv_cache* cache, attn_stream_t stream) {
  CacheView v;
  const attn_status st = check_cache(cache, &v);
  if (st != ATTN_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int32_t err = 0;
  cudaError_t e = cudaMemcpyAsync(&err, v.status, sizeof(err), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(v.status, 0, sizeof(err), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return record_cuda_error(e, "attn_cache_get_status");
  if (err & kErrTimeout) return ATTN_ERR_DEVICE_TIMEOUT;
  if (err & kErrCacheInput) return ATTN_ERR_DEVICE_INVALID_INPUT;
  return ATTN_OK;
}

}  // extern "C"
