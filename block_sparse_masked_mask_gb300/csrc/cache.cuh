// Internal declarations of the rotary and key / value cache operators
// (include/attn_cache.h): arguments, device-side checks and e4m3 arithmetic.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn_cache.h"
#include "common.cuh"

namespace attnmask {

constexpr uint32_t kRopeMagic = 0x45504F52u;  // "ROPE"

// Bits of the cache's status word (kErr* of common.cuh, and:)
enum : int32_t {
  kErrBadPage = 1 << 4,    // a page number outside the pool
  kErrTooManyNew = 1 << 5, // a sequence has more new tokens than max_new
  kErrHeld = 1 << 6,       // seq_lens negative, or below the new tokens of an append
  kErrBudget = 1 << 7,     // an eviction's budget negative or above max_keep
  kErrCacheInput = kErrInputMask | kErrBadPage | kErrTooManyNew | kErrHeld | kErrBudget,
};

// The cache as the kernels see it.
struct CacheView {
  uint8_t* k_pages;
  uint8_t* v_pages;
  float* k_scale;
  float* v_scale;
  const int32_t* table;
  int32_t* status;
  int num_pages, heads, page_log2, head_dim, batch, max_pages;
};

struct RopeArgs {
  const void* q;
  void* q_out;
  const void* k;
  void* k_out;
  int64_t q_stride, q_out_stride, k_stride, k_out_stride;
  int num_heads, num_kv_heads, total_tokens, head_dim, batch;
  const int32_t* positions;
  const int32_t* cu;
  const int32_t* lens;
  bool inverse, bf16;
};

struct AppendArgs {
  const void* k;
  const void* v;
  int64_t k_stride, v_stride;
  int total_tokens, max_new;
  const int32_t* cu;
  const int32_t* lens;
  bool bf16;
  CacheView cache;
};

// One call's queries over the cache (attention and weights).
struct CacheQueryArgs {
  const void* q;
  void* o;             // attention only
  float* lse;          // written by the attention, read by the weights
  const float* prev;   // weights only
  float* weights;
  int64_t weight_stride;
  int total_tokens, num_heads, max_new, max_seqlen;
  float scale;
  bool causal;
  const int32_t* cu;
  const int32_t* lens;
  CacheView cache;
  float* workspace;
};

// How attn_cache_fwd cuts its work, and where the pieces' results meet: rows (new
// token, query head of the group) in tiles and tokens in chunks
// (tcgen05 kernel), or share the line of all tokens evenly (mma.sync kernel).
struct CacheAttnParams {
  CacheQueryArgs a;
  int G;           // query heads per key / value head
  bool many;       // the tcgen05 kernel
  int row_tiles, chunk, splits;  // many: tiles of kManyRows rows, tokens per chunk, chunks
  int ctas;        // few: CTAs
  int team;        // few: CTAs per (sequence, head), a cluster; 0: the line is cut
  float scale_log2;
  // Results before the division, and (running maximum, sum).
  //   many: [splits][total_tokens * num_heads] rows
  //   few:  [2 * ctas][max_new * G] rows: of CTA c, 2 c a segment that goes on
  //         one of the CTA before, 2 c + 1 one that goes on in the next
  float* part_o;   // rows of head_dim
  float2* part_m;
};
constexpr int kFewRows = 16, kManyRows = 256;

struct EvictArgs {
  const float* weights;
  int64_t weight_stride, new_stride;
  const int32_t* lens;
  const int32_t* budgets;
  int recent, max_seqlen, max_keep;
  int32_t* kept;
  float* new_weights;
  int32_t* new_lens;
  CacheView src, dst;
};

attn_status launch_rope(const RopeArgs& a, const attn_rope_plan& plan, cudaStream_t s);
attn_status launch_cache_append(const AppendArgs& a, cudaStream_t s);
uint64_t cache_fwd_workspace(const CacheView& c, int total_tokens, int num_heads, int max_new, int max_seqlen);
attn_status launch_cache_fwd(const CacheQueryArgs& a, cudaStream_t s);
attn_status launch_cache_chunk(const CacheAttnParams& p, cudaStream_t s);
attn_status launch_cache_weights(const CacheQueryArgs& a, cudaStream_t s);
attn_status launch_cache_weights_many(const CacheQueryArgs& a, int sms, cudaStream_t s);
attn_status launch_cache_evict(const EvictArgs& a, cudaStream_t s);

// ---------------------------------------------------------------- device side

// New rows [q0, q0 + n) of a sequence that holds len tokens.
struct SeqRows {
  int q0, n, len;
};

// Reads and checks sequence b.  False where its numbers cannot be used: the
// status word then says why, and the caller leaves the sequence out, so no
// index below is ever formed from them.  max_new and max_len bound what the
// launch was sized for; max_len is at most max_pages * page_size.
__device__ __forceinline__ bool load_rows(const int32_t* cu, const int32_t* lens, int b, int total_tokens,
                                          int max_new, int max_len, int32_t* status, SeqRows& r,
                                          bool note = true) {
  const int q0 = cu[b], q1 = cu[b + 1];
  r.q0 = q0;
  r.len = lens[b];
  int err = 0;
  if (b == 0 && q0 != 0) err |= kErrCuFirst;
  if (q0 < 0 || q1 < q0) err |= kErrCuOrder;
  if (q1 > total_tokens) err |= kErrCuLast;
  r.n = err ? 0 : q1 - q0;
  if (r.n > max_new) err |= kErrTooManyNew;
  if (r.len < 0) err |= kErrHeld;
  if (r.len > max_len) err |= kErrSeqTooLong;
  if (err && note) atomicOr(status, err);
  return err == 0;
}

__device__ __forceinline__ float pow2f(int e) {  // -126 <= e <= 127
  return __int_as_float((e + 127) << 23);
}
// Exponent of a power of two (a scale).
__device__ __forceinline__ int exponent_of(float x) { return int((__float_as_uint(x) >> 23) & 255u) - 127; }

constexpr int kScaleExpMin = -80, kScaleExpMax = 120;

// The least e with amax <= 448 2^e = 1.75 2^(8 + e), within the scales' range:
// read from the exponent and mantissa of amax (finite, >= 0), so without rounding.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = int(b >> 23) - 127 - 8 + int((b & 0x7FFFFFu) > 0x600000u);
  return max(kScaleExpMin, min(kScaleExpMax, e));
}

// Two fp32 -> two e4m3 codes (nearest even, saturating, NaN kept); `lo` in bits 0-7.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes -> two fp16 (exact).
__device__ __forceinline__ uint32_t half2_of(uint32_t two_codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 c, d;\n\tmov.b32 {c, d}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(two_codes));
  return r;
}
__device__ __forceinline__ uint32_t half2_of_high(uint32_t four_codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 c, d;\n\tmov.b32 {c, d}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, d;\n\t}" : "=r"(r) : "r"(four_codes));
  return r;
}
// Four codes times 2^-shift, shift >= 0.  The product of a code (four
// significant bits) by 2^-shift is exact in fp16 while it is at least 2^-20;
// below that e4m3, whose smallest step is 2^-9, holds zero either way.  So
// each code is rounded once.
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, int shift) {
  const __half2 f = __float2half2_rn(pow2f(-min(shift, 24)));
  uint32_t lo = half2_of(codes), hi = half2_of_high(codes);
  __half2 a = __hmul2(*reinterpret_cast<__half2*>(&lo), f), b = __hmul2(*reinterpret_cast<__half2*>(&hi), f);
  uint16_t ca, cb;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(ca) : "r"(*reinterpret_cast<uint32_t*>(&a)));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(cb) : "r"(*reinterpret_cast<uint32_t*>(&b)));
  return uint32_t(ca) | (uint32_t(cb) << 16);
}

}  // namespace attnmask
