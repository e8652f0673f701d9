// What the mma.sync kernels over the cache (attention of few rows, weights) share:
// the query rows and their fp16 form, the queue of a warp's keys and values, and
// the even division of the tokens among the CTAs.
//
// Rows.  The queries of one sequence and key / value head are n * G rows, row
// r = new token r / G, query head h G + r % G.
//
// Operands.  m16n8k16 with the tokens as M, the rows as N: lane = 4 g + t holds,
// of a 16-wide step of the contracted dimension, the places 2t, 2t + 1, 2t + 8,
// 2t + 9 of tokens g, g + 8 and of row g.  The order of that dimension is free
// as long as both operands agree, so lane t takes two pieces of D / 8
// consecutive dimensions, at t D / 8 of each half of the head, four dimensions
// per step: a token's codes are then read as they lie, and the four lanes of a
// token read whole sectors.
//
// Division.  Tokens are counted in units of 64; the units of all sequences and
// heads form one line, which is cut into equal pieces, one per CTA.  So every
// CTA has the same work whatever the lengths, and a CTA's piece touches few
// (sequence, head)s.
#pragma once

#include "cache.cuh"

namespace attnmask {
namespace {

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// One row's dimensions of lane t (two pieces) as fp16 pairs, times a power of two
// that puts the row's largest magnitude into [1, 2): w[2 s], w[2 s + 1] belong to
// step s.  Returns that power's inverse.  A row past the last is zero.
template <int D>
__device__ __forceinline__ float load_query(const CacheQueryArgs& a, const SeqRows& r, int h, int G, int row, int t,
                                            uint32_t (&w)[D / 8]) {
  float f[D / 4];
  float amax = 0.f;
  if (row < r.n * G) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.q) +
                             (int64_t(r.q0 + row / G) * a.num_heads + h * G + row % G) * D + t * (D / 8);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint2 v = reinterpret_cast<const uint2*>(p + x * (D / 2))[i];
        float* at = f + x * (D / 8) + 4 * i;
        at[0] = __uint_as_float(v.x << 16);
        at[1] = __uint_as_float(v.x & 0xFFFF0000u);
        at[2] = __uint_as_float(v.y << 16);
        at[3] = __uint_as_float(v.y & 0xFFFF0000u);
      }
#pragma unroll
    for (int i = 0; i < D / 4; ++i) amax = fmaxf(amax, fabsf(f[i]));
  } else {
#pragma unroll
    for (int i = 0; i < D / 4; ++i) f[i] = 0.f;
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const int e = amax > 0.f ? max(-126, min(126, exponent_of(amax))) : 0;
  const float inv = pow2f(-e);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) w[i] = pack_half2(f[2 * i] * inv, f[2 * i + 1] * inv);
  return pow2f(e);
}

constexpr int kUnit = 64;    // tokens
constexpr int kGroup = 16;   // tokens a warp takes at a time
constexpr int kWarps = 4;    // per CTA; they take a segment's groups in turn
static_assert(kUnit == kGroup * kWarps, "a unit is one group per warp");

// A division of the line of units among the CTAs of a launch: `units(b)` is the
// number of sequence b, all heads.  Called by whole warps.
template <typename F>
__device__ __forceinline__ int total_units(const F& units, int batch, int lane) {
  int n = 0;
  for (int b = lane; b < batch; b += 32) n += units(b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}
// The sequence that unit `pos` belongs to (pos is below the total), and the units before it.
template <typename F>
__device__ __forceinline__ int find_unit(const F& units, int batch, int lane, int pos, int& before) {
  before = 0;
  for (int b0 = 0;; b0 += 32) {
    int n = b0 + lane < batch ? units(b0 + lane) : 0;
    const int mine = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + n > pos);
    if (past || b0 + 32 >= batch) {
      const int at = past ? __ffs(past) - 1 : 31;
      before += __shfl_sync(0xffffffffu, n - mine, at);
      return b0 + at;
    }
    before += __shfl_sync(0xffffffffu, n, 31);
  }
}

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool on) {
  const int n = on ? BYTES : 0;  // nothing read, zeros stored
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}

// Pages of a warp's groups, looked up by its lanes 32 at a time, a batch ahead;
// they travel by shuffle.  A page outside the pool is -1, with scales 0.
struct PageBatch {
  int page;
  float k_scale, v_scale;
};
__device__ __forceinline__ PageBatch look_up(const CacheView& c, int b, int h, int token, bool on, bool values) {
  PageBatch p{-1, 0.f, 0.f};
  if (on) {
    p.page = load_page(c, b, token >> c.page_log2);
    if (p.page >= 0) {
      const int64_t at = int64_t(p.page) * c.heads + h;
      p.k_scale = c.k_scale[at];
      if (values) p.v_scale = c.v_scale[at];
    }
  }
  return p;
}

// Tokens [0, visible) that row `row` sees (0 for a row past the last).
__device__ __forceinline__ int visible_tokens(const SeqRows& r, int G, int row, bool causal) {
  if (row >= r.n * G) return 0;
  return causal ? max(0, r.len - r.n + row / G + 1) : r.len;
}

}  // namespace
}  // namespace attnmask
