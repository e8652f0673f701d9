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
#include "ptx.cuh"

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
// step s.  (fp16's least step is 2^-24: with bf16's 8 bits, elements down to 2^-17 are
// exact, and smaller ones off by 2^-25 at most.)  Returns that power's inverse.  A row
// past the last is zero.
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

// The line of units: `units(b)` is the number of sequence b, all heads.  Called
// by whole warps; the first 128 sequences' numbers stay with the lanes.
struct UnitLine {
  int n[4];
  int total;

  template <typename F>
  __device__ __forceinline__ UnitLine(const F& units, int batch, int lane) {
    total = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) n[k] = 32 * k + lane < batch ? units(32 * k + lane) : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) total += n[k];
    for (int b = 128 + lane; b < batch; b += 32) total += units(b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }

  // The sequence that unit `pos` (below the total) belongs to, and the units before it.
  template <typename F>
  __device__ __forceinline__ int find(const F& units, int batch, int lane, int pos, int& before) const {
    before = 0;
    for (int b0 = 0;; b0 += 32) {
      int mine = 0;
      if (b0 < 128) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (b0 == 32 * k) mine = n[k];
      } else if (b0 + lane < batch) {
        mine = units(b0 + lane);
      }
      int sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, before + sum > pos);
      if (past || b0 + 32 >= batch) {
        const int at = past ? __ffs(past) - 1 : 31;
        before += __shfl_sync(0xffffffffu, sum - mine, at);
        return b0 + at;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
};

// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, bool on) {
  const int n = on ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// Sixteen tokens' codes in shared memory, rows of D bytes as they lie in the page.
// They are copied 512 consecutive bytes per instruction, lane by lane, and read
// by the lanes that use them, so a warp meets at a barrier of its own
// between the two.  (Copies straight to the lane that uses them need none, but
// the values' rows then come in four pieces of 32 bytes per eight lanes: 5.2
// instead of 7.0 TB/s.)  The pieces of 16 bytes of a row are permuted so that
// the readers of keys (lane 4 g + t: row g, D / 8 bytes at t D / 8 of a half) or
// of values (rows 2t, 2t + 1, piece g of D / 8 bytes) meet as few bank conflicts as
// the row's length allows.
template <int D>
struct GroupTile {
  static constexpr int BYTES = kGroup * D;
  template <bool VALUES>
  __device__ static int turn(int row) {
    if (VALUES) return D == 128 ? ((row >> 1) & 3) << 1 : D == 64 ? (row >> 1) & 3 : 0;
    return D == 128 ? (row & 1) << 2 : D == 64 ? ((row >> 1) & 1) << 1 : (row >> 2) & 1;
  }
  // Rows [0, left) of `src`; zeros behind them.
  template <bool VALUES>
  __device__ static void copy(uint32_t dst, const uint8_t* src, int left, int lane) {
#pragma unroll
    for (int j = 0; j < BYTES / 512; ++j) {
      const int at = j * 512 + lane * 16, row = at / D, unit = at % D / 16;
      copy16_async(dst + row * D + ((unit ^ turn<VALUES>(row)) << 4), src + at, row < left);
    }
  }
  // The D / 8 bytes at `at` of a row, as words.
  template <bool VALUES>
  __device__ static void read(const uint8_t* tile, int row, int at, uint32_t (&w)[D / 32]) {
    const uint8_t* from = tile + row * D + (((at >> 4) ^ turn<VALUES>(row)) << 4) + (at & 15);
    if constexpr (D == 128) {
      const uint4 v = *reinterpret_cast<const uint4*>(from);
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (D == 64) {
      const uint2 v = *reinterpret_cast<const uint2*>(from);
      w[0] = v.x; w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(from);
    }
  }
};

// Pages of a warp's groups, looked up by its lanes 32 at a time and a batch ahead;
// they travel by shuffle.  The numbers come first, so that copies can start;
// a page outside the pool has scales 0 (and is noted in the status word).
struct PageBatch {
  int number;
  float k_scale, v_scale;
};
__device__ __forceinline__ int page_number(const CacheView& c, int b, int token, bool on) {
  return on ? __ldg(c.table + int64_t(b) * c.max_pages + (token >> c.page_log2)) : 0;
}
__device__ __forceinline__ bool in_pool(const CacheView& c, int number) {
  return unsigned(number) < unsigned(c.num_pages);
}
__device__ __forceinline__ PageBatch with_scales(const CacheView& c, int h, int number, bool on, bool values) {
  PageBatch p{number, 0.f, 0.f};
  if (on && in_pool(c, number)) {
    const int64_t at = int64_t(number) * c.heads + h;
    p.k_scale = __ldg(c.k_scale + at);
    if (values) p.v_scale = __ldg(c.v_scale + at);
  } else if (on) {
    atomicOr(c.status, kErrBadPage);
  }
  return p;
}

// Weights as fp16, powers of two: the largest when the reference moves, and at most.
constexpr float kTopWeight = 7.f, kMostWeight = 15.f;

// A term of a softmax's sum is its weight without the value's exponent (cache_attn.cu).
// A weight is lost below 2^-126 of the reference: with value exponents this far apart
// that is at most 2^-53 of the sum; further apart its terms are formed without them.
constexpr int kSpread = 80;

// The square root of the factor that brings what refers to `m` to the reference `top`:
// sums are multiplied by it twice, since one may be 2^125 and the factor itself below
// what fp32 holds.
__device__ __forceinline__ float half_factor(float m, float top) {
  return m == -INFINITY ? 0.f : ptx::ex2(0.5f * (m - top));
}

// Tokens [0, visible) that row `row` sees (0 for a row past the last).
__device__ __forceinline__ int visible_tokens(const SeqRows& r, int G, int row, bool causal) {
  if (row >= r.n * G) return 0;
  return causal ? max(0, r.len - r.n + row / G + 1) : r.len;
}

}  // namespace
}  // namespace attnmask
