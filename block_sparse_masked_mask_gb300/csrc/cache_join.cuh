// How partial results of a row's attention over the cache, from several CTAs, become
// one: O before the division, and (running maximum, sum), in the order of the tokens.
#pragma once

#include "cache_rows.cuh"

namespace attnmask {
namespace {

constexpr float kLn2 = 0.69314718055994531f;

// Joins a row's partial results in their order: `n` of them, the i-th at row
// at(i).  W warps share a row (warp w takes w, w + W, ..), each lane D / 32
// dimensions.
template <int D, int W, typename P, typename At>
__device__ __forceinline__ void join_row(const P& p, int n, const At& at, int64_t token, int head, int w,
                                         int lane, float* shared) {
  constexpr int E = D / 32;
  const CacheQueryArgs& a = p.a;
  float m = -INFINITY, l = 0.f, x[E];
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = 0.f;
  for (int i0 = w; i0 < n; i0 += 32 * W) {
    // up to 32 partial results at a time: their statistics by lanes
    const int i = i0 + lane * W;
    const float2 s = i < n ? p.part_m[at(i)] : make_float2(-INFINITY, 0.f);
    float top = s.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(top, m);
    const float half = half_factor(s.x, top), f = half * half, old_half = half_factor(m, top), old = old_half * old_half;
    float sum = s.y != s.y ? s.y : s.y * half * half;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * old_half * old_half + sum;
    m = top;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= old;
    const int k = min(32, (n - i0 + W - 1) / W);
#pragma unroll 4
    for (int j = 0; j < k; ++j) {
      const float fj = __shfl_sync(0xffffffffu, f, j);
      const float* from = p.part_o + at(i0 + j * W) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = fmaf(fj, from[e], x[e]);
    }
  }
  if constexpr (W > 1) {
    float* mine = shared + w * (D + 2);
#pragma unroll
    for (int e = 0; e < E; ++e) mine[lane * E + e] = x[e];
    if (lane == 0) {
      mine[D] = m;
      mine[D + 1] = l;
    }
    __syncthreads();
    if (w > 0) return;
    float top = -INFINITY;
#pragma unroll
    for (int y = 0; y < W; ++y) top = fmaxf(top, shared[y * (D + 2) + D]);
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.f;
#pragma unroll
    for (int y = 0; y < W; ++y) {
      const float* from = shared + y * (D + 2);
      const float half = half_factor(from[D], top), f = half * half, s = from[D + 1];
      l += s != s ? s : s * half * half;
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = fmaf(f, from[lane * E + e], x[e]);
    }
    m = top;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < E; ++e)
    static_cast<__nv_bfloat16*>(a.o)[(token * a.num_heads + head) * D + lane * E + e] = __float2bfloat16_rn(x[e] * inv);
  if (lane == 0) a.lse[int64_t(head) * a.total_tokens + token] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace
}  // namespace attnmask
