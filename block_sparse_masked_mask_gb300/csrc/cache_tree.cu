// Attention of trees of drafted tokens over the 8-bit cache.
//
// A CTA takes eight rows of one sequence and key / value head and walks the tokens
// 128 at a time: each thread scores one token against every row, each warp settles
// the running maximum and sum of two rows, and each thread then adds up one
// dimension of O.  All in fp32.
#include <cmath>

#include "cache_rows.cuh"

namespace attnmask {
namespace {

constexpr int kTreeThreads = 128, kTreeRows = 8;

template <int D>
__global__ void __launch_bounds__(kTreeThreads) cache_tree_kernel(const TreeAttnArgs t) {
  __shared__ float q[kTreeRows][D], w[kTreeRows][kTreeThreads], factor[kTreeRows], sum[kTreeRows], top[kTreeRows];
  const CacheQueryArgs& a = t.a;
  const CacheView& c = a.cache;
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.num_heads / c.heads;
  SeqRows r;
  if (!load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, a.max_seqlen, c.status, r, tid == 0)) return;
  if (r.len < r.n) {
    if (tid == 0) atomicOr(c.status, kErrHeld);
    return;
  }
  const int row0 = blockIdx.x * kTreeRows, rows = min(kTreeRows, r.n * G - row0), base = r.len - r.n;
  if (rows <= 0) return;
  for (int x = tid; x < kTreeRows * D; x += kTreeThreads) {
    const int row = row0 + x / D;
    q[x / D][x % D] = x / D < rows ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[
        (int64_t(r.q0 + row / G) * a.num_heads + h * G + row % G) * D + x % D]) * a.scale * 1.4426950408889634f : 0.f;
  }
  if (tid < kTreeRows) {
    top[tid] = -INFINITY;
    sum[tid] = 0.f;
  }
  float o[kTreeRows];
#pragma unroll
  for (int i = 0; i < kTreeRows; ++i) o[i] = 0.f;
  for (int t0 = 0; t0 < r.len; t0 += kTreeThreads) {
    __syncthreads();
    const int token = t0 + tid;
    const int number = page_number(c, b, token, token < r.len);
    const bool here = token < r.len && in_pool(c, number);
    if (token < r.len && !here) atomicOr(c.status, kErrBadPage);
    float s[kTreeRows];
#pragma unroll
    for (int i = 0; i < kTreeRows; ++i) s[i] = 0.f;
    if (here) {
      const int64_t at = int64_t(number) * c.heads + h;
      const uint32_t* k = reinterpret_cast<const uint32_t*>(
          c.k_pages + ((at << c.page_log2) + (token & ((1 << c.page_log2) - 1))) * D);
      for (int x = 0; x < D / 4; ++x) {
        const uint32_t codes = k[x];
        uint32_t lo = half2_of(codes), hi = half2_of_high(codes);
        const float2 y = __half22float2(*reinterpret_cast<__half2*>(&lo)), z = __half22float2(*reinterpret_cast<__half2*>(&hi));
#pragma unroll
        for (int i = 0; i < kTreeRows; ++i)
          s[i] += q[i][4 * x] * y.x + q[i][4 * x + 1] * y.y + q[i][4 * x + 2] * z.x + q[i][4 * x + 3] * z.y;
      }
      const float ks = c.k_scale[at];
#pragma unroll
      for (int i = 0; i < kTreeRows; ++i) s[i] *= ks;
    }
    const int node = token - base;
#pragma unroll
    for (int i = 0; i < kTreeRows; ++i) {
      bool seen = here && i < rows;
      if (seen && node >= 0) seen = t.bits[int64_t(r.q0 + (row0 + i) / G) * t.words + (node >> 5)] >> (node & 31) & 1u;
      w[i][tid] = seen ? s[i] : -INFINITY;
    }
    __syncthreads();
    for (int i = warp; i < kTreeRows; i += kTreeThreads / 32) {
      float x[4], m = top[i];
#pragma unroll
      for (int y = 0; y < 4; ++y) m = fmaxf(m, x[y] = w[i][32 * y + lane]);
#pragma unroll
      for (int y = 16; y > 0; y >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, y));
      const float ref = m == -INFINITY ? 0.f : m;
      float l = 0.f;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        x[y] = exp2f(x[y] - ref);
        l += x[y];
        w[i][32 * y + lane] = x[y];
      }
#pragma unroll
      for (int y = 16; y > 0; y >>= 1) l += __shfl_xor_sync(0xffffffffu, l, y);
      const float f = exp2f(top[i] - ref);
      __syncwarp();
      if (lane == 0) {
        factor[i] = f;
        sum[i] = sum[i] * f + l;
        top[i] = m;
      }
    }
    __syncthreads();
    if (tid < D) {
#pragma unroll
      for (int i = 0; i < kTreeRows; ++i) o[i] *= factor[i];
      for (int x = 0; x < min(kTreeThreads, r.len - t0); ++x) {
        const int page = page_number(c, b, t0 + x, true);
        if (!in_pool(c, page)) continue;
        const int64_t at = int64_t(page) * c.heads + h;
        uint32_t y = half2_of(c.v_pages[((at << c.page_log2) + ((t0 + x) & ((1 << c.page_log2) - 1))) * D + tid]);
        const float v = __half22float2(*reinterpret_cast<__half2*>(&y)).x * c.v_scale[at];
#pragma unroll
        for (int i = 0; i < kTreeRows; ++i) o[i] = fmaf(w[i][x], v, o[i]);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kTreeRows; ++i) {
    if (i >= rows) break;
    const int row = row0 + i, head = h * G + row % G;
    const int64_t token = r.q0 + row / G;
    const float l = sum[i];
    if (tid < D)
      static_cast<__nv_bfloat16*>(a.o)[(token * a.num_heads + head) * D + tid] = __float2bfloat16_rn(l == 0.f ? 0.f : o[i] / l);
    if (tid == 0)
      a.lse[int64_t(head) * a.total_tokens + token] = l == 0.f ? -INFINITY : (top[i] + log2f(l)) * 0.69314718055994531f;
  }
}

}  // namespace

uint64_t cache_tree_workspace(const CacheView&, int, int, int, int) { return 0; }

attn_status launch_cache_tree(const TreeAttnArgs& t, cudaStream_t s) {
  const CacheQueryArgs& a = t.a;
  const int64_t rows = int64_t(a.max_new) * (a.num_heads / a.cache.heads);
  const dim3 grid(unsigned((rows + kTreeRows - 1) / kTreeRows), unsigned(a.cache.heads), unsigned(a.cache.batch));
  switch (a.cache.head_dim) {
    case 32: cache_tree_kernel<32><<<grid, kTreeThreads, 0, s>>>(t); break;
    case 64: cache_tree_kernel<64><<<grid, kTreeThreads, 0, s>>>(t); break;
    default: cache_tree_kernel<128><<<grid, kTreeThreads, 0, s>>>(t); break;
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_tree_fwd launch");
}

}  // namespace attnmask
