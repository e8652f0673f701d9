// The attention weight that each cached token receives from a call's queries:
// the columns of exp(scale q k - LSE) summed over the query rows that share a
// key / value head.
//
// The keys are read once (D bytes per token and head), which bounds it for a
// decode step; the LSE is known, so no second pass and no running maximum.  A
// warp owns 32 tokens: it holds their keys in registers as the B operand of
// mma.sync m16n8k16 and walks the query rows 16 at a time, which the CTA's
// four warps stage in shared memory in operand order.  Every token's sum is
// formed by one warp in a fixed order: no atomics, repeats are bit-identical.
#include "cache_rows.cuh"
#include "ptx.cuh"

namespace attnmask {
namespace {

constexpr int kWarps = 4;
constexpr int kWeightThreads = 32 * kWarps;
constexpr int kTokens = 32;  // per warp

struct WeightParams {
  CacheQueryArgs a;
  int G;
  float scale_log2;
};

template <int D>
__global__ void __launch_bounds__(kWeightThreads, 4) cache_weights_kernel(const WeightParams p) {
  constexpr int WORDS = D / 16;  // of a token, per lane
  const CacheQueryArgs& a = p.a;
  const CacheView& c = a.cache;
  __shared__ uint4 frag[kWarps][D / 16][32];
  __shared__ float row_scale[kWarps][16], row_lse[kWarps][16];
  const int h = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  SeqRows r;
  if (!load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, a.max_seqlen, c.status, r)) return;
  const int cta_tok = blockIdx.x * kWarps * kTokens;
  if (cta_tok >= r.len) return;
  const int tok0 = cta_tok + warp * kTokens;

  // keys of tokens tok0 + 8 nt + g, the lane's two pieces
  uint32_t w[4][WORDS];
  float ks[2] = {0.f, 0.f};
  bool fine[2] = {false, false};
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int tok = tok0 + 16 * half;
    int page = -1;
    if (tok < r.len) page = load_page(c, b, tok >> c.page_log2);
    fine[half] = page >= 0;
    if (page >= 0) ks[half] = c.k_scale[int64_t(page) * c.heads + h];
    const uint8_t* base = c.k_pages + (((int64_t(page >= 0 ? page : 0) * c.heads + h) << c.page_log2) +
                                       (tok & ((1 << c.page_log2) - 1))) * D;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int nt = 2 * half + n;
      const uint8_t* at = base + (8 * n + g) * D + t * (D / 8);
      const bool on = page >= 0 && tok + 8 * n + g < r.len;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t* to = w[nt] + x * (WORDS / 2);
        const uint8_t* from = at + x * (D / 2);
        if constexpr (D == 128) {
          const uint4 v = on ? *reinterpret_cast<const uint4*>(from) : make_uint4(0, 0, 0, 0);
          to[0] = v.x; to[1] = v.y; to[2] = v.z; to[3] = v.w;
        } else if constexpr (D == 64) {
          const uint2 v = on ? *reinterpret_cast<const uint2*>(from) : make_uint2(0, 0);
          to[0] = v.x; to[1] = v.y;
        } else {
          to[0] = on ? *reinterpret_cast<const uint32_t*>(from) : 0u;
        }
      }
    }
  }

  float sum[4][2];
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) sum[nt][0] = sum[nt][1] = 0.f;
  const int rows = r.n * p.G;
  for (int row0 = 0; row0 < rows; row0 += 16 * kWarps) {
    {
      uint32_t qa[D / 8], qb[D / 8];
      const int ra = row0 + warp * 16 + g, rb = ra + 8;
      const float sa = load_query<D>(a, r, h, p.G, ra, t, qa), sb = load_query<D>(a, r, h, p.G, rb, t, qb);
      __syncthreads();  // the last batch has been read
#pragma unroll
      for (int s = 0; s < D / 16; ++s) frag[warp][s][lane] = make_uint4(qa[2 * s], qb[2 * s], qa[2 * s + 1], qb[2 * s + 1]);
      if (t < 2) {
        const int row = t ? rb : ra;
        float l = INFINITY;  // a row that does not exist or sees nothing adds 0
        if (row < rows)
          l = a.lse[int64_t(h * p.G + row % p.G) * a.total_tokens + r.q0 + row / p.G] * 1.4426950408889634f;
        row_lse[warp][g + 8 * t] = l == -INFINITY ? INFINITY : l;
        row_scale[warp][g + 8 * t] = (t ? sb : sa) * p.scale_log2;
      }
      __syncthreads();
    }
    const int tiles = min(kWarps, (rows - row0 + 15) / 16);
    for (int tl = 0; tl < tiles; ++tl) {
      const int first = row0 + tl * 16, last = min(first + 15, rows - 1);
      if (visible_tokens(r, p.G, last, a.causal) <= tok0) continue;
      float s[4][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint4 q = frag[tl][k][lane];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) mma16816(s[nt], q.x, q.y, q.z, q.w, half2_of(w[nt][k]), half2_of_high(w[nt][k]));
      }
      const float fa = row_scale[tl][g], fb = row_scale[tl][g + 8];
      const float ea = row_lse[tl][g], eb = row_lse[tl][g + 8];
      const bool masked = tok0 + kTokens > visible_tokens(r, p.G, first, a.causal) || !fine[0] || !fine[1];
      const int va = visible_tokens(r, p.G, first + g, a.causal), vb = visible_tokens(r, p.G, first + g + 8, a.causal);
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        float x[4] = {fmaf(s[nt][0], fa * ks[nt >> 1], -ea), fmaf(s[nt][1], fa * ks[nt >> 1], -ea),
                      fmaf(s[nt][2], fb * ks[nt >> 1], -eb), fmaf(s[nt][3], fb * ks[nt >> 1], -eb)};
        if (masked) {
          const int col = tok0 + 8 * nt + 2 * t;
          if (!fine[nt >> 1] || col >= va) x[0] = -INFINITY;
          if (!fine[nt >> 1] || col + 1 >= va) x[1] = -INFINITY;
          if (!fine[nt >> 1] || col >= vb) x[2] = -INFINITY;
          if (!fine[nt >> 1] || col + 1 >= vb) x[3] = -INFINITY;
        }
        sum[nt][0] += ptx::ex2(x[0]) + ptx::ex2(x[2]);
        sum[nt][1] += ptx::ex2(x[1]) + ptx::ex2(x[3]);
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < 4; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = sum[nt][e];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      const int tok = tok0 + 8 * nt + 2 * t + e;
      if (g == nt && tok < r.len) {  // one lane of the eight that hold it
        const int64_t at = (int64_t(b) * c.heads + h) * a.weight_stride + tok;
        a.weights[at] = (a.prev ? a.prev[at] : 0.f) + x;
      }
    }
}

template <int D>
cudaError_t launch_d(const WeightParams& p, cudaStream_t s) {
  const CacheQueryArgs& a = p.a;
  const dim3 grid(unsigned((a.max_seqlen + kWarps * kTokens - 1) / (kWarps * kTokens)), unsigned(a.cache.heads),
                  unsigned(a.cache.batch));
  cache_weights_kernel<D><<<grid, kWeightThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

attn_status launch_cache_weights(const CacheQueryArgs& a, cudaStream_t s) {
  WeightParams p{a, a.num_heads / a.cache.heads, a.scale * 1.4426950408889634f};
  cudaError_t e = cudaErrorInvalidValue;
  switch (a.cache.head_dim) {
    case 32: e = launch_d<32>(p, s); break;
    case 64: e = launch_d<64>(p, s); break;
    case 128: e = launch_d<128>(p, s); break;
  }
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_weights launch");
}

}  // namespace attnmask
