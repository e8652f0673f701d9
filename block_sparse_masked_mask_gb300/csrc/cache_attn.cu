// Attention over the 8-bit cache for few query rows (decoding).
//
// Every cached byte is read once and used for at most 16 query rows, so the
// memory bounds it: 2 D bytes per token and key / value head.  The design is
// about keeping loads in flight:
//  * The tokens of all sequences and heads are divided evenly among the CTAs
//    (cache_rows.cuh).  A CTA walks its piece segment by segment (one sequence
//    and head each); its four warps take a segment's groups of 16 tokens in
//    turn and share nothing until the segment's end.
//  * Each warp has a queue of its own in shared memory, filled by cp.async
//    kStages - 1 groups ahead.
//  * Codes become fp16 in registers (exact) and feed mma.sync m16n8k16, with the
//    tokens (and then the dimensions) as M and the rows as N = 8 or 16: a
//    decode step's few rows waste little of a product.  Lanes take their
//    dimensions and tokens in the order of memory; the values' token pairs are
//    interleaved byte by byte, the weights turned by movmatrix.
// Scores s_j (base 2) are the product times the page's key scale.  The page's
// value scale 2^x is folded into the exponent, w_j = 2^(s_j + x_j - m), with m
// 2^7 below the running maximum of s_j + x_j: weights of all pages share one fp16
// range, and the sum of 2^(s_j - m) is that of w_j 2^-x_j, one multiplication.  m
// moves only when a weight would pass 2^15, the top of that range: the largest is
// between 2^7 and 2^15, and fp16's least step, 2^-24, is 2^-31 of it at most (with
// the largest at 1, thousands of tokens below 2^-25 of it would be lost in O).
// That sum does not depend on the values, and its terms span more
// than an exponential: where exponents of pages lie more than kSpread apart (a page of
// zeros has 2^-80) they are taken as squares of 2^((s_j - m) / 2), and so are the
// factors of sums whose reference moves (half_factor).  fp32 holds them: the
// largest sum, of 2^30 tokens, is 2^125, and one that a page of 2^120 dominates is 2^-113.
// A (sequence, head) that lies in one CTA's piece is finished there; the others
// meet in a second kernel through fp32 partial results, two per CTA at most.
// Few or short sequences go another way: a cluster of up to eight CTAs takes each
// (sequence, head) and joins its results through shared memory (team_of).
// Measured, 64 requests of 1024 to 16384 tokens, 8 heads, D = 128: 118 us, 84% of the
// copy rate; 16 of 8192, 16 rows 63 us, 63%; a single one of 2049 tokens 8.4 us.
#include <algorithm>
#include <cmath>

#include "cache_join.cuh"
#include "cache_rows.cuh"
#include "ptx.cuh"

namespace attnmask {
namespace {

constexpr int kAttnThreads = 32 * kWarps;
constexpr int kStages = 4;  // of the queue, groups
constexpr int kTeam = 8;    // CTAs of a cluster

template <int D>
struct AttnCfg {
  using Tile = GroupTile<D>;
  static constexpr int STAGE = 2 * Tile::BYTES;  // keys, values
  static constexpr int QUEUE = kWarps * kStages * STAGE;
  static constexpr int MERGE = kWarps * kFewRows * D * 4;  // over the queue
  static constexpr int STATS = QUEUE > MERGE ? QUEUE : MERGE;
  static constexpr int TEAM = STATS + kWarps * kFewRows * 8;  // the CTA's own, for its team
  static constexpr int SMEM = TEAM + kFewRows * 8;
};

// Units of sequence b and all heads: of the tokens that some row sees, at least
// one where there are rows (they get their zeros).
__device__ __forceinline__ int units_of(const SeqRows& r, int G, bool causal) {
  if (r.n == 0) return 0;
  return max(1, (visible_tokens(r, G, r.n * G - 1, causal) + kUnit - 1) / kUnit);
}
struct AttnUnits {
  const CacheAttnParams& p;
  bool note;
  __device__ int operator()(int b) const {
    const CacheQueryArgs& a = p.a;
    SeqRows r;
    if (!load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, a.max_seqlen, a.cache.status, r, note)) return 0;
    return units_of(r, p.G, a.causal) * a.cache.heads;
  }
};
// Units per CTA: an even share, but at least two, where a CTA's start and end
// cost as much as its reads.
__device__ __forceinline__ int share(int total, int ctas) { return max(2, (total + ctas - 1) / ctas); }

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A cluster's results meet in each other's shared memory: every CTA joins its share
// of the rows' elements, in the order of the ranks.
template <int D>
__device__ __forceinline__ void team_join(const CacheAttnParams& p, int b, int h, int rank, const float* mo,
                                          const float2* own) {
  const CacheQueryArgs& a = p.a;
  SeqRows r;
  load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, a.max_seqlen, a.cache.status, r, false);
  const int rows = r.n * p.G;
  ptx::cluster_sync();
  for (int at = (rank * kAttnThreads + threadIdx.x) * 4; at < rows * D; at += p.team * kAttnThreads * 4) {
    const int row = at / D, d = at % D;
    float2 s[kTeam];
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kTeam; ++k) {
      s[k] = k < p.team ? ptx::load_peer(own + row, k) : make_float2(-INFINITY, 0.f);
      top = fmaxf(top, s[k].x);
    }
    float sum = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kTeam; ++k) {
      const float half = half_factor(s[k].x, top), f = half * half;
      sum += s[k].y != s[k].y ? s[k].y : s[k].y * half * half;
      if (f > 0.f) {
        const float4 z = ptx::load_peer(reinterpret_cast<const float4*>(mo + row * D + d), k);
        y.x = fmaf(f, z.x, y.x);
        y.y = fmaf(f, z.y, y.y);
        y.z = fmaf(f, z.z, y.z);
        y.w = fmaf(f, z.w, y.w);
      }
    }
    const int head = h * p.G + row % p.G;
    const int64_t token = r.q0 + row / p.G;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + (token * a.num_heads + head) * D + d) =
        make_uint2(ptx::pack_bf16(y.x * inv, y.y * inv), ptx::pack_bf16(y.z * inv, y.w * inv));
    if (d == 0) a.lse[int64_t(head) * a.total_tokens + token] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
  ptx::cluster_sync();  // nobody leaves while others read
}

// NT: tiles of 8 rows
template <int D, int NT>
__global__ void __launch_bounds__(kAttnThreads, 3) cache_attn_kernel(const CacheAttnParams p) {
  using C = AttnCfg<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  const CacheQueryArgs& a = p.a;
  const CacheView& c = a.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int b, pos, stop, before = 0;
  const int rank = p.team > 1 ? blockIdx.x % p.team : 0;  // in the cluster
  if (p.team > 0) {
    const int item = blockIdx.x / p.team, h = item % c.heads;
    b = item / c.heads;
    const int U = AttnUnits{p, h == 0 && rank == 0}(b) / c.heads;
    if (U == 0) return;  // the whole team
    pos = h * U + int(int64_t(U) * rank / p.team);
    stop = h * U + int(int64_t(U) * (rank + 1) / p.team);
  } else {
    const AttnUnits units{p, blockIdx.x == 0};
    const UnitLine line(units, c.batch, lane);
    const int piece = share(line.total, p.ctas);
    pos = blockIdx.x * piece;
    stop = min(pos + piece, line.total);
    if (pos < stop) b = line.find(units, c.batch, lane, pos, before);
  }
  if (pos >= stop && p.team <= 1) return;

  uint8_t* queue = smem + warp * kStages * C::STAGE;
  const uint32_t queue_addr = ptx::smem_addr(queue);
  float* mo = reinterpret_cast<float*>(smem);                  // [warp][8 NT][D]
  float2* ml = reinterpret_cast<float2*>(smem + C::STATS);     // [warp][8 NT]
  float2* own = reinterpret_cast<float2*>(smem + C::TEAM);     // [8 NT]: of the CTA, with its O in mo's first part
  if (threadIdx.x < kFewRows) own[threadIdx.x] = make_float2(-INFINITY, 0.f);

  while (pos < stop) {
    // ---- the segment: units u0 .. u1 - 1 of sequence b, head h
    SeqRows r;
    const bool good = load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, a.max_seqlen, c.status, r, false);
    const int U = good ? units_of(r, p.G, a.causal) : 0;
    if (U == 0) {
      ++b;
      continue;
    }
    const int h = (pos - before) / U, u0 = (pos - before) - h * U, u1 = min(U, u0 + stop - pos);
    const int rows = r.n * p.G;
    const int limit = visible_tokens(r, p.G, rows - 1, a.causal);
    const int begin = u0 * kUnit, end = min(u1 * kUnit, limit);
    const int groups = end > begin ? (end - begin + kGroup - 1) / kGroup : 0;
    const int mine = groups > warp ? (groups - warp + kWarps - 1) / kWarps : 0;
    auto token_of = [&](int i) { return begin + (warp + i * kWarps) * kGroup; };

    // ---- the queue
    int number = page_number(c, b, token_of(lane), lane < mine);
    int number_next = page_number(c, b, token_of(32 + lane), 32 + lane < mine);
    auto issue = [&](int i, int numbers) {
      const int page = __shfl_sync(0xffffffffu, numbers, i & 31);
      if (i < mine) {
        const int tok = token_of(i);
        const bool fine = in_pool(c, page);
        const int64_t base = (((int64_t(fine ? page : 0) * c.heads + h) << c.page_log2) +
                              (tok & ((1 << c.page_log2) - 1))) * D;
        const int left = fine ? end - tok : 0;  // tokens of the group
        const uint32_t dst = queue_addr + (i % kStages) * C::STAGE;
        C::Tile::template copy<false>(dst, c.k_pages + base, left, lane);
        C::Tile::template copy<true>(dst + C::Tile::BYTES, c.v_pages + base, left, lane);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i, number);
    PageBatch now = with_scales(c, h, number, lane < mine, true);
    PageBatch next = with_scales(c, h, number_next, 32 + lane < mine, true);

    // ---- the queries: B operand of row 8 nt + g; scales and limits of rows 8 nt + 2t, + 1
    uint32_t q[NT][D / 8];
    float scale[NT][2], m[NT][2], l[NT][2];
    int visible[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float s = load_query<D>(a, r, h, p.G, 8 * nt + g, t, q[nt]) * p.scale_log2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        scale[nt][e] = __shfl_sync(0xffffffffu, s, 4 * (2 * t + e));
        visible[nt][e] = min(end, visible_tokens(r, p.G, 8 * nt + 2 * t + e, a.causal));
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
      }
    }
    const int least = visible_tokens(r, p.G, 0, a.causal);  // tokens that every row sees
    float o[D / 16][NT][4];
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[k][nt][0] = o[k][nt][1] = o[k][nt][2] = o[k][nt][3] = 0.f;

    int x_top = 0;  // largest exponent of the values so far, if above that of values up to 448
    bool far;       // some pages of this batch lie far below it
    auto compare = [&]() {
      const int x = exponent_of(now.v_scale);  // (-127: no page)
      if (__any_sync(0xffffffffu, x > x_top)) x_top = max(x_top, __reduce_max_sync(0xffffffffu, x));
      far = __any_sync(0xffffffffu, now.v_scale > 0.f && x < x_top - kSpread);
    };
    compare();
    for (int i = 0; i < mine; ++i) {
      if (i > 0 && (i & 31) == 0) {
        now = next;
        compare();
        const bool on = i + 32 + lane < mine;
        next = with_scales(c, h, page_number(c, b, token_of(i + 32 + lane), on), on, true);
      }
      __syncwarp();  // the slot's last group has been read
      issue(i + kStages - 1, (((i + kStages - 1) ^ i) >> 5) ? next.number : now.number);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();  // every lane's copies are here
      const uint8_t* keys = queue + (i % kStages) * C::STAGE;
      const uint8_t* values = keys + C::Tile::BYTES;
      const float ks = __shfl_sync(0xffffffffu, now.k_scale, i & 31), vs = __shfl_sync(0xffffffffu, now.v_scale, i & 31);
      const int tok = token_of(i);

      // S: tokens g, g + 8 by rows 2t, 2t + 1
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t w[2][D / 32];
#pragma unroll
        for (int half = 0; half < 2; ++half)
          C::Tile::template read<false>(keys, 8 * half + g, x * (D / 2) + t * (D / 8), w[half]);
#pragma unroll
        for (int y = 0; y < D / 32; ++y) {
          const int step = x * (D / 32) + y;
          const uint32_t a0 = half2_of(w[0][y]), a1 = half2_of(w[1][y]), a2 = half2_of_high(w[0][y]),
                         a3 = half2_of_high(w[1][y]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], a0, a1, a2, a3, q[nt][2 * step], q[nt][2 * step + 1]);
        }
      }
      const float x = float(exponent_of(vs));
      float inv_vs = pow2f(max(-126, -exponent_of(vs)));
      const bool masked = tok + kGroup > least || vs == 0.f;  // scale 0: the page was left out
      bool raise = far;  // (one check for both rare ways)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f = scale[nt][e] * ks;
          s[nt][e] = fmaf(s[nt][e], f, x);
          s[nt][2 + e] = fmaf(s[nt][2 + e], f, x);
          if (masked) {
            if (vs == 0.f || tok + g >= visible[nt][e]) s[nt][e] = -INFINITY;
            if (vs == 0.f || tok + g + 8 >= visible[nt][e]) s[nt][2 + e] = -INFINITY;
          }
          raise |= fmaxf(s[nt][e], s[nt][2 + e]) > m[nt][e] + kMostWeight;
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(s[nt][e], s[nt][2 + e]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            top = fmaxf(top - kTopWeight, m[nt][e]);
            const float half = half_factor(m[nt][e], top), f = half * half;
            m[nt][e] = top;
            l[nt][e] = l[nt][e] * half * half;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              o[k][nt][e] *= f;
              o[k][nt][2 + e] *= f;
            }
          }
        if (far) {  // the sums here, and not from the weights
          inv_vs = 0.f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float ref = (m[nt][e] == -INFINITY ? 0.f : m[nt][e]) + x;
              const float y0 = ptx::ex2(0.5f * (s[nt][e] - ref)), y1 = ptx::ex2(0.5f * (s[nt][2 + e] - ref));
              l[nt][e] = fmaf(y0, y0, fmaf(y1, y1, l[nt][e]));
            }
        }
      }
      uint32_t w0[NT], w1[NT];  // weights: tokens 2t, 2t + 1 (and + 8) of row g
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float ref = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
          s[nt][e] = ptx::ex2(s[nt][e] - ref);
          s[nt][2 + e] = ptx::ex2(s[nt][2 + e] - ref);
          l[nt][e] = fmaf(s[nt][e] + s[nt][2 + e], inv_vs, l[nt][e]);
        }
        w0[nt] = transposed(pack_half2(s[nt][0], s[nt][1]));
        w1[nt] = transposed(pack_half2(s[nt][2], s[nt][3]));
      }
      // O: dimensions g D/8 + 2k, + 1 by rows 2t, 2t + 1
      uint32_t v[4][D / 32];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        C::Tile::template read<true>(values, 8 * (j >> 1) + 2 * t + (j & 1), g * (D / 8), v[j]);
#pragma unroll
      for (int y = 0; y < D / 32; ++y)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const uint32_t lo = __byte_perm(v[0][y], v[1][y], z ? 0x7362 : 0x5140);
          const uint32_t hi = __byte_perm(v[2][y], v[3][y], z ? 0x7362 : 0x5140);
          const uint32_t a0 = half2_of(lo), a1 = half2_of_high(lo), a2 = half2_of(hi), a3 = half2_of_high(hi);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(o[2 * y + z][nt], a0, a1, a2, a3, w0[nt], w1[nt]);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");

    // ---- the warps' results meet in shared memory (their queues are empty)
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nt][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int row = warp * 8 * NT + 8 * nt + 2 * t + e;
        if (g == 0) ml[row] = make_float2(m[nt][e], sum);
        float2* to = reinterpret_cast<float2*>(mo + row * D + g * (D / 8));
#pragma unroll
        for (int k = 0; k < D / 16; ++k) to[k] = make_float2(o[k][nt][e], o[k][nt][2 + e]);
      }
    __syncthreads();
    const bool whole = p.team <= 1 && u0 == 0 && u1 == U;
    const int slot = 2 * blockIdx.x + (u0 > 0 ? 0 : 1);
    for (int at = threadIdx.x * 4; at < rows * D; at += kAttnThreads * 4) {
      const int row = at / D, d = at % D;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * 8 * NT + row].x);
      float sum = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 s = ml[w * 8 * NT + row];
        const float half = half_factor(s.x, top), f = half * half;
        sum += s.y != s.y ? s.y : s.y * half * half;  // a NaN sum stays one even where no maximum was found
        const float4 z = *reinterpret_cast<const float4*>(mo + (w * 8 * NT + row) * D + d);
        y.x = fmaf(f, z.x, y.x);
        y.y = fmaf(f, z.y, y.y);
        y.z = fmaf(f, z.z, y.z);
        y.w = fmaf(f, z.w, y.w);
      }
      if (whole) {
        const int head = h * p.G + row % p.G;
        const int64_t token = r.q0 + row / p.G;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + (token * a.num_heads + head) * D + d) =
            make_uint2(ptx::pack_bf16(y.x * inv, y.y * inv), ptx::pack_bf16(y.z * inv, y.w * inv));
        if (d == 0) a.lse[int64_t(head) * a.total_tokens + token] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
      } else if (p.team > 0) {
        *reinterpret_cast<float4*>(mo + row * D + d) = y;  // (read by this thread alone)
        if (d == 0) own[row] = make_float2(top, sum);
      } else {
        const int64_t to = int64_t(slot) * (a.max_new * p.G) + row;
        *reinterpret_cast<float4*>(p.part_o + to * D + d) = y;
        if (d == 0) p.part_m[to] = make_float2(top, sum);
      }
    }
    __syncthreads();  // before the next segment's copies
    pos += u1 - u0;
    if (pos == before + U * c.heads && p.team == 0) {
      before = pos;
      ++b;
    }
  }
  if (p.team > 1) team_join<D>(p, b, blockIdx.x / p.team % c.heads, rank, mo, own);
}

constexpr int kJoinWarps = 8;  // per CTA

// Both joining kernels start while the first one ends; every CTA waits for its
// end, those with nothing to join too, so that what follows on the stream does.
// Few rows: W warps per row share its partial results (1 or 8).
template <int D, int W>
__global__ void __launch_bounds__(32 * kJoinWarps) cache_join_few_kernel(const CacheAttnParams p) {
  __shared__ float shared[W > 1 ? W * (D + 2) : 1];
  const CacheQueryArgs& a = p.a;
  const int b = blockIdx.y, w = (threadIdx.x >> 5) % W, lane = threadIdx.x & 31;
  const int i = blockIdx.x * (kJoinWarps / W) + (threadIdx.x >> 5) / W;  // of the sequence: token, head
  SeqRows r;
  const bool good = load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, a.max_seqlen, a.cache.status, r, false);
  const bool mine = good && i < r.n * a.num_heads;
  const int head = i % a.num_heads, row = (i / a.num_heads) * p.G + head % p.G;
  const int U = mine ? units_of(r, p.G, a.causal) : 0;
  // the line before this (sequence, head); the division is the other kernel's
  const AttnUnits units{p, false};
  int all = 0, first = 0;
#pragma unroll 4
  for (int s = lane; s < a.cache.batch; s += 32) {
    const int n = units(s);
    all += n;
    first += s < b ? n : 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    first += __shfl_xor_sync(0xffffffffu, first, o);
  }
  first += (head / p.G) * U;
  const int piece = share(all, p.ctas);
  const int c0 = first / piece, c1 = (first + U - 1) / piece;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!mine || c0 == c1) return;  // finished by its CTA
  auto at = [&](int j) { return int64_t(2 * (c0 + j) + (j == 0 ? 1 : 0)) * (a.max_new * p.G) + row; };
  join_row<D, W>(p, c1 - c0 + 1, at, r.q0 + i / a.num_heads, head, w, lane, shared);
}

// Many rows: a warp per row, over the chunks that the row's tile had.
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) cache_join_many_kernel(const CacheAttnParams p) {
  const CacheQueryArgs& a = p.a;
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int i = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  SeqRows r;
  const bool good = load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, a.max_seqlen, a.cache.status, r, false);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!good || i >= r.n * a.num_heads) return;
  const int head = i % a.num_heads, row = (i / a.num_heads) * p.G + head % p.G;
  const int last = min(row / kManyRows * kManyRows + kManyRows - 1, r.n * p.G - 1);
  const int limit = visible_tokens(r, p.G, last, a.causal);
  const int64_t token = r.q0 + i / a.num_heads, step = int64_t(a.total_tokens) * a.num_heads;
  auto at = [&](int j) { return j * step + token * a.num_heads + head; };
  join_row<D, 1>(p, max(1, (limit + p.chunk - 1) / p.chunk), at, token, head, 0, lane, nullptr);
}

constexpr int64_t kMostPartial = int64_t(512) << 20;

// CTAs that take a (sequence, head) together, as one cluster whose results meet in
// shared memory, with one launch and no workspace; 0: the line of all tokens is cut
// and joined.  As many as the GPU holds at once (456), for up to 1024 tokens each:
// above that, and for sequences of which one alone is long, the line is more
// even.  Measured, line / cluster, D = 128, 8 heads: 1 sequence of 700 tokens 10.2 /
// 7.2 us, 2049 10.9 / 8.4, 8192 13.4 / 13.3, 16384 16.7 / 20.8; with 16 rows, 2049 15.6 /
// 10.8; 4 of 3000 14.0 / 9.9, of 6000 18.5 / 14.7; 8 of 3000 18.8 / 14.4; 16 of 2000 21.1 /
// 17.1.  (D = 32 and 64 follow the same numbers.)  Short sequences are quickest by one CTA: 8 of 300 tokens, by 4 CTAs 7.9 us, by
// one 6.9; 16 of 700, by two 10.0, by one 9.7; 64 of 700, by one 23, the line 27.
int team_of(const CacheQueryArgs& a) {
  const int64_t items = int64_t(a.cache.batch) * a.cache.heads;
  if (a.max_seqlen <= 384) return 1;
  int team = kTeam;
  while (team > 1 && items * team > 456) team /= 2;
  if (team <= 2 && a.max_seqlen <= 768) return 1;
  return items * team <= 456 && a.max_seqlen <= 1024 * team ? team : 0;
}

// Which kernel, and its cut.  More than 16 rows of a key / value head go to the
// tcgen05 kernel (cache_chunk.cu), which reads the cache once for 256, one CTA per
// SM: measured here / there, 16 sequences of 8192, 8 heads, 4 rows 54 / 88 us, 16 rows
// 63 / 89 (there 20 rows 90, 32 rows 91, 128 rows 108); one of 8192, 16 rows 18 / 19.
// Its chunks are of one size: the least number of chunks (of 4096 tokens at
// most), or as many as fill the SMs one to four times, whichever is quickest in
// this estimate, in tokens of a CTA's walk (11 to 20 ns each): a chunk with its
// start and end (384) times the waves, half rounded up, as sequences differ in
// length; and the join, with the bytes of its partial results (8 per element, at
// 5 TB/s).  Measured against chunks of work / SMs tokens: 2 sequences of 4096,
// 300 new, 4 heads 58 -> 43 us; 8 of up to 9000, up to 200 new, D = 64: 72 -> 46;
// 1 of 32768, 512 new, 8 heads 303 -> 284.
// However long the sequences, the partial results stay within kMostPartial bytes,
// about what the backward of the masked attention takes at 32768 tokens: a call whose
// rows need more has over 4000 CTAs (tiles of rows times chunks), 26 per SM, by then.
// (32 / 8 heads, D = 128, behind a bound of 131072: 2048 new tokens 1.09 GB and 4.0
// ms -> 0.51 GB and 3.6 ms; 16384 new 8.7 GB and 30.3 ms -> none and 24.9 ms.)
// The number of SMs only sizes the work, and the size query runs without a
// device, so it is that of the GPU this library is built for.
void plan(CacheAttnParams* p) {
  constexpr int kSms = 152;
  const CacheQueryArgs& a = p->a;
  p->G = a.num_heads / a.cache.heads;
  const int64_t rows = int64_t(a.max_new) * p->G;
  p->many = rows > kFewRows;
  p->team = team_of(a);
  p->ctas = p->team ? a.cache.batch * a.cache.heads * p->team : 3 * kSms;  // (three per SM are resident at once)
  p->row_tiles = int((rows + kManyRows - 1) / kManyRows);
  const int64_t items = int64_t(p->row_tiles) * a.cache.heads * a.cache.batch;
  p->chunk = 256;
  p->splits = 1;
  if (!p->many || items == 0) return;
  const int64_t row_bytes = int64_t(a.total_tokens) * a.num_heads * (4 * a.cache.head_dim + 8);
  const int64_t most = std::max<int64_t>(1, kMostPartial / row_bytes);  // (items > 0: there are rows)
  const int64_t least = std::min((int64_t(a.max_seqlen) + 4095) / 4096, most);
  double best = INFINITY;
  for (int fill = 0; fill <= 4; ++fill) {
    const int64_t n = fill == 0 ? least : std::min<int64_t>(fill * kSms / items, most);
    if (n < least || n < 1) continue;
    int64_t chunk = (int64_t(a.max_seqlen) + n - 1) / n;
    chunk = (chunk + kTile - 1) / kTile * kTile;
    if (chunk < 256) chunk = 256;
    const int64_t splits = a.max_seqlen > 0 ? (int64_t(a.max_seqlen) + chunk - 1) / chunk : 1;
    const double ctas = double(items) * double(splits), waves = ctas / kSms;
    double cost = (waves > 1 ? (waves + ceil(waves)) / 2 : 1) * double(chunk + 384);
    if (splits > 1) cost += 400 + double(splits) * a.total_tokens * a.num_heads * a.cache.head_dim / 6400;
    if (cost >= best) continue;
    best = cost;
    p->chunk = int(chunk);
    p->splits = int(splits);
  }
}

// Rows of partial results.
uint64_t partial_rows(const CacheAttnParams& p) {
  if (p.many) return p.splits == 1 ? 0 : uint64_t(p.splits) * uint64_t(p.a.total_tokens) * uint64_t(p.a.num_heads);
  return p.team ? 0 : 2 * uint64_t(p.ctas) * uint64_t(p.a.max_new) * uint64_t(p.G);
}

template <int D>
cudaError_t launch_few(const CacheAttnParams& p, cudaStream_t s) {
  using C = AttnCfg<D>;
  auto kernel = p.a.max_new * p.G <= 8 ? cache_attn_kernel<D, 1> : cache_attn_kernel<D, 2>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.ctas));
  cfg.blockDim = dim3(kAttnThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(p.team > 1 ? p.team : 1);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// The joining kernel is launched early and waits for the first one's end.
template <int D>
cudaError_t launch_join(const CacheAttnParams& p, cudaStream_t s) {
  const int64_t rows = int64_t(p.a.max_new) * p.a.num_heads;
  // A (sequence, head) meets about ctas / (their number) CTAs; where those are
  // many, a CTA joins each row (one request of 131072 tokens and one head: 128
  // us with a warp per row, 25 us), else a warp does (64 requests of 8 heads: the
  // join takes 12 us with a CTA per row, 5 us with a warp).
  const bool wide = !p.many && int64_t(p.ctas) > 8 * int64_t(p.a.cache.batch) * p.a.cache.heads;
  const int per_cta = wide ? 1 : kJoinWarps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((rows + per_cta - 1) / per_cta), unsigned(p.a.cache.batch));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, p.many ? cache_join_many_kernel<D>
                                         : wide ? cache_join_few_kernel<D, kJoinWarps> : cache_join_few_kernel<D, 1>, p);
}

}  // namespace

uint64_t cache_fwd_workspace(const CacheView& c, int total_tokens, int num_heads, int max_new, int max_seqlen) {
  CacheAttnParams p;
  p.a.cache = c;
  p.a.total_tokens = total_tokens;
  p.a.num_heads = num_heads;
  p.a.max_new = max_new;
  p.a.max_seqlen = max_seqlen;
  plan(&p);
  return partial_rows(p) * (uint64_t(c.head_dim) * 4 + 8);
}

attn_status launch_cache_fwd(const CacheQueryArgs& a, cudaStream_t s) {
  CacheAttnParams p;
  p.a = a;
  plan(&p);
  p.scale_log2 = a.scale * 1.4426950408889634f;
  const uint64_t partial = partial_rows(p);
  p.part_o = a.workspace;
  p.part_m = reinterpret_cast<float2*>(a.workspace + partial * uint64_t(a.cache.head_dim));
  const int d = a.cache.head_dim;
  cudaError_t e = cudaSuccess;
  if (p.many) {
    const attn_status st = launch_cache_chunk(p, s);
    if (st != ATTN_OK) return st;
  } else {
    e = d == 32 ? launch_few<32>(p, s) : d == 64 ? launch_few<64>(p, s) : launch_few<128>(p, s);
  }
  if (e == cudaSuccess && partial > 0)
    e = d == 32 ? launch_join<32>(p, s) : d == 64 ? launch_join<64>(p, s) : launch_join<128>(p, s);
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_fwd launch");
}

}  // namespace attnmask
