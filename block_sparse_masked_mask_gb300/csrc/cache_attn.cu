// Attention over the 8-bit cache for few query rows (decoding).
//
// Every cached byte is read once and used for at most 16 query rows, so the
// memory bounds it: 2 D bytes per token and key / value head.  The design is
// about keeping loads in flight:
//  * A CTA takes one sequence, key / value head, tile of 16 rows and chunk of
//    the tokens; its four warps take the chunk's groups of 16 tokens in turn
//    and share nothing until the end.
//  * Each lane copies (cp.async) exactly the bytes that it will use itself,
//    kStages groups ahead, into its own places in shared memory: a queue that
//    needs no barrier.
//  * Codes become fp16 in registers (exact) and feed mma.sync m16n8k16.  Lanes
//    take their dimensions and tokens in the order of memory
//    (cache_rows.cuh), so nothing is shuffled; only the values' token pairs are
//    interleaved byte by byte.
// Scores s_j (base 2) are the product times the page's key scale.  The page's
// value scale 2^x is folded into the exponent, w_j = 2^(s_j + x_j - m), with m
// the running maximum of s_j + x_j: weights of all pages share one fp16 range
// in which those that matter to O are near 1, and the sum of 2^(s_j - m) is that
// of w_j 2^-x_j, one multiplication.  m moves only when it would grow by
// more than 2^8.
// Chunks of a long sequence meet in a second kernel through fp32 partial results.
#include "cache_rows.cuh"
#include "ptx.cuh"

namespace attnmask {
namespace {

constexpr int kWarps = 4;
constexpr int kAttnThreads = 32 * kWarps;
constexpr int kStages = 4;  // groups in flight per warp
constexpr int kGroup = 16;  // tokens per group
constexpr int kMost = 32;   // groups per warp at most: a chunk has 2048 tokens or less
constexpr float kRaise = 8.f;

template <int D>
struct AttnCfg {
  // A lane copies a group in eight pieces: two of the keys of two tokens each,
  // one of the values of four tokens.
  static constexpr int PIECE = D / 8;
  static constexpr int STAGE = 32 * 8 * PIECE;  // per warp
  static constexpr int QUEUE = kWarps * kStages * STAGE;
  static constexpr int MERGE = kWarps * 16 * (D + 2) * 4;
  static constexpr int SMEM = QUEUE > MERGE ? QUEUE : MERGE;
};

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool on) {
  const int n = on ? BYTES : 0;  // nothing read, zeros stored
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kAttnThreads, 3) cache_attn_kernel(const CacheAttnParams p) {
  using C = AttnCfg<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  const CacheQueryArgs& a = p.a;
  const CacheView& c = a.cache;
  const int split = blockIdx.x / p.row_tiles, row0 = (blockIdx.x % p.row_tiles) * 16;
  const int h = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  SeqRows r;
  if (!load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, a.max_seqlen, c.status, r)) return;
  const int rows = min(16, r.n * p.G - row0);
  if (rows <= 0) return;
  // tokens that some row of the tile sees: the last row sees most
  const int limit = visible_tokens(r, p.G, row0 + rows - 1, a.causal);
  const int begin = split * p.chunk, end = min(begin + p.chunk, limit);
  if (split > 0 && begin >= end) return;  // chunk 0 also answers for rows that see nothing

  const uint32_t queue = ptx::smem_addr(smem) + warp * kStages * C::STAGE;
  const uint8_t* queue_ptr = smem + warp * kStages * C::STAGE;
  const int groups = end > begin ? (end - begin + kGroup - 1) / kGroup : 0;
  const int mine = groups > warp ? (groups - warp + kWarps - 1) / kWarps : 0;
  const int64_t page_bytes = int64_t(D) << c.page_log2;

  // Lane i looks up the page of the warp's i-th group and its scales (at most
  // kMost groups per warp), once; they travel by shuffle.  A page that is left
  // out has scale 0: none of its tokens is visible.
  int my_page = -1;
  float my_ks = 0.f, my_vs = 0.f;
  if (lane < mine) {
    my_page = load_page(c, b, (begin + (warp + lane * kWarps) * kGroup) >> c.page_log2);
    if (my_page >= 0) {
      my_ks = c.k_scale[int64_t(my_page) * c.heads + h];
      my_vs = c.v_scale[int64_t(my_page) * c.heads + h];
    }
  }
  auto issue = [&](int i) {
    const int page = __shfl_sync(0xffffffffu, my_page, i & 31);
    if (i < mine) {
      const int tok = begin + (warp + i * kWarps) * kGroup;
      const int slot = tok & ((1 << c.page_log2) - 1);
      const int64_t base = (int64_t(max(page, 0)) * c.heads + h) * page_bytes + int64_t(slot) * D;
      const uint8_t* kp = c.k_pages + base + g * D + t * C::PIECE;
      const uint8_t* vp = c.v_pages + base + 2 * t * D + g * C::PIECE;
      const uint32_t dst = queue + (i % kStages) * C::STAGE + lane * C::PIECE;
      const int left = page >= 0 ? end - tok : 0;  // tokens of the group; zeros behind them
      // piece j of lane l at (j * 32 + l) * PIECE: no bank conflicts either way
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          copy_async<C::PIECE>(dst + (2 * nt + x) * 32 * C::PIECE, kp + nt * 8 * D + x * (D / 2), 8 * nt + g < left);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int tk = 8 * (q >> 1) + (q & 1);
        copy_async<C::PIECE>(dst + (4 + q) * 32 * C::PIECE, vp + tk * D, tk + 2 * t < left);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);

  // the queries of rows g and g + 8
  uint32_t qa[D / 8], qb[D / 8];
  const float sa = load_query<D>(a, r, h, p.G, row0 + g, t, qa) * p.scale_log2;
  const float sb = load_query<D>(a, r, h, p.G, row0 + g + 8, t, qb) * p.scale_log2;
  const int va = visible_tokens(r, p.G, row0 + g, a.causal), vb = visible_tokens(r, p.G, row0 + g + 8, a.causal);
  const int least = visible_tokens(r, p.G, row0, a.causal);  // tokens that every row sees

  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;

  for (int i = 0; i < mine; ++i) {
    issue(i + kStages - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    const uint8_t* st = queue_ptr + (i % kStages) * C::STAGE + lane * C::PIECE;
    const float ks = __shfl_sync(0xffffffffu, my_ks, i), vs = __shfl_sync(0xffffffffu, my_vs, i);
    const int tok = begin + (warp + i * kWarps) * kGroup;

    float s[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t w[C::PIECE / 4];
#pragma unroll
        for (int y = 0; y < C::PIECE / 4; ++y)
          w[y] = reinterpret_cast<const uint32_t*>(st + (2 * nt + x) * 32 * C::PIECE)[y];
#pragma unroll
        for (int y = 0; y < C::PIECE / 4; ++y) {
          const int step = x * (C::PIECE / 4) + y;
          mma16816(s[nt], qa[2 * step], qb[2 * step], qa[2 * step + 1], qb[2 * step + 1], half2_of(w[y]),
                   half2_of_high(w[y]));
        }
      }
    }
    const float x = float(exponent_of(vs)), inv_vs = pow2f(max(-126, -exponent_of(vs)));
    const float fa = sa * ks, fb = sb * ks;
    float pw[2][4];
    const bool masked = tok + kGroup > least || vs == 0.f;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      pw[nt][0] = fmaf(s[nt][0], fa, x);
      pw[nt][1] = fmaf(s[nt][1], fa, x);
      pw[nt][2] = fmaf(s[nt][2], fb, x);
      pw[nt][3] = fmaf(s[nt][3], fb, x);
      if (masked) {
        const int col = tok + 8 * nt + 2 * t;
        if (vs == 0.f || col >= min(va, end)) pw[nt][0] = -INFINITY;
        if (vs == 0.f || col + 1 >= min(va, end)) pw[nt][1] = -INFINITY;
        if (vs == 0.f || col >= min(vb, end)) pw[nt][2] = -INFINITY;
        if (vs == 0.f || col + 1 >= min(vb, end)) pw[nt][3] = -INFINITY;
      }
    }
    float xa = fmaxf(fmaxf(pw[0][0], pw[0][1]), fmaxf(pw[1][0], pw[1][1]));
    float xb = fmaxf(fmaxf(pw[0][2], pw[0][3]), fmaxf(pw[1][2], pw[1][3]));
    if (__any_sync(0xffffffffu, xa > ma + kRaise || xb > mb + kRaise)) {
      xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 1));
      xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 2));
      xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 1));
      xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 2));
      const float na = fmaxf(ma, xa), nb = fmaxf(mb, xb);
      const float ra = ma == -INFINITY ? 0.f : ptx::ex2(ma - na), rb = mb == -INFINITY ? 0.f : ptx::ex2(mb - nb);
      ma = na;
      mb = nb;
      la *= ra;
      lb *= rb;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        o[k][0] *= ra;
        o[k][1] *= ra;
        o[k][2] *= rb;
        o[k][3] *= rb;
      }
    }
    const float ua = ma == -INFINITY ? 0.f : ma, ub = mb == -INFINITY ? 0.f : mb;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      pw[nt][0] = ptx::ex2(pw[nt][0] - ua);
      pw[nt][1] = ptx::ex2(pw[nt][1] - ua);
      pw[nt][2] = ptx::ex2(pw[nt][2] - ub);
      pw[nt][3] = ptx::ex2(pw[nt][3] - ub);
    }
    la = fmaf((pw[0][0] + pw[0][1]) + (pw[1][0] + pw[1][1]), inv_vs, la);
    lb = fmaf((pw[0][2] + pw[0][3]) + (pw[1][2] + pw[1][3]), inv_vs, lb);
    const uint32_t a0 = pack_half2(pw[0][0], pw[0][1]), a1 = pack_half2(pw[0][2], pw[0][3]);
    const uint32_t a2 = pack_half2(pw[1][0], pw[1][1]), a3 = pack_half2(pw[1][2], pw[1][3]);
    // values: tokens 2t, 2t + 1 and 2t + 8, 2t + 9, dimensions g D/8 ..
    uint32_t v[4][C::PIECE / 4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int y = 0; y < C::PIECE / 4; ++y)
        v[q][y] = reinterpret_cast<const uint32_t*>(st + (4 + q) * 32 * C::PIECE)[y];
#pragma unroll
    for (int y = 0; y < C::PIECE / 4; ++y) {
      const uint32_t l0 = __byte_perm(v[0][y], v[1][y], 0x5140), l1 = __byte_perm(v[0][y], v[1][y], 0x7362);
      const uint32_t h0 = __byte_perm(v[2][y], v[3][y], 0x5140), h1 = __byte_perm(v[2][y], v[3][y], 0x7362);
      mma16816(o[4 * y], a0, a1, a2, a3, half2_of(l0), half2_of(h0));
      mma16816(o[4 * y + 1], a0, a1, a2, a3, half2_of_high(l0), half2_of_high(h0));
      mma16816(o[4 * y + 2], a0, a1, a2, a3, half2_of(l1), half2_of(h1));
      mma16816(o[4 * y + 3], a0, a1, a2, a3, half2_of_high(l1), half2_of_high(h1));
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  la += __shfl_xor_sync(0xffffffffu, la, 1);
  la += __shfl_xor_sync(0xffffffffu, la, 2);
  lb += __shfl_xor_sync(0xffffffffu, lb, 1);
  lb += __shfl_xor_sync(0xffffffffu, lb, 2);

  // ---- the warps' results meet in shared memory (the queues are done)
  __syncthreads();
  float* mo = reinterpret_cast<float*>(smem);               // [warp][16][D]
  float* ml = mo + kWarps * 16 * D;                         // [warp][16][2]
  float* mine_o = mo + warp * 16 * D;
#pragma unroll
  for (int k = 0; k < D / 8; ++k) {
    // column 2t (2t + 1) of product k is dimension (2t) D/8 + k ((2t + 1) D/8 + k)
    mine_o[g * D + 2 * t * C::PIECE + k] = o[k][0];
    mine_o[g * D + (2 * t + 1) * C::PIECE + k] = o[k][1];
    mine_o[(g + 8) * D + 2 * t * C::PIECE + k] = o[k][2];
    mine_o[(g + 8) * D + (2 * t + 1) * C::PIECE + k] = o[k][3];
  }
  if (t == 0) {
    ml[(warp * 16 + g) * 2] = ma;
    ml[(warp * 16 + g) * 2 + 1] = la;
    ml[(warp * 16 + g + 8) * 2] = mb;
    ml[(warp * 16 + g + 8) * 2 + 1] = lb;
  }
  __syncthreads();
  for (int at = threadIdx.x * 2; at < rows * D; at += kAttnThreads * 2) {
    const int row = at / D, d = at % D;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml[(w * 16 + row) * 2]);
    float l = 0.f, x0 = 0.f, x1 = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = ml[(w * 16 + row) * 2];
      const float f = mw == -INFINITY ? 0.f : ptx::ex2(mw - m);
      // a NaN sum stays one even where no maximum was found
      const float lw = ml[(w * 16 + row) * 2 + 1];
      l += lw != lw ? lw : f * lw;
      const float2 y = *reinterpret_cast<const float2*>(mo + (w * 16 + row) * D + d);
      x0 = fmaf(f, y.x, x0);
      x1 = fmaf(f, y.y, x1);
    }
    const int rg = row0 + row;
    const int head = h * p.G + rg % p.G;
    const int64_t token = r.q0 + rg / p.G;
    if (p.splits == 1) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.o) + (token * a.num_heads + head) * D + d);
      *out = ptx::pack_bf16(x0 * inv, x1 * inv);
      if (d == 0) a.lse[int64_t(head) * a.total_tokens + token] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    } else {
      const int64_t at_row = (int64_t(split) * a.total_tokens + token) * a.num_heads + head;
      *reinterpret_cast<float2*>(p.part_o + at_row * D + d) = make_float2(x0, x1);
      if (d == 0) p.part_m[at_row] = make_float2(m, l);
    }
  }
}

// Joins the chunks of each row, one warp per row, in the order of the chunks.
template <int D>
__global__ void __launch_bounds__(128) cache_combine_kernel(const CacheAttnParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const CacheQueryArgs& a = p.a;
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int i = blockIdx.x * 4 + (threadIdx.x >> 5);  // row of the sequence: token i / H, head i % H
  SeqRows r;
  if (!load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, a.max_seqlen, a.cache.status, r)) return;
  if (i >= r.n * a.num_heads) return;
  const int head = i % a.num_heads;
  const int64_t token = r.q0 + i / a.num_heads;
  // the chunks that this row's tile had
  const int rg = (i / a.num_heads) * p.G + head % p.G;
  const int last = min(rg / p.tile_rows * p.tile_rows + p.tile_rows - 1, r.n * p.G - 1);
  const int limit = visible_tokens(r, p.G, last, a.causal);
  const int n = max(1, (limit + p.chunk - 1) / p.chunk);
  const int64_t step = int64_t(a.total_tokens) * a.num_heads;
  const int64_t at = token * a.num_heads + head;
  float m = -INFINITY;
  for (int s = lane; s < n; s += 32) m = fmaxf(m, p.part_m[s * step + at].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.f, x[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) x[e] = 0.f;
  for (int s = 0; s < n; ++s) {
    const float2 ml = p.part_m[s * step + at];
    const float f = ml.x == -INFINITY ? 0.f : ptx::ex2(ml.x - m);
    l += ml.y != ml.y ? ml.y : f * ml.y;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) x[e] = fmaf(f, p.part_o[(s * step + at) * D + e * 32 + lane], x[e]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < D / 32; ++e)
    static_cast<__nv_bfloat16*>(a.o)[at * D + e * 32 + lane] = __float2bfloat16_rn(x[e] * inv);
  if (lane == 0)
    a.lse[int64_t(head) * a.total_tokens + token] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// Tiles, chunks and their number.  More than 16 rows of a key / value head go to
// the tcgen05 kernel (cache_chunk.cu), which reads the cache once for 256.
// Chunks: enough CTAs to fill the GPU about twice over; for few rows none below
// 256 tokens, where a CTA's start and end cost more than its reads, and none above
// 1024, so that sequences of different lengths spread evenly; for many rows, one
// CTA per SM, 1024 to 4096.  The number of SMs only sizes the work, and the
// size query runs without a device, so it is that of the GPU this library is
// built for.
void plan(CacheAttnParams* p) {
  constexpr int64_t kSms = 152;
  const CacheQueryArgs& a = p->a;
  p->G = a.num_heads / a.cache.heads;
  const int64_t rows = int64_t(a.max_new) * p->G;
  const bool many = rows > kFewRows;
  p->tile_rows = many ? kManyRows : kFewRows;
  p->row_tiles = int((rows + p->tile_rows - 1) / p->tile_rows);
  const int64_t items = int64_t(p->row_tiles) * a.cache.heads * a.cache.batch;
  const int64_t fill = (many ? 2 : 6) * kSms, least = many ? 1024 : 256, most = many ? 4096 : 1024;
  static_assert(1024 <= kMost * kWarps * kGroup, "a warp's groups fit its lanes");
  const int64_t want = items > 0 ? (fill + items - 1) / items : 1;
  int64_t chunk = (int64_t(a.max_seqlen) + want - 1) / want;
  chunk = (chunk + kTile - 1) / kTile * kTile;
  chunk = chunk < least ? least : (chunk > most ? most : chunk);
  p->chunk = int(chunk);
  p->splits = int((int64_t(a.max_seqlen) + chunk - 1) / chunk);
  if (p->splits < 1) p->splits = 1;
}

template <int D>
cudaError_t launch_few(const CacheAttnParams& p, cudaStream_t s) {
  using C = AttnCfg<D>;
  cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const dim3 grid(unsigned(p.splits) * unsigned(p.row_tiles), unsigned(p.a.cache.heads), unsigned(p.a.cache.batch));
  cache_attn_kernel<D><<<grid, kAttnThreads, C::SMEM, s>>>(p);
  return cudaGetLastError();
}

// The joining kernel is launched early and waits for the first one's end.
template <int D>
cudaError_t launch_combine(const CacheAttnParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((int64_t(p.a.max_new) * p.a.num_heads + 3) / 4), unsigned(p.a.cache.batch));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_combine_kernel<D>, p);
}

}  // namespace

uint64_t cache_fwd_workspace(const CacheView& c, int total_tokens, int num_heads, int max_new, int max_seqlen) {
  CacheAttnParams p;
  p.a.cache = c;
  p.a.num_heads = num_heads;
  p.a.max_new = max_new;
  p.a.max_seqlen = max_seqlen;
  plan(&p);
  if (p.splits == 1) return 0;
  const uint64_t rows = uint64_t(p.splits) * uint64_t(total_tokens) * uint64_t(num_heads);
  return rows * uint64_t(c.head_dim) * 4 + rows * 8;
}

attn_status launch_cache_fwd(const CacheQueryArgs& a, cudaStream_t s) {
  CacheAttnParams p;
  p.a = a;
  plan(&p);
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.part_o = a.workspace;
  p.part_m = reinterpret_cast<float2*>(a.workspace + uint64_t(p.splits) * uint64_t(a.total_tokens) *
                                                         uint64_t(a.num_heads) * uint64_t(a.cache.head_dim));
  const int d = a.cache.head_dim;
  cudaError_t e = cudaSuccess;
  if (p.tile_rows == kManyRows) {
    const attn_status st = launch_cache_chunk(p, s);
    if (st != ATTN_OK) return st;
  } else {
    e = d == 32 ? launch_few<32>(p, s) : d == 64 ? launch_few<64>(p, s) : launch_few<128>(p, s);
  }
  if (e == cudaSuccess && p.splits > 1)
    e = d == 32 ? launch_combine<32>(p, s) : d == 64 ? launch_combine<64>(p, s) : launch_combine<128>(p, s);
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_fwd launch");
}

}  // namespace attnmask
