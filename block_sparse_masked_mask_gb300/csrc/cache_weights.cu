// The attention weight that each cached token receives from a call's queries:
// the columns of exp(scale q k - LSE) summed over the query rows that share a
// key / value head.
//
// The keys are read once (D bytes per token and head), which bounds it for a
// decode step; the LSE is known, so no second pass and no running maximum.  The
// tokens are divided evenly among the CTAs and queued as in cache_attn.cu; a warp
// takes 32 of them at a time, holds their keys as fp16 A operands of mma.sync
// m16n8k16 and walks the query rows 8 at a time, which the CTA has staged in
// shared memory in operand order.
// Up to 24 rows of a key / value head.  More go to cache_weights_many.cu: measured
// there / here, D = 128, 32 sequences of 8 heads, 16 rows 46 / 38 us, 24 rows 47 /
// 43, 32 rows 47 / 52; 8 sequences of 16 heads, 16 rows 18.7 / 17.1, 32 rows 18.9 /
// 21.4, 64 rows 22 / 32; 4 sequences of 8192, 512 rows 81 / 158.
// 32 sequences of 1024 to 16384 tokens, 4 rows: 35 us, 26 at the copy rate.
// Every token's sum is formed by one warp in a fixed order: no atomics, repeats
// are bit-identical.
#include "cache_rows.cuh"
#include "ptx.cuh"

namespace attnmask {
namespace {

constexpr int kWeightThreads = 32 * kWarps;
constexpr int kCtas = 4;       // per SM; 3 with a third stage: 38 us where 4 take 35
constexpr int kStages = 2;     // of the queue, blocks
constexpr int kBlock = 32;     // tokens a warp takes at a time
constexpr int kRowTiles = 3;   // of 8 query rows
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct WeightCfg {
  using Tile = GroupTile<D>;
  static constexpr int STAGE = 2 * Tile::BYTES;  // two groups' keys, per warp
  static constexpr int QUEUE = kWarps * kStages * STAGE;
  static constexpr int FRAG = D / 16 * 32 * 8;  // a row tile's B operands
  static constexpr int OFF_FRAG = QUEUE;
  static constexpr int OFF_ROWS = OFF_FRAG + kRowTiles * FRAG;  // per row: scale, LSE, visible
  static constexpr int SMEM = OFF_ROWS + kRowTiles * 8 * 16;
};

struct WeightParams {
  CacheQueryArgs a;
  int G, ctas;
  float scale_log2;
};

// Units of sequence b and all heads (its tokens, also where it has no query).
struct WeightUnits {
  const WeightParams& p;
  bool note;
  __device__ int operator()(int b) const {
    const CacheQueryArgs& a = p.a;
    SeqRows r;
    if (!load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, a.max_seqlen, a.cache.status, r, note)) return 0;
    return (r.len + kUnit - 1) / kUnit * a.cache.heads;
  }
};

template <int D>
__global__ void __launch_bounds__(kWeightThreads, kCtas) cache_weights_kernel(const WeightParams p) {
  using C = WeightCfg<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  const CacheQueryArgs& a = p.a;
  const CacheView& c = a.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const WeightUnits units{p, blockIdx.x == 0};
  const UnitLine line(units, c.batch, lane);
  const int piece = (line.total + p.ctas - 1) / p.ctas;
  int pos = blockIdx.x * piece;
  const int stop = min(pos + piece, line.total);
  if (pos >= stop) return;
  int before;
  int b = line.find(units, c.batch, lane, pos, before);

  uint8_t* queue = smem + warp * kStages * C::STAGE;
  const uint32_t queue_addr = ptx::smem_addr(queue);
  uint2* frag = reinterpret_cast<uint2*>(smem + C::OFF_FRAG);    // [row tile][step][lane]
  float4* row_of = reinterpret_cast<float4*>(smem + C::OFF_ROWS);  // scale, LSE (base 2), visible

  while (pos < stop) {
    // ---- the segment: units u0 .. u1 - 1 of sequence b, head h
    SeqRows r;
    const bool good = load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, a.max_seqlen, c.status, r, false);
    const int U = good ? (r.len + kUnit - 1) / kUnit : 0;
    if (U == 0) {
      ++b;
      continue;
    }
    const int h = (pos - before) / U, u0 = (pos - before) - h * U, u1 = min(U, u0 + stop - pos);
    const int rows = r.n * p.G;
    const int begin = u0 * kUnit, end = min(u1 * kUnit, r.len);
    const int blocks = (end - begin + kBlock - 1) / kBlock;
    const int mine = blocks > warp ? (blocks - warp + kWarps - 1) / kWarps : 0;
    auto token_of = [&](int i) { return begin + (warp + i * kWarps) * kBlock; };
    const int64_t out = (int64_t(b) * c.heads + h) * a.weight_stride;

    // lane 2 i + x: the x-th 16 tokens of the i-th block; 16 blocks at a time, a batch ahead
    auto has = [&](int first) {
      const int i = first + lane / 2;
      return i < mine && token_of(i) + (lane & 1) * kGroup < end;
    };
    auto numbers = [&](int first) {
      return page_number(c, b, token_of(first + lane / 2) + (lane & 1) * kGroup, has(first));
    };
    auto issue = [&](int i, int from) {
      const int page[2] = {__shfl_sync(0xffffffffu, from, (2 * i) & 31), __shfl_sync(0xffffffffu, from, (2 * i + 1) & 31)};
      if (i < mine) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int tok = token_of(i) + half * kGroup;
          const bool fine = in_pool(c, page[half]);
          const int64_t base = (((int64_t(fine ? page[half] : 0) * c.heads + h) << c.page_log2) +
                                (tok & ((1 << c.page_log2) - 1))) * D;
          C::Tile::template copy<false>(queue_addr + (i % kStages) * C::STAGE + half * C::Tile::BYTES,
                                        c.k_pages + base, fine ? end - tok : 0, lane);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int number = numbers(0), number_next = numbers(16);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i, number);
    PageBatch now = with_scales(c, h, number, has(0), false);
    PageBatch next = with_scales(c, h, number_next, has(16), false);

    // ---- the rows: warp w stages tiles w, w + 4
    const int tiles = (rows + 7) / 8;
    __syncthreads();  // the last segment's rows have been read
    for (int x = warp; x < tiles; x += kWarps) {
      uint32_t q[D / 8];
      const int row = 8 * x + g;
      const float s = load_query<D>(a, r, h, p.G, row, t, q) * p.scale_log2;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) frag[(x * (D / 16) + k) * 32 + lane] = make_uint2(q[2 * k], q[2 * k + 1]);
      if (t == 0) {
        float e = INFINITY;  // a row that does not exist or sees nothing adds 0
        if (row < rows) e = a.lse[int64_t(h * p.G + row % p.G) * a.total_tokens + r.q0 + row / p.G] * kLog2e;
        row_of[8 * x + g] = make_float4(s, e == -INFINITY ? INFINITY : e,
                                        __int_as_float(visible_tokens(r, p.G, row, a.causal)), 0.f);
      }
    }
    __syncthreads();
    const int least = visible_tokens(r, p.G, 0, a.causal);  // tokens that all rows see
    const int most = rows > 0 ? visible_tokens(r, p.G, rows - 1, a.causal) : 0;

    for (int i = 0; i < mine; ++i) {
      if (i > 0 && (i & 15) == 0) {
        now = next;
        next = with_scales(c, h, numbers(i + 16), has(i + 16), false);
      }
      __syncwarp();  // the slot's last block has been read
      issue(i + kStages - 1, (((i + kStages - 1) ^ i) >> 4) ? next.number : now.number);
      const int tok = token_of(i);
      // what the sums are added to: tokens tok + lane, read early
      float was = 0.f;
      if (a.prev && tok + lane < end) was = a.prev[out + tok + lane];
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();  // every lane's copies are here
      const uint8_t* st = queue + (i % kStages) * C::STAGE;
      const float ks[2] = {__shfl_sync(0xffffffffu, now.k_scale, (2 * i) & 31),
                           __shfl_sync(0xffffffffu, now.k_scale, (2 * i + 1) & 31)};
      uint32_t k[2][D / 16][4];  // A operands: tokens 16 half + g, + 8
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t w0[D / 32], w1[D / 32];
          const int at = x * (D / 2) + t * (D / 8);
          C::Tile::template read<false>(st + half * C::Tile::BYTES, g, at, w0);
          C::Tile::template read<false>(st + half * C::Tile::BYTES, 8 + g, at, w1);
#pragma unroll
          for (int y = 0; y < D / 32; ++y) {
            uint32_t* to = k[half][x * (D / 32) + y];
            to[0] = half2_of(w0[y]);
            to[1] = half2_of(w1[y]);
            to[2] = half2_of_high(w0[y]);
            to[3] = half2_of_high(w1[y]);
          }
        }
      float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};  // tokens 16 half + g, + 8
      if (tok < most) {
        const bool masked = tok + kBlock > least || ks[0] == 0.f || ks[1] == 0.f;  // scale 0: left out
        for (int x = 0; x < tiles; ++x) {
          float s[2][4];
#pragma unroll
          for (int half = 0; half < 2; ++half) s[half][0] = s[half][1] = s[half][2] = s[half][3] = 0.f;
#pragma unroll
          for (int y = 0; y < D / 16; ++y) {
            const uint2 q = frag[(x * (D / 16) + y) * 32 + lane];
#pragma unroll
            for (int half = 0; half < 2; ++half)
              mma16816(s[half], k[half][y][0], k[half][y][1], k[half][y][2], k[half][y][3], q.x, q.y);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 row = row_of[8 * x + 2 * t + e];
            const int visible = __float_as_int(row.z);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const float f = row.x * ks[half];
              float w0 = fmaf(s[half][e], f, -row.y), w1 = fmaf(s[half][2 + e], f, -row.y);
              if (masked) {
                const bool gone = ks[half] == 0.f;
                if (gone || tok + 16 * half + g >= visible) w0 = -INFINITY;
                if (gone || tok + 16 * half + g + 8 >= visible) w1 = -INFINITY;
              }
              sum[half][0] += ptx::ex2(w0);
              sum[half][1] += ptx::ex2(w1);
            }
          }
        }
      }
      // over the four lanes of a token; lane 4 g + t then stores token 8 t + g
      float mine_sum = 0.f;
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = sum[half][e];
          x += __shfl_xor_sync(0xffffffffu, x, 1);
          x += __shfl_xor_sync(0xffffffffu, x, 2);
          if (t == 2 * half + e) mine_sum = x;
        }
      const int at = 8 * t + g;
      was = __shfl_sync(0xffffffffu, was, at);
      if (tok + at < end) a.weights[out + tok + at] = was + mine_sum;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    pos += u1 - u0;
    if (pos == before + U * c.heads) {
      before = pos;
      ++b;
    }
  }
}

template <int D>
cudaError_t launch_d(const WeightParams& p, cudaStream_t s) {
  using C = WeightCfg<D>;
  const cudaError_t e =
      cudaFuncSetAttribute(cache_weights_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  cache_weights_kernel<D><<<unsigned(p.ctas), kWeightThreads, C::SMEM, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

attn_status launch_cache_weights(const CacheQueryArgs& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return record_cuda_error(e, "attn_cache_weights device query");
  if (int64_t(a.max_new) * (a.num_heads / a.cache.heads) > 8 * kRowTiles) return launch_cache_weights_many(a, sms, s);
  WeightParams p{a, a.num_heads / a.cache.heads, kCtas * sms, a.scale * kLog2e};
  e = cudaErrorInvalidValue;
  switch (a.cache.head_dim) {
    case 32: e = launch_d<32>(p, s); break;
    case 64: e = launch_d<64>(p, s); break;
    case 128: e = launch_d<128>(p, s); break;
  }
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_weights launch");
}

}  // namespace attnmask
