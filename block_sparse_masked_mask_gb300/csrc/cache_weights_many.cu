// The attention weight received per cached token (cache_weights.cu) from many
// query rows, on the tcgen05 tensor cores.
//
// The products bound it: 2 D operations per row and token, twice, for the two
// halves of a query; and an exponential each.  So S^T = K Q^T has the tokens as its rows:
// the codes as they lie are the A operand (kind::f8f6f4, brought by TMA), up to
// 128 queries as hi + lo (split_query) the B operand, and one thread of the
// epilogue owns one token.  It walks the token's scores in TMEM, adds up
// ex2(s scale - LSE) in registers and writes one number: no maximum, no
// exchange between threads, no atomics, and a fixed order.
// More than 128 rows take the tokens again for each 128 (keys from L2) and add to
// what the last ones left, which the same thread wrote.
// Work: tiles of 128 tokens of all sequences and heads form a line that is cut
// evenly among two CTAs per SM (one's exponentials run beside the other's
// products and its change of queries).
// Warps (192 threads): 0-3 queries and epilogue, 4 pages, scales and TMA of the
// keys (three slots), 5 tcgen05 issuer and owner of TMEM (two S buffers of 128 columns).
// Scales lie in a ring of eight slots without a barrier for their reuse: the keys
// of tile j have waited for the products of j - 3, those for the epilogue of j - 5.
// Measured (there: with mma.sync, cache_weights.cu), D = 128: 8 sequences of 16 heads,
// 32 rows 18 us (there 21), 64 rows 22 (32); 4 of 8192, 8 heads, 512 rows 81 (158).
// The starts bound it: a change of queries costs 3 to 4 us, a tile about 0.6.
// Every wait is bounded and ends in ATTN_ERR_DEVICE_TIMEOUT; each is for an
// earlier tile's event of the others, or for this tile's by a role that comes
// before it (queries, keys, S, epilogue).
#include "cache_tiles.cuh"

namespace attnmask {
namespace {

constexpr int kManyThreads = 192;
constexpr int kWarpKeys = 4, kWarpS = 5;
constexpr int kRows = 128;  // query rows at a time

template <int D>
struct ManyCfg {
  static constexpr int KT = CodeTile<D>::BYTES;
  static constexpr int NK = 3, NSCL = 8;
  static constexpr int OFF_Q = 0;                    // [hi, lo]
  static constexpr int OFF_K = OFF_Q + 2 * KT;
  static constexpr int OFF_ROWS = OFF_K + NK * KT;   // per two rows: scales, -LSE (base 2)
  static constexpr int OFF_SEEN = OFF_ROWS + kRows * 8;  // per row: visible tokens
  static constexpr int OFF_SCL = OFF_SEEN + kRows * 4;   // [slot][8 blocks of 16 tokens]: scale, or -1
  static constexpr int OFF_BAR = OFF_SCL + NSCL * 8 * 4;
  static constexpr int B_Q = 0, B_ROWS = 1, B_KFULL = 2, B_KEMPTY = B_KFULL + NK, B_SCL = B_KEMPTY + NK,
                       B_SFULL = B_SCL + NSCL, B_SEMPTY = B_SFULL + 2, B_DRAIN = B_SEMPTY + 2, NBAR = B_DRAIN + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;  // the base is aligned to 1024
  static_assert(2 * SMEM <= 226 * 1024, "two CTAs per SM");
};

struct ManyParams {
  CacheQueryArgs a;
  int G;
  float scale_log2;
};

__device__ __forceinline__ int tiles_of(const SeqRows& r) { return (r.len + kTile - 1) / kTile; }

// Tiles of sequence b and all heads (its tokens, also where it has no query).
struct TileCount {
  const ManyParams& p;
  bool note;
  __device__ int operator()(int b) const {
    const CacheQueryArgs& a = p.a;
    SeqRows r;
    if (!load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, a.max_seqlen, a.cache.status, r, note)) return 0;
    return tiles_of(r) * a.cache.heads;
  }
};

// One role's walk over the CTA's tiles: `visit(r, b, h, first token, tiles, row0)` for
// every segment (tiles of one sequence and head) and every 128 of its rows, until
// it returns false.
template <typename F>
__device__ __forceinline__ void walk(const ManyParams& p, const UnitLine& line, const TileCount& count, int lane,
                                     int pos, int stop, F&& visit) {
  const CacheQueryArgs& a = p.a;
  int before;
  int b = line.find(count, a.cache.batch, lane, pos, before);
  while (pos < stop) {
    SeqRows r;
    const bool good = load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, a.max_seqlen, a.cache.status, r, false);
    const int U = good ? tiles_of(r) : 0;
    if (U == 0) {
      ++b;
      continue;
    }
    const int h = (pos - before) / U, u0 = (pos - before) - h * U, n = min(U - u0, stop - pos);
    int row0 = 0;
    do {
      if (!visit(r, b, h, u0 * kTile, n, row0)) return;
      row0 += kRows;
    } while (row0 < r.n * p.G);
    pos += n;
    if (pos == before + U * a.cache.heads) {
      before = pos;
      ++b;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kManyThreads, 2)
    cache_weights_many_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ ManyParams p) {
  using C = ManyCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const CacheQueryArgs& a = p.a;
  const CacheView& c = a.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const TileCount count{p, blockIdx.x == 0};
  const UnitLine line(count, c.batch, lane);
  const int piece = (line.total + int(gridDim.x) - 1) / int(gridDim.x);
  const int pos = blockIdx.x * piece, stop = min(pos + piece, line.total);
  if (pos >= stop) return;
  int32_t* err = c.status;

  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base - raw);
  auto bar = [&](int i) { return base + C::OFF_BAR + 8u * uint32_t(i); };
  uint32_t* misc = reinterpret_cast<uint32_t*>(sbase + C::OFF_MISC);
  volatile uint32_t* abort_flag = misc + 1;
  float* scl = reinterpret_cast<float*>(sbase + C::OFF_SCL);

  if (threadIdx.x == 0) {
    ptx::mbar_init(bar(C::B_Q), 4);
    ptx::mbar_init(bar(C::B_ROWS), 4);
    for (int i = 0; i < C::NK; ++i) {
      ptx::mbar_init(bar(C::B_KFULL + i), 1);
      ptx::mbar_init(bar(C::B_KEMPTY + i), 1);
    }
    for (int i = 0; i < C::NSCL; ++i) ptx::mbar_init(bar(C::B_SCL + i), 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(C::B_SFULL + i), 1);
      ptx::mbar_init(bar(C::B_SEMPTY + i), 4);
    }
    ptx::mbar_init(bar(C::B_DRAIN), 1);
    // an earlier CTA that gave up on a wait makes every later one skip its work (the second
    // word, which no wait writes: all warps start or none does)
    misc[2] = *abort_flag = (*reinterpret_cast<volatile int32_t*>(err) & kErrTimeout) ? 1u : 0u;
    ptx::fence_mbar_init();
  }
  if (warp == kWarpS) {
    ptx::tmem_alloc(ptx::smem_addr(misc), 256);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];
  int j = 0;  // tiles so far

  if (misc[2] != 0u) {
    // nothing issued, nothing to drain
  } else if (warp == kWarpKeys) {
    // -------------------------------------------------------------- pages, scales, keys
    // Eight lanes a tile, one per 16 tokens: lanes 8 q .. 8 q + 7 look up the q-th
    // tile of four.  Page numbers are read two fours ahead, scales one, so that
    // neither read is waited for.
    const int step = (1 << c.page_log2) / 16;  // lanes per page
    if (lane == 0) ptx::prefetch_tensormap(&tmK);
    int done = 0;
    walk(p, line, count, lane, pos, stop, [&](const SeqRows& r, int b, int h, int begin, int n, int) {
      const int end = min(begin + n * kTile, r.len);
      auto token = [&](int i) { return begin + i * kTile + lane * 16; };  // of the four from i
      auto number = [&](int i) { return page_number(c, b, token(i), token(i) < end); };
      auto scale = [&](int i, int id) {
        const bool fine = token(i) < end && in_pool(c, id);
        return fine ? __ldg(c.k_scale + int64_t(id) * c.heads + h) : 0.f;
      };
      int id = 0, id_next = number(0), id_after = number(4);
      float sc = 0.f, sc_next = scale(0, id_next);
      for (int i = 0; i < n; ++i, ++j) {
        if ((i & 3) == 0) {
          id = id_next;
          id_next = id_after;
          id_after = number(i + 8);
          sc = sc_next;
          sc_next = scale(i + 4, id_next);
        }
        const bool mine = lane >> 3 == (i & 3), here = mine && token(i & ~3) < end, fine = here && in_pool(c, id);
        if (here && !fine) atomicOr(err, kErrBadPage);
        const int slot = j % C::NK, ss = j % C::NSCL;
        if (j >= C::NK && !wait_warp(bar(C::B_KEMPTY + slot), uint32_t(j / C::NK - 1) & 1u, abort_flag, err, 21))
          return false;
        if (mine) scl[ss * 8 + (lane & 7)] = fine ? sc : -1.f;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(C::B_SCL + ss));
        const bool load = fine && lane % step == 0;  // one lane per page (eight lanes are whole pages)
        const uint32_t loads = __ballot_sync(0xffffffffu, load);
        if (lane == 0)
          ptx::mbar_arrive_expect_tx(bar(C::B_KFULL + slot), (uint32_t(D) << c.page_log2) * __popc(loads));
        __syncwarp();
        if (load)
          ptx::tma_load_4d(base + C::OFF_K + slot * C::KT + (lane & 7) * 16 * D, &tmK, bar(C::B_KFULL + slot), 0, 0, h, id);
        done = j + 1;
      }
      return true;
    });
    // do not leave while a copy may still be writing shared memory
    if (lane == 0) {
      for (int s = 0; s < min(done, C::NK); ++s) {
        const int last = s + C::NK * ((done - 1 - s) / C::NK);
        drain_bar(bar(C::B_KFULL + s), uint32_t(last / C::NK) & 1u, err);
      }
    }
    __syncwarp();
  } else if (warp == kWarpS) {
    // -------------------------------------------------------------- S issuer
    const uint64_t qhi = ptx::smem_desc(base + C::OFF_Q, 16u, 8 * D, CodeTile<D>::SW);
    const uint64_t qlo = ptx::smem_desc(base + C::OFF_Q + C::KT, 16u, 8 * D, CodeTile<D>::SW);
    const uint64_t kd = ptx::smem_desc(base + C::OFF_K, 16u, 8 * D, CodeTile<D>::SW);
    uint32_t turn = 0;
    walk(p, line, count, lane, pos, stop, [&](const SeqRows& r, int, int, int, int n, int row0) {
      const int cols = max(32, (min(kRows, r.n * p.G - row0) + 31) & ~31);
      const uint32_t idesc = ptx::idesc_e4m3_f32(128, cols);
      bool ok = true;
      if (lane == 0) {
        ok = wait_lane(bar(C::B_Q), turn & 1u, abort_flag, err, 22);
        for (int i = 0; ok && i < n; ++i) {
          const int x = j + i, slot = x % C::NK, buf = x & 1;
          ok = wait_lane(bar(C::B_KFULL + slot), uint32_t(x / C::NK) & 1u, abort_flag, err, 23) &&
               (x < 2 || wait_lane(bar(C::B_SEMPTY + buf), uint32_t(x / 2 - 1) & 1u, abort_flag, err, 24));
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t s_tmem = tmem + uint32_t(kRows * buf);
          const uint64_t ki = kd + uint64_t((slot * C::KT) >> 4);
#pragma unroll
          for (int k = 0; k < D / 32; ++k) ptx::mma_f8_ss(s_tmem, ki + 2 * k, qhi + 2 * k, idesc, k > 0);
#pragma unroll
          for (int k = 0; k < D / 32; ++k) ptx::mma_f8_ss(s_tmem, ki + 2 * k, qlo + 2 * k, idesc, 1);
          ptx::mma_commit(bar(C::B_SFULL + buf));
          ptx::mma_commit(bar(C::B_KEMPTY + slot));
        }
      }
      j += n;
      ++turn;
      return __shfl_sync(0xffffffffu, int(ok), 0) != 0;
    });
    if (lane == 0) {
      // every product this thread issued has finished once this arrives
      ptx::mma_commit(bar(C::B_DRAIN));
      drain_bar(bar(C::B_DRAIN), 0, err);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- queries, epilogue
    const int row = warp * 32 + lane;  // a query's, and then the token's of a tile
    const uint32_t lane_base = tmem + (uint32_t(warp * 32) << 16);
    float* rows_at = reinterpret_cast<float*>(sbase + C::OFF_ROWS);
    int* seen_at = reinterpret_cast<int*>(sbase + C::OFF_SEEN);
    const float4* pairs = reinterpret_cast<const float4*>(rows_at);
    uint32_t met = 0;
    auto meet = [&]() {  // the four warps
      warp_arrive(bar(C::B_ROWS), lane);
      return wait_warp(bar(C::B_ROWS), met++ & 1u, abort_flag, err, 27);
    };
    walk(p, line, count, lane, pos, stop, [&](const SeqRows& r, int b, int h, int begin, int n, int row0) {
      const int rows = min(kRows, r.n * p.G - row0);
      const int cols = max(32, (rows + 31) & ~31);
      const int end = min(begin + n * kTile, r.len);
      {
        const bool real = row < rows;
        const int rg = row0 + row, i = real ? rg / p.G : 0, head = h * p.G + (real ? rg % p.G : 0);
        const int64_t token = r.q0 + i;
        float e = INFINITY;  // a row that does not exist or sees nothing adds 0
        if (real) e = a.lse[int64_t(head) * a.total_tokens + token] * 1.4426950408889634f;
        if (e == -INFINITY) e = INFINITY;
        // the last rows' scores have been used by all four warps, so their products
        // have ended, too
        if (!meet()) return false;
        const float s = split_query<D>(static_cast<const __nv_bfloat16*>(a.q) + (token * a.num_heads + head) * D, real,
                                       sbase + C::OFF_Q, row);
        ptx::fence_proxy_async_smem();
        rows_at[(row >> 1) * 4 + (row & 1)] = s * p.scale_log2;
        rows_at[(row >> 1) * 4 + 2 + (row & 1)] = -e;
        seen_at[row] = real ? visible_tokens(r, p.G, rg, a.causal) : 0;
        warp_arrive(bar(C::B_Q), lane);
        if (!meet()) return false;
      }
      const int least = visible_tokens(r, p.G, row0, a.causal);  // tokens that all these rows see
      const float* prev = row0 == 0 ? a.prev : a.weights;
      const int64_t out = (int64_t(b) * c.heads + h) * a.weight_stride;
      for (int i = 0; i < n; ++i, ++j) {
        const int first = begin + i * kTile, tok = first + row, ss = j % C::NSCL, buf = j & 1;
        const float was = prev && tok < end ? prev[out + tok] : 0.f;
        if (!wait_warp(bar(C::B_SCL + ss), uint32_t(j / C::NSCL) & 1u, abort_flag, err, 25) ||
            !wait_warp(bar(C::B_SFULL + buf), uint32_t(j / 2) & 1u, abort_flag, err, 26))
          return false;
        ptx::tc_fence_after();
        const float ks = scl[ss * 8 + (row >> 4)];
        const float2 ks2 = make_float2(ks, ks);
        const bool masked = first + kTile > least;
        float2 sum = make_float2(0.f, 0.f);
        for (int x = 0; x < cols; x += 32) {
          uint32_t s[32];
          ptx::tmem_ld32(lane_base + uint32_t(kRows * buf + x), s);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            const float4 q = pairs[x / 2 + y];
            float2 w = ptx::ffma2(make_float2(__uint_as_float(s[2 * y]), __uint_as_float(s[2 * y + 1])),
                                  ptx::fmul2(make_float2(q.x, q.y), ks2), make_float2(q.z, q.w));
            if (masked) {
              if (tok >= seen_at[x + 2 * y]) w.x = -INFINITY;
              if (tok >= seen_at[x + 2 * y + 1]) w.y = -INFINITY;
            }
            sum = ptx::fadd2(sum, make_float2(ptx::ex2(w.x), ptx::ex2(w.y)));
          }
          __syncwarp();
        }
        ptx::tc_fence_before();
        warp_arrive(bar(C::B_SEMPTY + buf), lane);
        // a page outside the pool receives nothing
        if (tok < end) a.weights[out + tok] = was + (ks < 0.f ? 0.f : sum.x + sum.y);
      }
      return true;
    });
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kWarpS) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 256);
  }
}

template <int D>
attn_status launch_d(const ManyParams& p, int sms, cudaStream_t s) {
  using C = ManyCfg<D>;
  CUtensorMap map;
  if (!encode_pages<D>(&map, p.a.cache, p.a.cache.k_pages, true))
    return record_cuda_error(cudaErrorInvalidValue, "attn_cache_weights tensor map encoding");
  cudaError_t e =
      cudaFuncSetAttribute(cache_weights_many_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e == cudaSuccess) {
    cache_weights_many_kernel<D><<<unsigned(2 * sms), kManyThreads, C::SMEM, s>>>(map, p);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_weights launch");
}

}  // namespace

attn_status launch_cache_weights_many(const CacheQueryArgs& a, int sms, cudaStream_t s) {
  const ManyParams p{a, a.num_heads / a.cache.heads, a.scale * 1.4426950408889634f};
  switch (a.cache.head_dim) {
    case 32: return launch_d<32>(p, sms, s);
    case 64: return launch_d<64>(p, sms, s);
    case 128: return launch_d<128>(p, sms, s);
  }
  return ATTN_ERR_UNSUPPORTED;
}

}  // namespace attnmask
