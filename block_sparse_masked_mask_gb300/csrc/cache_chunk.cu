// Attention over the 8-bit cache for many query rows (chunks of prompts), on
// the tcgen05 tensor cores.
//
// An item is one sequence and key / value head and 256 query rows (two M tiles
// of 128; rows are numbered new token * G + query head), over the tokens that
// some of its rows see, 128 at a time.  The products bound it: 4 D operations
// per row and token, while a tile's bytes serve 256 rows.  The tiles of all items
// form one line, cut into equal pieces, one per CTA and SM (as cache_rows.cuh
// does for few rows); a CTA walks its piece item by item, and an item that lies in
// several pieces is joined by a second kernel.  Every role runs on from one item to
// the next with its own ring positions: the next item's keys, values and
// queries are there before the last one's results are stored.  (One CTA per
// item and chunk of tokens instead paid 15 us per CTA, as much as eight tiles.)
//  * S = Q K^T runs on the codes as they lie (kind::f8f6f4): the keys need no
//    conversion.  A bf16 query has 8 significant bits and e4m3 4, so each row,
//    scaled by a power of two to a largest value in [128, 256), is the sum of two
//    e4m3 numbers, q = hi + lo, exact down to 2^-10 of that value and within
//    2^-18 of it below; S is hi K^T + lo K^T in one accumulator, at the cost
//    of one fp16 product (e4m3 runs at twice the rate).
//  * O += P V runs in fp16: weights keep 11 bits, the values are exact.  One
//    warpgroup turns the codes into fp16 tiles in shared memory, once
//    for both M tiles.
//  * The pages' scales and the running maximum are those of cache_attn.cu.
// Warps (512 threads):
//   0-3, 4-7   softmax of M tile 0 and 1, one thread per row
//   8-11       values: codes to fp16 tiles (two slots)
//   12         pages, scales (four slots) and TMA of the keys (three slots)
//   13, 14     tcgen05 issuers of S, one per M tile
//   15         tcgen05 issuer of P V for both M tiles (also owns TMEM)
// Keys and values come in tiles of 128 tokens; the products and the softmax go
// in steps of 64, with two S buffers per M tile: S of the next step is there
// when a softmax ends its step, so the softmax and the tensor cores both run
// without a pause.  P of a step is written over its S; S(i + 2) waits for P V(i).
// (With one S buffer of 128 tokens per M tile the chain S, softmax, P V of a
// tile took 6200 cycles, most of it with the tensor cores idle.)
// TMEM columns: S of M tile m, buffer f at 128 m + 64 f; O at 256 + 128 m.
// Every wait is bounded, as in the other tcgen05 kernels, and ends in
// ATTN_ERR_DEVICE_TIMEOUT in the cache's status word.  Each role walks the same
// items and steps and waits only for an earlier step's events of the others, or
// for this step's by a role that comes before it (pages, keys / values and
// queries, S, softmax, P V), so the order of steps carries every wait to its end.
#include "cache_rows.cuh"
#include "tile_pipeline.cuh"

namespace attnmask {
namespace {

constexpr int kChunkThreads = 512;
constexpr int kWarpValues = 8, kWarpKeys = 12, kWarpS = 13, kWarpPV = 15;
constexpr int kStep = 64;  // tokens per step

// The bounded waits of tile_pipeline.cuh behind one inlined try: five roles run
// at once, and their loops are fastest when they are short (the instruction
// caches; with the whole wait inlined everywhere the kernel ran 20% slower).
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, int32_t* err,
                                       int site) {
  return wait_bar(bar, parity, abort_flag, err, site);
}
__device__ __forceinline__ bool wait_lane(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, int32_t* err,
                                          int site) {
  return ptx::mbar_try_wait(bar, parity) || wait_long(bar, parity, abort_flag, err, site);
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, int32_t* err,
                                          int site) {
  return __all_sync(0xffffffffu, wait_lane(bar, parity, abort_flag, err, site));
}

template <int D>
struct ChunkCfg {
  using V = TileLayout<D>;                     // fp16 value tile: the 16-bit layout
  static constexpr int KT = kTile * D;         // bytes of a tile of codes (keys, or half a query)
  static constexpr int VT = V::TILE;
  static constexpr int NK = 3, NV = 2, NSCL = 4;
  static constexpr int OFF_Q = 0;              // [M tile][hi, lo]
  static constexpr int OFF_K = OFF_Q + 4 * KT;
  static constexpr int OFF_V = OFF_K + NK * KT;
  // [slot][8 blocks of 16 tokens]: key scale, exponent of the value scale, its
  // inverse, the page (as an int; -1: none)
  static constexpr int OFF_SCL = OFF_V + NV * VT;
  // B_SFULL, B_PFULL, B_PDONE: per M tile and S buffer
  static constexpr int B_Q = 0, B_KFULL = 2, B_KEMPTY = B_KFULL + NK, B_VFULL = B_KEMPTY + NK,
                       B_VEMPTY = B_VFULL + NV, B_SCLFULL = B_VEMPTY + NV, B_SCLFREE = B_SCLFULL + NSCL,
                       B_SFULL = B_SCLFREE + NSCL, B_PFULL = B_SFULL + 4, B_PDONE = B_PFULL + 4,
                       B_DRAIN = B_PDONE + 4, NBAR = B_DRAIN + 3;
  static constexpr int STAGE = 16 * D * 2;                // rows of O on their way out, per softmax warp
  static constexpr int OFF_STAGE = OFF_SCL + NSCL * 8 * 16;
  static constexpr int OFF_BAR = (OFF_STAGE + 8 * STAGE + 15) & ~15;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int USED = OFF_MISC + 16 + 1024;        // the base is aligned to 1024
  // one CTA per SM: it takes all of TMEM
  static constexpr int SMEM = USED > 116 * 1024 ? USED : 116 * 1024;
  static_assert(SMEM <= 232448, "shared memory budget");
  // rows of D bytes, swizzled over their own width
  static constexpr uint32_t SW8 = D == 128 ? ptx::kSwizzle128B : D == 64 ? ptx::kSwizzle64B : ptx::kSwizzle32B;
  __device__ static uint32_t unit8(int row, int u) {  // byte offset of 16-byte unit u of a row
    const int x = D == 128 ? (row & 7) : D == 64 ? ((row >> 1) & 3) : ((row >> 2) & 1);
    return uint32_t(row * D + ((u ^ x) << 4));
  }
  __device__ static uint32_t unit16(int row, int u) {  // of the fp16 layout's row chunk
    const int x = V::ROWB == 128 ? (row & 7) : ((row >> 1) & 3);
    return uint32_t(row * V::ROWB + ((u ^ x) << 4));
  }
};

// What a CTA does next: units u0 .. u1 - 1 (tiles of 128 tokens) of an item.
struct Segment {
  SeqRows r;
  int b, h, row0, nm;       // first row; M tiles in use
  int begin, end, tiles;    // tokens [begin, end)
  bool whole;               // all of the item
  int slot;                 // else: where its partial result goes
};

// The line as a CTA walks it.  Called by whole warps; every role walks alike.
struct Walk {
  const CacheAttnParams& p;
  int lane, pos, stop, b, before;
  SeqRows r;
  int known, all;  // the sequence that r and its units of one head belong to

  __device__ __forceinline__ Walk(const CacheAttnParams& params, int lane_id)
      : p(params), lane(lane_id), b(0), before(0), known(-1) {
    const ManyUnits units{p, blockIdx.x == 0 && threadIdx.x < 32};
    const UnitLine line(units, p.a.cache.batch, lane);
    const int piece = share_many(line.total, p.ctas);
    pos = blockIdx.x * piece;
    stop = min(pos + piece, line.total);
    if (pos < stop) b = line.find(units, p.a.cache.batch, lane, pos, before);
  }

  __device__ __noinline__ bool next(Segment& s) {
    const CacheQueryArgs& a = p.a;
    while (pos < stop) {
      if (b != known) {
        const bool good = load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, a.max_seqlen, a.cache.status, r, false);
        all = good ? item_units_warp(r, p.G, a.causal, lane) : 0;
        known = b;
      }
      s.r = r;
      if (all == 0) {
        ++b;
        continue;
      }
      s.b = b;
      s.h = (pos - before) / all;
      int rest = pos - before - s.h * all, tile = 0, U = 0;
      // the row tile: 32 at a time
      for (int t0 = 0;; t0 += 32) {
        const int mine = tile_units(s.r, p.G, a.causal, t0 + lane);
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, sum > rest);
        if (past) {
          const int at = __ffs(past) - 1;
          tile = t0 + at;
          U = __shfl_sync(0xffffffffu, mine, at);
          rest -= __shfl_sync(0xffffffffu, sum - mine, at);
          break;
        }
        rest -= __shfl_sync(0xffffffffu, sum, 31);
      }
      const int u0 = rest, u1 = min(U, u0 + stop - pos);
      s.row0 = tile * kManyRows;
      const int rows = min(kManyRows, s.r.n * p.G - s.row0);
      s.nm = rows > kTile ? 2 : 1;
      const int limit = visible_tokens(s.r, p.G, s.row0 + rows - 1, a.causal);
      s.begin = u0 * kTile;
      s.end = min(u1 * kTile, limit);
      s.tiles = s.end > s.begin ? (s.end - s.begin + kTile - 1) / kTile : 0;
      s.whole = u0 == 0 && u1 == U;
      s.slot = 2 * blockIdx.x + (u0 > 0 ? 0 : 1);
      pos += u1 - u0;
      if (pos == before + all * a.cache.heads) {
        before = pos;
        ++b;
      }
      return true;
    }
    return false;
  }
};

// One row's query as hi + lo in shared memory (tile m's row `row`, by the thread
// whose row it is); arrives on `full` and returns the row's scale.
template <int D>
__device__ __noinline__ float put_query(const CacheAttnParams& p, const Segment& s, int m, int row, uint8_t* sbase,
                                        uint32_t full) {
  using C = ChunkCfg<D>;
  const CacheQueryArgs& a = p.a;
  const int rg = s.row0 + m * kTile + row;  // of the sequence and head
  const bool real = rg < s.r.n * p.G;
  const int64_t at_q = int64_t(s.r.q0 + (real ? rg / p.G : 0)) * a.num_heads + s.h * p.G + (real ? rg % p.G : 0);
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + at_q * D);
  uint4 q[D / 8];  // all reads in flight at once
#pragma unroll
  for (int i = 0; i < D / 8; ++i) q[i] = real ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xFFFF0000u))));
  }
  const int e = amax > 0.f ? max(-119, min(126, exponent_of(amax))) : 0;
  const float f = pow2f(7 - e);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e4 = 0; e4 < 4; ++e4) {
      const uint4 v = q[2 * i + (e4 >> 1)];
      const uint32_t w0 = (e4 & 1) ? v.z : v.x, w1 = (e4 & 1) ? v.w : v.y;
      const float x0 = __uint_as_float(w0 << 16) * f, x1 = __uint_as_float(w0 & 0xFFFF0000u) * f;
      const float x2 = __uint_as_float(w1 << 16) * f, x3 = __uint_as_float(w1 & 0xFFFF0000u) * f;
      const uint32_t h0 = e4m3_pair(x0, x1), h1 = e4m3_pair(x2, x3);
      uint32_t y0 = half2_of(h0), y1 = half2_of(h1);
      const float2 z0 = __half22float2(*reinterpret_cast<__half2*>(&y0));
      const float2 z1 = __half22float2(*reinterpret_cast<__half2*>(&y1));
      hi[e4] = h0 | (h1 << 16);
      lo[e4] = e4m3_pair(x0 - z0.x, x1 - z0.y) | (e4m3_pair(x2 - z1.x, x3 - z1.y) << 16);
    }
    const uint32_t at = C::OFF_Q + (2 * m) * C::KT + C::unit8(row, i);
    *reinterpret_cast<uint4*>(sbase + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(sbase + at + C::KT) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  ptx::fence_proxy_async_smem();
  warp_arrive(full, threadIdx.x & 31);
  // an infinite query has no scores
  return (amax < INFINITY ? pow2f(e - 7) : __int_as_float(0x7FC00000)) * p.scale_log2;
}

template <int D>
__global__ void __launch_bounds__(kChunkThreads, 1)
    cache_chunk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CacheAttnParams p) {
  using C = ChunkCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const CacheQueryArgs& a = p.a;
  const CacheView& c = a.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Walk walk(p, lane);
  if (walk.pos >= walk.stop) return;
  int32_t* err = c.status;

  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base - raw);
  const uint32_t bars = base + C::OFF_BAR;
  auto bar = [&](int i) { return bars + 8u * uint32_t(i); };
  uint32_t* misc = reinterpret_cast<uint32_t*>(sbase + C::OFF_MISC);
  volatile uint32_t* abort_flag = misc + 1;
  float4* scl = reinterpret_cast<float4*>(sbase + C::OFF_SCL);

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NK; ++i) {
      ptx::mbar_init(bar(C::B_KFULL + i), 1);
      ptx::mbar_init(bar(C::B_KEMPTY + i), 2);  // both S issuers
    }
    for (int i = 0; i < C::NV; ++i) {
      ptx::mbar_init(bar(C::B_VFULL + i), 4);
      ptx::mbar_init(bar(C::B_VEMPTY + i), 1);
    }
    for (int i = 0; i < C::NSCL; ++i) {
      ptx::mbar_init(bar(C::B_SCLFULL + i), 1);
      ptx::mbar_init(bar(C::B_SCLFREE + i), 12);  // softmax and value warps
    }
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(bar(C::B_SFULL + i), 1);
      ptx::mbar_init(bar(C::B_PFULL + i), 4);
      ptx::mbar_init(bar(C::B_PDONE + i), 1);
    }
    for (int i = 0; i < 2; ++i) ptx::mbar_init(bar(C::B_Q + i), 4);
    for (int i = 0; i < 3; ++i) ptx::mbar_init(bar(C::B_DRAIN + i), 1);
    // an earlier CTA that gave up on a wait makes every later one skip its work
    *abort_flag = (*reinterpret_cast<volatile int32_t*>(err) & kErrTimeout) ? 1u : 0u;
    ptx::fence_mbar_init();
  }
  if (warp == kWarpPV) {
    ptx::tmem_alloc(ptx::smem_addr(misc), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];
  const bool skip = *abort_flag != 0u;
  Segment g;

  // Ring positions run on across items: T counts the tiles that a role has
  // passed, Tm those of its M tile (an item of one M tile does not use the second).
  if (skip) {
    // nothing issued, nothing to drain
  } else if (warp == kWarpKeys) {
    // -------------------------------------------------------------- pages, scales, keys
    // Lane i < 8: the i-th 16 tokens of a tile.  Page numbers are read two tiles
    // ahead, scales one, so that neither read is waited for.
    const int step = (1 << c.page_log2) / 16;  // lanes per page
    if (lane == 0) ptx::prefetch_tensormap(&tmK);
    int T = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      auto here = [&](int j) { return lane < 8 && g.begin + j * kTile + lane * 16 < g.end; };
      auto number = [&](int j) { return page_number(c, g.b, g.begin + j * kTile + lane * 16, here(j)); };
      int id = number(0), id_next = number(1);
      PageBatch sc = with_scales(c, g.h, id, here(0), true);
      for (int j = 0; j < g.tiles; ++j, ++T) {
        const int id_after = number(j + 2);
        const PageBatch sc_next = with_scales(c, g.h, id_next, here(j + 1), true);
        const int ss = T % C::NSCL, slot = T % C::NK;
        const bool fine = here(j) && in_pool(c, id);
        if (T >= C::NSCL &&
            !wait_warp(bar(C::B_SCLFREE + ss), uint32_t(T / C::NSCL - 1) & 1u, abort_flag, err, 1)) {
          ok = false;
          break;
        }
        if (lane < 8) {
          const int x = exponent_of(sc.v_scale);
          scl[ss * 8 + lane] = fine ? make_float4(sc.k_scale, float(x), pow2f(max(-126, -x)), __int_as_float(id))
                                    : make_float4(0.f, 0.f, 0.f, __int_as_float(-1));
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(C::B_SCLFULL + ss));
        if (T >= C::NK && !wait_warp(bar(C::B_KEMPTY + slot), uint32_t(T / C::NK - 1) & 1u, abort_flag, err, 2)) {
          ok = false;
          break;
        }
        const bool load = fine && lane % step == 0;  // one lane per page
        const uint32_t loads = __ballot_sync(0xffffffffu, load);
        const uint32_t piece = uint32_t(D) << c.page_log2;  // bytes of a page's keys
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar(C::B_KFULL + slot), piece * __popc(loads));
        __syncwarp();
        if (load)
          ptx::tma_load_4d(base + C::OFF_K + slot * C::KT + lane * 16 * D, &tmK, bar(C::B_KFULL + slot), 0, 0, g.h, id);
        id = id_next;
        id_next = id_after;
        sc = sc_next;
      }
    }
    // do not leave while a copy may still be writing shared memory
    if (lane == 0) {
      for (int s = 0; s < C::NK; ++s) {
        if (T <= s) continue;
        const int last = s + C::NK * ((T - 1 - s) / C::NK);
        drain_bar(bar(C::B_KFULL + s), uint32_t(last / C::NK) & 1u, err);
      }
    }
    __syncwarp();
  } else if (warp == kWarpPV) {
    // -------------------------------------------------------------- P V issuer
    constexpr uint32_t IDESC = ptx::idesc_f16_f32(128, D, false, true);
    const uint64_t vd = v_base<D>(base + C::OFF_V);
    int T = 0, Tm[2] = {0, 0};
    bool ok = true;
    while (ok && walk.next(g)) {
      if (lane == 0) {
        for (int i = 0; ok && i < 2 * g.tiles; ++i) {
          const int j = i >> 1, f = i & 1, vs = (T + j) % C::NV;
          if (f == 0 && !wait_lane(bar(C::B_VFULL + vs), uint32_t((T + j) / C::NV) & 1u, abort_flag, err, 6)) {
            ok = false;
            break;
          }
          const uint64_t vi = vd + uint64_t(vs) * (C::VT >> 4) + v_step<D>(f * (kStep / 16));
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (m >= g.nm) continue;
            ok = ok && wait_lane(bar(C::B_PFULL + 2 * m + f), uint32_t(Tm[m] + j) & 1u, abort_flag, err, 7);
            if (!ok) continue;
            ptx::tc_fence_after();
            const uint32_t p_tmem = tmem + uint32_t(128 * m + kStep * f), o_tmem = tmem + uint32_t(256 + 128 * m);
#pragma unroll
            for (int kk = 0; kk < kStep / 16; ++kk)
              ptx::mma_ts(o_tmem, p_tmem + uint32_t(kk) * 8u, vi + v_step<D>(kk), IDESC, (i > 0 || kk > 0) ? 1u : 0u);
            ptx::mma_commit(bar(C::B_PDONE + 2 * m + f));
          }
          if (ok && f == 1) ptx::mma_commit(bar(C::B_VEMPTY + vs));
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      T += g.tiles;
      Tm[0] += g.tiles;
      if (g.nm == 2) Tm[1] += g.tiles;
    }
    if (lane == 0) {
      // every product this thread issued has finished once this arrives
      ptx::mma_commit(bar(C::B_DRAIN + 2));
      drain_bar(bar(C::B_DRAIN + 2), 0, err);
    }
    __syncwarp();
  } else if (warp >= kWarpS) {
    // -------------------------------------------------------------- S issuers
    const int m = warp - kWarpS;
    constexpr uint32_t IDESC = ptx::idesc_e4m3_f32(128, kStep);
    const uint64_t qhi = ptx::smem_desc(base + C::OFF_Q + 2 * m * C::KT, 16u, 8 * D, C::SW8);
    const uint64_t qlo = ptx::smem_desc(base + C::OFF_Q + (2 * m + 1) * C::KT, 16u, 8 * D, C::SW8);
    const uint64_t kd = ptx::smem_desc(base + C::OFF_K, 16u, 8 * D, C::SW8);
    int T = 0, Tm = 0, items = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      const bool mine = m < g.nm;
      if (lane == 0) {
        if (mine) ok = wait_lane(bar(C::B_Q + m), uint32_t(items) & 1u, abort_flag, err, 3);
        for (int i = 0; ok && i < 2 * g.tiles; ++i) {
          const int j = i >> 1, ks = (T + j) % C::NK, f = i & 1, use = Tm + j;
          if (f == 0 && !wait_lane(bar(C::B_KFULL + ks), uint32_t((T + j) / C::NK) & 1u, abort_flag, err, 4)) {
            ok = false;
            break;
          }
          if (!mine) {  // the tile is not read for this M tile
            if (f == 1) ptx::mbar_arrive(bar(C::B_KEMPTY + ks));
            continue;
          }
          // P of two steps before lies over this S: its product has read it
          if (use > 0 && !wait_lane(bar(C::B_PDONE + 2 * m + f), uint32_t(use - 1) & 1u, abort_flag, err, 5)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t s_tmem = tmem + uint32_t(128 * m + kStep * f);
          const uint64_t ki = kd + uint64_t((ks * C::KT + f * kStep * D) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) ptx::mma_f8_ss(s_tmem, qhi + 2 * kk, ki + 2 * kk, IDESC, kk > 0);
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) ptx::mma_f8_ss(s_tmem, qlo + 2 * kk, ki + 2 * kk, IDESC, 1);
          ptx::mma_commit(bar(C::B_SFULL + 2 * m + f));
          if (f == 1) ptx::mma_commit(bar(C::B_KEMPTY + ks));
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      T += g.tiles;
      if (mine) {
        Tm += g.tiles;
        ++items;
      }
    }
    if (lane == 0) {
      ptx::mma_commit(bar(C::B_DRAIN + m));
      drain_bar(bar(C::B_DRAIN + m), 0, err);
    }
    __syncwarp();
  } else if (warp >= kWarpValues) {
    // -------------------------------------------------------------- values
    constexpr int PPT = D / 16;  // 16-byte pieces per token = pieces per thread
    const int ct = threadIdx.x - kWarpValues * 32;
    uint4 next[PPT];
    int T = 0;  // tiles stored
    auto fetch = [&](int j, int t) -> bool {  // tile j of the item, the t-th of all
      if (j >= g.tiles) return true;
      const int ss = t % C::NSCL;
      if (!wait_warp(bar(C::B_SCLFULL + ss), uint32_t(t / C::NSCL) & 1u, abort_flag, err, 12)) return false;
#pragma unroll
      for (int i = 0; i < PPT; ++i) {
        const int x = i * 128 + ct, row = x / PPT, piece = x % PPT;
        const int tok = g.begin + j * kTile + row;
        const int id = __float_as_int(scl[ss * 8 + row / 16].w);
        next[i] = make_uint4(0, 0, 0, 0);  // behind the end, or without a page: weights of 0 times 0
        if (tok < g.end && id >= 0)
          next[i] = __ldg(reinterpret_cast<const uint4*>(
              c.v_pages + (((int64_t(id) * c.heads + g.h) << c.page_log2) + (tok & ((1 << c.page_log2) - 1))) * D +
              piece * 16));
      }
      warp_arrive(bar(C::B_SCLFREE + ss), lane);
      return true;
    };
    bool ok = true;
    while (ok && walk.next(g)) {
      ok = fetch(0, T);
      for (int j = 0; ok && j < g.tiles; ++j, ++T) {
        const int slot = T % C::NV;
        if (T >= C::NV && !wait_warp(bar(C::B_VEMPTY + slot), uint32_t(T / C::NV - 1) & 1u, abort_flag, err, 8)) {
          ok = false;
          break;
        }
        uint8_t* tile = sbase + C::OFF_V + slot * C::VT;
#pragma unroll
        for (int i = 0; i < PPT; ++i) {
          const int x = i * 128 + ct, row = x / PPT, piece = x % PPT;
          uint8_t* chunk = tile + (piece * 16 / C::V::CE) * C::V::CHUNK;
          const int u = (piece * 16 % C::V::CE) / 8;  // two units: u, u + 1
          const uint4 w = next[i];
          const uint4 lo = make_uint4(half2_of(w.x), half2_of_high(w.x), half2_of(w.y), half2_of_high(w.y));
          const uint4 hi = make_uint4(half2_of(w.z), half2_of_high(w.z), half2_of(w.w), half2_of_high(w.w));
          // pieces of the second row chunk store their halves the other way
          // round: eight lanes of a token then meet eight different bank groups
          const bool flip = piece * 16 >= C::V::CE;
          *reinterpret_cast<uint4*>(chunk + C::unit16(row, u + (flip ? 1 : 0))) = flip ? hi : lo;
          *reinterpret_cast<uint4*>(chunk + C::unit16(row, u + (flip ? 0 : 1))) = flip ? lo : hi;
        }
        ptx::fence_proxy_async_smem();
        warp_arrive(bar(C::B_VFULL + slot), lane);
        ok = fetch(j + 1, T + 1);
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    const int m = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;  // of the M tile, its TMEM lane
    const uint32_t lane_base = tmem + (uint32_t(quarter * 32) << 16);
    const uint32_t o_col = lane_base + 256u + uint32_t(m) * 128u;

    int T = 0, Tm = 0;
    bool ok = true, more = walk.next(g);
    float qscale = more && m < g.nm ? put_query<D>(p, g, m, row, sbase, bar(C::B_Q + m)) : 0.f;
    while (ok && more) {
      if (m >= g.nm) {
        // no second M tile: the scales are passed on
        for (int j = 0; j < g.tiles; ++j, ++T) {
          const int ss = T % C::NSCL;
          if (!wait_warp(bar(C::B_SCLFULL + ss), uint32_t(T / C::NSCL) & 1u, abort_flag, err, 9)) {
            ok = false;
            break;
          }
          warp_arrive(bar(C::B_SCLFREE + ss), lane);
        }
        if (!ok) break;
        more = walk.next(g);
        if (more && m < g.nm) qscale = put_query<D>(p, g, m, row, sbase, bar(C::B_Q + m));
        continue;
      }
      const int rg = g.row0 + m * kTile + row;
      const int visible = visible_tokens(g.r, p.G, rg, a.causal);
      float mx = -INFINITY;               // running maximum (of score + value exponent)
      float2 l2 = make_float2(0.f, 0.f);  // two halves of the sum
      for (int i = 0; i < 2 * g.tiles; ++i) {
        const int j = i >> 1, f = i & 1, ss = (T + j) % C::NSCL;
        if (f == 0 && !wait_warp(bar(C::B_SCLFULL + ss), uint32_t((T + j) / C::NSCL) & 1u, abort_flag, err, 9)) {
          ok = false;
          break;
        }
        if (!wait_warp(bar(C::B_SFULL + 2 * m + f), uint32_t(Tm + j) & 1u, abort_flag, err, 10)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t s_col = lane_base + uint32_t(128 * m + kStep * f);
        const int first = g.begin + i * kStep;  // token of column 0
        const float4* sc = scl + ss * 8 + 4 * f;
        const int seen = visible - first;  // columns [0, seen) are visible
        bool masked = seen < kStep;
#pragma unroll
        for (int q = 0; q < 4; ++q) masked |= __float_as_int(sc[q].w) < 0;
        masked = __any_sync(0xffffffffu, masked);

        // 32 columns at a time: weights 2^(t - ref) against the running maximum so
        // far, and the largest t - ref beside them.  Only where that passes 2^8 (or
        // on the first visible token) the reference moves: what was formed with
        // the old one is scaled, and these columns are formed once more.  P of columns
        // [32 q, 32 q + 32) goes over S columns [16 q, 16 q + 16), which have been read.
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          const float4* sq = sc + 2 * q;
          uint32_t s[32];
          ptx::tmem_ld32(s_col + 32 * q, s);
          ptx::tmem_wait_ld();
          if (masked) {
            // hidden: the lowest score, whatever lay there
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int n = __float_as_int(sq[z].w) < 0 ? 0 : seen - 32 * q - 16 * z;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (e >= n) s[16 * z + e] = 0xFF800000u;  // -inf
            }
          }
          uint32_t pk[16];
          float2 sum2;
#pragma unroll 1
          for (bool again = false;; again = true) {
            const float ref = mx == -INFINITY ? 0.f : mx;
            float top = -INFINITY;
            sum2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const float4 k = sq[z];
              // -inf * 0 (a page left out) would be NaN
              const float kf = __float_as_int(k.w) < 0 ? 1.f : qscale * k.x, kx = k.y - ref;
              const float2 f2 = make_float2(kf, kf), x2 = make_float2(kx, kx);
              float2 part = make_float2(0.f, 0.f);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float2 w = ptx::ffma2(make_float2(__uint_as_float(s[16 * z + 2 * e]), __uint_as_float(s[16 * z + 2 * e + 1])),
                                      f2, x2);
                top = ptx::fmax3(top, w.x, w.y);
                w.x = ptx::ex2(w.x);
                w.y = ptx::ex2(w.y);
                part = ptx::fadd2(part, w);
                pk[8 * z + e] = pack_half2(w.x, w.y);
              }
              sum2 = ptx::ffma2(part, make_float2(k.z, k.z), sum2);
            }
            const bool raise = mx == -INFINITY ? top > -INFINITY : top > 8.f;
            if (again || !__any_sync(0xffffffffu, raise)) break;
            const float alpha = raise && mx != -INFINITY ? ptx::ex2(-top) : 1.f;  // (no sum yet where it is -inf)
            if (raise) mx = ref + top;
            l2.x *= alpha;
            l2.y *= alpha;
            if (q > 0) {  // this step's earlier weights
              uint32_t v[16];
              ptx::tmem_ld16(s_col, v);
              ptx::tmem_wait_ld();
              const __half2 a2 = __float2half2_rn(alpha);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const __half2 x = __hmul2(*reinterpret_cast<__half2*>(&v[e]), a2);
                v[e] = *reinterpret_cast<const uint32_t*>(&x);
              }
              ptx::tmem_st16(s_col, v);
            }
            if (i > 0) {  // O holds the earlier steps' products once the last of them has ended
              const int was = i - 1;
              if (!wait_warp(bar(C::B_PDONE + 2 * m + (was & 1)), uint32_t(Tm + (was >> 1)) & 1u, abort_flag, err, 13)) {
                ok = false;
                break;
              }
              ptx::tc_fence_after();
#pragma unroll 1
              for (int d = 0; d < D / 16; ++d) {
                uint32_t v[16];
                ptx::tmem_ld16(o_col + d * 16, v);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
                ptx::tmem_st16(o_col + d * 16, v);
              }
            }
          }
          l2 = ptx::fadd2(l2, sum2);
          ptx::tmem_st16(s_col + 16 * q, pk);
        }
        if (!ok) break;
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(bar(C::B_PFULL + 2 * m + f));
          if (f == 1) ptx::mbar_arrive(bar(C::B_SCLFREE + ss));
        }
      }
      if (!ok) break;
      T += g.tiles;
      Tm += g.tiles;

      // The next item's query first (every S of this one has been read, so its
      // place is free): its products run while this item's results are stored.
      const Segment done = g;
      more = walk.next(g);
      if (more && m < g.nm) qscale = put_query<D>(p, g, m, row, sbase, bar(C::B_Q + m));

      if (done.tiles > 0 &&
          !wait_warp(bar(C::B_PDONE + 2 * m + 1), uint32_t(Tm - 1) & 1u, abort_flag, err, 11)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      const float l = l2.x + l2.y;
      const bool real = rg < done.r.n * p.G;
      const int64_t token = done.r.q0 + (real ? rg / p.G : 0);
      const int head = done.h * p.G + (real ? rg % p.G : 0);
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (done.whole) {
        // rows of O as whole rows, 16 at a time through the warp's stage
        constexpr int CPR = D / 8, RPI = 32 / CPR;  // 16-byte pieces per row, rows per store
        uint8_t* stage = sbase + C::OFF_STAGE + warp * C::STAGE;
        uint32_t pk[D / 2];
#pragma unroll
        for (int q = 0; q < D / 16; ++q) {
          uint32_t v[16];
          if (done.tiles > 0) {
            ptx::tmem_ld16(o_col + q * 16, v);
            ptx::tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            pk[8 * q + e] = ptx::pack_bf16(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv);
        }
        const int row_first = done.row0 + m * kTile + quarter * 32;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if ((lane >> 4) == half) {
#pragma unroll
            for (int x = 0; x < CPR; ++x)
              *reinterpret_cast<uint4*>(stage + (lane & 15) * D * 2 + ((x ^ lane) & (CPR - 1)) * 16) =
                  make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
          }
          __syncwarp();
#pragma unroll 1
          for (int x = 0; x < 16 / RPI; ++x) {
            const int r16 = x * RPI + lane / CPR, piece = lane % CPR;
            const uint4 val = *reinterpret_cast<const uint4*>(stage + r16 * D * 2 + ((piece ^ r16) & (CPR - 1)) * 16);
            const int rr = row_first + half * 16 + r16;
            if (rr < done.r.n * p.G)
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) +
                                        (int64_t(done.r.q0 + rr / p.G) * a.num_heads + done.h * p.G + rr % p.G) * D +
                                        piece * 8) = val;
          }
          __syncwarp();
        }
        if (real)
          a.lse[int64_t(head) * a.total_tokens + token] =
              l == 0.f ? -INFINITY : (mx + log2f(l)) * 0.69314718055994531f;
      } else {
        // four dimensions of all rows together: lanes are rows
        const int per_slot = min(kManyRows, a.max_new * p.G), x = m * kTile + row;
        float4* to = reinterpret_cast<float4*>(p.part_o) + int64_t(done.slot) * per_slot * (D / 4) + x;
#pragma unroll
        for (int q = 0; q < D / 16; ++q) {
          uint32_t v[16];
          ptx::tmem_ld16(o_col + q * 16, v);
          ptx::tmem_wait_ld();
          if (real) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              to[int64_t(4 * q + e) * per_slot] =
                  make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]), __uint_as_float(v[4 * e + 2]),
                              __uint_as_float(v[4 * e + 3]));
          }
          __syncwarp();
        }
        if (real) p.part_m[int64_t(done.slot) * per_slot + x] = make_float2(mx, l);
      }
      // O has been read before the next item's first weights arrive
      ptx::tc_fence_before();
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kWarpPV) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int D>
attn_status launch_d(const CacheAttnParams& p, cudaStream_t s) {
  using C = ChunkCfg<D>;
  const CacheView& c = p.a.cache;
  // the keys' pages as rows of D bytes: (dimension, slot, head, page), one page
  // and head per copy
  CUtensorMap map;
  auto fn = encode_fn();
  const int page_size = 1 << c.page_log2;
  cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(page_size), cuuint64_t(c.heads), cuuint64_t(c.num_pages)};
  cuuint64_t strides[3] = {cuuint64_t(D), cuuint64_t(D) * page_size, cuuint64_t(D) * page_size * c.heads};
  cuuint32_t box[4] = {cuuint32_t(D), cuuint32_t(page_size), 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapSwizzle sw = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                : D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
  if (!fn || fn(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, c.k_pages, dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return record_cuda_error(cudaErrorInvalidValue, "attn_cache_fwd tensor map encoding");
  cudaError_t e = cudaFuncSetAttribute(cache_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return record_cuda_error(e, "attn_cache_fwd configure");
  cache_chunk_kernel<D><<<unsigned(p.ctas), kChunkThreads, C::SMEM, s>>>(map, p);
  e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_fwd launch");
}

}  // namespace

attn_status launch_cache_chunk(const CacheAttnParams& p, cudaStream_t s) {
  switch (p.a.cache.head_dim) {
    case 32: return launch_d<32>(p, s);
    case 64: return launch_d<64>(p, s);
    case 128: return launch_d<128>(p, s);
  }
  return ATTN_ERR_UNSUPPORTED;
}

}  // namespace attnmask
