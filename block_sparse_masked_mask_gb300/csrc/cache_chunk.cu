// Attention over the 8-bit cache for many query rows (chunks of prompts), on
// the tcgen05 tensor cores.
//
// A CTA takes one sequence and key / value head, 256 query rows (two M tiles of
// 128; rows are numbered new token * G + query head) and a chunk of the
// tokens, which it walks 128 at a time.  The products bound it: 4 D operations
// per row and token, while a tile's bytes serve 256 rows.
//  * S = Q K^T runs on the codes as they lie (kind::f8f6f4): the keys need no
//    conversion.  A bf16 query has 8 significant bits and e4m3 4, so each row,
//    scaled by a power of two to a largest value in [128, 256), is the sum of two
//    e4m3 numbers, q = hi + lo, exact down to 2^-9 of that value and within
//    2^-17 of it below; S is hi K^T + lo K^T in one accumulator, at the cost
//    of one fp16 product (e4m3 runs at twice the rate).
//  * O += P V runs in fp16: weights keep 11 bits, the values are exact.  One
//    warpgroup turns the codes into fp16 tiles in shared memory, once
//    for both M tiles.
//  * Up to 128 rows (a draft, the end of a prompt) both M tiles hold the same
//    queries and take the tiles of tokens in turn, each with its own running
//    maximum, and the CTA joins them at its end; warps without rows only pass the
//    steps on.  Such a CTA waits for latencies, and two chains hide each other's:
//    16 sequences of 8192, 32 rows of 8 heads 137 -> 108 us.
//  * The pages' scales, the running maximum and the far pages' sums are those of
//    cache_attn.cu.
// Warps (512 threads):
//   0-3, 4-7   softmax of M tile 0 and 1, one thread per row
//   8-11       values: codes to fp16 tiles (two slots)
//   12         pages, scales (four slots) and TMA of the codes (two slots each
//              of keys and values; reads by the value warps themselves came a
//              latency late: the 32 rows above 108 -> 91 us)
//   13, 14     tcgen05 issuers of S, one per M tile
//   15         tcgen05 issuer of P V for both M tiles (also owns TMEM)
// Keys and values come in tiles of 128 tokens; the products and the softmax go
// in steps of 64, with two S buffers per M tile: S of the next step is there
// when a softmax ends its step, so the softmax and the tensor cores both run
// without a pause.  P of a step is written over its S; S(i + 2) waits for P V(i).
// (With one S buffer of 128 tokens per M tile the chain S, softmax, P V of a
// tile took 6200 cycles, most of it with the tensor cores idle.)
// TMEM columns: S of M tile m, buffer f at 128 m + 64 f; O at 256 + 128 m.
// Measured, D = 128: 4 prompts of 300 to 512 new tokens behind 4096 to 16384, 32 / 8
// heads 334 us, 44% of the bf16 rate; one of 2048 behind 14336 530 us, 51%.  A tile of
// 256 rows and 128 tokens takes about 3700 cycles: its score products 1570 (49 each,
// their operands from shared memory; the pipe alone 32), its weight products 1040, and
// each M tile's chain of products and softmax (1000 cycles per step) goes on through them.
// Every wait is bounded, as in the other tcgen05 kernels, and ends in
// ATTN_ERR_DEVICE_TIMEOUT in the cache's status word.  Each role waits only for
// an earlier step's events of the others, or for this step's by a role that
// comes before it (pages, keys / values, S, softmax, P V), so the order of steps
// carries every wait to its end.
#include "cache_tiles.cuh"

namespace attnmask {
namespace {

constexpr int kChunkThreads = 512;
constexpr int kWarpValues = 8, kWarpKeys = 12, kWarpS = 13, kWarpPV = 15;
constexpr int kStep = 64;  // tokens per step
constexpr int kNoPage = INT_MIN;  // a block without a page
constexpr int kFar = 1;           // one whose value exponent lies kSpread below the largest so far

template <int D>
struct ChunkCfg {
  using V = TileLayout<D>;                     // fp16 value tile: the 16-bit layout
  static constexpr int KT = CodeTile<D>::BYTES;  // a tile of codes: keys, values or half a query
  static constexpr int VT = V::TILE;
  static constexpr int NK = 2, NR = 2, NV = 2, NSCL = 4;
  static constexpr int OFF_Q = 0;              // [M tile][hi, lo]
  static constexpr int OFF_K = OFF_Q + 4 * KT;
  static constexpr int OFF_R = OFF_K + NK * KT;  // the values' codes
  static constexpr int OFF_V = OFF_R + NR * KT;
  // [slot][8 blocks of 16 tokens]: key scale, exponent of the value scale, its
  // inverse (0: far), and as an int kNoPage, kFar or 0
  static constexpr int OFF_SCL = OFF_V + NV * VT;
  // B_SFULL, B_PFULL, B_PDONE: per M tile and S buffer
  static constexpr int B_Q = 0, B_KFULL = 2, B_KEMPTY = B_KFULL + NK, B_RFULL = B_KEMPTY + NK, B_REMPTY = B_RFULL + NR, B_VFULL = B_REMPTY + NR,
                       B_VEMPTY = B_VFULL + NV, B_SCLFULL = B_VEMPTY + NV, B_SCLFREE = B_SCLFULL + NSCL,
                       B_SFULL = B_SCLFREE + NSCL, B_PFULL = B_SFULL + 4, B_PDONE = B_PFULL + 4,
                       B_DRAIN = B_PDONE + 4, NBAR = B_DRAIN + 3;
  static constexpr int OFF_BAR = (OFF_SCL + NSCL * 8 * 16 + 15) & ~15;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int USED = OFF_MISC + 16 + 1024;        // the base is aligned to 1024
  // one CTA per SM: it takes all of TMEM
  static constexpr int SMEM = USED > 116 * 1024 ? USED : 116 * 1024;
  static_assert(SMEM <= 232448, "shared memory budget");
  __device__ static uint32_t unit16(int row, int u) {  // of the fp16 layout's row chunk
    const int x = V::ROWB == 128 ? (row & 7) : ((row >> 1) & 3);
    return uint32_t(row * V::ROWB + ((u ^ x) << 4));
  }
};

// The sums of a step's far blocks, from the scores as they lie; not inlined, to keep
// the softmax's loop short.
__device__ __noinline__ float far_sums(uint32_t s_col, const float4* sc, float qscale, float ref, int seen) {
  float sum = 0.f;
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    if (__float_as_int(sc[q].w) != kFar) continue;
    const float f = qscale * sc[q].x;
    uint32_t v[16];
    ptx::tmem_ld16(s_col + 16 * q, v);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float y = ptx::ex2(0.5f * fmaf(__uint_as_float(v[e]), f, -ref));
      if (16 * q + e < seen) sum = fmaf(y, y, sum);
    }
  }
  return sum;
}

template <int D>
__global__ void __launch_bounds__(kChunkThreads, 1)
    cache_chunk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CacheAttnParams p) {
  using C = ChunkCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const CacheQueryArgs& a = p.a;
  const CacheView& c = a.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x / p.row_tiles, row0 = (blockIdx.x % p.row_tiles) * kManyRows;
  const int h = blockIdx.y, b = blockIdx.z;
  SeqRows r;
  if (!load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, a.max_seqlen, c.status, r)) return;
  const int rows = min(kManyRows, r.n * p.G - row0);
  if (rows <= 0) return;
  const int limit = visible_tokens(r, p.G, row0 + rows - 1, a.causal);
  const int begin = split * p.chunk, end = min(begin + p.chunk, limit);
  if (split > 0 && begin >= end) return;  // chunk 0 also answers for rows that see nothing
  const int steps = end > begin ? (end - begin + kStep - 1) / kStep : 0;
  const int tiles = (steps + 1) / 2;
  // up to 128 rows: both M tiles hold them, and take the tiles of tokens in turn
  const bool twin = rows <= kTile;
  const int users = twin ? 1 : 2;  // M tiles per tile of tokens
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
      ptx::mbar_init(bar(C::B_KEMPTY + i), users);
    }
    for (int i = 0; i < C::NR; ++i) {
      ptx::mbar_init(bar(C::B_RFULL + i), 1);
      ptx::mbar_init(bar(C::B_REMPTY + i), 4);
    }
    for (int i = 0; i < C::NV; ++i) {
      ptx::mbar_init(bar(C::B_VFULL + i), 4);
      ptx::mbar_init(bar(C::B_VEMPTY + i), 1);
    }
    for (int i = 0; i < C::NSCL; ++i) {
      ptx::mbar_init(bar(C::B_SCLFULL + i), 1);
      ptx::mbar_init(bar(C::B_SCLFREE + i), 4 * users + 4);  // softmax and value warps
    }
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(bar(C::B_SFULL + i), 1);
      ptx::mbar_init(bar(C::B_PFULL + i), 4);
      ptx::mbar_init(bar(C::B_PDONE + i), 1);
    }
    for (int i = 0; i < 2; ++i) ptx::mbar_init(bar(C::B_Q + i), 4);
    for (int i = 0; i < 3; ++i) ptx::mbar_init(bar(C::B_DRAIN + i), 1);
    // An earlier CTA that gave up on a wait makes every later one skip its work.  No
    // wait writes the second word, so all warps start or none does: a wait that
    // runs out while a slower warp is still on its way here must not keep that warp
    // from the softmax warps' meetings, which have no bound of their own.
    misc[2] = *abort_flag = (*reinterpret_cast<volatile int32_t*>(err) & kErrTimeout) ? 1u : 0u;
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
  const bool skip = misc[2] != 0u;

  if (skip) {
    // nothing issued, nothing to drain
  } else if (warp == kWarpKeys) {
    // -------------------------------------------------------------- pages, scales, keys
    // Eight lanes a tile, one per 16 tokens: lanes 8 q .. 8 q + 7 look up the q-th
    // tile of four.  Page numbers are read two fours ahead, scales one, so that
    // neither read is waited for.
    const int step = (1 << c.page_log2) / 16;  // lanes per page
    auto token = [&](int j) { return begin + j * kTile + lane * 16; };  // of the four from j
    auto number = [&](int j) { return page_number(c, b, token(j), token(j) < end); };
    auto scales = [&](int j, int id) {
      const bool fine = token(j) < end && in_pool(c, id);
      const int64_t at = fine ? int64_t(id) * c.heads + h : 0;
      return make_float2(fine ? __ldg(c.k_scale + at) : 0.f, fine ? __ldg(c.v_scale + at) : 0.f);
    };
    if (lane == 0) {
      ptx::prefetch_tensormap(&tmK);
      ptx::prefetch_tensormap(&tmV);
    }
    int id = 0, id_next = number(0), id_after = number(4);
    float2 sc = make_float2(0.f, 0.f), sc_next = scales(0, id_next);
    int x_top = 0;  // largest exponent of the values so far, if above that of values up to 448
    int done = 0, done_v = 0;
    for (int j = 0; j < tiles; ++j) {
      if ((j & 3) == 0) {
        id = id_next;
        id_next = id_after;
        id_after = number(j + 8);
        sc = sc_next;
        sc_next = scales(j + 4, id_next);
      }
      const int ss = j % C::NSCL, slot = j % C::NK;
      const bool mine = lane >> 3 == (j & 3), here = mine && token(j & ~3) < end, fine = here && in_pool(c, id);
      if (here && !fine) atomicOr(err, kErrBadPage);
      if (j >= C::NSCL && !wait_warp(bar(C::B_SCLFREE + ss), uint32_t(j / C::NSCL - 1) & 1u, abort_flag, err, 1))
        break;
      const int x = exponent_of(sc.y);
      if (__any_sync(0xffffffffu, fine && x > x_top)) x_top = max(x_top, __reduce_max_sync(0xffffffffu, fine ? x : 0));
      if (mine) {
        const bool far = x < x_top - kSpread;
        scl[ss * 8 + (lane & 7)] =
            fine ? make_float4(sc.x, float(x), far ? 0.f : pow2f(max(-126, -x)), __int_as_float(far ? kFar : 0))
                 : make_float4(0.f, 0.f, 0.f, __int_as_float(kNoPage));
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(C::B_SCLFULL + ss));
      if (j >= C::NK && !wait_warp(bar(C::B_KEMPTY + slot), uint32_t(j / C::NK - 1) & 1u, abort_flag, err, 2)) break;
      const bool load = fine && lane % step == 0;  // one lane per page (eight lanes are whole pages)
      const uint32_t loads = __ballot_sync(0xffffffffu, load);
      const uint32_t piece = uint32_t(D) << c.page_log2;  // bytes of a page's keys
      if (lane == 0) ptx::mbar_arrive_expect_tx(bar(C::B_KFULL + slot), piece * __popc(loads));
      __syncwarp();
      if (load)
        ptx::tma_load_4d(base + C::OFF_K + slot * C::KT + (lane & 7) * 16 * D, &tmK, bar(C::B_KFULL + slot), 0, 0, h, id);
      done = j + 1;
      const int rs = j % C::NR;
      if (j >= C::NR && !wait_warp(bar(C::B_REMPTY + rs), uint32_t(j / C::NR - 1) & 1u, abort_flag, err, 12)) break;
      if (lane == 0) ptx::mbar_arrive_expect_tx(bar(C::B_RFULL + rs), piece * __popc(loads));
      __syncwarp();
      if (load)
        ptx::tma_load_4d(base + C::OFF_R + rs * C::KT + (lane & 7) * 16 * D, &tmV, bar(C::B_RFULL + rs), 0, 0, h, id);
      done_v = j + 1;
    }
    // do not leave while a copy may still be writing shared memory
    if (lane == 0) {
      for (int s = 0; s < C::NK; ++s) {
        if (done <= s) continue;
        const int last = s + C::NK * ((done - 1 - s) / C::NK);
        drain_bar(bar(C::B_KFULL + s), uint32_t(last / C::NK) & 1u, err);
      }
      for (int s = 0; s < C::NR; ++s) {
        if (done_v <= s) continue;
        const int last = s + C::NR * ((done_v - 1 - s) / C::NR);
        drain_bar(bar(C::B_RFULL + s), uint32_t(last / C::NR) & 1u, err);
      }
    }
    __syncwarp();
  } else if (warp == kWarpPV) {
    // -------------------------------------------------------------- P V issuer
    if (lane == 0) {
      constexpr uint32_t IDESC = ptx::idesc_f16_f32(128, D, false, true);
      const uint64_t vd = v_base<D>(base + C::OFF_V);
      bool ok = true;
      for (int i = 0; ok && i < steps; ++i) {
        const int j = i >> 1, vs = j % C::NV, f = i & 1;
        if (f == 0 && !wait_lane(bar(C::B_VFULL + vs), uint32_t(j / C::NV) & 1u, abort_flag, err, 6)) break;
        const uint64_t vi = vd + uint64_t(vs) * (C::VT >> 4) + v_step<D>(f * (kStep / 16));
        const int turn = twin ? j >> 1 : j;  // of the M tile's own
        for (int m = twin ? j & 1 : 0; m < 2; m += twin ? 2 : 1) {
          ok = wait_lane(bar(C::B_PFULL + 2 * m + f), uint32_t(turn) & 1u, abort_flag, err, 7);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t p_tmem = tmem + uint32_t(128 * m + kStep * f), o_tmem = tmem + uint32_t(256 + 128 * m);
#pragma unroll
          for (int kk = 0; kk < kStep / 16; ++kk)
            ptx::mma_ts(o_tmem, p_tmem + uint32_t(kk) * 8u, vi + v_step<D>(kk), IDESC,
                        (turn > 0 || f > 0 || kk > 0) ? 1u : 0u);
          ptx::mma_commit(bar(C::B_PDONE + 2 * m + f));
        }
        if (ok && (f == 1 || i == steps - 1)) ptx::mma_commit(bar(C::B_VEMPTY + vs));
      }
      // every product this thread issued has finished once this arrives
      ptx::mma_commit(bar(C::B_DRAIN + 2));
      drain_bar(bar(C::B_DRAIN + 2), 0, err);
    }
    __syncwarp();
  } else if (warp >= kWarpS) {
    // -------------------------------------------------------------- S issuers
    const int m = warp - kWarpS;
    if (lane == 0) {
      constexpr uint32_t IDESC = ptx::idesc_e4m3_f32(128, kStep);
      const uint64_t qhi = ptx::smem_desc(base + C::OFF_Q + 2 * m * C::KT, 16u, 8 * D, CodeTile<D>::SW);
      const uint64_t qlo = ptx::smem_desc(base + C::OFF_Q + (2 * m + 1) * C::KT, 16u, 8 * D, CodeTile<D>::SW);
      const uint64_t kd = ptx::smem_desc(base + C::OFF_K, 16u, 8 * D, CodeTile<D>::SW);
      const bool ok = steps == 0 || wait_lane(bar(C::B_Q + m), 0, abort_flag, err, 3);
      for (int i = twin ? 2 * m : 0; ok && i < steps; i += twin && (i & 1) ? 3 : 1) {
        const int j = i >> 1, ks = j % C::NK, f = i & 1, turn = twin ? j >> 1 : j;
        if (f == 0 && !wait_lane(bar(C::B_KFULL + ks), uint32_t(j / C::NK) & 1u, abort_flag, err, 4)) break;
        // the P before lies over this S: its product has read it
        if (turn >= 1 && !wait_lane(bar(C::B_PDONE + 2 * m + f), uint32_t(turn - 1) & 1u, abort_flag, err, 5)) break;
        ptx::tc_fence_after();
        const uint32_t s_tmem = tmem + uint32_t(128 * m + kStep * f);
        const uint64_t ki = kd + uint64_t((ks * C::KT + f * kStep * D) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) ptx::mma_f8_ss(s_tmem, qhi + 2 * kk, ki + 2 * kk, IDESC, kk > 0);
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) ptx::mma_f8_ss(s_tmem, qlo + 2 * kk, ki + 2 * kk, IDESC, 1);
        ptx::mma_commit(bar(C::B_SFULL + 2 * m + f));
        if (f == 1 || i == steps - 1) ptx::mma_commit(bar(C::B_KEMPTY + ks));
      }
      ptx::mma_commit(bar(C::B_DRAIN + m));
      drain_bar(bar(C::B_DRAIN + m), 0, err);
    }
    __syncwarp();
  } else if (warp >= kWarpValues) {
    // ------------------------------------------------------------ values
    constexpr int PPT = D / 16;  // 16-byte pieces per token = pieces per thread
    const int ct = threadIdx.x - kWarpValues * 32;
    for (int j = 0; j < tiles; ++j) {
      const int rs = j % C::NR, ss = j % C::NSCL, slot = j % C::NV;
      // (the scales' slot was written before this arrived)
      if (!wait_warp(bar(C::B_RFULL + rs), uint32_t(j / C::NR) & 1u, abort_flag, err, 12)) break;
      uint4 next[PPT];
#pragma unroll
      for (int i = 0; i < PPT; ++i)
        next[i] = *reinterpret_cast<const uint4*>(sbase + C::OFF_R + rs * C::KT + (i * 128 + ct) * 16);
      const bool gone = __float_as_int(scl[ss * 8 + (lane & 7)].w) < 0;
      if (__any_sync(0xffffffffu, gone) || begin + (j + 1) * kTile > end) {
        // behind the end, or without a page: weights of 0 times 0
#pragma unroll
        for (int i = 0; i < PPT; ++i) {
          const int row = (i * 128 + ct) / PPT;
          if (begin + j * kTile + row >= end || __float_as_int(scl[ss * 8 + row / 16].w) < 0)
            next[i] = make_uint4(0, 0, 0, 0);
        }
      }
      warp_arrive(bar(C::B_REMPTY + rs), lane);
      if (lane == 0) ptx::mbar_arrive(bar(C::B_SCLFREE + ss));
      if (j >= C::NV && !wait_warp(bar(C::B_VEMPTY + slot), uint32_t(j / C::NV - 1) & 1u, abort_flag, err, 8)) break;
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
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int m = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;          // of the M tile, its TMEM lane
    const int rg = row0 + (twin ? 0 : m * kTile) + row;  // of the sequence and head
    const uint32_t lane_base = tmem + (uint32_t(quarter * 32) << 16);
    const uint32_t o_col = lane_base + 256u + uint32_t(m) * 128u;
    const bool real = rg < r.n * p.G;
    const int64_t token = r.q0 + (real ? rg / p.G : 0);
    const int head = h * p.G + (real ? rg % p.G : 0);
    // (a lane without a row hides nothing: one hidden score sends its warp the slow way)
    const int visible = real ? visible_tokens(r, p.G, rg, a.causal) : limit;
    const bool idle = rg - lane >= r.n * p.G;     // a warp without rows only keeps the steps' order

    const float qscale =
        p.scale_log2 * split_query<D>(static_cast<const __nv_bfloat16*>(a.q) + (token * a.num_heads + head) * D, real,
                                      sbase + C::OFF_Q + 2 * m * C::KT, row);
    ptx::fence_proxy_async_smem();
    warp_arrive(bar(C::B_Q + m), lane);

    float mx = -INFINITY;                    // running maximum (of score + value exponent)
    float2 l2 = make_float2(0.f, 0.f);       // two halves of the sum
    bool ok = true;
    int last = -1;                           // step of this M tile: its turns' 2 t and 2 t + 1
    for (int i = twin ? 2 * m : 0; i < steps; i += twin && (i & 1) ? 3 : 1) {
      const int j = i >> 1, f = i & 1, ss = j % C::NSCL, turn = twin ? j >> 1 : j;
      if (f == 0 && !wait_warp(bar(C::B_SCLFULL + ss), uint32_t(j / C::NSCL) & 1u, abort_flag, err, 9)) {
        ok = false;
        break;
      }
      if (!wait_warp(bar(C::B_SFULL + 2 * m + f), uint32_t(turn) & 1u, abort_flag, err, 10)) { ok = false; break; }
      if (idle) {
        if (lane == 0) {
          ptx::mbar_arrive(bar(C::B_PFULL + 2 * m + f));
          if (f == 1 || i == steps - 1) ptx::mbar_arrive(bar(C::B_SCLFREE + ss));
        }
        __syncwarp();
        last = 2 * turn + f;
        continue;
      }
      ptx::tc_fence_after();
      const uint32_t s_col = lane_base + uint32_t(128 * m + kStep * f);
      uint32_t s[2][32];
      ptx::tmem_ld32(s_col, s[0]);
      ptx::tmem_ld32(s_col + 32, s[1]);
      const float4* sc = scl + ss * 8 + 4 * f;
      const int seen = visible - (begin + i * kStep);  // columns [0, seen) are visible
      const int odd = __float_as_int(sc[0].w) | __float_as_int(sc[1].w) | __float_as_int(sc[2].w) | __float_as_int(sc[3].w);
      ptx::tmem_wait_ld();
      if (__any_sync(0xffffffffu, seen < kStep) || odd < 0) {
        // hidden: the lowest score, whatever lay there
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = __float_as_int(sc[q].w) < 0 ? 0 : seen - 16 * q;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (e >= n) s[q >> 1][(q & 1) * 16 + e] = 0xFF800000u;  // -inf
        }
      }
      // a block's largest score: its factor is not negative, so the largest product
      float top = -INFINITY;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t* v = s[q >> 1] + (q & 1) * 16;
        float t = ptx::fmax3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
#pragma unroll
        for (int e = 3; e < 15; e += 2) t = ptx::fmax3(t, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
        t = fmaxf(t, __uint_as_float(v[15]));
        if (t > -INFINITY) top = fmaxf(top, fmaf(t, qscale * sc[q].x, sc[q].y));
      }
      // the reference moves on the first visible token and when a weight would
      // pass 2^15
      const bool raise = top > mx + kMostWeight;
      top -= kTopWeight;
      if (__any_sync(0xffffffffu, raise || (odd & kFar))) {
        const float half = raise ? half_factor(mx, top) : 1.f, alpha = half * half;
        if (raise) mx = top;
        l2.x = l2.x * half * half;
        l2.y = l2.y * half * half;
        if (last >= 0) {  // O holds the earlier steps' products once the last of them has ended
          if (!wait_warp(bar(C::B_PDONE + 2 * m + (last & 1)), uint32_t(last >> 1) & 1u, abort_flag, err, 13)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < D / 16; ++q) {
            uint32_t v[16];
            ptx::tmem_ld16(o_col + q * 16, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
            ptx::tmem_st16(o_col + q * 16, v);
          }
        }
        if (odd & kFar) l2.x += far_sums(s_col, sc, qscale, mx == -INFINITY ? 0.f : mx, seen);
      }
      const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 k = sc[q];
        // never 0, where a page is left out or the product is below fp32: a hidden score is
        // -inf, and times 0 it would be NaN
        const float kf = fmaf(qscale, k.x, 0x1p-126f), kx = k.y - ref;
        const float2 f2 = make_float2(kf, kf), x2 = make_float2(kx, kx);
        float2 part = make_float2(0.f, 0.f);
        uint32_t* v = s[q >> 1] + (q & 1) * 16;
        uint32_t pk[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float2 w = ptx::ffma2(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), f2, x2);
          w.x = ptx::ex2(w.x);
          w.y = ptx::ex2(w.y);
          part = ptx::fadd2(part, w);
          pk[e] = pack_half2(w.x, w.y);
        }
        l2 = ptx::ffma2(part, make_float2(k.z, k.z), l2);
        ptx::tmem_st8(s_col + 8 * q, pk);  // over S columns read already
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(bar(C::B_PFULL + 2 * m + f));
        if (f == 1 || i == steps - 1) ptx::mbar_arrive(bar(C::B_SCLFREE + ss));
      }
      last = 2 * turn + f;
    }
    float l = l2.x + l2.y;
    if (ok && last >= 0)
      ok = wait_warp(bar(C::B_PDONE + 2 * m + (last & 1)), uint32_t(last >> 1) & 1u, abort_flag, err, 11);
    ptx::tc_fence_after();
    // Both M tiles' results become the first's, through shared memory: once
    // every softmax warp is here, all scores are read, and so are the queries and
    // keys.  Four dimensions of all rows together: lanes are rows.
    float4* const other = reinterpret_cast<float4*>(sbase + C::OFF_Q);
    float2* const other_m = reinterpret_cast<float2*>(sbase + C::OFF_K);
    float mine = 1.f, its = 0.f;  // factors of the two
    if (twin) {
      ptx::named_barrier(1, 256);
      if (m == 1) {
        other_m[row] = make_float2(mx, l);
        if (ok && last >= 0) {
#pragma unroll 1
          for (int q = 0; q < D / 16; ++q) {
            uint32_t v[16];
            ptx::tmem_ld16(o_col + q * 16, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e)
              other[(4 * q + e) * kTile + row] =
                  make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]), __uint_as_float(v[4 * e + 2]),
                              __uint_as_float(v[4 * e + 3]));
          }
        }
      }
      ptx::named_barrier(1, 256);
      if (m == 0) {
        const float2 ml = other_m[row];
        const float top = fmaxf(mx, ml.x);
        const float half = half_factor(mx, top), other_half = half_factor(ml.x, top);
        mine = half * half;
        its = other_half * other_half;
        l = l * half * half + ml.y * other_half * other_half;
        mx = top;
      }
    }
    if (ok && (m == 0 || !twin)) {
      const bool single = p.splits == 1;
      const float inv = single ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      const int64_t at = (int64_t(single ? 0 : split) * a.total_tokens + token) * a.num_heads + head;
#pragma unroll
      for (int q = 0; q < D / 16; ++q) {
        uint32_t v[16];
        if (steps > 0) {
          ptx::tmem_ld16(o_col + q * 16, v);
          ptx::tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0u;
        }
        if (twin) {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * mine);
          if (its > 0.f) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 x = other[(4 * q + e) * kTile + row];
              v[4 * e] = __float_as_uint(fmaf(x.x, its, __uint_as_float(v[4 * e])));
              v[4 * e + 1] = __float_as_uint(fmaf(x.y, its, __uint_as_float(v[4 * e + 1])));
              v[4 * e + 2] = __float_as_uint(fmaf(x.z, its, __uint_as_float(v[4 * e + 2])));
              v[4 * e + 3] = __float_as_uint(fmaf(x.w, its, __uint_as_float(v[4 * e + 3])));
            }
          }
        }
        if (real && single) {
          uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + at * D + q * 16);
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            w[i] = ptx::pack_bf16(__uint_as_float(v[2 * i]) * inv, __uint_as_float(v[2 * i + 1]) * inv);
          out[0] = make_uint4(w[0], w[1], w[2], w[3]);
          out[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else if (real) {
          uint4* out = reinterpret_cast<uint4*>(p.part_o + at * D + q * 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) out[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
        __syncwarp();
      }
      if (real) {
        if (single)
          a.lse[int64_t(head) * a.total_tokens + token] =
              l == 0.f ? -INFINITY : (mx + log2f(l)) * 0.69314718055994531f;
        else
          p.part_m[at] = make_float2(mx, l);
      }
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
  CUtensorMap map, map_v;
  if (!encode_pages<D>(&map, c, c.k_pages, true) || !encode_pages<D>(&map_v, c, c.v_pages, false))
    return record_cuda_error(cudaErrorInvalidValue, "attn_cache_fwd tensor map encoding");
  cudaError_t e = cudaFuncSetAttribute(cache_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return record_cuda_error(e, "attn_cache_fwd configure");
  const dim3 grid(unsigned(p.splits) * unsigned(p.row_tiles), unsigned(c.heads), unsigned(c.batch));
  cache_chunk_kernel<D><<<grid, kChunkThreads, C::SMEM, s>>>(map, map_v, p);
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
