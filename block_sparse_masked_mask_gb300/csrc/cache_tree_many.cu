// Attention of drafted trees over the 8-bit cache for more than 64 rows (nodes times query
// heads of the group), on the tcgen05 tensor cores.
//
// The products are those of cache_chunk.cu: rows are their M, in two tiles of 128;
// S = Q K^T on the codes as they lie, a query as the sum of two e4m3 numbers; the weights,
// fp16, written over their S in tensor memory, times the values' codes as fp16 tiles in shared
// memory.  Up to 128 rows both M tiles hold them and take the tiles of tokens in turn.  A thread
// of the softmax owns a row, with its maximum and sum; scales and far pages are those of
// cache_attn.cu.
// What differs is the division.  Tiles of 128 tokens of all (sequence, head, 256 rows)s form one
// line, counted by what they cost, that is cut evenly among one CTA per SM (TreeLine in cache_tree.cuh).  A CTA
// walks its piece segment by segment: page numbers, keys and values of the next one are under way while
// the last one ends.  Segments that are not whole meet in a second kernel, two per CTA at most.
// 32 trees of 17 to 32 nodes behind 1024 to 16384 tokens, 32 query and 8 key heads of 128, take 114 us, and
// 8 trees of 48 to 64 nodes, 64 and 8 heads, behind 4096 to 16384 tokens 126 us (the kernel of
// cache_chunk.cu with these masks, a CTA for 4096 tokens, took 155 and 157: starts and ends were a quarter of
// it, and uneven).  Products of 128 rows fill the tensor cores to a half there; a tile takes about 1.4 us, most of it
// the softmax's, which waits for its scores, its exponentials and the other warps' instructions in
// turn; a segment's start and end about 9 us (queries as two numbers, O, the first scores).
// Every tile is two steps of 64 tokens, whatever lies behind a sequence's end (weights of 0
// times 0), so that each barrier's phases go on by one a tile.
// Warps (640 threads):
//   0-3, 4-7   softmax of M tile 0 and 1, one thread per row; its queries
//   8-11       values: codes to fp16 tiles
//   12         pages, scales and TMA of the codes
//   13, 14     tcgen05 issuers of S, one per M tile
//   15         tcgen05 issuer of P V for both M tiles (also owns TMEM)
//   16         the line: the CTA's segments (17-19 idle)
// TMEM columns: S of M tile m, step f of a tile at 128 m + 64 f; O at 256 + 128 m.
// Waits are those of cache_tree.cuh; each role waits only for an earlier tile's events of the
// others, or for this tile's by a role that comes before it (line, pages, queries and keys, S,
// softmax, values, P V).  No barrier's phase ends a second time before all who wait for it have seen the
// first: they bring something, or free a place, that the second one needs.  Warps of the softmax meet
// without a bound at a segment's beginning and end: all come there, whatever ran out, and leave together.
#include <algorithm>
#include <cmath>

#include "cache_join.cuh"
#include "cache_tree.cuh"

namespace attnmask {
namespace {

constexpr int kTreeRows = 256;          // of a segment
// What a tile of tokens costs, with up to 256 rows and with up to 128, and a segment's start and end
// (32 trees of 17 to 32 nodes, heads of 128 / 64 / 32: 10 128 / 93 / 83 us, 16 119 / 88 / 81, 20 114 / 88 / 83,
// 26 115 / 91 / 86).
using Line = TreeLine<kTreeRows, 5, 3, 20, 5>;
constexpr int kStep = 64;

// A piece of the line in one (sequence, head, 256 rows).
struct Segment {
  int tiles;  // 0: there is no further one
  int b, h, row0, rows, q0, n, len, token, slot;  // slot of the partial result, -1: whole
};

// The tokens of a step of 64 from `first` on that a row sees: the text, and of the nodes, numbers
// from first - text on, those of its bits.
__device__ __forceinline__ uint64_t tree_step(const uint32_t* bits, int first, int text, int nodes) {
  uint64_t seen = first >= text ? 0ull : text - first >= kStep ? ~0ull : (1ull << (text - first)) - 1;
  const int node = first - text;  // of the first token; negative in the text
#pragma unroll 1
  for (int w = max(node, 0) / 32; 32 * w < min(node + kStep, nodes); ++w) {
    uint64_t x = __ldg(bits + w);
    if (nodes - 32 * w < 32) x &= (1ull << (nodes - 32 * w)) - 1;
    const int to = 32 * w - node;  // its first bit's place
    seen |= to >= 0 ? x << to : x >> -to;
  }
  return seen;
}

template <int D>
struct ManyCfg {
  static constexpr int THREADS = 640;
  static constexpr int VALUES = 8, PAGES = 12, ISSUE_S = 13, ISSUE_O = 15, LINE = 16;
  // Registers for each thread of the softmax, the values and the others, of the launch's 96 for all (with which
  // the compiler spills 72 bytes a thread)
  static constexpr int REG_SOFTMAX = 144, REG_VALUES = 80, REG_OTHERS = 56;
  static_assert(2 * REG_SOFTMAX + REG_VALUES + 2 * REG_OTHERS == 5 * 96, "registers");
  using V = TileLayout<D>;                       // fp16 value tile: the 16-bit layout
  static constexpr int KT = CodeTile<D>::BYTES;  // a tile of codes: keys, values or half a query
  static constexpr int VT = V::TILE;
  static constexpr int NK = 2, NR = 2, NV = 2, NSCL = 8, NSEG = 4;
  static constexpr int OFF_Q = 0;                // [M tile][hi, lo]
  static constexpr int OFF_K = OFF_Q + 4 * KT;
  static constexpr int OFF_R = OFF_K + NK * KT;  // the values' codes
  static constexpr int OFF_V = OFF_R + NR * KT;
  static constexpr int OFF_SCL = OFF_V + NV * VT;          // as in cache_chunk.cu
  static constexpr int OFF_STATS = OFF_SCL + NSCL * 8 * 16;  // [M tile][row]: maximum and sum
  static constexpr int OFF_ROWS = OFF_STATS + 2 * kTile * 8;  // [M tile][row]: the queries' factors
  static constexpr int OFF_SEG = OFF_ROWS + 2 * kTile * 4;
  static constexpr int OFF_BAR = OFF_SEG + NSEG * 48;
  static constexpr int B_SEGFULL = 0, B_SEGFREE = B_SEGFULL + NSEG, B_Q = B_SEGFREE + NSEG, B_KFULL = B_Q + 2 * NSEG,
                       B_KFREE = B_KFULL + NK, B_RFULL = B_KFREE + NK, B_RFREE = B_RFULL + NR, B_VFULL = B_RFREE + NR,
                       B_VFREE = B_VFULL + NV, B_SCLFULL = B_VFREE + NV, B_SCLFREE = B_SCLFULL + NSCL,
                       B_SFULL = B_SCLFREE + NSCL, B_PFULL = B_SFULL + 4, B_PDONE = B_PFULL + 4, B_OFREE = B_PDONE + 4,
                       B_DRAIN = B_OFREE + 1, NBAR = B_DRAIN + 3;
  static_assert(NBAR <= THREADS, "a thread for each");
  __device__ static int arrivals(int i) {
    return i >= B_OFREE ? (i >= B_DRAIN ? 1 : 8)
           : i >= B_PFULL ? (i >= B_PDONE ? 1 : 4)
           : i >= B_SCLFREE ? (i >= B_SFULL ? 1 : 12)  // softmax (twice by those of one M tile alone) and value warps
           : i >= B_SCLFULL ? 1
           : i >= B_VFULL ? (i >= B_VFREE ? 1 : 4)
           : i >= B_RFULL ? (i >= B_RFREE ? 4 : 1)
           : i >= B_KFULL ? (i >= B_KFREE ? 2 : 1)     // (twice by one issuer alone)
           : i >= B_Q ? 4
           : i >= B_SEGFREE ? LINE : 1;  // the warps before that one
  }
  // The queries of segment s and M tile m: a barrier for each place of the segments' ring.  An issuer frees the
  // place only once it has seen them, so that no phase can end twice while it looks for it, in a segment
  // without a tile of its own too.
  __device__ static int queries(int s, int m) { return B_Q + 2 * (s % NSEG) + m; }
  __device__ static uint32_t queries_parity(int s) { return uint32_t(s / NSEG) & 1u; }
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

template <int D>
__global__ void __launch_bounds__(ManyCfg<D>::THREADS, 1)
    cache_tree_many_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                           const __grid_constant__ TreeParams p) {
  using C = ManyCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const CacheQueryArgs& a = p.a;
  const CacheView& c = a.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t* err = c.status;

  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base - raw);
  const uint32_t bars = base + C::OFF_BAR;
  auto bar = [&](int i) { return bars + 8u * uint32_t(i); };
  uint32_t* misc = reinterpret_cast<uint32_t*>(sbase + C::OFF_MISC);
  volatile uint32_t* abort_flag = misc + 1;
  float4* scl = reinterpret_cast<float4*>(sbase + C::OFF_SCL);

  if (threadIdx.x < C::NBAR) {
    ptx::mbar_init(bar(threadIdx.x), C::arrivals(threadIdx.x));
    ptx::fence_mbar_init();
  }
  if (threadIdx.x == 0) *abort_flag = 0u;
  if (warp == C::ISSUE_O) {
    ptx::tmem_alloc(ptx::smem_addr(misc), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];

  // The s-th segment, copied from its place in the ring; one arrival frees that (an issuer of S brings it later).
  auto segment = [&](int s, Segment& g, bool single, bool later = false) {
    const int at = s % C::NSEG;
    const bool ok = single ? tree_wait(bar(C::B_SEGFULL + at), uint32_t(s / C::NSEG) & 1u, abort_flag, 1)
                           : tree_warp_wait(bar(C::B_SEGFULL + at), uint32_t(s / C::NSEG) & 1u, abort_flag, 1);
    g.tiles = 0;
    if (!ok) return false;
    const int4* w = reinterpret_cast<const int4*>(sbase + C::OFF_SEG + at * 48);
    const int4 x = w[0], y = w[1], z = w[2];
    g = Segment{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, z.x, z.y};
    if (later) return true;
    if (single) ptx::mbar_arrive(bar(C::B_SEGFREE + at));
    else warp_arrive(bar(C::B_SEGFREE + at), lane);
    return true;
  };

  // (the registers are split in each branch: where they meet, the least would hold for all)
  if (warp >= C::PAGES) {
    ptx::regs_dec<C::REG_OTHERS>();
    if (warp == C::LINE) {
      // ------------------------------------------------------------ segments
      const int64_t total = Line::total(p, lane), piece = Line::share(total, p);
      int64_t pos = min(int64_t(blockIdx.x) * piece, total);
      const int64_t stop = min(pos + piece, total);
      // (after a wait that ran out in an earlier CTA there is nothing to do)
      if (*reinterpret_cast<volatile int32_t*>(err) & kErrTimeout) pos = stop;
      int64_t before = 0;
      int b = pos < stop ? Line::find(p, pos, lane, before) : 0;
      TreeCut cut{};
#pragma unroll 1
      for (int s = 0;; ++s) {
        Segment g{};
#pragma unroll 1
        while (pos < stop) {
          const int64_t all = Line::of(p, b);
          if (pos >= before + all) {
            before += all;
            ++b;
            continue;
          }
          const int q0 = a.cu[b], n = a.cu[b + 1] - q0, len = a.lens[b];
          const Line::Seq l(n, p.G, len);
          const Line::Item it(l, before, pos);
          const int u0 = it.tiles(pos, l.U), u1 = it.tiles(stop, l.U);
          pos = min(stop, it.end);
          if (u1 <= u0) continue;
          g.tiles = u1 - u0;
          g.b = b;
          g.h = it.h;
          g.row0 = it.rt * kTreeRows;
          g.rows = int(min(int64_t(kTreeRows), int64_t(n) * p.G - g.row0));
          g.q0 = q0;
          g.n = n;
          g.len = len;
          g.token = u0 * kTile;
          g.slot = u0 == 0 && u1 == l.U ? -1 : 2 * int(blockIdx.x) + (u0 > 0 ? 0 : 1);
          if (u0 == 0 && u1 < l.U)
            cut = TreeCut{int((it.end - it.w) / piece) - int(blockIdx.x) + 1, g.h, g.row0, g.rows, g.q0};
          break;
        }
        const int at = s % C::NSEG;
        if (s >= C::NSEG && !tree_warp_wait(bar(C::B_SEGFREE + at), uint32_t(s / C::NSEG - 1) & 1u, abort_flag, 2)) break;
        if (lane == 0) {
          int4* w = reinterpret_cast<int4*>(sbase + C::OFF_SEG + at * 48);
          w[0] = make_int4(g.tiles, g.b, g.h, g.row0);
          w[1] = make_int4(g.rows, g.q0, g.n, g.len);
          w[2] = make_int4(g.token, g.slot, 0, 0);
          ptx::mbar_arrive(bar(C::B_SEGFULL + at));
        }
        __syncwarp();
        if (g.tiles == 0) break;
        // queries and masks on their way to L2
#pragma unroll 1
        for (int x = lane; x < g.rows; x += 32) {
          const int rg = g.row0 + x, node = rg / p.G;
          const int64_t token = g.q0 + node;
          const char* row = static_cast<const char*>(a.q) + (token * a.num_heads + g.h * p.G + rg - node * p.G) * (2 * D);
#pragma unroll
          for (int y = 0; y < 2 * D; y += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + y));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(p.tree.bits + token * p.tree.words));
        }
      }
      if (lane == 0) p.cuts[blockIdx.x] = cut;
      // what is wrong with the sequences is noted once, when nobody waits for it
      if (blockIdx.x == 0) {
#pragma unroll 1
        for (int x = lane; x < c.batch; x += 32) {
          SeqRows r;
          if (load_rows(a.cu, a.lens, x, a.total_tokens, a.max_new, a.max_seqlen, err, r) && r.len < r.n) atomicOr(err, kErrHeld);
        }
      }
    } else if (warp == C::PAGES) {
      // ------------------------------------------------------------ pages, scales, codes
      // As in cache_tree.cu: eight lanes a tile, one per 16 tokens; page numbers are read two
      // fours of tiles ahead, scales one.
      const int step = (1 << c.page_log2) / 16;  // lanes per page
      const uint32_t bytes = uint32_t(D) << c.page_log2;  // of a page's keys
      if (lane == 0) {
        ptx::prefetch_tensormap(&tmK);
        ptx::prefetch_tensormap(&tmV);
      }
      Segment g;
      int T = 0, done = 0, done_v = 0;
      bool ok = true;
#pragma unroll 1
      for (int s = 0; ok && segment(s, g, false) && g.tiles; ++s) {
        const int end = min(g.token + g.tiles * kTile, g.len);
        auto token = [&](int j) { return g.token + j * kTile + lane * 16; };  // of the four from j
        auto number = [&](int j) { return page_number(c, g.b, token(j), token(j) < end); };
        auto scales = [&](int j, int id) {
          const bool fine = token(j) < end && in_pool(c, id);
          const int64_t at = fine ? int64_t(id) * c.heads + g.h : 0;
          return make_float2(fine ? __ldg(c.k_scale + at) : 0.f, fine ? __ldg(c.v_scale + at) : 0.f);
        };
        int id = 0, id_next = number(0), id_after = number(4);
        float2 sc = make_float2(0.f, 0.f), sc_next = scales(0, id_next);
        int x_top = 0;  // largest exponent of the values so far, if above that of values up to 448
#pragma unroll 1
        for (int j = 0; j < g.tiles; ++j, ++T) {
          if ((j & 3) == 0) {
            id = id_next;
            id_next = id_after;
            id_after = number(j + 8);
            sc = sc_next;
            sc_next = scales(j + 4, id_next);
          }
          const int ss = T % C::NSCL, ks = T % C::NK, rs = T % C::NR;
          const bool mine = lane >> 3 == (j & 3), here = mine && token(j & ~3) < end, fine = here && in_pool(c, id);
          if (here && !fine) atomicOr(err, kErrBadPage);
          // keys first: they need no scales yet
          if (T >= C::NK && !tree_warp_wait(bar(C::B_KFREE + ks), uint32_t(T / C::NK - 1) & 1u, abort_flag, 4)) { ok = false; break; }
          const bool load = fine && lane % step == 0;  // one lane per page (eight lanes are whole pages)
          const uint32_t loads = __popc(__ballot_sync(0xffffffffu, load));
          if (lane == 0) ptx::mbar_arrive_expect_tx(bar(C::B_KFULL + ks), bytes * loads);
          __syncwarp();
          if (load)
            ptx::tma_load_4d(base + C::OFF_K + ks * C::KT + (lane & 7) * 16 * D, &tmK, bar(C::B_KFULL + ks), 0, 0, g.h, id);
          done = T + 1;
          if (T >= C::NSCL && !tree_warp_wait(bar(C::B_SCLFREE + ss), uint32_t(T / C::NSCL - 1) & 1u, abort_flag, 3)) { ok = false; break; }
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
          if (T >= C::NR && !tree_warp_wait(bar(C::B_RFREE + rs), uint32_t(T / C::NR - 1) & 1u, abort_flag, 5)) { ok = false; break; }
          if (lane == 0) ptx::mbar_arrive_expect_tx(bar(C::B_RFULL + rs), bytes * loads);
          __syncwarp();
          if (load)
            ptx::tma_load_4d(base + C::OFF_R + rs * C::KT + (lane & 7) * 16 * D, &tmV, bar(C::B_RFULL + rs), 0, 0, g.h, id);
          done_v = T + 1;
        }
      }
      // do not leave while a copy may still be writing shared memory
      if (lane == 0) {
#pragma unroll 1
        for (int i = 0; i < C::NK; ++i) {
          if (done <= i) continue;
          const int last = i + C::NK * ((done - 1 - i) / C::NK);
          drain_bar(bar(C::B_KFULL + i), uint32_t(last / C::NK) & 1u, err);
        }
#pragma unroll 1
        for (int i = 0; i < C::NR; ++i) {
          if (done_v <= i) continue;
          const int last = i + C::NR * ((done_v - 1 - i) / C::NR);
          drain_bar(bar(C::B_RFULL + i), uint32_t(last / C::NR) & 1u, err);
        }
      }
      __syncwarp();
    } else if (warp < C::ISSUE_O) {
      // ------------------------------------------------------------ S issuers
      const int m = warp - C::ISSUE_S;
      if (lane == 0) {
        constexpr uint32_t IDESC = ptx::idesc_e4m3_f32(128, kStep);
        const uint64_t qd = ptx::smem_desc(base + C::OFF_Q, 16u, 8 * D, CodeTile<D>::SW);
        const uint64_t kd = ptx::smem_desc(base + C::OFF_K, 16u, 8 * D, CodeTile<D>::SW);
        Segment g;
        int T0 = 0, turn = 0;  // turn: this M tile's tiles so far
        bool ok = true;
#pragma unroll 1
        for (int s = 0; ok && segment(s, g, true, true) && g.tiles; ++s) {
          const bool twin = g.rows <= kTile;
          // (A build may hold back the second M tile's issuer in every segment, to test that the others do not
          // get ahead of a phase that it still waits for.)
#ifdef ATTN_TREE_LATE_NS
          for (const uint64_t t0 = ptx::globaltimer(); m == 1 && ptx::globaltimer() - t0 < ATTN_TREE_LATE_NS;) {
          }
#endif
          // (Behind both M tiles' end of the segment before.  Sooner, the tile two places before this one's first, the
          // other issuer's, may be on its way still, and a wait for a phase's parity would not tell it from it.)
          ok = tree_wait(bar(C::queries(s, m)), C::queries_parity(s), abort_flag, 6) &&
               (!twin || tree_wait(bar(C::queries(s, 1 - m)), C::queries_parity(s), abort_flag, 6));
          if (ok) ptx::mbar_arrive(bar(C::B_SEGFREE + s % C::NSEG));
          const uint64_t qhi = qd + (twin ? 0 : uint64_t(m) * (2 * C::KT >> 4)), qlo = qhi + (C::KT >> 4);
#pragma unroll 1
          for (int j = twin ? m : 0; ok && j < g.tiles; j += twin ? 2 : 1, ++turn) {
            const int T = T0 + j, ks = T % C::NK;
            ok = tree_wait(bar(C::B_KFULL + ks), uint32_t(T / C::NK) & 1u, abort_flag, 7);
#pragma unroll 1
            for (int f = 0; ok && f < 2; ++f) {
              // the P before lies over this S: its product has read it
              if (turn >= 1 && !tree_wait(bar(C::B_PDONE + 2 * m + f), uint32_t(turn - 1) & 1u, abort_flag, 8)) { ok = false; break; }
              ptx::tc_fence_after();
              const uint32_t s_tmem = tmem + uint32_t(128 * m + kStep * f);
              const uint64_t ki = kd + uint64_t((ks * C::KT + f * kStep * D) >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk) ptx::mma_f8_ss(s_tmem, qhi + 2 * kk, ki + 2 * kk, IDESC, kk > 0);
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk) ptx::mma_f8_ss(s_tmem, qlo + 2 * kk, ki + 2 * kk, IDESC, 1);
              ptx::mma_commit(bar(C::B_SFULL + 2 * m + f));
            }
            if (!ok) break;
            ptx::mma_commit(bar(C::B_KFREE + ks));
            if (twin) ptx::mma_commit(bar(C::B_KFREE + ks));
          }
          T0 += g.tiles;
        }
        // every product this thread issued has finished once this arrives
        ptx::mma_commit(bar(C::B_DRAIN + m));
        drain_bar(bar(C::B_DRAIN + m), 0, err);
      }
      __syncwarp();
    } else if (warp == C::ISSUE_O) {
      // ------------------------------------------------------------ P V issuer
      if (lane == 0) {
        constexpr uint32_t IDESC = ptx::idesc_f16_f32(128, D, false, true);
        const uint64_t vd = v_base<D>(base + C::OFF_V);
        Segment g;
        int T = 0, turn[2] = {0, 0};
        bool ok = true;
#pragma unroll 1
        for (int s = 0; ok && segment(s, g, true) && g.tiles; ++s) {
          const bool twin = g.rows <= kTile;
          // the segment before has read its O
          if (s > 0) ok = tree_wait(bar(C::B_OFREE), uint32_t(s - 1) & 1u, abort_flag, 9);
#pragma unroll 1
          for (int j = 0; ok && j < g.tiles; ++j, ++T) {
            const int vs = T % C::NV, first = twin ? j & 1 : 0, last = twin ? first : 1;
            ok = tree_wait(bar(C::B_VFULL + vs), uint32_t(T / C::NV) & 1u, abort_flag, 10);
#pragma unroll 1
            for (int f = 0; ok && f < 2; ++f) {
              const uint64_t vi = vd + uint64_t(vs) * (C::VT >> 4) + v_step<D>(f * (kStep / 16));
#pragma unroll 1
              for (int m = first; m <= last; ++m) {
                ok = tree_wait(bar(C::B_PFULL + 2 * m + f), uint32_t(m ? turn[1] : turn[0]) & 1u, abort_flag, 11);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t p_tmem = tmem + uint32_t(128 * m + kStep * f), o_tmem = tmem + uint32_t(256 + 128 * m);
#pragma unroll
                for (int kk = 0; kk < kStep / 16; ++kk)
                  ptx::mma_ts(o_tmem, p_tmem + uint32_t(kk) * 8u, vi + v_step<D>(kk), IDESC,
                              (j > (twin ? 1 : 0) || f > 0 || kk > 0) ? 1u : 0u);
                ptx::mma_commit(bar(C::B_PDONE + 2 * m + f));
              }
            }
            if (!ok) break;
            ptx::mma_commit(bar(C::B_VFREE + vs));
            turn[0] += first == 0;
            turn[1] += last == 1;
          }
        }
        ptx::mma_commit(bar(C::B_DRAIN + 2));
        drain_bar(bar(C::B_DRAIN + 2), 0, err);
      }
      __syncwarp();
    }
  } else if (warp >= C::VALUES) {
    ptx::regs_dec<C::REG_VALUES>();
    // -------------------------------------------------------------- values
    constexpr int PPT = D / 16;  // 16-byte pieces per token = pieces per thread
    const int ct = threadIdx.x - C::VALUES * 32;
    Segment g;
    int T = 0;
    bool ok = true;
#pragma unroll 1
    for (int s = 0; ok && segment(s, g, false) && g.tiles; ++s) {
      const int end = min(g.token + g.tiles * kTile, g.len);
#pragma unroll 1
      for (int j = 0; j < g.tiles; ++j, ++T) {
        const int rs = T % C::NR, ss = T % C::NSCL, slot = T % C::NV;
        // (the scales' slot was written before this arrived)
        if (!tree_warp_wait(bar(C::B_RFULL + rs), uint32_t(T / C::NR) & 1u, abort_flag, 12)) { ok = false; break; }
        uint4 next[PPT];
#pragma unroll
        for (int i = 0; i < PPT; ++i)
          next[i] = *reinterpret_cast<const uint4*>(sbase + C::OFF_R + rs * C::KT + (i * 128 + ct) * 16);
        const bool gone = __float_as_int(scl[ss * 8 + (lane & 7)].w) < 0;
        if (__any_sync(0xffffffffu, gone) || g.token + (j + 1) * kTile > end) {
          // behind the end, or without a page: weights of 0 times 0
#pragma unroll
          for (int i = 0; i < PPT; ++i) {
            const int row = (i * 128 + ct) / PPT;
            if (g.token + j * kTile + row >= end || __float_as_int(scl[ss * 8 + row / 16].w) < 0)
              next[i] = make_uint4(0, 0, 0, 0);
          }
        }
        warp_arrive(bar(C::B_RFREE + rs), lane);
        if (lane == 0) ptx::mbar_arrive(bar(C::B_SCLFREE + ss));
        if (T >= C::NV && !tree_warp_wait(bar(C::B_VFREE + slot), uint32_t(T / C::NV - 1) & 1u, abort_flag, 13)) { ok = false; break; }
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
    }
  } else {
    ptx::regs_inc<C::REG_SOFTMAX>();
    // -------------------------------------------------------------- softmax
    const int m = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;          // of the M tile, its TMEM lane
    const uint32_t lane_base = tmem + (uint32_t(quarter * 32) << 16);
    const uint32_t o_col = lane_base + 256u + uint32_t(m) * 128u;
    float2* const stats = reinterpret_cast<float2*>(sbase + C::OFF_STATS);
    auto meet = [&](bool x) { return ptx::named_barrier_or(5, 256, x); };
    Segment g;
    int T0 = 0, turn = 0;  // turn: this M tile's tiles so far
    bool ok = true;
#pragma unroll 1
    for (int s = 0;; ++s) {
      ok = ok && segment(s, g, false);
      // (and both M tiles' products have used the queries)
      if (meet(!ok) || g.tiles == 0) break;
      const bool twin = g.rows <= kTile;
      const int mine = (twin ? 0 : m * kTile) + row;  // of the segment's rows
      const bool real = mine < g.rows;
      const bool idle = mine - lane >= g.rows;        // a warp without rows only keeps the steps' order
      const int rg = g.row0 + (real ? mine : 0), node = rg / p.G;
      const int64_t token = g.q0 + node;
      const int head = g.h * p.G + rg - node * p.G;
      const int text = g.len - g.n;
      // Queries: D / 16 lanes per row, rows on their way two turns ahead (the whole row by its own
      // lane took 16 KB of code, which a CTA met anew at every segment).
      // Rows that both M tiles hold lie in the first one's place, half of them brought by each.
      const int place = twin ? 0 : m;
      const float* const factors = reinterpret_cast<const float*>(sbase + C::OFF_ROWS) + place * kTile;
      {
        constexpr int PARTS = D / 16, STEP = 32 / PARTS;
        const int share = twin ? 16 : 32, begin = twin ? m * 64 + quarter * 16 : quarter * 32;
        auto fetch = [&](int r, uint4 (&q)[2]) {
          const int x = (twin ? 0 : m * kTile) + begin + r;
          if (r < share && x < g.rows) {
            const int at = g.row0 + x, node = at / p.G;
            const uint4* src = reinterpret_cast<const uint4*>(
                static_cast<const __nv_bfloat16*>(a.q) +
                (int64_t(g.q0 + node) * a.num_heads + g.h * p.G + at - node * p.G) * D) + 2 * (lane % PARTS);
            q[0] = src[0];
            q[1] = src[1];
          } else {
            q[0] = q[1] = make_uint4(0, 0, 0, 0);
          }
        };
        uint4 q[3][2];
        fetch(lane / PARTS, q[0]);
        fetch(lane / PARTS + STEP, q[1]);
#pragma unroll 1
        for (int r = lane / PARTS; r < share; r += STEP) {
          fetch(r + 2 * STEP, q[2]);
          const float f = p.scale_log2 * split_held<D, PARTS>(q[0], sbase + C::OFF_Q + 2 * place * C::KT, begin + r, C::KT, lane % PARTS);
          if (lane % PARTS == 0) const_cast<float*>(factors)[begin + r] = f;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            q[0][x] = q[1][x];
            q[1][x] = q[2][x];
          }
        }
      }
      ptx::fence_proxy_async_smem();
      warp_arrive(bar(C::queries(s, m)), lane);
      // (brought by other warps)
      if (twin)
        ok = tree_warp_wait(bar(C::queries(s, 0)), C::queries_parity(s), abort_flag, 18) &&
             tree_warp_wait(bar(C::queries(s, 1)), C::queries_parity(s), abort_flag, 18);
      const float qscale = factors[row];

      float mx = kNoReference;                 // the weights' reference (a score + value exponent)
      float2 l2 = make_float2(0.f, 0.f);       // two halves of the sum
      bool some = false;                       // O holds products of this segment
#pragma unroll 1
      for (int j = twin ? m : 0; ok && j < g.tiles; j += twin ? 2 : 1, ++turn) {
        const int T = T0 + j, ss = T % C::NSCL;
        ok = tree_warp_wait(bar(C::B_SCLFULL + ss), uint32_t(T / C::NSCL) & 1u, abort_flag, 14);
#pragma unroll 1
        for (int f = 0; f < 2; ++f) {
          ok = ok && tree_warp_wait(bar(C::B_SFULL + 2 * m + f), uint32_t(turn) & 1u, abort_flag, 15);
          if (!ok) break;
          if (!idle) {
            ptx::tc_fence_after();
            const uint32_t s_col = lane_base + uint32_t(128 * m + kStep * f);
            const float4* sc = scl + ss * 8 + 4 * f;
            const int first = g.token + j * kTile + f * kStep;
            const int odd = __float_as_int(sc[0].w) | __float_as_int(sc[1].w) | __float_as_int(sc[2].w) | __float_as_int(sc[3].w);
            uint64_t see = ~0ull;
            if (__builtin_expect(text - first < kStep || odd < 0, 0)) {
              // Hidden scores to -inf, in tensor memory and rolled up: few steps have any, and the code that
              // all run is the faster for being short.  (A lane without a row hides nothing.)
              if (real) see = tree_step(p.tree.bits + token * p.tree.words, first, text, g.n);
#pragma unroll 1
              for (int q = 0; q < 4; ++q) {
                const uint32_t part = __float_as_int(sc[q].w) < 0 ? 0u : uint32_t(see >> (16 * q)) & 0xFFFFu;
                uint32_t v[16];
                ptx::tmem_ld16(s_col + 16 * q, v);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if (!(part >> e & 1u)) v[e] = 0xFF800000u;
                ptx::tmem_st16(s_col + 16 * q, v);
              }
              ptx::tmem_wait_st();
            }
            uint32_t w[2][32];
            ptx::tmem_ld32(s_col, w[0]);
            ptx::tmem_ld32(s_col + 32, w[1]);
            ptx::tmem_wait_ld();
            // The weights under the present reference, and the sum with them.  Eight of them together above
            // 2^15 (or a segment's first step, or a far page) send the warp to the rows' maxima, and the
            // weights are repeated: scores without a maximum to wait for come through that much sooner.
            float2 lt;
#pragma unroll 1
            for (bool need = !some || (odd & kFar);;) {
              if (__builtin_expect(need, 0)) {
                // a block's largest score: its factor is not negative, so the largest product
                float top = -INFINITY;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const uint32_t* v = w[q >> 1] + (q & 1) * 16;
                  float t = ptx::fmax3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
#pragma unroll
                  for (int e = 3; e < 15; e += 2) t = ptx::fmax3(t, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                  t = fmaxf(t, __uint_as_float(v[15]));
                  if (t > -INFINITY) top = fmaxf(top, fmaf(t, qscale * sc[q].x, sc[q].y));
                }
                // (eight weights of 2^12 do not come here again)
                const bool raise = top > mx + (kMostWeight - 3.f);
                top -= kTopWeight;
                const float half = raise ? half_factor(mx, top) : 1.f, alpha = half * half;
                if (raise) mx = top;
                l2.x = l2.x * half * half;
                l2.y = l2.y * half * half;
                if (some) {  // O holds the earlier steps' products once the last of them has ended
                  ok = tree_warp_wait(bar(C::B_PDONE + 2 * m + (f ^ 1)), uint32_t(turn - (f ^ 1)) & 1u, abort_flag, 16);
                  if (!ok) break;
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
                if (odd & kFar) {  // sums that do not go through the weights, from the scores as they lie
#pragma unroll 1
                  for (int q = 0; q < 4; ++q) {
                    if (__float_as_int(sc[q].w) != kFar) continue;
                    const float by = fmaf(qscale, sc[q].x, 0x1p-126f);
                    uint32_t v[16];
                    ptx::tmem_ld16(s_col + 16 * q, v);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                      const float y = ptx::ex2(0.5f * fmaf(__uint_as_float(v[e]), by, -mx));
                      l2.x = fmaf(y, y, l2.x);
                    }
                  }
                }
              }
              lt = l2;
              float hot = 0.f;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float4 k = sc[q];
                // never 0, where a page is left out or the product is below fp32: a hidden score is
                // -inf, and times 0 it would be NaN
                const float kf = fmaf(qscale, k.x, 0x1p-126f), kx = k.y - mx;
                const float2 f2 = make_float2(kf, kf), x2 = make_float2(kx, kx);
                float2 part = make_float2(0.f, 0.f);
                uint32_t* v = w[q >> 1] + (q & 1) * 16;
                uint32_t pk[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  float2 y = ptx::ffma2(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), f2, x2);
                  y.x = ptx::ex2(y.x);
                  y.y = ptx::ex2(y.y);
                  part = ptx::fadd2(part, y);
                  pk[e] = pack_half2(y.x, y.y);
                }
                lt = ptx::ffma2(part, make_float2(k.z, k.z), lt);
                hot = ptx::fmax3(hot, part.x, part.y);
                ptx::tmem_st8(s_col + 8 * q, pk);  // over S columns read already
              }
              if (__builtin_expect(need || !__any_sync(0xffffffffu, hot > 0x1p15f), 1)) break;
              need = true;
            }
            if (!ok) break;
            l2 = lt;
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            some = true;
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(C::B_PFULL + 2 * m + f));
        }
        if (!ok) break;
        if (lane == 0) {
          ptx::mbar_arrive(bar(C::B_SCLFREE + ss));
          if (twin) ptx::mbar_arrive(bar(C::B_SCLFREE + ss));
        }
      }
      // ---- the segment's end
      T0 += g.tiles;
      const bool had = twin ? m < g.tiles : true;  // this M tile had a tile, the last one's second step the last
      ok = ok && (!had || tree_warp_wait(bar(C::B_PDONE + 2 * m + 1), uint32_t(turn - 1) & 1u, abort_flag, 17));
      ptx::tc_fence_after();
      float l = l2.x + l2.y;
      // Of rows that both M tiles hold, in the same lanes of tensor memory, each ends half of the dimensions.
      float ours = 1.f, theirs = 0.f;  // factors of the two
      if (twin) {
        stats[m * kTile + row] = make_float2(mx, l);
        if (meet(!ok)) break;
        ptx::tc_fence_after();
        const float2 ml = stats[(1 - m) * kTile + row];
        const float top = fmaxf(mx, ml.x);
        const float half = half_factor(mx, top), other_half = half_factor(ml.x, top);
        ours = half * half;
        theirs = other_half * other_half;
        l = l * half * half + ml.y * other_half * other_half;
        mx = top;
      } else if (!ok) {
        continue;  // to the meeting
      }
      const bool whole = g.slot < 0;
      const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
      ours *= inv;
      theirs *= inv;
      const int from = twin ? m * (D / 2) : 0, count = twin ? D / 32 : D / 16;
#pragma unroll 1
      for (int q = 0; q < count; ++q) {
        uint32_t v[16], y[16];
        ptx::tmem_ld16(o_col + uint32_t(from + q * 16), v);
        if (twin) ptx::tmem_ld16((o_col ^ 128u) + uint32_t(from + q * 16), y);
        ptx::tmem_wait_ld();
        if (q == count - 1) {
          ptx::tc_fence_before();
          warp_arrive(bar(C::B_OFREE), lane);
        }
        // (nothing has been written where an M tile had no tile, or has no weight yet)
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = had && ours != 0.f ? __float_as_uint(__uint_as_float(v[e]) * ours) : 0u;
        if (twin && theirs != 0.f && 1 - m < g.tiles) {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(fmaf(__uint_as_float(y[e]), theirs, __uint_as_float(v[e])));
        }
        if (real && whole) {
          uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + (token * a.num_heads + head) * D + from + q * 16);
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = ptx::pack_bf16(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
          out[0] = make_uint4(w[0], w[1], w[2], w[3]);
          out[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else if (real) {
          // four dimensions of all rows together
          uint4* out = reinterpret_cast<uint4*>(p.part_o) + (int64_t(g.slot) * (D / 4) + from / 4 + q * 4) * kTreeRows + mine;
#pragma unroll
          for (int i = 0; i < 4; ++i) out[i * kTreeRows] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
      if (real && (m == 0 || !twin)) {
        if (whole)
          a.lse[int64_t(head) * a.total_tokens + token] = l == 0.f ? -INFINITY : (mx + log2f(l)) * kLn2;
        else
          p.part_m[int64_t(g.slot) * kTreeRows + mine] = make_float2(mx, l);
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) atomicOr(err, kErrTimeout | int(*abort_flag - 1u) << 9);
  if (warp == C::ISSUE_O) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

constexpr int kJoinWarps = 8, kJoinRows = 32;  // per CTA: a lane per row, a warp per eighth of the dimensions

// Starts while the first kernel ends, and waits for it.
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) cache_tree_many_join_kernel(const __grid_constant__ TreeParams p) {
  constexpr int E = D / kJoinWarps / 4;  // of four dimensions
  const CacheQueryArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, x = blockIdx.x, row = blockIdx.y * kJoinRows + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const TreeCut cut = p.cuts[x];
  if (cut.parts < 2 || row >= cut.rows) return;
  float m = -INFINITY, sum = 0.f;
  float4 o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int i = 0; i < cut.parts; ++i) {
    const int64_t slot = 2 * (x + i) + (i == 0 ? 1 : 0);
    const float2 s = p.part_m[slot * kTreeRows + row];
    float4 v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = reinterpret_cast<const float4*>(p.part_o)[(slot * (D / 4) + warp * E + e) * kTreeRows + row];
    const float top = fmaxf(m, s.x), was = half_factor(m, top), now = half_factor(s.x, top);
    const float old = was * was, f = now * now;
    m = top;
    sum = sum * was * was + (s.y != s.y ? s.y : s.y * now * now);
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = make_float4(fmaf(v[e].x, f, o[e].x * old), fmaf(v[e].y, f, o[e].y * old), fmaf(v[e].z, f, o[e].z * old),
                         fmaf(v[e].w, f, o[e].w * old));
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int rg = cut.row0 + row, node = rg / p.G, head = cut.h * p.G + rg - node * p.G;
  const int64_t at = cut.q0 + node;
  uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + (at * a.num_heads + head) * D + warp * (E * 4));
#pragma unroll
  for (int e = 0; e < E; ++e)
    out[e] = make_uint2(ptx::pack_bf16(o[e].x * inv, o[e].y * inv), ptx::pack_bf16(o[e].z * inv, o[e].w * inv));
  if (warp == 0) a.lse[int64_t(head) * a.total_tokens + at] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
}

template <int D>
attn_status launch_d(const TreeParams& p, cudaStream_t s) {
  using C = ManyCfg<D>;
  const CacheView& c = p.a.cache;
  CUtensorMap map, map_v;
  if (!encode_pages<D>(&map, c, c.k_pages, true) || !encode_pages<D>(&map_v, c, c.v_pages, false))
    return record_cuda_error(cudaErrorInvalidValue, "attn_cache_tree_fwd tensor map encoding");
  cudaError_t e = cudaFuncSetAttribute(cache_tree_many_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return record_cuda_error(e, "attn_cache_tree_fwd configure");
  cache_tree_many_kernel<D><<<unsigned(p.ctas), C::THREADS, C::SMEM, s>>>(map, map_v, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return record_cuda_error(e, "attn_cache_tree_fwd launch");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.ctas), kTreeRows / kJoinRows);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, cache_tree_many_join_kernel<D>, p);
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_tree_fwd join launch");
}

uint64_t partial_bytes(int D) { return 2ull * kTreeSms * kTreeRows * (uint64_t(D) * 4 + 8); }

}  // namespace

uint64_t cache_tree_many_workspace(const CacheView& c) {
  return partial_bytes(c.head_dim) + kTreeSms * sizeof(TreeCut);
}

attn_status launch_cache_tree_many(const CacheQueryArgs& a, const TreeMasks& tree, cudaStream_t s) {
  TreeParams p;
  p.a = a;
  p.tree = tree;
  p.G = a.num_heads / a.cache.heads;
  p.ctas = kTreeSms;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.part_o = a.workspace;
  p.part_m = reinterpret_cast<float2*>(a.workspace + 2ull * kTreeSms * kTreeRows * a.cache.head_dim);
  p.cuts = reinterpret_cast<TreeCut*>(a.workspace + partial_bytes(a.cache.head_dim) / 4);
  switch (a.cache.head_dim) {
    case 32: return launch_d<32>(p, s);
    case 64: return launch_d<64>(p, s);
    default: return launch_d<128>(p, s);
  }
}

}  // namespace attnmask
