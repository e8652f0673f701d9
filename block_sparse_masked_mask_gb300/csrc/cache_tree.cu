// Attention of trees of drafted tokens over the 8-bit cache, on the tcgen05 tensor
// cores: up to 64 rows (nodes times query heads of the group) share each cached byte.
//
// That is too few to fill the 128 lanes of a product, so the products are turned round: tokens are
// their M, rows their N, padded to 16, 32 or 64 only.
//  * S^T = K Q^T on the codes as they lie (kind::f8f6f4), a query as the sum of two
//    e4m3 numbers (cache_tiles.cuh).
//  * O^T += V^T P^T in fp16.  One warpgroup turns the values' codes into fp16 in tensor memory,
//    dimensions in its lanes (a transposed load of bytes); the softmax writes its weights to
//    shared memory, rows along the tokens (stmatrix).
//  * Scores, scales, references and far pages are those of cache_attn.cu: the weight is
//    2^(s + x - m), x the exponent of the page's value scale.  A page has one scale for 16 tokens at
//    least, which a warp's loads from tensor memory are arranged by, so it is uniform there; m, the
//    row's factor and its sum stay in the registers of the lanes that hold the row.
//  * References move when the sum of two weights of any row passes 2^15.  The warps vote on that with
//    a barrier's OR, once a tile, behind the weights; a tile that moves them repeats its weights.
//  * Two warpgroups take tiles in turn, each with references, sums and O of its own, which meet
//    at a segment's end.
//  * The masks matter in the tiles that hold the tree (and at the end of a sequence): only there
//    hidden scores are overwritten, in tensor memory, before the loop that all tiles share.
// Work: tiles of 128 tokens of all (sequence, head)s form one line that is cut evenly among one
// CTA per SM (TreeLine in cache_tree.cuh); a CTA's piece is walked segment by segment without a pause between them: the
// rings of tiles run on, queries and O have two buffers each.  Segments that are
// not whole meet in a second kernel (cache_join.cuh), two per CTA at most.
// Warps (512 threads):
//   0-3, 4-7   softmax of every other tile
//   8-11       queries; values: codes to fp16
//   12         pages, scales and TMA of the codes
//   13, 14     tcgen05 issuers of S^T and of O^T (which also owns TMEM)
//   15         the line: the CTA's segments
//
// What bounds it: 64 trees of 4 to 8 nodes behind 1024 to 16384 tokens, 32 query and 8 key heads of
// 128, take 137 us where the bytes take 108 at the rate of a copy; 16 sequences of 8192 tokens, 16 / 32 / 64
// rows a head, 55 / 59 / 71 us (40).  Heads of 64 or 32 take as long as those of 128 (139 us both): it is
// not the bytes but the softmax, a score as dear as any other, and the instructions'
// supply more than their issue: with five roles' loops at once, warps wait for instructions
// more than for anything else, and each step that made the code shorter (loops rolled up, one form of
// waits, rare paths out of line) was worth more than one that took operations out.  Four
// warpgroups for the softmax, or factors held ready across its loop, were no faster.
// One tree of 16 nodes behind 2049 tokens takes 18 us: the kernels' start, one tile, the join.
//
// Every wait is bounded and ends in ATTN_ERR_DEVICE_TIMEOUT in the cache's status word.
// Each role waits only for an earlier tile's events of the others, or for this
// tile's by a role that comes before it (line, pages, queries and keys, S^T, softmax,
// values, O^T), so the order of tiles carries every wait to its end.  Warps of the softmax
// meet at barriers without a bound: a wait that ran out counts in the vote behind it, and
// they leave together.
#include <algorithm>
#include <cmath>

#include "cache_join.cuh"
#include "cache_tree.cuh"

namespace attnmask {
namespace {

// A piece of the line in one (sequence, head).
struct Segment {
  int tiles;  // 0: there is no further one
  int b, h, rows, q0, n, len, token, slot;  // slot of the partial result, -1: whole
};

// A segment's start and end cost as much as three tiles (64 trees of 4 to 8 nodes, heads of 128 / 64 / 32: taken for 0
// 154 / 154 / 152 us, 2 137 / 143 / 140, 3 137 / 139 / 139, 4 138 / 141 / 141, 7 144 / 146 / 145); pieces of less than two tiles' cost gain nothing (a tree of 16 nodes behind 1024
// tokens: from 1 17.4 us, 2 16.5, 4 17.9, 6 19.4).
template <int N>
using Line = TreeLine<N, 1, 1, 3, 2>;

// E 16-bit rows of 128 tokens (P^T): MN-major, swizzled over a token's width.
template <int E>
struct WeightTile {
  static constexpr int ROWB = E * 2, BYTES = kTile * ROWB;
  static constexpr uint32_t SW = ROWB == 128 ? ptx::kSwizzle128B : ROWB == 64 ? ptx::kSwizzle64B : ptx::kSwizzle32B;
  __device__ static uint32_t unit(int token, int u) {  // byte offset of 16-byte unit u of the token
    const int x = ROWB == 128 ? (token & 7) : ROWB == 64 ? ((token >> 1) & 3) : ((token >> 2) & 1);
    return uint32_t(token * ROWB + ((u ^ x) << 4));
  }
  __device__ static uint64_t desc(uint32_t addr) { return ptx::smem_desc(addr, BYTES, 8 * ROWB, SW); }
  __host__ __device__ static constexpr uint64_t step(int kk) { return uint64_t(kk * 16 * ROWB) >> 4; }
};

template <int D, int N>
struct TreeCfg {
  using P = WeightTile<N>;
  // Warpgroups of the softmax, and the warps behind them
  static constexpr int GROUPS = 2, THREADS = 128 * GROUPS + 256;
  static constexpr int CONVERT = 4 * GROUPS, PAGES = CONVERT + 4, ISSUE_S = PAGES + 1, ISSUE_O = PAGES + 2, LINE = PAGES + 3;
  // Registers for each thread of the softmax, the conversion and the others, of the launch's 128 for all
  static constexpr int REG_SOFTMAX = 168, REG_CONVERT = 104, REG_OTHERS = 72;
  static_assert(GROUPS * REG_SOFTMAX + REG_CONVERT + REG_OTHERS == (GROUPS + 2) * 128, "registers");
  static constexpr int KT = CodeTile<D>::BYTES;   // a tile of codes
  static constexpr int QT = 2 * N * D;            // queries: hi, lo
  static constexpr int NB = N <= 32 ? 3 : 2;      // of scores and of weights
  static constexpr int NO = 2;                    // segments' O
  static constexpr int NK = N <= 32 ? 5 : 4, NR = NK;
  static constexpr int NSCL = 8, NSEG = 4;
  static constexpr int OFF_P = 0;
  static constexpr int OFF_Q = OFF_P + NB * P::BYTES;
  static constexpr int OFF_K = OFF_Q + (2 * QT + 1023) / 1024 * 1024;
  static constexpr int OFF_R = OFF_K + NK * KT;
  static constexpr int OFF_SCL = OFF_R + NR * KT;          // as in cache_chunk.cu
  static constexpr int OFF_ROWS = OFF_SCL + NSCL * 8 * 16; // [2][N]: the rows' factors
  static constexpr int OFF_MAX = OFF_ROWS + 2 * N * 4;     // [warpgroup][4 warps][N]: maxima, then sums
  static constexpr int OFF_REF = OFF_MAX + GROUPS * 4 * N * 4;  // [warpgroup][N]: negative references
  static constexpr int OFF_MOVE = OFF_REF + GROUPS * N * 4;     // [warp][N]: negative reference, half the factor's exponent
  static constexpr int OFF_OUT = OFF_MOVE + GROUPS * 4 * N * 8;      // [N]: factors of the two warpgroups' O, place in the outputs
  static constexpr int OFF_SEG = OFF_OUT + N * 16;
  static constexpr int OFF_BAR = OFF_SEG + NSEG * 48;
  static constexpr int B_SEGFULL = 0, B_SEGFREE = B_SEGFULL + NSEG, B_QFULL = B_SEGFREE + NSEG, B_QFREE = B_QFULL + 2,
                       B_KFULL = B_QFREE + 2, B_KFREE = B_KFULL + NK, B_RFULL = B_KFREE + NK, B_RFREE = B_RFULL + NR,
                       B_VFULL = B_RFREE + NR, B_VFREE = B_VFULL + 2, B_SCLFULL = B_VFREE + 2,
                       B_SCLFREE = B_SCLFULL + NSCL, B_SFULL = B_SCLFREE + NSCL, B_PFULL = B_SFULL + NB,
                       B_PDONE = B_PFULL + NB, B_OFREE = B_PDONE + NB, B_USED = B_OFREE + NO,
                       B_DRAIN = B_USED + 2, NBAR = B_DRAIN + 2;
  static_assert(NBAR <= THREADS, "a thread for each");
  __device__ static int arrivals(int i) {
    constexpr int ALL = 4 * GROUPS, EACH = 4;  // warps of the softmax, and of those with a tile
    return i >= B_OFREE ? (i >= B_DRAIN ? 1 : ALL)
           : i >= B_PFULL ? (i >= B_PDONE ? 1 : EACH)
           : i >= B_SCLFREE ? (i >= B_SFULL ? 1 : 4 + EACH)  // value and softmax warps
           : i >= B_SCLFULL ? 1
           : i >= B_VFULL ? (i >= B_VFREE ? 1 : 4)
           : i >= B_RFREE ? 4
           : i >= B_QFULL ? (i >= B_QFREE ? 1 : 4)
           : i >= B_SEGFREE ? LINE : 1;  // the warps before that one
  }
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int USED = OFF_MISC + 16 + 1024;        // the base is aligned to 1024
  // one CTA per SM: it takes all of TMEM
  static constexpr int SMEM = USED > 116 * 1024 ? USED : 116 * 1024;
  static_assert(SMEM <= 232448, "shared memory budget");
  // TMEM columns
  static constexpr int S = 0, O = NB * N, OSEG = GROUPS * N, V = O + NO * OSEG;
  static_assert(V + 2 * 64 <= 512, "tensor memory");
};

template <int D, int N>
__global__ void __launch_bounds__(TreeCfg<D, N>::THREADS, 1)
    cache_tree_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ TreeParams p) {
  using C = TreeCfg<D, N>;
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

  // The s-th segment, copied from its place in the ring; one arrival frees that.
  auto segment = [&](int s, Segment& g, bool single) {
    const int at = s % C::NSEG;
    const bool ok = single ? tree_wait(bar(C::B_SEGFULL + at), uint32_t(s / C::NSEG) & 1u, abort_flag, 1)
                           : tree_warp_wait(bar(C::B_SEGFULL + at), uint32_t(s / C::NSEG) & 1u, abort_flag, 1);
    g.tiles = 0;
    if (!ok) return false;
    const int4* w = reinterpret_cast<const int4*>(sbase + C::OFF_SEG + at * 48);
    const int4 x = w[0], y = w[1];
    const int slot = w[2].x;
    g = Segment{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, slot};
    if (single) ptx::mbar_arrive(bar(C::B_SEGFREE + at));
    else warp_arrive(bar(C::B_SEGFREE + at), lane);
    return true;
  };

  // (the registers are split in each branch: where they meet, the least would hold for all)
  if (warp >= C::PAGES) {
   ptx::regs_dec<C::REG_OTHERS>();
   if (warp == C::LINE) {
    // -------------------------------------------------------------- segments
    const int64_t total = Line<N>::total(p, lane), piece = Line<N>::share(total, p);
    int64_t pos = min(int64_t(blockIdx.x) * piece, total);
    const int64_t stop = min(pos + piece, total);
    // (after a wait that ran out in an earlier CTA there is nothing to do)
    if (*reinterpret_cast<volatile int32_t*>(err) & kErrTimeout) pos = stop;
    int64_t before = 0;
    int b = pos < stop ? Line<N>::find(p, pos, lane, before) : 0;
    TreeCut cut{};
#pragma unroll 1
    for (int s = 0;; ++s) {
      Segment g{};
#pragma unroll 1
      while (pos < stop) {
        const int64_t all = Line<N>::of(p, b);
        if (pos >= before + all) {
          before += all;
          ++b;
          continue;
        }
        const int q0 = a.cu[b], n = a.cu[b + 1] - q0, len = a.lens[b];
        const typename Line<N>::Seq l(n, p.G, len);
        const typename Line<N>::Item it(l, before, pos);
        const int u0 = it.tiles(pos, l.U), u1 = it.tiles(stop, l.U);
        pos = min(stop, it.end);
        if (u1 <= u0) continue;
        g.tiles = u1 - u0;
        g.b = b;
        g.h = it.h;
        g.rows = n * p.G;
        g.q0 = q0;
        g.n = n;
        g.len = len;
        g.token = u0 * kTile;
        g.slot = u0 == 0 && u1 == l.U ? -1 : 2 * int(blockIdx.x) + (u0 > 0 ? 0 : 1);
        if (u0 == 0 && u1 < l.U)
          cut = TreeCut{int((it.end - it.w) / piece) - int(blockIdx.x) + 1, g.h, 0, g.rows, g.q0};
        break;
      }
      const int at = s % C::NSEG;
      if (s >= C::NSEG && !tree_warp_wait(bar(C::B_SEGFREE + at), uint32_t(s / C::NSEG - 1) & 1u, abort_flag, 2)) break;
      if (lane == 0) {
        int4* w = reinterpret_cast<int4*>(sbase + C::OFF_SEG + at * 48);
        w[0] = make_int4(g.tiles, g.b, g.h, g.rows);
        w[1] = make_int4(g.q0, g.n, g.len, g.token);
        w[2].x = g.slot;
        ptx::mbar_arrive(bar(C::B_SEGFULL + at));
      }
      __syncwarp();
      if (g.tiles == 0) break;
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
    // -------------------------------------------------------------- pages, scales, codes
    // Eight lanes a tile, one per 16 tokens: lanes 8 q .. 8 q + 7 look up the q-th
    // tile of four.  Page numbers are read two fours ahead, scales one.
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
  } else if (warp == C::ISSUE_S) {
    // -------------------------------------------------------------- S^T issuer
    if (lane == 0) {
      constexpr uint32_t IDESC = ptx::idesc_e4m3_f32(128, N);
      const uint64_t qd = ptx::smem_desc(base + C::OFF_Q, 16u, 8 * D, CodeTile<D>::SW);
      const uint64_t kd = ptx::smem_desc(base + C::OFF_K, 16u, 8 * D, CodeTile<D>::SW);
      Segment g;
      int T = 0;
      bool ok = true;
#pragma unroll 1
      for (int s = 0; ok && segment(s, g, true) && g.tiles; ++s) {
        ok = tree_wait(bar(C::B_QFULL + (s & 1)), uint32_t(s >> 1) & 1u, abort_flag, 6);
        const uint64_t qhi = qd + uint64_t((s & 1) * C::QT >> 4), qlo = qhi + uint64_t(N * D >> 4);
#pragma unroll 1
        for (int j = 0; ok && j < g.tiles; ++j, ++T) {
          const int ks = T % C::NK, f = T % C::NB;
          ok = tree_wait(bar(C::B_KFULL + ks), uint32_t(T / C::NK) & 1u, abort_flag, 7) &&
               // the softmax has read the scores that lie there
               (T < C::NB || tree_wait(bar(C::B_PFULL + f), uint32_t(T / C::NB - 1) & 1u, abort_flag, 8));
          if (!ok) break;
          ptx::tc_fence_after();
          const uint64_t ki = kd + uint64_t(ks * C::KT >> 4);
          const uint32_t s_tmem = tmem + uint32_t(C::S + f * N);
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) ptx::mma_f8_ss(s_tmem, ki + 2 * kk, qhi + 2 * kk, IDESC, kk > 0);
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) ptx::mma_f8_ss(s_tmem, ki + 2 * kk, qlo + 2 * kk, IDESC, 1);
          ptx::mma_commit(bar(C::B_SFULL + f));
          ptx::mma_commit(bar(C::B_KFREE + ks));
          if (j == g.tiles - 1) ptx::mma_commit(bar(C::B_QFREE + (s & 1)));
        }
      }
      // every product this thread issued has finished once this arrives
      ptx::mma_commit(bar(C::B_DRAIN));
      drain_bar(bar(C::B_DRAIN), 0, err);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- O^T issuer
    if (lane == 0) {
      constexpr uint32_t IDESC = ptx::idesc_f16_f32(128, N, false, true);
      const uint64_t pd = C::P::desc(base + C::OFF_P);
      Segment g;
      int T = 0;
      bool ok = true;
#pragma unroll 1
      for (int s = 0; ok && segment(s, g, true) && g.tiles; ++s) {
        if (s >= C::NO) ok = tree_wait(bar(C::B_OFREE + s % C::NO), uint32_t(s / C::NO - 1) & 1u, abort_flag, 9);
        const uint32_t o_seg = tmem + uint32_t(C::O + s % C::NO * C::OSEG);
#pragma unroll 1
        for (int j = 0; ok && j < g.tiles; ++j, ++T) {
          const int f = T % C::NB, vs = T & 1;
          ok = tree_wait(bar(C::B_VFULL + vs), uint32_t(T >> 1) & 1u, abort_flag, 11) &&
               tree_wait(bar(C::B_PFULL + f), uint32_t(T / C::NB) & 1u, abort_flag, 10);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t o_tmem = o_seg + uint32_t(T & 1) * N, v_tmem = tmem + uint32_t(C::V + vs * 64);
          const uint64_t pi = pd + uint64_t(f * C::P::BYTES >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            ptx::mma_ts(o_tmem, v_tmem + uint32_t(kk) * 8u, pi + C::P::step(kk), IDESC, (j > 1 || kk > 0) ? 1u : 0u);
          ptx::mma_commit(bar(C::B_PDONE + f));
          ptx::mma_commit(bar(C::B_VFREE + vs));
        }
      }
      ptx::mma_commit(bar(C::B_DRAIN + 1));
      drain_bar(bar(C::B_DRAIN + 1), 0, err);
    }
    __syncwarp();
   }
  } else if (warp >= C::CONVERT) {
    ptx::regs_dec<C::REG_CONVERT>();
    // -------------------------------------------------------------- queries, values
    const int ct = threadIdx.x - C::CONVERT * 32, cw = warp - C::CONVERT;
    Segment g;
    int T = 0;
    bool ok = true;
#pragma unroll 1
    for (int s = 0; ok && segment(s, g, false) && g.tiles; ++s) {
      // the queries two segments back are used, and so are their factors
      if (s >= 2) ok = tree_warp_wait(bar(C::B_QFREE + (s & 1)), uint32_t((s >> 1) - 1) & 1u, abort_flag, 12);
      if (ok && s >= 2) ok = tree_warp_wait(bar(C::B_USED + (s & 1)), uint32_t((s >> 1) - 1) & 1u, abort_flag, 13);
      if (!ok) break;
      // D / 16 lanes per row, rows on their way two turns ahead
      constexpr int PARTS = D / 16, STEP = 128 / PARTS;
      auto fetch = [&](int row, uint4 (&q)[2]) {
        if (row < g.rows) {
          const uint4* src = reinterpret_cast<const uint4*>(
              static_cast<const __nv_bfloat16*>(a.q) +
              (int64_t(g.q0 + row / p.G) * a.num_heads + g.h * p.G + row % p.G) * D) + 2 * (ct % PARTS);
          q[0] = src[0];
          q[1] = src[1];
        } else {
          q[0] = q[1] = make_uint4(0, 0, 0, 0);
        }
      };
      uint4 q[3][2];
      fetch(ct / PARTS, q[0]);
      fetch(ct / PARTS + STEP, q[1]);
#pragma unroll 1
      for (int row = ct / PARTS; row < N; row += STEP) {  // (whole warps)
        fetch(row + 2 * STEP, q[2]);
        const float f = p.scale_log2 * split_held<D, PARTS>(q[0], sbase + C::OFF_Q + (s & 1) * C::QT, row, N * D, ct % PARTS);
        if (ct % PARTS == 0) reinterpret_cast<float*>(sbase + C::OFF_ROWS)[(s & 1) * N + row] = f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          q[0][x] = q[1][x];
          q[1][x] = q[2][x];
        }
      }
      ptx::fence_proxy_async_smem();
      warp_arrive(bar(C::B_QFULL + (s & 1)), lane);
      const int end = min(g.token + g.tiles * kTile, g.len);
#pragma unroll 1
      for (int j = 0; j < g.tiles; ++j, ++T) {
        const int rs = T % C::NR, ss = T % C::NSCL;
        // (the scales' slot was written before this arrived)
        if (!tree_warp_wait(bar(C::B_RFULL + rs), uint32_t(T / C::NR) & 1u, abort_flag, 14)) { ok = false; break; }
        const bool gone = __float_as_int(scl[ss * 8 + (lane & 7)].w) < 0;
        const bool ragged = __any_sync(0xffffffffu, gone) || g.token + (j + 1) * kTile > end;
        if (T >= 2 && !tree_warp_wait(bar(C::B_VFREE + (T & 1)), uint32_t((T >> 1) - 1) & 1u, abort_flag, 15)) { ok = false; break; }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int u = 2 * cw + z;  // 16 dimensions
          if (u >= D / 16) break;
          uint32_t w[16];  // tokens 16 b + 4 i .. + 3 of dimensions g and g + 8, i and g of the lane
#pragma unroll
          for (int x = 0; x < 4; ++x)
            ptx::ldmatrix_bytes(base + C::OFF_R + rs * C::KT + CodeTile<D>::unit(32 * x + lane, u), w[4 * x], w[4 * x + 1],
                                w[4 * x + 2], w[4 * x + 3]);
          if (__builtin_expect(ragged, 0)) {
            // behind the end, or without a page: weights of 0 times 0
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const int first = g.token + j * kTile + 16 * x + 4 * (lane & 3);
              const int n = __float_as_int(scl[ss * 8 + x].w) < 0 ? 0 : min(max(end - first, 0), 4);
              const uint32_t keep = n == 4 ? ~0u : (1u << (8 * n)) - 1u;
              w[2 * x] &= keep;
              w[2 * x + 1] &= keep;
            }
          }
          const uint32_t to = tmem + (uint32_t(16 * u) << 16) + uint32_t(C::V + (T & 1) * 64);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t v[16];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              v[2 * y] = half2_of(w[8 * x + y]);
              v[2 * y + 1] = half2_of_high(w[8 * x + y]);
            }
            ptx::tmem_st16x256(to + uint32_t(32 * x), v);
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        warp_arrive(bar(C::B_VFULL + (T & 1)), lane);
        if (lane == 0) {
          ptx::mbar_arrive(bar(C::B_RFREE + rs));
          ptx::mbar_arrive(bar(C::B_SCLFREE + ss));
        }
      }
    }
  } else {
    ptx::regs_inc<C::REG_SOFTMAX>();
    // -------------------------------------------------------------- softmax
    // A warp takes 32 tokens, in two blocks of 16 (of one page each); of a block, lane
    // 4 g + i holds tokens g and g + 8 and rows 8 k + 2 i, + 1.  What a tile costs besides its
    // scores (waits, the vote) is paid by each warpgroup for every other one.
    // The weights are formed and stored before the vote on the references; a tile whose
    // references move repeats them.
    constexpr int K = N / 8, STRIDE = C::GROUPS;
    const int wg = warp >> 2, w4 = warp & 3, g4 = lane >> 2, i4 = lane & 3;
    const uint32_t lanes = tmem + (uint32_t(w4 * 32) << 16);
    float* const warps = reinterpret_cast<float*>(sbase + C::OFF_MAX) + wg * 4 * N;  // [warp][row]: maxima, then sums
    float* const refs = reinterpret_cast<float*>(sbase + C::OFF_REF);                   // [warpgroup][row]
    float4* const out = reinterpret_cast<float4*>(sbase + C::OFF_OUT);
    auto meet = [&](bool x) { return ptx::named_barrier_or(1 + wg, 128, x); };
    auto meet_all = [&](bool x) { return ptx::named_barrier_or(5, 256, x); };
    // Scores of this warp's tokens to -inf where the row does not see the token, for which
    // `see` of the token's lane has no bit.  In tensor memory, and rolled up: few tiles have any, and
    // the loop over the others is the faster for being short.
    auto hide = [&](uint32_t s_col, uint64_t see) {
#pragma unroll 1
      for (int x = 0; x < 2 * K; ++x) {
        const uint32_t at = s_col + (uint32_t(16 * (x / K)) << 16) + uint32_t(8 * (x % K));
        uint32_t v[4];
        ptx::tmem_ld16x256(at, v);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint64_t seen = __shfl_sync(0xffffffffu, see, 16 * (x / K) + 8 * e + g4) >> (8 * (x % K) + 2 * i4);
          if (!(seen & 1u)) v[2 * e] = 0xFF800000u;
          if (!(seen & 2u)) v[2 * e + 1] = 0xFF800000u;
        }
        ptx::tmem_st16x256(at, v);
      }
      ptx::tmem_wait_st();
    };
    // (never 0, where a page is left out or the product is below fp32: a hidden score is -inf, and
    // times 0 it would be NaN)
    auto factor = [](float2 f, float2 ks) { return ptx::ffma2(f, ks, make_float2(0x1p-126f, 0x1p-126f)); };
    float2* const move = reinterpret_cast<float2*>(sbase + C::OFF_MOVE) + warp * N;
    // The scales of this warp's two blocks of tile T, which has no further use for its slot.
    float4 of[2];
    auto scales = [&](int T) {
      const int ss = T % C::NSCL;
      if (!tree_warp_wait(bar(C::B_SCLFULL + ss), uint32_t(T / C::NSCL) & 1u, abort_flag, 17)) return false;
      of[0] = scl[ss * 8 + w4 * 2];
      of[1] = scl[ss * 8 + w4 * 2 + 1];
      warp_arrive(bar(C::B_SCLFREE + ss), lane);
      return true;
    };
    // where this lane's row of a matrix of weights goes: a token, and the first or second
    // eight rows of the query of sixteen
    const int to_token = w4 * 32 + (lane & 15), to_unit = lane >> 4;
    // Before the first segment is there, one tile of nothing (on what lies in this warpgroup's O):
    // the instructions of the loop arrive while the first keys do, and not after them.
    Segment g{wg + 1, 0, 0, 0, 0, 0, 1 << 30, 0, 0};
    of[0] = of[1] = make_float4(1.f, 0.f, 1.f, 0.f);
    bool dry = opaque(1) != 0;
#pragma unroll 1
    for (int s = 0, T0 = 0;;) {
      bool ok = true;
      if (!dry) {
        ok = segment(s, g, false);
        if (ok && g.tiles) ok = tree_warp_wait(bar(C::B_QFULL + (s & 1)), uint32_t(s >> 1) & 1u, abort_flag, 16);
        if (meet_all(!ok) || g.tiles == 0) break;
      }
      const int text = g.len - g.n;
      const uint32_t o_seg = lanes + uint32_t(C::O + s % C::NO * C::OSEG), o_col = o_seg + uint32_t(wg * N);
      const float* factors = reinterpret_cast<const float*>(sbase + C::OFF_ROWS) + (s & 1) * N;
      float2 f2[K], m2[K], l2[K];  // of the rows: factor, negative reference, sum
#pragma unroll
      for (int k = 0; k < K; ++k) {
        f2[k] = *reinterpret_cast<const float2*>(factors + 8 * k + 2 * i4);
        m2[k] = make_float2(-kNoReference, -kNoReference);
        l2[k] = make_float2(0.f, 0.f);
      }

      const int mine = (T0 ^ wg) & 1;  // the first tile of this warpgroup's
      if (mine < g.tiles && !dry) ok = scales(T0 + mine);
      bool left = false;
#pragma unroll 1
      for (int j = mine; j < g.tiles; j += STRIDE) {
        const int T = T0 + j, f = T % C::NB;
        const uint32_t s_col = dry ? o_col : lanes + uint32_t(C::S + f * N), weights = base + C::OFF_P + f * C::P::BYTES;
        const int token = g.token + j * kTile + w4 * 32 + lane;
        const int flags = __float_as_int(of[0].w) | __float_as_int(of[1].w);
        // which rows see this lane's token
        const bool masked = __any_sync(0xffffffffu, token >= text) || flags < 0;
        uint64_t see = ~0ull;
        if (__builtin_expect(masked, 0)) {
          const bool here = token < g.len && __float_as_int(lane < 16 ? of[0].w : of[1].w) >= 0;
          see = here && token < text ? ~0ull : 0ull;
          if (here && token >= text) {
            const int node = token - text;
            const uint32_t* word = p.tree.bits + int64_t(g.q0) * p.tree.words + (node >> 5);
#pragma unroll 4
            for (int i = 0; i < g.n; ++i) {
              const uint32_t bit = __ldg(word + int64_t(i) * p.tree.words) >> (node & 31) & 1u;
              // (the last row may be the 64th)
              const uint64_t span = (i + 1) * p.G >= 64 ? ~0ull << i * p.G : ((1ull << p.G) - 1) << i * p.G;
              see |= bit ? span : 0ull;
            }
          }
        }
        // the scores, and room for the weights
        ok = ok && (dry || tree_warp_wait(bar(C::B_SFULL + f), uint32_t(T / C::NB) & 1u, abort_flag, 18)) &&
             (T < C::NB || tree_warp_wait(bar(C::B_PDONE + f), uint32_t(T / C::NB - 1) & 1u, abort_flag, 19));
        ptx::tc_fence_after();
        if (__builtin_expect(masked, 0)) hide(s_col, see);
        float2 lt[K];  // the sums with this tile's
        float top;
        // The weights under the present references, into shared memory, and the largest sum of two.
        auto weigh = [&]() {
          top = 0.f;
#pragma unroll
          for (int k = 0; k < K; ++k) lt[k] = l2[k];
          // (rolled up: the second block's instructions are still at hand)
#pragma unroll 1
          for (int z = 0; z < 2; ++z) {
            uint32_t v[4 * K];
            ptx::tmem_ld16x256(s_col + (uint32_t(16 * z) << 16), v);
            const float2 ks = z ? make_float2(of[1].x, of[1].x) : make_float2(of[0].x, of[0].x);
            const float2 x = z ? make_float2(of[1].y, of[1].y) : make_float2(of[0].y, of[0].y);
            const float2 inv = z ? make_float2(of[1].z, of[1].z) : make_float2(of[0].z, of[0].z);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int k0 = 0; k0 < K; k0 += 2) {
              uint32_t pk[4];
#pragma unroll
              for (int kk = 0; kk < 2; ++kk) {
                const int k = k0 + kk;
                const float2 by = factor(f2[k], ks), at = ptx::fadd2(m2[k], x);
                float2 y[2];  // of tokens g and g + 8
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t* const w = v + 4 * k + 2 * e;
                  y[e] = ptx::ffma2(make_float2(__uint_as_float(w[0]), __uint_as_float(w[1])), by, at);
                  y[e] = make_float2(ptx::ex2(y[e].x), ptx::ex2(y[e].y));
                  pk[2 * kk + e] = pack_half2(y[e].x, y[e].y);
                }
                const float2 sum = ptx::fadd2(y[0], y[1]);
                top = ptx::fmax3(top, sum.x, sum.y);
                lt[k] = ptx::ffma2(sum, inv, lt[k]);
              }
              // (the 16 tokens of the second block are 16 rows on, whatever the swizzle)
              ptx::stmatrix(weights + C::P::unit(to_token, to_unit + k0) + z * 16 * C::P::ROWB, pk[0], pk[1], pk[2], pk[3]);
            }
          }
        };
#pragma unroll 1
        for (bool moved = opaque(0) != 0;; moved = true) {
          // (the first tile sets the references)
          if (j >= STRIDE || moved) {
            weigh();
            if (__builtin_expect(moved || !meet(!ok || top > 0x1p15f), 1)) break;
          }
          // two weights together pass 2^15 (or a wait ran out): references move where one may have
#pragma unroll 2
          for (int k = 0; k < K; ++k) {
            uint32_t v[2][4];
#pragma unroll
            for (int z = 0; z < 2; ++z) ptx::tmem_ld16x256(s_col + (uint32_t(16 * z) << 16) + uint32_t(8 * k), v[z]);
            ptx::tmem_wait_ld();
            const float2 row = *reinterpret_cast<const float2*>(factors + 8 * k + 2 * i4);
            float2 most = make_float2(-INFINITY, -INFINITY);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const float2 by = factor(row, make_float2(of[z].x, of[z].x)), x = make_float2(of[z].y, of[z].y);
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                const float2 y = ptx::ffma2(make_float2(__uint_as_float(v[z][e]), __uint_as_float(v[z][e + 1])), by, x);
                most = make_float2(fmaxf(most.x, y.x), fmaxf(most.y, y.y));
              }
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              most.x = fmaxf(most.x, __shfl_xor_sync(0xffffffffu, most.x, o));
              most.y = fmaxf(most.y, __shfl_xor_sync(0xffffffffu, most.y, o));
            }
            if (g4 == 0) *reinterpret_cast<float2*>(warps + w4 * N + 8 * k + 2 * i4) = most;
          }
          const int before = T - STRIDE;  // this warpgroup's last tile
          if (j >= STRIDE)
            ok = ok && tree_warp_wait(bar(C::B_PDONE + before % C::NB), uint32_t(before / C::NB) & 1u, abort_flag, 20);
          if (meet(!ok)) {
            left = true;  // all of them
            break;
          }
          ptx::tc_fence_after();
          // A lane per row, every warp for itself with the same result (in little code, as
          // all that runs once a segment: instructions from far away cost more than their work)
          if (lane < N) {
#pragma unroll 1
            for (int x = lane; x < N; x += 32) {
              const float now = fmaxf(fmaxf(warps[x], warps[N + x]), fmaxf(warps[2 * N + x], warps[3 * N + x]));
              const float was = j >= STRIDE ? -move[x].x : kNoReference;
              const bool raise = now > was + (kMostWeight - 1.f);
              move[x] = make_float2(raise ? kTopWeight - now : -was, raise ? half_factor(was, now - kTopWeight) : 1.f);
            }
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const float4 y = *reinterpret_cast<const float4*>(move + 8 * k + 2 * i4);
            const float2 h = make_float2(y.y, y.w);
            m2[k] = make_float2(y.x, y.z);
            l2[k] = ptx::fmul2(ptx::fmul2(l2[k], h), h);
          }
          if (j >= STRIDE) {  // O holds the earlier tiles' products, which have ended
#pragma unroll 1
            for (int k = 0; k < K; ++k) {
              const float4 y = *reinterpret_cast<const float4*>(move + 8 * k + 2 * i4);
              const float2 h = make_float2(y.y * y.y, y.w * y.w);
              uint32_t w[2][4];
#pragma unroll
              for (int z = 0; z < 2; ++z) ptx::tmem_ld16x256(o_col + (uint32_t(16 * z) << 16) + uint32_t(8 * k), w[z]);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int z = 0; z < 2; ++z) {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[z][e] = __float_as_uint(__uint_as_float(w[z][e]) * (e & 1 ? h.y : h.x));
                ptx::tmem_st16x256(o_col + (uint32_t(16 * z) << 16) + uint32_t(8 * k), w[z]);
              }
            }
          }
          __syncwarp();  // the table is read before it changes again
          ptx::tmem_wait_st();
        }
        if (left) break;
        if (__builtin_expect(flags & kFar, 0)) {  // sums that do not go through the weights
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            if (__float_as_int(of[z].w) != kFar) continue;
#pragma unroll
            for (int k = 0; k < K; ++k) {
              uint32_t v[4];
              ptx::tmem_ld16x256(s_col + (uint32_t(16 * z) << 16) + uint32_t(8 * k), v);
              ptx::tmem_wait_ld();
              const float2 by = factor(f2[k], make_float2(of[z].x, of[z].x));
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                float2 y = ptx::ffma2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), by, m2[k]);
                y = make_float2(ptx::ex2(0.5f * y.x), ptx::ex2(0.5f * y.y));
                lt[k] = ptx::ffma2(y, y, lt[k]);
              }
            }
          }
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0 && !dry) ptx::mbar_arrive(bar(C::B_PFULL + f));
#pragma unroll
        for (int k = 0; k < K; ++k) l2[k] = lt[k];
        if (j + STRIDE < g.tiles) ok = scales(T + STRIDE);
      }
      if (dry) {
        dry = false;
        continue;
      }
      // ---- the segment's end: sums over the tokens, O
      const int end = T0 + g.tiles - 1, last = end - ((end ^ wg) & 1);  // this warpgroup's last tile
      if (last >= T0) ok = ok && !left && tree_warp_wait(bar(C::B_PDONE + last % C::NB), uint32_t(last / C::NB) & 1u, abort_flag, 21);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float2 y = l2[k];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          y.x += __shfl_xor_sync(0xffffffffu, y.x, o);
          y.y += __shfl_xor_sync(0xffffffffu, y.y, o);
        }
        if (g4 == 0) *reinterpret_cast<float2*>(warps + w4 * N + 8 * k + 2 * i4) = y;
        if (g4 == 0 && w4 == 0) *reinterpret_cast<float2*>(refs + wg * N + 8 * k + 2 * i4) = m2[k];
      }
      if (meet_all(!ok)) break;
      constexpr int OUT = N / C::GROUPS;  // rows that a warpgroup writes
      const bool whole = g.slot < 0;
      const int tid = w4 * 32 + lane, row = wg * OUT + tid;  // of the tile, for the first OUT threads
      if (tid < OUT) {
        float m = -INFINITY, sum = 0.f, part[2];
        const float* const all = reinterpret_cast<const float*>(sbase + C::OFF_MAX);
        float its[2], half[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float* const w = all + x * 4 * N + row;
          its[x] = (w[0] + w[N]) + (w[2 * N] + w[3 * N]);
          half[x] = -refs[x * N + row];
          m = fmaxf(m, half[x]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          half[x] = half_factor(half[x], m);
          sum += its[x] * half[x] * half[x];
          part[x] = half[x] * half[x];
        }
        const int node = row / p.G, head = g.h * p.G + row - node * p.G, at = g.q0 + node;
        if (row < g.rows) {
          if (whole)
            a.lse[int64_t(head) * a.total_tokens + at] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
          else
            p.part_m[int64_t(g.slot) * N + row] = make_float2(m == kNoReference ? -INFINITY : m, sum);
        }
        const float inv = !whole ? 1.f : sum == 0.f ? 0.f : __fdividef(1.f, sum);
        const uint64_t to = whole ? (uint64_t(at) * a.num_heads + head) * (2 * D) : uint64_t(g.slot * N + row) * (4 * D);  // bytes
        out[row] = make_float4(part[0] * inv, part[1] * inv, __uint_as_float(uint32_t(to)), __uint_as_float(uint32_t(to >> 32)));
      }
      meet(false);  // (a warpgroup reads the rows that it wrote)
      if (lane == 0) ptx::mbar_arrive(bar(C::B_USED + (s & 1)));
      ptx::tc_fence_after();
      const int first = row - tid;
      // (the other warpgroup's O, of which its factor is 0 where it had no tile and there is nothing)
      const uint32_t o_mine = o_seg + uint32_t((T0 & 1) * N);
      const uint32_t o_other = o_seg + uint32_t(((T0 + (g.tiles > 1)) & 1) * N);
      uint8_t* const to = (whole ? static_cast<uint8_t*>(a.o) : reinterpret_cast<uint8_t*>(p.part_o)) + tid * (whole ? 2 : 4);
#pragma unroll 1
      for (int q = first; q < first + OUT; q += 4) {
        uint32_t w[2][4];
        ptx::tmem_ld4(o_mine + q, w[0]);
        ptx::tmem_ld4(o_other + q, w[1]);
        ptx::tmem_wait_ld();
        if (q + 4 == first + OUT) {
          ptx::tc_fence_before();
          warp_arrive(bar(C::B_OFREE + s % C::NO), lane);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 x = out[q + i];
          float y = __uint_as_float(w[0][i]) * (T0 & 1 ? x.y : x.x);
          y = fmaf(__uint_as_float(w[1][i]), g.tiles == 1 ? 0.f : (T0 & 1) ? x.x : x.y, y);
          uint8_t* const at = to + (uint64_t(__float_as_uint(x.w)) << 32 | __float_as_uint(x.z));
          const bool on = q + i < g.rows && w4 * 32 < D;
          if (on && whole) *reinterpret_cast<__nv_bfloat16*>(at) = __float2bfloat16_rn(y);
          if (on && !whole) *reinterpret_cast<float*>(at) = y;
        }
      }
      ++s;
      T0 += g.tiles;
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

constexpr int kJoinWarps = 8;  // per CTA

// Starts while the first kernel ends, and waits for it.  W warps per row of a cut segment; where few sequences
// are cut often, a CTA per row for every eight CTAs of the line (one for each: 16 nodes behind 2049 tokens 18 us, 22).
constexpr int kCutsWide = 8;

template <int D, int N, int W>
__global__ void __launch_bounds__(32 * kJoinWarps) cache_tree_join_kernel(const __grid_constant__ TreeParams p) {
  __shared__ float shared[W > 1 ? W * (D + 2) : 1];
  constexpr int CUTS = W > 1 ? kCutsWide : 1;
  const int w = (threadIdx.x >> 5) % W, lane = threadIdx.x & 31, x0 = blockIdx.x * CUTS;
  const int row = blockIdx.y * (kJoinWarps / W) + (threadIdx.x >> 5) / W;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool here = lane < CUTS && x0 + lane < p.ctas && p.cuts[x0 + lane].parts >= 2 && row < p.cuts[x0 + lane].rows;
#pragma unroll 1
  for (uint32_t left = __ballot_sync(0xffffffffu, here); left; left &= left - 1) {
    const int x = x0 + __ffs(left) - 1;
    const TreeCut cut = p.cuts[x];
    const int node = row / p.G;
    auto at = [&](int j) { return int64_t(2 * (x + j) + (j == 0 ? 1 : 0)) * N + row; };
    join_row<D, W>(p, cut.parts, at, cut.q0 + node, cut.h * p.G + row - node * p.G, w, lane, shared);
    if (W > 1) __syncthreads();
  }
}

// Rows are padded to the least of these; 0: cache_tree_many.cu takes them, 128 or 256 rows of a sequence
// and head at a time (16 sequences of 8192 tokens, 8 heads: 64 rows 71 us here, 128 rows 87 us there; 128 rows
// as N of the products here took 112).
int padded_rows(const CacheView& c, int num_heads, int max_new) {
  const int64_t rows = int64_t(max_new) * (num_heads / c.heads);
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 0;
}
uint64_t partial_rows(int N) { return 2ull * kTreeSms * N; }
uint64_t partial_bytes(int N, int D) { return partial_rows(N) * (uint64_t(D) * 4 + 8); }

template <int D, int N>
attn_status launch_dn(TreeParams& p, cudaStream_t s) {
  using C = TreeCfg<D, N>;
  const CacheView& c = p.a.cache;
  CUtensorMap map, map_v;
  if (!encode_pages<D>(&map, c, c.k_pages, true) || !encode_pages<D>(&map_v, c, c.v_pages, true))
    return record_cuda_error(cudaErrorInvalidValue, "attn_cache_tree_fwd tensor map encoding");
  cudaError_t e = cudaFuncSetAttribute(cache_tree_kernel<D, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return record_cuda_error(e, "attn_cache_tree_fwd configure");
  cache_tree_kernel<D, N><<<unsigned(p.ctas), C::THREADS, C::SMEM, s>>>(map, map_v, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return record_cuda_error(e, "attn_cache_tree_fwd launch");
  // One warp or a CTA joins a row, as in cache_attn.cu.
  const bool wide = int64_t(p.ctas) > 8 * int64_t(c.batch) * c.heads;
  const int per_cta = wide ? 1 : kJoinWarps;
  cudaLaunchConfig_t cfg = {};
  const int cuts = wide ? kCutsWide : 1;
  cfg.gridDim = dim3(unsigned((p.ctas + cuts - 1) / cuts), unsigned(N / per_cta));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, wide ? cache_tree_join_kernel<D, N, kJoinWarps> : cache_tree_join_kernel<D, N, 1>, p);
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_tree_fwd join launch");
}

template <int D>
attn_status launch_d(TreeParams& p, int N, cudaStream_t s) {
  switch (N) {
    case 16: return launch_dn<D, 16>(p, s);
    case 32: return launch_dn<D, 32>(p, s);
    default: return launch_dn<D, 64>(p, s);
  }
}

}  // namespace

uint64_t cache_tree_workspace(const CacheView& c, int total_tokens, int num_heads, int max_new, int max_seqlen) {
  if (total_tokens == 0 || max_new == 0) return 0;
  const int N = padded_rows(c, num_heads, max_new);
  if (N == 0) return cache_tree_many_workspace(c);
  return partial_bytes(N, c.head_dim) + kTreeSms * sizeof(TreeCut);
}

attn_status launch_cache_tree(const CacheQueryArgs& a, const TreeMasks& tree, cudaStream_t s) {
  const int N = padded_rows(a.cache, a.num_heads, a.max_new);
  if (N == 0) return launch_cache_tree_many(a, tree, s);
  TreeParams p;
  p.a = a;
  p.tree = tree;
  p.G = a.num_heads / a.cache.heads;
  p.ctas = kTreeSms;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.part_o = a.workspace;
  p.part_m = reinterpret_cast<float2*>(a.workspace + partial_rows(N) * a.cache.head_dim);
  p.cuts = reinterpret_cast<TreeCut*>(a.workspace + partial_bytes(N, a.cache.head_dim) / 4);
  switch (a.cache.head_dim) {
    case 32: return launch_d<32>(p, N, s);
    case 64: return launch_d<64>(p, N, s);
    default: return launch_d<128>(p, N, s);
  }
}

}  // namespace attnmask
