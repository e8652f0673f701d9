// What the two kernels of attention over drafted trees (cache_tree.cu, cache_tree_many.cu) share.
#pragma once

#include "cache_tiles.cuh"

namespace attnmask {
namespace {

constexpr int kNoPage = INT_MIN, kFar = 1;  // of a block of 16 tokens, as in cache_chunk.cu
constexpr int kTreeSms = 152;
constexpr float kNoReference = -0x1.8p127f;  // of a row that has seen nothing yet: any score moves it

// A constant that the compiler does not see: it would else copy a loop's body for its first turn.
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  asm volatile("" : "+r"(x));
  return x;
}

// The bounded waits of tile_pipeline.cuh in the few instructions that five roles at once
// leave room for: with 100 KB of code in all, warps waited for instructions more than for
// anything else.  What runs out is left in *abort_flag, the site plus 1, and
// becomes the status at the kernel's end.
__device__ __forceinline__ bool tree_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, int site) {
  bool ok = ptx::mbar_try_wait(bar, parity);
  if (__builtin_expect(!ok, 0)) {
    const uint32_t t0 = ptx::globaltimer_lo();
    while (true) {
      ok = ptx::mbar_try_wait(bar, parity);
      if (ok || *abort_flag) break;
      if (ptx::globaltimer_lo() - t0 > uint32_t(kWaitTimeoutNs)) {
        *abort_flag = uint32_t(site) + 1u;
        break;
      }
    }
  }
  return ok;
}
static_assert(kWaitTimeoutNs < (1ull << 32), "of a 32-bit clock");
__device__ __forceinline__ bool tree_warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, int site) {
  return __all_sync(0xffffffffu, tree_wait(bar, parity, abort_flag, site));
}

struct TreeParams {
  CacheQueryArgs a;
  TreeMasks tree;
  int G;
  int ctas;
  float scale_log2;
  float* part_o;    // [2 * ctas][rows of a segment] of head_dim, as for few rows in cache_attn.cu
  float2* part_m;
  struct TreeCut* cuts;  // [ctas]
};

// What the line of a CTA leaves for the second kernel: the segment that begins in its piece and ends in
// a later one's.
struct alignas(16) TreeCut {
  int parts;  // CTAs that hold a part of it, this one the first; 0: there is no such segment
  int h, row0, rows, q0, unused[3];
};

// The line of work: tiles of tokens of all (sequence, head, ROWS rows)s, one behind the other, in units
// of cost: FULL for a tile with all rows, HALF with up to half of them, ITEM for what begins and ends a segment.
// It is cut evenly among the CTAs.  The numbers are the device's alone.
template <int ROWS, int FULL, int HALF, int ITEM, int LEAST>
struct TreeLine {
  // One sequence's part of it.
  struct Seq {
    int U, row_tiles, last;  // tiles of tokens, of rows; the cost of the last one's tiles

    __device__ __forceinline__ Seq(int n, int G, int len) {
      const int64_t rows = int64_t(n) * G;
      U = (len + kTile - 1) / kTile;
      row_tiles = int((rows + ROWS - 1) / ROWS);
      last = rows - int64_t(row_tiles - 1) * ROWS <= ROWS / 2 ? HALF : FULL;
    }
    // of one tile of rows but the last, and of one head
    __device__ __forceinline__ int64_t item() const { return int64_t(U) * FULL + ITEM; }
    __device__ __forceinline__ int64_t head() const { return (row_tiles - 1) * item() + int64_t(U) * last + ITEM; }
    __device__ __forceinline__ int cost(int rt) const { return rt == row_tiles - 1 ? last : FULL; }
  };

  // One (head, tile of rows) of a sequence: where its first tile of tokens begins.
  struct Item {
    int h, rt, w;   // w: cost of a tile
    int64_t first, end;

    __device__ __forceinline__ Item(const Seq& l, int64_t before, int64_t pos) {
      h = int((pos - before) / l.head());
      int64_t start = before + h * l.head();
      rt = int(min((pos - start) / l.item(), int64_t(l.row_tiles - 1)));
      start += rt * l.item();
      w = l.cost(rt);
      first = start + ITEM;
      end = first + int64_t(l.U) * w;
    }
    // The tiles that begin before `pos`.
    __device__ __forceinline__ int tiles(int64_t pos, int U) const {
      return pos <= first ? 0 : int(min(int64_t(U), (pos - first + w - 1) / w));
    }
  };

  // Sequence b's, all heads; 0 where its numbers cannot be used.
  __device__ static __forceinline__ int64_t of(const TreeParams& p, int b) {
    const CacheQueryArgs& a = p.a;
    if (b >= a.cache.batch) return 0;
    const int q0 = a.cu[b], q1 = a.cu[b + 1], len = a.lens[b], n = q1 - q0;
    const bool good = q0 >= 0 && q1 > q0 && q1 <= a.total_tokens && (b > 0 || q0 == 0) && n <= a.max_new && len >= n &&
                      len <= a.max_seqlen;
    return good ? Seq(n, p.G, len).head() * a.cache.heads : 0;
  }
  // Its length, by whole warps, and a CTA's piece of it: LEAST or more, so that at least a tile begins in each
  // piece of an item that goes on behind it.
  static_assert(LEAST >= FULL && FULL >= HALF, "a tile begins in every piece of an item");
  __device__ static __forceinline__ int64_t total(const TreeParams& p, int lane) {
    int64_t sum = 0;
#pragma unroll 1
    for (int b = lane; b < p.a.cache.batch; b += 32) sum += of(p, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
  }
  __device__ static __forceinline__ int64_t share(int64_t total, const TreeParams& p) {
    return max(int64_t(LEAST), (total + p.ctas - 1) / p.ctas);
  }
  // The sequence that `pos` (below the total) belongs to, and the line before it.
  __device__ static __forceinline__ int find(const TreeParams& p, int64_t pos, int lane, int64_t& before) {
    before = 0;
#pragma unroll 1
    for (int b = 0;; b += 32) {
      const int64_t n = of(p, b + lane);
      int64_t sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, before + sum > pos);
      if (past || b + 32 >= p.a.cache.batch) {
        const int at = past ? __ffs(past) - 1 : 31;
        before += __shfl_sync(0xffffffffu, sum - n, at);
        return b + at;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
};

}  // namespace
}  // namespace attnmask
