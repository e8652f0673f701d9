// What the two kernels of attention over drafted trees (cache_tree.cu, cache_tree_many.cu) share.
#pragma once

#include "cache_tiles.cuh"

namespace attnmask {
namespace {

constexpr int kNoPage = INT_MIN, kFar = 1;  // of a block of 16 tokens, as in cache_chunk.cu
constexpr int kTreeSms = 152;

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
};

}  // namespace
}  // namespace attnmask
