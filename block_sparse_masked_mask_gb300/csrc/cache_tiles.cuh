// What the tcgen05 kernels over the cache (attention and weights of many rows)
// share: tiles of 128 tokens' codes as TMA brings them, the queries as two e4m3
// numbers, and bounded waits in few instructions.
#pragma once

#include "cache_rows.cuh"
#include "tile_pipeline.cuh"

namespace attnmask {
namespace {

// The bounded waits of tile_pipeline.cuh behind one inlined try: five roles run
// at once, and their loops are fastest when they are short (the instruction
// caches; with the whole wait inlined everywhere 4 prompts of 300 to 512 tokens
// took 378 us, so 358).
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

// 128 rows of D bytes, swizzled over their own width (K-major operands).
template <int D>
struct CodeTile {
  static constexpr int BYTES = kTile * D;
  static constexpr uint32_t SW = D == 128 ? ptx::kSwizzle128B : D == 64 ? ptx::kSwizzle64B : ptx::kSwizzle32B;
  __device__ static uint32_t unit(int row, int u) {  // byte offset of 16-byte unit u of a row
    const int x = D == 128 ? (row & 7) : D == 64 ? ((row >> 1) & 3) : ((row >> 2) & 1);
    return uint32_t(row * D + ((u ^ x) << 4));
  }
};

// A bf16 query as the sum of two e4m3 numbers.  Scaled by a power of two to a
// largest magnitude in [128, 256), its 8 significant bits are hi + lo exactly down
// to 2^-9 of that magnitude, and within 2^-17 of it below.  Writes `row` of the
// tile of hi at `tiles` and of the tile of lo behind it (zeros if not `real`);
// returns the scale's inverse, NaN for an infinite query, which has no scores.
template <int D>
__device__ __forceinline__ float split_query(const __nv_bfloat16* query, bool real, uint8_t* tiles, int row) {
  uint4 q[D / 8];
  float amax = 0.f;
  const uint4* src = reinterpret_cast<const uint4*>(query);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    q[i] = real ? src[i] : make_uint4(0, 0, 0, 0);
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
    const uint32_t at = CodeTile<D>::unit(row, i);
    *reinterpret_cast<uint4*>(tiles + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(tiles + CodeTile<D>::BYTES + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  return amax < INFINITY ? pow2f(e - 7) : __int_as_float(0x7FC00000);
}

// Pages as rows of D bytes, (dimension, slot, head, page), one page and head per copy.
template <int D>
bool encode_pages(CUtensorMap* map, const CacheView& c, void* pages, bool swizzled) {
  auto fn = encode_fn();
  const int page_size = 1 << c.page_log2;
  const cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(page_size), cuuint64_t(c.heads), cuuint64_t(c.num_pages)};
  const cuuint64_t strides[3] = {cuuint64_t(D), cuuint64_t(D) * page_size, cuuint64_t(D) * page_size * c.heads};
  const cuuint32_t box[4] = {cuuint32_t(D), cuuint32_t(page_size), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapSwizzle sw = !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE
                                : D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                : D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, pages, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace attnmask
