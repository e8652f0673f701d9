// Trees of drafted tokens: their ancestor masks and positions, and the accepted
// path moved together in the cache.
//
// Masks.  A thread takes a node and walks up to its root; the words of its row are collected
// in shared memory, eight at a time from the last down, since a parent's number is below
// the node's own, and a CTA's rows are written together.  Every CTA checks the parents of the
// whole sequence first, so every walk ends.  What bounds it is the walk, one load behind the
// other, and with few nodes the launch: 512 trees of 128 to 256 nodes 3.8 us.  (A warp per node, a lane per
// word, had the walks of a warp's nodes one behind the other: 15.8 us.)
//
// Path.  A warp owns one (sequence, head) of the keys or of the values and takes the
// tokens in their order: the node of a path's j-th token is at least j, so what a slot
// receives lies in it or behind it and has not been written yet, whatever number of slots
// is loaded at once, as long as their stores come behind.  No thread waits for another warp;
// the lookups of a page (path, table) are all that stands before its loads, and the scales
// arrive with the tokens.  Tokens go through shared memory by copies that need no registers, in loops of
// little code.  256 sequences of 16 heads of 128, 16 to 64 of their 128 to 256 nodes kept, take 21 us where
// the bytes take 12.5: rows of 128 bytes, scattered.  (A CTA per head and side, a barrier between a page's loads and
// stores: 39 us.)
#include "cache_rows.cuh"

namespace attnmask {
namespace {

constexpr int kBuildThreads = 128;  // a node each
constexpr int kBuildWords = 8;      // of a row at a time

__global__ void __launch_bounds__(kBuildThreads) tree_build_kernel(const TreeBuildArgs a) {
  __shared__ uint32_t rows[kBuildThreads][kBuildWords + 1];
  const int b = blockIdx.y, tid = threadIdx.x;
  const CacheView& c = a.cache;
  SeqRows r;
  const bool note = blockIdx.x == 0 && tid == 0;
  if (!load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, c.max_pages << c.page_log2, c.status, r, note)) return;
  const int first = blockIdx.x * kBuildThreads, nodes = min(r.n - first, kBuildThreads);
  if (nodes <= 0) return;
  const int32_t* parents = a.parents + r.q0;
  bool bad = r.len < r.n;
#pragma unroll 4
  for (int i = tid; i < r.n; i += kBuildThreads) {
    const int p = __ldg(parents + i);
    bad |= p < -1 || p >= i;
  }
  if (__syncthreads_or(bad)) {
    if (note) atomicOr(c.status, r.len < r.n ? kErrHeld : kErrTree);
    return;
  }
  int p = tid < nodes ? first + tid : -1, depth = -1;
  uint32_t* const bits = a.bits + int64_t(r.q0 + first) * a.words;
  for (int w0 = (a.words - 1) / kBuildWords * kBuildWords; w0 >= 0; w0 -= kBuildWords) {
    const int width = min(kBuildWords, a.words - w0);
#pragma unroll
    for (int w = 0; w < kBuildWords; ++w) rows[tid][w] = 0;
    while (p >= w0 * 32) {
      rows[tid][(p >> 5) - w0] |= 1u << (p & 31);
      p = __ldg(parents + p);
      ++depth;
    }
    __syncthreads();
    for (int x = tid; x < nodes * kBuildWords; x += kBuildThreads) {
      const int row = x / kBuildWords, w = x % kBuildWords;
      if (w < width) bits[int64_t(row) * a.words + w0 + w] = rows[row][w];
    }
    __syncthreads();
  }
  if (tid < nodes && a.positions) a.positions[r.q0 + first + tid] = r.len - r.n + depth;
}

constexpr int kKeepWarps = 4, kKeepThreads = 32 * kKeepWarps;

__global__ void __launch_bounds__(kKeepThreads) tree_keep_kernel(const TreeKeepArgs a) {
  __shared__ __align__(16) uint4 staged[kKeepWarps][32 * 128 / 16];  // 32 rows
  const CacheView& c = a.cache;
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int log2 = c.page_log2, page_size = 1 << log2, D = c.head_dim;
  const int row_log2 = 31 - __clz(D / 16);  // pieces of 16 bytes of a row
  const bool note = blockIdx.x == 0 && tid == 0;
  SeqRows r;
  const int m = __ldg(a.counts + b);
  if (!load_rows(a.cu, a.lens, b, INT_MAX, a.max_new, c.max_pages << c.page_log2, c.status, r, note)) return;
  const int base = r.len - r.n;
  const int32_t* path = a.path + int64_t(b) * a.path_stride;
  bool bad = base < 0 || m < 0 || m > r.n || m > a.path_stride;
  if (!bad) {
#pragma unroll 1
    for (int j = tid; j < m; j += kKeepThreads) {
      const int p = __ldg(path + j);
      bad |= p < 0 || p >= r.n || (j > 0 && __ldg(path + j - 1) >= p);
    }
  }
  if (__syncthreads_or(bad)) {
    if (note) atomicOr(c.status, base < 0 ? kErrHeld : kErrTree);
    return;
  }
  if (note) a.new_lens[b] = base + m;
  const int head = blockIdx.x * kKeepWarps + warp, h = head >> 1, values = head & 1;
  if (h >= c.heads) return;
  uint4* const pages = reinterpret_cast<uint4*>(values ? c.v_pages : c.k_pages);
  float* const scales = values ? c.v_scale : c.k_scale;
  const int32_t* table = c.table + int64_t(b) * c.max_pages;
  uint4* const stage = staged[warp];
  const uint32_t stage_at = ptx::smem_addr(stage);
  const int mask = (1 << row_log2) - 1;
  auto number_of = [&](int i) { return i << log2 < base + m ? __ldg(table + i) : 0; };
  int next = number_of(base >> log2);
#pragma unroll 1
  for (int i = base >> log2; i << log2 < base + m; ++i) {
    const int number = next;
    next = number_of(i + 1);
    if (!in_pool(c, number)) {
      if (lane == 0) atomicOr(c.status, kErrBadPage);
      continue;
    }
    const int64_t at = int64_t(number) * c.heads + h;
    const int t0 = i << log2;                     // its first token
    const int j0 = max(t0 - base, 0), j1 = min(t0 + page_size - base, m);  // of the path, its new tokens
    const float own_scale = scales[at];
    // The row that token j comes from, or -1 if it stays where it is or has no page; its scale (which is looked
    // at only once the tokens are on their way).
    float scale;
    auto source = [&](int j) -> int64_t {
      scale = own_scale;
      if (j >= j1) return -1;
      const int src = base + __ldg(path + j);
      if (src == base + j) return -1;
      const int from = __ldg(table + (src >> log2));
      if (!in_pool(c, from)) {
        atomicOr(c.status, kErrBadPage);
        return -1;
      }
      const int64_t row = int64_t(from) * c.heads + h;
      scale = scales[row];
      return (row << log2) + (src & (page_size - 1));
    };
    auto fetch = [&](int j, int64_t row) {
      const int n = min(32, j1 - j) << row_log2;
#pragma unroll 1
      for (int x = lane; x < ((n + 31) & ~31); x += 32) {
        const int64_t from = __shfl_sync(0xffffffffu, row, x >> row_log2);
        copy16_async(stage_at + x * 16, pages + ((from < 0 ? 0 : from) << row_log2) + (x & mask), from >= 0);
      }
    };
    int64_t row = source(j0 + lane);
    fetch(j0, row);
    const int own = exponent_of(own_scale), e0 = exponent_of(scale);
    int to = max(own, e0), e = e0;
#pragma unroll 1
    for (int j = j0 + 32; j < j1; j += 32) {
      source(j + lane);
      to = max(to, exponent_of(scale));
    }
    to = __reduce_max_sync(0xffffffffu, to);
#pragma unroll 1
    for (int j = j0; j < j1; j += 32) {
      if (j > j0) {
        row = source(j + lane);
        fetch(j, row);
        e = exponent_of(scale);
      }
      asm volatile("cp.async.commit_group;\n\tcp.async.wait_all;" ::: "memory");
      __syncwarp();
      const int n = min(32, j1 - j) << row_log2;
      uint4* const out = pages + (((at << log2) + base + j - t0) << row_log2);
#pragma unroll 1
      for (int x = lane; x < ((n + 31) & ~31); x += 32) {
        const int down = __shfl_sync(0xffffffffu, row < 0 ? -1 : to - e, x >> row_log2);
        if (down < 0) continue;
        uint4 w = stage[x];
        if (down > 0) {
          w.x = rescale4(w.x, down);
          w.y = rescale4(w.y, down);
          w.z = rescale4(w.z, down);
          w.w = rescale4(w.w, down);
        }
        out[x] = w;
      }
      __syncwarp();
    }
    if (__builtin_expect(to > own, 0)) {
      // the page's other tokens take the new scale
      uint4* const all = pages + (at << log2 << row_log2);
      const int n = min(page_size, r.len - t0) << row_log2;
#pragma unroll 1
      for (int x = lane; x < n; x += 32) {
        const int j = (x >> row_log2) + t0 - base;
        if (j >= 0 && j < m && __ldg(path + j) != j) continue;
        uint4 w = all[x];
        w.x = rescale4(w.x, to - own);
        w.y = rescale4(w.y, to - own);
        w.z = rescale4(w.z, to - own);
        w.w = rescale4(w.w, to - own);
        all[x] = w;
      }
      if (lane == 0) scales[at] = pow2f(to);
    }
    __syncwarp();  // before the reads of what was written here
  }
}

}  // namespace

attn_status launch_tree_build(const TreeBuildArgs& a, cudaStream_t s) {
  const dim3 grid(unsigned((a.max_new + kBuildThreads - 1) / kBuildThreads), unsigned(a.cache.batch));
  tree_build_kernel<<<grid, kBuildThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_tree_build launch");
}

attn_status launch_tree_keep(const TreeKeepArgs& a, cudaStream_t s) {
  const dim3 grid(unsigned((2 * a.cache.heads + kKeepWarps - 1) / kKeepWarps), unsigned(a.cache.batch));
  tree_keep_kernel<<<grid, kKeepThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_tree_keep launch");
}

}  // namespace attnmask
