// Trees of drafted tokens: their ancestor masks and positions, and the accepted
// path moved together in the cache.
//
// Masks.  A warp takes a node and walks up to its root; lane w collects word w of
// the node's row.  A parent's number is below the node's own, which every
// CTA checks for the whole sequence first, so every walk ends.
//
// Path.  A CTA owns one (sequence, head) of the keys or of the values and takes the
// pages that receive tokens in their order: the node of a path's j-th token is at
// least j, so what a page receives lies in it or behind it and has not been written
// yet.  All of a page's loads are in flight at once, and a barrier
// stands between them and the page's stores.
#include "cache_rows.cuh"

namespace attnmask {
namespace {

constexpr int kBuildThreads = 256, kBuildWarps = kBuildThreads / 32;
constexpr int kBuildNodes = 64;  // of one CTA

__global__ void __launch_bounds__(kBuildThreads) tree_build_kernel(const TreeBuildArgs a) {
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheView& c = a.cache;
  SeqRows r;
  const bool note = blockIdx.x == 0 && threadIdx.x == 0;
  if (!load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, c.max_pages << c.page_log2, c.status, r, note)) return;
  const int first = blockIdx.x * kBuildNodes, last = min(r.n, first + kBuildNodes);
  if (first >= r.n) return;
  const int32_t* parents = a.parents + r.q0;
  bool bad = r.len < r.n;
  for (int i = threadIdx.x; i < r.n; i += kBuildThreads) {
    const int p = __ldg(parents + i);
    bad |= p < -1 || p >= i;
  }
  if (__syncthreads_or(bad)) {
    if (note) atomicOr(c.status, r.len < r.n ? kErrHeld : kErrTree);
    return;
  }
  for (int i = first + warp; i < last; i += kBuildWarps) {
    for (int w0 = 0; w0 < a.words; w0 += 32) {
      uint32_t word = 0;
      int depth = -1;
      for (int p = i; p >= 0; p = __ldg(parents + p)) {
        if ((p >> 5) - w0 == lane) word |= 1u << (p & 31);
        ++depth;
      }
      if (w0 + lane < a.words) a.bits[int64_t(r.q0 + i) * a.words + w0 + lane] = word;
      if (w0 == 0 && lane == 0 && a.positions) a.positions[r.q0 + i] = r.len - r.n + depth;
    }
  }
}

constexpr int kKeepThreads = 128;

// N: 16-byte pieces per thread of a page.
template <int N>
__global__ void __launch_bounds__(kKeepThreads) tree_keep_kernel(const TreeKeepArgs a) {
  __shared__ int src_page[128], src_slot[128], shift[128];
  __shared__ int top;
  const CacheView& c = a.cache;
  const int h = blockIdx.x >> 1, values = blockIdx.x & 1, b = blockIdx.y, tid = threadIdx.x;
  const int log2 = c.page_log2, page_size = 1 << log2, D = c.head_dim, per_row = D / 16;
  const bool note = blockIdx.x == 0 && tid == 0;
  SeqRows r;
  if (!load_rows(a.cu, a.lens, b, INT_MAX, a.max_new, c.max_pages << c.page_log2, c.status, r, note)) return;
  const int m = a.counts[b], base = r.len - r.n;
  const int32_t* path = a.path + int64_t(b) * a.path_stride;
  bool bad = base < 0 || m < 0 || m > r.n || m > a.path_stride;
  if (!bad)
    for (int j = tid; j < m; j += kKeepThreads) {
      const int p = __ldg(path + j);
      bad |= p < 0 || p >= r.n || (j > 0 && __ldg(path + j - 1) >= p);
    }
  if (__syncthreads_or(bad)) {
    if (note) atomicOr(c.status, base < 0 ? kErrHeld : kErrTree);
    return;
  }
  if (note) a.new_lens[b] = base + m;
  uint8_t* pages = values ? c.v_pages : c.k_pages;
  float* scales = values ? c.v_scale : c.k_scale;
  const int32_t* table = c.table + int64_t(b) * c.max_pages;
  for (int i = base >> log2; i << log2 < base + m; ++i) {
    const int number = __ldg(table + i);
    const bool fine = in_pool(c, number);
    const int t0 = i << log2, live = min(page_size, r.len - t0);  // its slots that hold tokens
    const int64_t at = int64_t(fine ? number : 0) * c.heads + h;
    const int own = fine ? exponent_of(scales[at]) : 0;
    if (tid == 0) top = own;
    __syncthreads();
    int e = own;
    if (tid < live) {
      // slot tid receives a token, or keeps its own
      const int j = t0 + tid - base;
      const bool moves = j >= 0 && j < m;
      const int src = moves ? base + __ldg(path + j) : t0 + tid;
      const int from = moves ? __ldg(table + (src >> log2)) : number;
      const bool good = fine && in_pool(c, from);
      if (!good) atomicOr(c.status, kErrBadPage);
      src_page[tid] = good ? from : -1;
      src_slot[tid] = src & (page_size - 1);
      if (good && from != number) {
        e = exponent_of(scales[int64_t(from) * c.heads + h]);
        atomicMax(&top, e);
      }
    }
    __syncthreads();
    const int to = top;
    if (tid < live) {
      shift[tid] = to - e;
      if (src_page[tid] == number && src_slot[tid] == tid && to == e) src_page[tid] = -1;  // stays as it is
    }
    __syncthreads();
    uint4 w[N];
#pragma unroll
    for (int y = 0; y < N; ++y) {
      const int x = y * kKeepThreads + tid, slot = x / per_row, piece = x % per_row;
      if (slot < live && src_page[slot] >= 0)
        w[y] = *reinterpret_cast<const uint4*>(
            pages + (((int64_t(src_page[slot]) * c.heads + h) << log2) + src_slot[slot]) * D + piece * 16);
    }
    __syncthreads();
#pragma unroll
    for (int y = 0; y < N; ++y) {
      const int x = y * kKeepThreads + tid, slot = x / per_row, piece = x % per_row;
      if (slot >= live || src_page[slot] < 0) continue;
      if (shift[slot] > 0) {
        w[y].x = rescale4(w[y].x, shift[slot]);
        w[y].y = rescale4(w[y].y, shift[slot]);
        w[y].z = rescale4(w[y].z, shift[slot]);
        w[y].w = rescale4(w[y].w, shift[slot]);
      }
      *reinterpret_cast<uint4*>(pages + ((at << log2) + slot) * D + piece * 16) = w[y];
    }
    if (tid == 0 && fine && to > own) scales[at] = pow2f(to);
    __syncthreads();  // before the next page's numbers, and its reads of what was written here
  }
}

}  // namespace

attn_status launch_tree_build(const TreeBuildArgs& a, cudaStream_t s) {
  const dim3 grid(unsigned((a.max_new + kBuildNodes - 1) / kBuildNodes), unsigned(a.cache.batch));
  tree_build_kernel<<<grid, kBuildThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_tree_build launch");
}

attn_status launch_tree_keep(const TreeKeepArgs& a, cudaStream_t s) {
  const dim3 grid(unsigned(2 * a.cache.heads), unsigned(a.cache.batch));
  switch ((a.cache.head_dim << a.cache.page_log2) / 16 / kKeepThreads) {
    case 8: tree_keep_kernel<8><<<grid, kKeepThreads, 0, s>>>(a); break;
    case 4: tree_keep_kernel<4><<<grid, kKeepThreads, 0, s>>>(a); break;
    case 2: tree_keep_kernel<2><<<grid, kKeepThreads, 0, s>>>(a); break;
    default: tree_keep_kernel<1><<<grid, kKeepThreads, 0, s>>>(a); break;
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_tree_keep launch");
}

}  // namespace attnmask
