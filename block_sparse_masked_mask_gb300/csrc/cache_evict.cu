// Eviction: choose the tokens that a sequence keeps, then copy them together.
//
// Choice, one CTA per (sequence, head): the last tokens are kept in any case;
// of the others the `want` largest weights.  Weights become 32-bit keys of the
// same order, and a radix selection fixes the want-th largest key eight bits
// at a time (a histogram per pass over the weights, which stay in L2).  A last
// pass in the order of the tokens writes those above the border key, and of
// those at it the first ones, at the places that a running count gives.
// Copy, one CTA per (page of the destination, head): the page's scale is the
// largest of its tokens' scales; codes of smaller scales are shifted.
#include "cache.cuh"

namespace attnmask {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kGatherThreads = 128;

// Whole numbers in the order of the weights; NaN counts as -inf, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// What a sequence keeps; false where its numbers cannot be used (noted in status).
__device__ __forceinline__ bool load_kept(const EvictArgs& a, int b, int& len, int& keep) {
  len = a.lens[b];
  const int budget = a.budgets[b];
  keep = min(len, budget);
  int err = 0;
  if (len < 0) err |= kErrHeld;
  if (len > a.max_seqlen) err |= kErrSeqTooLong;
  if (budget < 0 || keep > a.max_keep) err |= kErrBudget;
  if (err) atomicOr(a.src.status, err);
  return err == 0;
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int hist[256];
  __shared__ int warp_sum[32];
  __shared__ uint32_t border;
  __shared__ int left;  // keys still wanted among those that match the border so far
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int len, keep;
  if (!load_kept(a, b, len, keep)) return;
  const float* w = a.weights + (int64_t(b) * a.src.heads + h) * a.weight_stride;
  int32_t* kept = a.kept + (int64_t(b) * a.src.heads + h) * a.max_keep;
  float* out = a.new_weights + (int64_t(b) * a.src.heads + h) * a.new_stride;
  if (h == 0 && tid == 0) a.new_lens[b] = keep;
  const int tail = min(a.recent, keep), others = len - tail, want = keep - tail;

  if (tid == 0) {
    border = 0;
    left = want;
  }
  __syncthreads();
  if (want < others && want > 0) {
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t prefix = border;
      for (int j = tid; j < others; j += kSelectThreads) {
        const uint32_t k = order_key(w[j]);
        if (pass == 0 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1);
      }
      __syncthreads();
      if (warp == 0) {
        // digits from 255 down, eight per lane: the one where the count reaches `left`
        int n[8], mine = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) mine += n[i] = hist[255 - (8 * lane + i)];
        int before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += y;
        }
        before -= mine;
        const int need = left;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < need && before + n[i] >= need) {
            border = prefix | uint32_t(255 - (8 * lane + i)) << shift;
            left = need - before;
          }
          before += n[i];
        }
      }
      __syncthreads();
    }
  }
  const bool all = want >= others;
  const uint32_t edge = border;
  const int ties = left;  // of the keys equal to the border, the first `ties`
  __syncthreads();

  // in the order of the tokens: (kept, at the border) counts in one word
  int64_t base = 0;  // low half: kept so far; high half: border keys so far
  for (int j0 = 0; j0 < len; j0 += kSelectThreads) {
    const int j = j0 + tid;
    uint32_t k = 0;
    float x = 0.f;
    bool above = false, at = false;
    if (j < len) {
      x = w[j];
      k = order_key(x);
      above = j >= others || all || (want > 0 && k > edge);
      at = !above && want > 0 && k == edge;
    }
    // border keys before this one
    const uint32_t lower = (1u << lane) - 1u;
    const uint32_t tie_mask = __ballot_sync(0xffffffffu, at);
    if (lane == 0) warp_sum[warp] = __popc(tie_mask);
    __syncthreads();
    int tie_before = 0, tie_all = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int n = warp_sum[i];
      tie_before += i < warp ? n : 0;
      tie_all += n;
    }
    __syncthreads();
    const int tie_rank = int(base >> 32) + tie_before + __popc(tie_mask & lower);
    const bool take = above || (at && tie_rank < ties);
    const uint32_t take_mask = __ballot_sync(0xffffffffu, take);
    if (lane == 0) warp_sum[warp] = __popc(take_mask);
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int n = warp_sum[i];
      before += i < warp ? n : 0;
      total += n;
    }
    __syncthreads();
    if (take) {
      const int place = int(uint32_t(base)) + before + __popc(take_mask & lower);
      kept[place] = j;
      out[place] = x;
    }
    base += (int64_t(tie_all) << 32) + total;
  }
  for (int j = keep + tid; j < a.max_keep; j += kSelectThreads) kept[j] = -1;
  for (int64_t j = keep + tid; j < a.new_stride; j += kSelectThreads) out[j] = 0.f;
}

__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const EvictArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ int src_page[128], src_slot[128];
  __shared__ int exps[2][128];
  __shared__ int top[2];
  const int page_size = 1 << a.src.page_log2, D = a.src.head_dim;
  const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  int len, keep;
  if (!load_kept(a, b, len, keep)) return;
  const int n = min(page_size, keep - (i << a.src.page_log2));  // tokens of this page
  if (n <= 0) return;
  const int dst = load_page(a.dst, b, i);
  if (dst < 0) {
    if (tid == 0) atomicOr(a.src.status, kErrBadPage);
    return;
  }
  if (tid < 2) top[tid] = -1000;
  __syncthreads();
  if (tid < n) {
    const int j = a.kept[(int64_t(b) * a.src.heads + h) * a.max_keep + (i << a.src.page_log2) + tid];
    const int page = load_page(a.src, b, j >> a.src.page_log2);
    src_page[tid] = page;
    src_slot[tid] = j & (page_size - 1);
    if (page >= 0) {
      const int64_t at = int64_t(page) * a.src.heads + h;
      exps[0][tid] = exponent_of(a.src.k_scale[at]);
      exps[1][tid] = exponent_of(a.src.v_scale[at]);
      atomicMax(&top[0], exps[0][tid]);
      atomicMax(&top[1], exps[1][tid]);
    }
  }
  __syncthreads();
  const int pieces = D / 16;  // 16-byte pieces per token
  for (int x = tid; x < 2 * n * pieces; x += kGatherThreads) {
    const int side = x >= n * pieces, y = x - side * n * pieces;
    const int slot = y / pieces, piece = y % pieces;
    const int page = src_page[slot];
    if (page < 0) continue;
    const uint8_t* from = (side ? a.src.v_pages : a.src.k_pages) +
                          (((int64_t(page) * a.src.heads + h) << a.src.page_log2) + src_slot[slot]) * D + piece * 16;
    uint8_t* to = (side ? a.dst.v_pages : a.dst.k_pages) +
                  (((int64_t(dst) * a.dst.heads + h) << a.dst.page_log2) + slot) * D + piece * 16;
    uint4 v = *reinterpret_cast<const uint4*>(from);
    const int shift = top[side] - exps[side][slot];
    if (shift > 0) {
      v.x = rescale4(v.x, shift);
      v.y = rescale4(v.y, shift);
      v.z = rescale4(v.z, shift);
      v.w = rescale4(v.w, shift);
    }
    *reinterpret_cast<uint4*>(to) = v;
  }
  if (tid < 2 && top[tid] > -1000)
    (tid ? a.dst.v_scale : a.dst.k_scale)[int64_t(dst) * a.dst.heads + h] = pow2f(max(-126, top[tid]));
}

}  // namespace

attn_status launch_cache_evict(const EvictArgs& a, cudaStream_t s) {
  evict_select_kernel<<<dim3(unsigned(a.src.heads), unsigned(a.src.batch)), kSelectThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return record_cuda_error(e, "attn_cache_evict select launch");
  if (a.max_keep == 0) return ATTN_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((a.max_keep + (1 << a.src.page_log2) - 1) >> a.src.page_log2), unsigned(a.src.heads),
                     unsigned(a.src.batch));
  cfg.blockDim = dim3(kGatherThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_gather_kernel, a);
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_evict copy launch");
}

}  // namespace attnmask
