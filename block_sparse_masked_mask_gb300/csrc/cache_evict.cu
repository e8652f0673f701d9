// Eviction: choose the tokens that a sequence keeps, then copy them together.
//
// Choice, one CTA per (sequence, head): the last tokens are kept in any case;
// of the others the `want` largest weights.  Weights become 32-bit keys of the
// same order, held in shared memory (as many as fit, else read again), and a radix
// selection fixes the want-th largest key in digits of 11, 11 and 10 bits: the
// first digit is the exponent and two bits more, so that weights of one size
// still spread over a few counters.  Each warp then takes a run of consecutive
// tokens, counts what it keeps (above the border key, and of those at it the first
// ones) and, knowing the counts of the warps before it, writes it in order.
// Copy, a CTA per page of the destination and head, 16 bytes per lane and all of
// a page's loads in flight at once: the page's scale is the largest of its
// tokens' scales; codes of smaller scales are shifted.
#include "cache_rows.cuh"

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

constexpr int kBins = 2048;
constexpr int kStageMost = 48 * 1024;  // keys in shared memory

// Sum of `x` over the threads before this one (1024 threads), and over all.
// `sums` holds 32 words; the caller puts a barrier between two uses of it.
__device__ __forceinline__ int sum_before(int x, int* sums, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int up = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += y;
  }
  if (lane == 31) sums[warp] = up;
  __syncthreads();
  const int s = sums[lane];
  int w = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  all = __shfl_sync(0xffffffffu, w, 31);
  return __shfl_sync(0xffffffffu, w - s, warp) + up - x;
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictArgs a, int stage) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint32_t keys[];  // of the first `stage` tokens
  __shared__ int hist[kBins];
  __shared__ int sums[32];
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
  const bool all = want >= others;
  auto key_of = [&](int j) { return j < stage ? keys[j] : order_key(w[j]); };

  if (!all && want > 0) {
#pragma unroll 8
    for (int j = tid; j < min(others, stage); j += kSelectThreads) keys[j] = order_key(__ldg(w + j));
    uint32_t prefix = 0;
    int need = want;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
      for (int j = tid; j < others; j += kSelectThreads) {
        const uint32_t k = key_of(j);
        if (pass == 0 || (k >> (shift + bits)) == (prefix >> (shift + bits)))
          atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
      }
      __syncthreads();
      // digits from the highest down, two per thread: the one where the count reaches `need`
      const int n0 = hist[kBins - 1 - 2 * tid], n1 = hist[kBins - 2 - 2 * tid];
      int total;
      const int before = sum_before(n0 + n1, sums, total);
      if (before < need && before + n0 >= need) {
        border = prefix | uint32_t(kBins - 1 - 2 * tid) << shift;
        left = need - before;
      } else if (before + n0 < need && before + n0 + n1 >= need) {
        border = prefix | uint32_t(kBins - 2 - 2 * tid) << shift;
        left = need - before - n0;
      }
      __syncthreads();
      prefix = border;
      need = left;
    }
  }
  const uint32_t edge = all || want == 0 ? 0u : border;
  const int ties = all || want == 0 ? 0 : left;  // of the keys equal to the border, the first `ties`

  // warp w: a run of consecutive tokens, 32 at a time
  const int run = ((len + kSelectThreads - 1) / kSelectThreads) * 32;
  const int j0 = warp * run, j1 = min(len, j0 + run);
  auto classify = [&](int j, uint32_t& above, uint32_t& at) {
    bool up = false, tie = false;
    if (j < j1) {
      if (all || j >= others) {
        up = true;
      } else if (want > 0) {
        const uint32_t k = key_of(j);
        up = k > edge;
        tie = k == edge;
      }
    }
    above = __ballot_sync(0xffffffffu, up);
    at = __ballot_sync(0xffffffffu, tie);
  };
  int n_above = 0, n_tie = 0;
  for (int j = j0; j < j1; j += 32) {
    uint32_t above, at;
    classify(j + lane, above, at);
    n_above += __popc(above);
    n_tie += __popc(at);
  }
  int unused;
  __syncthreads();
  int tie = sum_before(lane == 0 ? n_tie : 0, sums, unused);  // border keys before this warp's
  tie = __shfl_sync(0xffffffffu, tie, 0);
  const int taken = max(0, min(n_tie, ties - tie));           // of this warp's, the first `taken`
  __syncthreads();
  int place = sum_before(lane == 0 ? n_above + taken : 0, sums, unused);
  place = __shfl_sync(0xffffffffu, place, 0);
  const uint32_t lower = (1u << lane) - 1u;
  for (int j8 = j0; j8 < j1; j8 += 256) {
    float x[8];  // weights, read together
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = j8 + 32 * u + lane < j1 ? __ldg(w + j8 + 32 * u + lane) : 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = j8 + 32 * u + lane;
      uint32_t above, at;
      classify(j, above, at);
      const bool first = (at >> lane & 1u) && tie + __popc(at & lower) < ties;
      const uint32_t take = above | __ballot_sync(0xffffffffu, first);
      if (take >> lane & 1u) {
        const int to = place + __popc(take & lower);
        kept[to] = j;
        out[to] = x[u];
      }
      place += __popc(take);
      tie += __popc(at);
    }
  }
  for (int j = keep + tid; j < a.max_keep; j += kSelectThreads) kept[j] = -1;
  for (int64_t j = keep + tid; j < a.new_stride; j += kSelectThreads) out[j] = 0.f;
}

// Pages of the destination that a sequence fills.
struct KeptPages {
  const EvictArgs& a;
  __device__ int operator()(int b) const {
    const int len = a.lens[b], budget = a.budgets[b], keep = min(len, budget);
    if (len < 0 || len > a.max_seqlen || budget < 0 || keep > a.max_keep) return 0;
    return (keep + (1 << a.src.page_log2) - 1) >> a.src.page_log2;
  }
};

// N: 16-byte pieces per thread of a page's keys (and as many of its values).
// A CTA takes destination pages in turn (one, up to 64 pages and heads per SM); the kept
// tokens' numbers are read two pages ahead and the source pages' one, so that a page waits
// for its own codes only.
template <int N>
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const EvictArgs a) {
  __shared__ uint4 moved[2 * N * kGatherThreads];  // each thread's own pieces
  __shared__ int src_page[2][128], src_slot[2][128];
  __shared__ int exps[2][2][128];
  __shared__ int top[2][2];
  const uint32_t codes = uint32_t(__cvta_generic_to_shared(moved + threadIdx.x));
  const int log2 = a.src.page_log2, page_size = 1 << log2, D = a.src.head_dim, per_row = D / 16;
  const int h = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const KeptPages pages{a};
  const UnitLine line(pages, a.src.batch, lane);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // The page at a place of the line: its sequence, number, tokens (0: none), and the
  // token that this thread looks up (-1: none).
  struct Place {
    int b, i, n, token;
  };
  auto place_at = [&](int pos) {
    Place p{0, 0, 0, -1};
    if (pos >= line.total) return p;
    int before;
    p.b = line.find(pages, a.src.batch, lane, pos, before);
    p.i = pos - before;
    p.n = min(page_size, min(a.lens[p.b], a.budgets[p.b]) - (p.i << log2));
    if (tid < p.n) p.token = a.kept[(int64_t(p.b) * a.src.heads + h) * a.max_keep + (p.i << log2) + tid];
    return p;
  };
  auto number_of = [&](const Place& p) {
    return p.token < 0 ? 0 : __ldg(a.src.table + int64_t(p.b) * a.src.max_pages + (p.token >> log2));
  };
  int pos = blockIdx.x;
  Place here = place_at(pos), next = place_at(pos + gridDim.x);
  int number = number_of(here);
  for (int turn = 0; pos < line.total; turn ^= 1) {  // the shared arrays alternate
    const int dst = __ldg(a.dst.table + int64_t(here.b) * a.dst.max_pages + here.i);
    if (tid < 2) top[turn][tid] = -1000;
    if (tid < here.n) {
      const bool fine = unsigned(number) < unsigned(a.src.num_pages);
      if (!fine) atomicOr(a.src.status, kErrBadPage);
      src_page[turn][tid] = fine ? number : -1;
      src_slot[turn][tid] = here.token & (page_size - 1);
    }
    __syncthreads();
    const bool fine = unsigned(dst) < unsigned(a.dst.num_pages);
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll
      for (int y = 0; y < N; ++y) {
        const int x = y * kGatherThreads + tid, slot = x / per_row, piece = x % per_row;
        if (slot >= here.n || src_page[turn][slot] < 0) continue;
        copy16_async(codes + (side * N + y) * kGatherThreads * 16,
                     (side ? a.src.v_pages : a.src.k_pages) +
                         (((int64_t(src_page[turn][slot]) * a.src.heads + h) << log2) + src_slot[turn][slot]) * D + piece * 16,
                     true);
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (tid < here.n && src_page[turn][tid] >= 0) {
      const int64_t at = int64_t(number) * a.src.heads + h;
      const int ek = exponent_of(a.src.k_scale[at]), ev = exponent_of(a.src.v_scale[at]);
      exps[turn][0][tid] = ek;
      exps[turn][1][tid] = ev;
      atomicMax(&top[turn][0], ek);
      atomicMax(&top[turn][1], ev);
    }
    const Place after = place_at(pos + 2 * gridDim.x);
    const int number_next = number_of(next);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (!fine) {
      if (tid == 0) {
        atomicOr(a.src.status, kErrBadPage);
        atomicOr(a.dst.status, kErrBadPage);
      }
    } else {
#pragma unroll
      for (int side = 0; side < 2; ++side)
#pragma unroll
        for (int y = 0; y < N; ++y) {
          const int x = y * kGatherThreads + tid, slot = x / per_row, piece = x % per_row;
          if (slot >= here.n || src_page[turn][slot] < 0) continue;
          uint4 w = moved[((side * N + y) * kGatherThreads + tid)];
          const int shift = top[turn][side] - exps[turn][side][slot];
          if (shift > 0) {
            w.x = rescale4(w.x, shift);
            w.y = rescale4(w.y, shift);
            w.z = rescale4(w.z, shift);
            w.w = rescale4(w.w, shift);
          }
          *reinterpret_cast<uint4*>((side ? a.dst.v_pages : a.dst.k_pages) +
                                    (((int64_t(dst) * a.dst.heads + h) << log2) + slot) * D + piece * 16) = w;
        }
      if (tid < 2 && top[turn][tid] > -1000)
        (tid ? a.dst.v_scale : a.dst.k_scale)[int64_t(dst) * a.dst.heads + h] = pow2f(max(-126, top[turn][tid]));
    }
    pos += gridDim.x;
    here = next;
    next = after;
    number = number_next;
  }
}

}  // namespace

attn_status launch_cache_evict(const EvictArgs& a, cudaStream_t s) {
  const int stage = a.max_seqlen < kStageMost ? a.max_seqlen : kStageMost;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageMost * 4);
  if (e != cudaSuccess) return record_cuda_error(e, "attn_cache_evict configure");
  evict_select_kernel<<<dim3(unsigned(a.src.heads), unsigned(a.src.batch)), kSelectThreads, unsigned(stage) * 4, s>>>(a, stage);
  e = cudaGetLastError();
  if (e != cudaSuccess) return record_cuda_error(e, "attn_cache_evict select launch");
  if (a.max_keep == 0) return ATTN_OK;
  // 64 CTAs per SM at most, four times what is resident: later ones even out the pages'
  // different waits.  (16 per SM, all at work at once: 95 us where 64 take 92, and 106 where
  // 86, 32 and 16 sequences of 1024 to 16384 tokens with pages of 64 x 128 and 16 x 64.)
  const int page_size = 1 << a.src.page_log2;
  const int64_t pages = int64_t(a.src.batch) * ((int64_t(a.max_keep) + page_size - 1) / page_size);
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return record_cuda_error(e, "attn_cache_evict device query");
  const int64_t most = (64ll * sms + a.src.heads - 1) / a.src.heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(pages < most ? pages : most), unsigned(a.src.heads));
  cfg.blockDim = dim3(kGatherThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (page_size * a.src.head_dim / 16 / kGatherThreads) {
    case 8: e = cudaLaunchKernelEx(&cfg, evict_gather_kernel<8>, a); break;
    case 4: e = cudaLaunchKernelEx(&cfg, evict_gather_kernel<4>, a); break;
    case 2: e = cudaLaunchKernelEx(&cfg, evict_gather_kernel<2>, a); break;
    default: e = cudaLaunchKernelEx(&cfg, evict_gather_kernel<1>, a); break;
  }
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_evict copy launch");
}

}  // namespace attnmask
