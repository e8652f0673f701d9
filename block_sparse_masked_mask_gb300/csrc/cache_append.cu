// Appending to the 8-bit cache: new keys and values become e4m3 codes with one
// power-of-two scale per page and head.
//
// A team of threads owns one page and head of the keys or of the values: it
// copies the page's new tokens once into shared memory (each thread what it will
// read itself, up to 64 elements in flight), takes their largest finite magnitude, settles the scale (the larger of the page's and the new tokens'
// where the page already holds tokens, whose codes are then re-scaled) and
// writes the codes.  Nobody else writes the page, so there are no atomics and
// the result does not depend on any order.  Bound: each new element is read
// once (2 or 4 bytes) and written once (1 byte).  A CTA's teams take different
// heads of one page.  (Held in registers instead, the elements leave room for
// two CTAs per SM and the latencies of the lookups show: 47 us instead of 36
// for 14000 tokens of 16 heads.)  The pages of all
// sequences form one line (cache_rows.cuh), a CTA per page, so that ragged
// batches launch few empty CTAs.
#include "cache_rows.cuh"

namespace attnmask {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kChunk = 8;   // elements of one access
constexpr int kChunks = 8;  // accesses per thread

// Eight elements (a chunk) in shared memory: 16-byte piece p of a thread's j-th
// chunk at ((j * PIECES + p) * kAppendThreads + thread) * 16.
template <typename T>
struct Chunk {
  static constexpr int PIECES = sizeof(T) * kChunk / 16;
  static constexpr int SMEM = kChunks * PIECES * kAppendThreads * 16;
  __device__ static void get(const uint8_t* smem, int j, float (&f)[kChunk]) {
    uint32_t w[4 * PIECES];
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const uint4 v = *reinterpret_cast<const uint4*>(smem + ((j * PIECES + p) * kAppendThreads + threadIdx.x) * 16);
      w[4 * p] = v.x; w[4 * p + 1] = v.y; w[4 * p + 2] = v.z; w[4 * p + 3] = v.w;
    }
#pragma unroll
    for (int e = 0; e < kChunk; ++e) {
      if constexpr (sizeof(T) == 4) f[e] = __uint_as_float(w[e]);
      else f[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
    }
  }
};

// Pages that a sequence's new tokens touch.
struct NewPages {
  const AppendArgs& a;
  bool note;
  __device__ int operator()(int b) const {
    const CacheView& c = a.cache;
    SeqRows r;
    if (!load_rows(a.cu, a.lens, b, a.total_tokens, a.max_new, c.max_pages << c.page_log2, c.status, r, note)) return 0;
    if (r.len < r.n) {
      if (note) atomicOr(c.status, kErrHeld);
      return 0;
    }
    return r.n == 0 ? 0 : ((r.len - 1) >> c.page_log2) - ((r.len - r.n) >> c.page_log2) + 1;
  }
};

// CTAs per SM: bf16 six (36.0 us for those 14000 tokens; five, as the compiler would have
// it, 36.9, seven 38.4); fp32 three, as many as its 64 KB of shared memory each allow
// (the same tokens 68.8 us, floor 40; held to the registers of six 69.8).
template <typename T>
__global__ void __launch_bounds__(kAppendThreads, sizeof(T) == 4 ? 3 : 6) append_kernel(const AppendArgs a, int team_log2) {
  using C = Chunk<T>;
  extern __shared__ __align__(16) uint8_t smem[];
  const CacheView& c = a.cache;
  const NewPages pages{a, blockIdx.x == 0 && blockIdx.y == 0};
  const UnitLine line(pages, c.batch, threadIdx.x & 31);
  const int pos = blockIdx.x;
  if (pos >= line.total) return;
  int before;
  const int b = line.find(pages, c.batch, threadIdx.x & 31, pos, before);
  const int q0 = a.cu[b], len = a.lens[b];
  const int held = len - (a.cu[b + 1] - q0);  // tokens that are there already
  const int page_size = 1 << c.page_log2;
  const int i = (held >> c.page_log2) + pos - before;  // this CTA's page of the sequence
  const int first = max(held - (i << c.page_log2), 0);  // slots [first, last) are new
  const int last = min(len - (i << c.page_log2), page_size);
  const int per_row = c.head_dim / kChunk;
  // the team's head: the keys' heads, then the values'
  const int team = threadIdx.x >> team_log2, tid = threadIdx.x & ((1 << team_log2) - 1);
  const int hv = blockIdx.y * (kAppendThreads >> team_log2) + team;
  const bool on = hv < 2 * c.heads, values = hv >= c.heads;
  const int h = on ? (values ? hv - c.heads : hv) : 0;
  const T* src = static_cast<const T*>(values ? a.v : a.k);
  const int64_t stride = values ? a.v_stride : a.k_stride;
  const int number = __ldg(c.table + int64_t(b) * c.max_pages + i);  // needed only behind the loads

  const uint32_t mine = uint32_t(__cvta_generic_to_shared(smem)) + threadIdx.x * 16;
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const int ch = (j << team_log2) + tid;
    const int slot = ch / per_row, d = (ch % per_row) * kChunk;
    const bool fresh = on && slot >= first && slot < last;  // else zeros
    const T* from = fresh ? src + (q0 + (i << c.page_log2) + slot - held) * stride + int64_t(h) * c.head_dim + d : src;
#pragma unroll
    for (int p = 0; p < C::PIECES; ++p)
      copy16_async(mine + (j * C::PIECES + p) * kAppendThreads * 16, from + p * 16 / sizeof(T), fresh);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  float amax = 0.f;
  if (!in_pool(c, number)) {
    atomicOr(c.status, kErrBadPage);
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  uint8_t* codes = (values ? c.v_pages : c.k_pages) + ((int64_t(number) * c.heads + h) << c.page_log2) * c.head_dim;
  float* scale = (values ? c.v_scale : c.k_scale) + int64_t(number) * c.heads + h;
  asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    float f[kChunk];
    C::get(smem, j, f);
#pragma unroll
    for (int e = 0; e < kChunk; ++e) {
      const float m = fabsf(f[e]);
      if (m < INFINITY) amax = fmaxf(amax, m);  // false for NaN too
    }
  }
  __shared__ float warp_max[kAppendThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  const float was = first > 0 ? *scale : 0.f;  // read before the team's first thread replaces it
  __syncthreads();
  if (!on) return;
  const int warps = 1 << (team_log2 - 5);  // of the team
  for (int w = 0; w < warps; ++w) amax = fmaxf(amax, warp_max[team * warps + w]);

  int e = scale_exponent(amax);
  if (first > 0) {
    // a scale outside the range (the caller's memory) is taken into it
    const int e0 = max(kScaleExpMin, min(kScaleExpMax, exponent_of(was)));
    if (e0 < e) {
      const int bytes = first * c.head_dim;  // codes of the earlier tokens
      for (int at = tid * 8; at < bytes; at += 8 << team_log2) {
        uint2 w = *reinterpret_cast<uint2*>(codes + at);
        w.x = rescale4(w.x, e - e0);
        w.y = rescale4(w.y, e - e0);
        *reinterpret_cast<uint2*>(codes + at) = w;
      }
    }
    e = max(e, e0);
  }
  const float inv = pow2f(-e);
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const int ch = (j << team_log2) + tid;
    const int slot = ch / per_row;
    if (slot < first || slot >= last) continue;
    float f[kChunk];
    C::get(smem, j, f);
    uint2 w;
    w.x = e4m3_pair(f[0] * inv, f[1] * inv) | (e4m3_pair(f[2] * inv, f[3] * inv) << 16);
    w.y = e4m3_pair(f[4] * inv, f[5] * inv) | (e4m3_pair(f[6] * inv, f[7] * inv) << 16);
    *reinterpret_cast<uint2*>(codes + int64_t(ch) * kChunk) = w;
  }
  if (tid == 0) *scale = pow2f(e);
}

template <typename T>
cudaError_t launch_t(const AppendArgs& a, cudaStream_t s) {
  const int page_size = 1 << a.cache.page_log2;
  int team_log2 = 5;  // threads of a team: a page's elements, 64 each
  while ((kChunks * kChunk << team_log2) < page_size * a.cache.head_dim) ++team_log2;
  const int teams = kAppendThreads >> team_log2;
  // n tokens touch at most (n + page_size - 2) / page_size + 1 pages; all of them
  // together at most T / page_size whole ones and two more per sequence
  const int64_t each = (int64_t(a.max_new) + page_size - 2) / page_size + 1;
  const int64_t most = a.total_tokens / page_size + 2ll * a.cache.batch;
  const int64_t pages = each * a.cache.batch < most ? each * a.cache.batch : most;
  const dim3 grid(unsigned(pages), unsigned((2 * a.cache.heads + teams - 1) / teams));
  const cudaError_t e =
      cudaFuncSetAttribute(append_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Chunk<T>::SMEM);
  if (e != cudaSuccess) return e;
  append_kernel<T><<<grid, kAppendThreads, Chunk<T>::SMEM, s>>>(a, team_log2);
  return cudaGetLastError();
}

}  // namespace

attn_status launch_cache_append(const AppendArgs& a, cudaStream_t s) {
  const cudaError_t e = a.bf16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_append launch");
}

}  // namespace attnmask
