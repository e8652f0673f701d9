// Appending to the 8-bit cache: new keys and values become e4m3 codes with one
// power-of-two scale per page and head.
//
// A team of threads owns one page and head of the keys or of the values: it
// reads the page's new tokens once into registers, takes their largest finite
// magnitude, settles the scale (the larger of the page's and the new tokens'
// where the page already holds tokens, whose codes are then re-scaled) and
// writes the codes.  Nobody else writes the page, so there are no atomics and
// the result does not depend on any order.  Bound: each new element is read
// once (2 or 4 bytes) and written once (1 byte).  A thread has up to 64 elements
// in flight; a CTA's teams take different heads of one page.  The pages of all
// sequences form one line (cache_rows.cuh), a CTA per page, so that ragged
// batches launch few empty CTAs.
#include "cache_rows.cuh"

namespace attnmask {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kChunk = 8;   // elements of one access
constexpr int kChunks = 8;  // accesses per thread

// Eight elements as they lie in memory.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 v;
  __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ void get(float (&f)[kChunk]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ void get(float (&f)[kChunk]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
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

template <typename T>
__global__ void __launch_bounds__(kAppendThreads, sizeof(T) == 2 ? 4 : 2) append_kernel(const AppendArgs a, int team_log2) {
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

  Raw<T> x[kChunks];
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const int ch = (j << team_log2) + tid;
    const int slot = ch / per_row, d = (ch % per_row) * kChunk;
    if (on && slot >= first && slot < last)
      x[j].load(src + (q0 + (i << c.page_log2) + slot - held) * stride + int64_t(h) * c.head_dim + d);
    else
      x[j].zero();
  }
  if (!in_pool(c, number)) {
    atomicOr(c.status, kErrBadPage);
    return;
  }
  uint8_t* codes = (values ? c.v_pages : c.k_pages) + ((int64_t(number) * c.heads + h) << c.page_log2) * c.head_dim;
  float* scale = (values ? c.v_scale : c.k_scale) + int64_t(number) * c.heads + h;
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    float f[kChunk];
    x[j].get(f);
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
    x[j].get(f);
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
  append_kernel<T><<<grid, kAppendThreads, 0, s>>>(a, team_log2);
  return cudaGetLastError();
}

}  // namespace

attn_status launch_cache_append(const AppendArgs& a, cudaStream_t s) {
  const cudaError_t e = a.bf16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_append launch");
}

}  // namespace attnmask
