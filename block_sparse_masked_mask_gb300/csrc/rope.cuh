// Rotary positions: each pair of a head's leading rotary_dim dimensions is
// turned by position * theta_i, (x, y) -> (x cos a - y sin a, y cos a + x sin a);
// the gradient is the same with -a.
//
// One pass: every element is read and written once, so the memory bounds it.
// A warp takes one token and a share of its heads.  Its lanes compute the
// token's sines and cosines once, two or so each, and exchange them through
// shared memory; a lane then keeps those of its own pairs in registers, for it
// meets the same pairs in every head.  No CTA-wide barrier: the loads of the
// first heads are in flight while the angles are computed.
//
// The angle in turns is position * theta / (2 pi) modulo 1.  The plan holds
// theta / (2 pi) as a 64-bit fixed-point fraction, and an integer product
// modulo 2^64 drops the whole turns exactly, however far the position; the top
// 32 bits, read as signed, are the turn in [-1/2, 1/2) to 2^-33.
#pragma once

#include "cache.cuh"

namespace attnmask {
namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeUnroll = 4;  // units in flight per lane (even)

struct RopeParams {
  RopeArgs a;
  int rot;         // rotated dimensions
  int unit_log2;   // log2 of the units per head
  int slices;      // warps per token
  int passes;      // passes of a warp over its heads (32 units each)
  float factor;
  uint64_t turn[ATTN_ROPE_MAX_PAIRS];
  RopeCheck check;  // CHECKED only
};

// E elements of one memory access, E * sizeof(T) a power of two up to 16 bytes.
template <typename T, int E>
struct alignas(sizeof(T) * E) Vec {
  T x[E];
};

// One access of a whole Vec, marked as streaming: nothing is read twice, and the
// L2 keeps its lines for others (32768 tokens of 64 heads: 220 us with plain
// accesses, 156 us with these).
template <int BYTES>
struct Words;
template <>
struct Words<16> { using type = uint4; };
template <>
struct Words<8> { using type = uint2; };
template <>
struct Words<4> { using type = uint32_t; };
template <>
struct Words<2> { using type = uint16_t; };
template <typename T, int E>
__device__ __forceinline__ void load_vec(Vec<T, E>& v, const T* p) {
  using W = typename Words<sizeof(T) * E>::type;
  const W w = __ldcs(reinterpret_cast<const W*>(p));
  *reinterpret_cast<W*>(&v) = w;
}
template <typename T, int E>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, E>& v) {
  using W = typename Words<sizeof(T) * E>::type;
  __stcs(reinterpret_cast<W*>(p), *reinterpret_cast<const W*>(&v));
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

// A turned pair, c = (cos, sin), with the roundings fixed: what goes into the cache does not depend on
// how it was read.
__device__ __forceinline__ float turned_x(float x, float y, float2 c) { return __fmaf_rn(x, c.x, -__fmul_rn(y, c.y)); }
__device__ __forceinline__ float turned_y(float x, float y, float2 c) { return __fmaf_rn(y, c.x, __fmul_rn(x, c.y)); }

// The slot of row t's token in sequence b; -1 where that is not used or does not hold the row.
__device__ __forceinline__ int slot_of(const int32_t* cu, const int32_t* lens, int t, int b, int total_tokens, int max_new,
                                       int max_len) {
  SeqRows r;
  const bool mine = load_rows(cu, lens, b, total_tokens, max_new, max_len, nullptr, r, false) && r.len >= r.n && t >= r.q0 &&
                    t < r.q0 + r.n;
  return mine ? r.len - r.n + t - r.q0 : -1;
}

// The same in any of them, by a whole warp: for a row of none, and where a cu that does not ascend leads a search
// astray.  (Out of line: 12 prompts 55 us, 58 with its code among what all run.)
__device__ __noinline__ int slot_of_any(const int32_t* cu, const int32_t* lens, int t, int batch, int total_tokens, int max_new,
                                        int max_len) {
  const int lane = int(threadIdx.x & 31u);
  bool some = false;  // most often none
#pragma unroll 8
  for (int b = lane; b < batch; b += 32) some |= __ldg(cu + b) <= t && t < __ldg(cu + b + 1);
  if (!__any_sync(0xffffffffu, some)) return -1;
  int slot = -1;
#pragma unroll 1
  for (int b = lane; b < batch; b += 32) slot = max(slot, slot_of(cu, lens, t, b, total_tokens, max_new, max_len));
  return __reduce_max_sync(0xffffffffu, slot);
}

// The position of row t and whether it has one.  CHECKED: only rows of sequences that
// an append would use have one, positions given or not, and all of those do, whatever stands
// beside them in a malformed cu.  Called by whole warps.
template <bool CHECKED>
__device__ __forceinline__ bool position_of(const RopeParams& p, int t, int& pos) {
  const RopeArgs& a = p.a;
  if (!CHECKED && a.positions) {
    pos = a.positions[t];
    return true;
  }
  // the last sequence that starts at or before the row
  int b0 = 0, b1 = a.batch;
  while (b0 + 1 < b1) {
    const int m = (b0 + b1) >> 1;
    if (a.cu[m] <= t) b0 = m; else b1 = m;
  }
  if (CHECKED) {
    int slot = slot_of(a.cu, a.lens, t, b0, a.total_tokens, p.check.max_new, p.check.max_len);
    if (__builtin_expect(slot < 0, 0))
      slot = slot_of_any(a.cu, a.lens, t, a.batch, a.total_tokens, p.check.max_new, p.check.max_len);
    if (slot < 0) return false;
    pos = a.positions ? a.positions[t] : slot;
    return true;
  }
  const int s0 = a.cu[b0], s1 = a.cu[b0 + 1];
  pos = t - s0 + (a.lens ? a.lens[b0] - (s1 - s0) : 0);
  return t >= s0 && t < s1;
}

// The warp's table of (cos, sin) for row t, the factor multiplied in; false if the row has no position.
template <bool CHECKED>
__device__ __forceinline__ bool angles(const RopeParams& p, int t, int lane, float2* cs) {
  int pos;
  if (!position_of<CHECKED>(p, t, pos)) return false;
  for (int c = lane; c < p.rot / 2; c += 32) {
    const int64_t turn = int64_t(uint64_t(int64_t(pos)) * p.turn[c]);
    float sn, cn;
    sincospif(float(int32_t(turn >> 32)) * 0x1p-31f, &sn, &cn);
    cs[c] = make_float2(cn * p.factor, (p.a.inverse ? -sn : sn) * p.factor);
  }
  __syncwarp();
  return true;
}

// A unit is VP pairs: for the half layout VP elements of each half, for the
// interleaved one 2 VP consecutive elements.  What lies behind rot is copied.  A
// pass of a warp covers 32 units: whole heads, or half a head where a head has 64.
// PART: an interleaved unit lies partly behind rot, so that any rot is taken by
// wide accesses (rot = 50, 10400 tokens of 40 heads of 128 bf16: 37 us; by the
// accesses that divide rot 133).
// (Three CTAs per SM fit fp32 without spills and are 5% faster; bf16 needs the registers.)
template <typename T, int VP, bool INTER, bool PART, bool CHECKED>
__device__ __forceinline__ void rope_rows(const RopeParams& p, int block_of_jobs) {
  __shared__ float2 cs[kRopeWarps][ATTN_ROPE_MAX_PAIRS];
  const RopeArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t job = int64_t(block_of_jobs) * kRopeWarps + warp;
  const int t = int(job / p.slices), slice = int(job % p.slices);
  if (t >= a.total_tokens) return;
  const int heads = a.num_heads + a.num_kv_heads;
  // units of a head that are rotated; the last interleaved one may be in part
  const int turned = (p.rot + (PART ? 2 * VP - 1 : 0)) / (2 * VP);
  const int units = 1 << p.unit_log2;
  const T* q = static_cast<const T*>(a.q) + int64_t(t) * a.q_stride;
  const T* k = static_cast<const T*>(a.k) + int64_t(t) * a.k_stride;
  T* qo = static_cast<T*>(a.q_out) + int64_t(t) * a.q_out_stride;
  T* ko = static_cast<T*>(a.k_out) + int64_t(t) * a.k_out_stride;

  // 64 units per head (VP = 1, 128 dimensions): the lane's unit alternates; else
  // it is the same in every pass
  const int blocks = units > 32 ? units / 32 : 1;
  const int per_pass = units > 32 ? 1 : 32 >> p.unit_log2;  // heads
  const int first = slice * p.passes * per_pass, last = min(heads, first + p.passes * per_pass);
  for (int block = 0; block < blocks; ++block) {
    const int u = block * 32 + (lane & (units - 1));
    int d0, d1;
    if (INTER) {
      d0 = u * 2 * VP;
      d1 = d0 + VP;
    } else if (u >= turned) {
      d0 = p.rot + (u - turned) * 2 * VP;
      d1 = d0 + VP;
    } else {
      d0 = u * VP;
      d1 = p.rot / 2 + d0;
    }
    const int h0 = first + (units > 32 ? 0 : lane >> p.unit_log2);
    Vec<T, VP> x[kRopeUnroll], y[kRopeUnroll];
    auto load = [&](int j, int i) {
      if (i >= last) return;
      const T* src = i < a.num_heads ? q + i * a.head_dim : k + (i - a.num_heads) * a.head_dim;
      load_vec(x[j], src + d0);
      load_vec(y[j], src + d1);
    };
#pragma unroll
    for (int j = 0; j < kRopeUnroll; ++j) load(j, h0 + j * per_pass);
    if (block == 0 && !angles<CHECKED>(p, t, lane, cs[warp])) return;  // the whole warp
    float2 c[VP];
#pragma unroll
    for (int e = 0; e < VP; ++e) c[e] = (PART ? u * VP + e < p.rot / 2 : u < turned) ? cs[warp][u * VP + e] : make_float2(1.f, 0.f);
    for (int h = h0; h < last; h += kRopeUnroll * per_pass) {
#pragma unroll
      for (int j = 0; j < kRopeUnroll; ++j) {
        const int i = h + j * per_pass;
        if (i >= last) continue;
        if (u < turned) {
#pragma unroll
          for (int e = 0; e < VP; ++e) {
            // the half layout pairs x with y; the interleaved one neighbours
            T* px = INTER ? (2 * e < VP ? &x[j].x[2 * e] : &y[j].x[2 * e - VP]) : &x[j].x[e];
            T* py = INTER ? (2 * e + 1 < VP ? &x[j].x[2 * e + 1] : &y[j].x[2 * e + 1 - VP]) : &y[j].x[e];
            if (PART && u * VP + e >= p.rot / 2) continue;  // copied
            const float fx = to_f(*px), fy = to_f(*py);
            from_f(*px, CHECKED ? turned_x(fx, fy, c[e]) : fx * c[e].x - fy * c[e].y);
            from_f(*py, CHECKED ? turned_y(fx, fy, c[e]) : fy * c[e].x + fx * c[e].y);
          }
        }
        T* dst = i < a.num_heads ? qo + i * a.head_dim : ko + (i - a.num_heads) * a.head_dim;
        store_vec(dst + d0, x[j]);
        store_vec(dst + d1, y[j]);
        load(j, i + kRopeUnroll * per_pass);  // the next unit takes its place
      }
    }
  }
}

// The half layout where rot / 2 is no multiple of a wide access: a lane takes W
// consecutive elements as they lie, and finds each one's partner, rot / 2 away, in
// a copy of the warp's heads in shared memory.
template <typename T, int W, bool CHECKED>
__device__ __forceinline__ void rope_halves(const RopeParams& p, int block_of_jobs) {
  __shared__ float2 cs[kRopeWarps][ATTN_ROPE_MAX_PAIRS];
  __shared__ alignas(16) T copies[kRopeWarps][2][32 * W];
  const RopeArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t job = int64_t(block_of_jobs) * kRopeWarps + warp;
  const int t = int(job / p.slices), slice = int(job % p.slices);
  if (t >= a.total_tokens) return;
  const int heads = a.num_heads + a.num_kv_heads, half = p.rot / 2;
  const int per_pass = 32 >> p.unit_log2;  // heads
  const int first = slice * p.passes * per_pass, last = min(heads, first + p.passes * per_pass);
  const int d0 = (lane & ((1 << p.unit_log2) - 1)) * W, h0 = first + (lane >> p.unit_log2);
  const T* q = static_cast<const T*>(a.q) + int64_t(t) * a.q_stride + d0;
  const T* k = static_cast<const T*>(a.k) + int64_t(t) * a.k_stride + d0;
  T* qo = static_cast<T*>(a.q_out) + int64_t(t) * a.q_out_stride + d0;
  T* ko = static_cast<T*>(a.k_out) + int64_t(t) * a.k_out_stride + d0;
  Vec<T, W> x[kRopeUnroll];
  auto load = [&](int j, int i) {
    if (i < last) load_vec(x[j], i < a.num_heads ? q + i * a.head_dim : k + (i - a.num_heads) * a.head_dim);
  };
#pragma unroll
  for (int j = 0; j < kRopeUnroll; ++j) load(j, h0 + j * per_pass);
  if (!angles<CHECKED>(p, t, lane, cs[warp])) return;  // the whole warp
  float2 c[W];  // y = x c.x + partner c.y
  int from[W];  // the partner's place in the copy
#pragma unroll
  for (int e = 0; e < W; ++e) {
    const int d = d0 + e, i = d < half ? d : d - half;
    c[e] = d < p.rot ? cs[warp][i] : make_float2(1.f, 0.f);
    if (d < half) c[e].y = -c[e].y;
    from[e] = lane * W + e + (d < half ? half : d < p.rot ? -half : 0);
  }
  const int rounds = (last - first + per_pass - 1) / per_pass;
  for (int r = 0; r < rounds; r += kRopeUnroll) {
#pragma unroll
    for (int j = 0; j < kRopeUnroll; ++j) {
      if (r + j >= rounds) break;  // the whole warp
      T* copy = copies[warp][j & 1];
      *reinterpret_cast<Vec<T, W>*>(copy + lane * W) = x[j];
      __syncwarp();  // (and the copy before the last one has been read)
      const int i = h0 + (r + j) * per_pass;
      Vec<T, W> y;
#pragma unroll
      for (int e = 0; e < W; ++e) {
        y.x[e] = x[j].x[e];
        if (d0 + e < p.rot) {
          const float a = to_f(x[j].x[e]), b = to_f(copy[from[e]]);
          from_f(y.x[e], CHECKED ? turned_y(b, a, c[e]) : a * c[e].x + b * c[e].y);
        }
      }
      if (i < last) store_vec(i < a.num_heads ? qo + i * a.head_dim : ko + (i - a.num_heads) * a.head_dim, y);
      load(j, i + kRopeUnroll * per_pass);
    }
  }
}

// Which of the two, as a type: KIND 0 halves, 1 interleaved, 2 interleaved with a unit in part,
// 3 halves through shared memory; W elements of an access.
template <typename T_, int KIND, int W, bool CHECKED>
struct RopeWay {
  using T = T_;
  static constexpr int kPerSM = KIND < 3 && sizeof(T) == 4 ? 3 : 1;  // CTAs, at least
  __device__ __forceinline__ static void run(const RopeParams& p, int block) {
    if constexpr (KIND == 3) rope_halves<T, W, CHECKED>(p, block);
    else rope_rows<T, W, KIND != 0, KIND == 2, CHECKED>(p, block);
  }
};

// Settles how the rows are read and divided, and calls launch(way, CTAs).
template <typename T, bool CHECKED, typename F>
cudaError_t with_way(RopeParams& p, bool interleaved, const F& launch) {
  const RopeArgs& a = p.a;
  // The widest access (up to 16 bytes) that the halves, addresses and strides allow.
  constexpr int kMost = 16 / sizeof(T);
  uint64_t bits = uint64_t(reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.q_out));
  bits |= uint64_t(a.q_stride | a.q_out_stride) * sizeof(T);
  if (a.num_kv_heads) {
    bits |= uint64_t(reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.k_out));
    bits |= uint64_t(a.k_stride | a.k_out_stride) * sizeof(T);
  }
  int wide = kMost, vp = kMost;
  while (wide > 1 && (bits & (wide * sizeof(T) - 1))) wide >>= 1;
  if (!interleaved) bits |= uint64_t(p.rot / 2) * sizeof(T);
  while (vp > 1 && (bits & (vp * sizeof(T) - 1))) vp >>= 1;
  // Halves at odd places: by wide accesses and shared memory, where pairs would be read
  // one or two at a time (16 x 650 tokens of 40 heads of 128, pairs / copies: rot = 50 bf16
  // 71 / 53 us, fp32 82 / 78; rot = 52 78 / 53, 96 / 78; but rot = 40 bf16, by fours, 37 / 52).
  const bool halves = vp < 4 && wide >= 4 && wide * 32 >= a.head_dim;
  const int unit = halves ? wide : 2 * vp;  // elements
  p.unit_log2 = 0;
  while ((unit << p.unit_log2) < a.head_dim) ++p.unit_log2;
  // Warps per token: one, or more while there are fewer warps than the GPU
  // holds (32 per SM), down to one pass each.  Beside an append's pages (CHECKED) 8 per SM: a
  // warp's start costs more than a pass of its loop there (32 trees of 17 to 64 tokens, 32 heads of 128:
  // 17.3 / 13.9 us).
  const int units = 1 << p.unit_log2, heads = a.num_heads + a.num_kv_heads;
  const int all = units > 32 ? heads : int((int64_t(heads) * units + 31) / 32);  // passes over a token
  int sms = 0, dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int want = ((CHECKED ? 8 : 32) * sms + a.total_tokens - 1) / a.total_tokens;
  p.passes = (all + want - 1) / want;
  p.slices = (all + p.passes - 1) / p.passes;
  const int64_t ctas = (int64_t(a.total_tokens) * p.slices + kRopeWarps - 1) / kRopeWarps;
  if (halves) {
    if constexpr (kMost >= 8)
      if (wide == 8) return launch(RopeWay<T, 3, 8, CHECKED>{}, ctas);
    return launch(RopeWay<T, 3, 4, CHECKED>{}, ctas);
  }
  const bool part = p.rot % (2 * vp) != 0;
  switch (vp) {
    case 8:
      if constexpr (kMost >= 8)
        return !interleaved ? launch(RopeWay<T, 0, 8, CHECKED>{}, ctas)
               : part ? launch(RopeWay<T, 2, 8, CHECKED>{}, ctas) : launch(RopeWay<T, 1, 8, CHECKED>{}, ctas);
    case 4:
      return !interleaved ? launch(RopeWay<T, 0, 4, CHECKED>{}, ctas)
             : part ? launch(RopeWay<T, 2, 4, CHECKED>{}, ctas) : launch(RopeWay<T, 1, 4, CHECKED>{}, ctas);
    case 2:
      return !interleaved ? launch(RopeWay<T, 0, 2, CHECKED>{}, ctas)
             : part ? launch(RopeWay<T, 2, 2, CHECKED>{}, ctas) : launch(RopeWay<T, 1, 2, CHECKED>{}, ctas);
    default:
      return !interleaved ? launch(RopeWay<T, 0, 1, CHECKED>{}, ctas) : launch(RopeWay<T, 1, 1, CHECKED>{}, ctas);
  }
}

inline RopeParams rope_params(const RopeArgs& a, const attn_rope_plan& plan) {
  RopeParams p;
  p.a = a;
  p.rot = plan.rotary_dim;
  p.factor = plan.result_factor;
  for (int i = 0; i < ATTN_ROPE_MAX_PAIRS; ++i) p.turn[i] = plan.turn[i];
  p.check = RopeCheck{};
  return p;
}

}  // namespace
}  // namespace attnmask
