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

// The position of row t and whether it has one.
__device__ __forceinline__ bool position_of(const RopeArgs& a, int t, int& pos) {
  if (a.positions) {
    pos = a.positions[t];
    return true;
  }
  // the last sequence that starts at or before the row
  int b0 = 0, b1 = a.batch;
  while (b0 + 1 < b1) {
    const int m = (b0 + b1) >> 1;
    if (a.cu[m] <= t) b0 = m; else b1 = m;
  }
  const int s0 = a.cu[b0], s1 = a.cu[b0 + 1];
  pos = t - s0 + (a.lens ? a.lens[b0] - (s1 - s0) : 0);
  return t >= s0 && t < s1;
}

// The warp's table of (cos, sin) for row t, the factor multiplied in; false if the row has no position.
__device__ __forceinline__ bool angles(const RopeParams& p, int t, int lane, float2* cs) {
  int pos;
  if (!position_of(p.a, t, pos)) return false;
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
template <typename T, int VP, bool INTER, bool PART>
__global__ void __launch_bounds__(32 * kRopeWarps, sizeof(T) == 4 ? 3 : 1) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 cs[kRopeWarps][ATTN_ROPE_MAX_PAIRS];
  const RopeArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t job = int64_t(blockIdx.x) * kRopeWarps + warp;
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
    if (block == 0 && !angles(p, t, lane, cs[warp])) return;  // the whole warp
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
            from_f(*px, fx * c[e].x - fy * c[e].y);
            from_f(*py, fy * c[e].x + fx * c[e].y);
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
template <typename T, int W>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_halves_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 cs[kRopeWarps][ATTN_ROPE_MAX_PAIRS];
  __shared__ alignas(16) T copies[kRopeWarps][2][32 * W];
  const RopeArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t job = int64_t(blockIdx.x) * kRopeWarps + warp;
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
  if (!angles(p, t, lane, cs[warp])) return;  // the whole warp
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
        if (d0 + e < p.rot) from_f(y.x[e], to_f(x[j].x[e]) * c[e].x + to_f(copy[from[e]]) * c[e].y);
      }
      if (i < last) store_vec(i < a.num_heads ? qo + i * a.head_dim : ko + (i - a.num_heads) * a.head_dim, y);
      load(j, i + kRopeUnroll * per_pass);
    }
  }
}

template <typename T, int W>
cudaError_t launch_halves(const RopeParams& p, cudaStream_t s) {
  const unsigned grid = unsigned((int64_t(p.a.total_tokens) * p.slices + kRopeWarps - 1) / kRopeWarps);
  rope_halves_kernel<T, W><<<grid, 32 * kRopeWarps, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int VP>
cudaError_t launch_vp(const RopeParams& p, bool interleaved, cudaStream_t s) {
  const unsigned grid = unsigned((int64_t(p.a.total_tokens) * p.slices + kRopeWarps - 1) / kRopeWarps);
  const bool part = p.rot % (2 * VP) != 0;
  auto kernel = !interleaved ? rope_kernel<T, VP, false, false>
                             : part ? rope_kernel<T, VP, true, VP != 1> : rope_kernel<T, VP, true, false>;
  kernel<<<grid, 32 * kRopeWarps, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(RopeParams& p, bool interleaved, cudaStream_t s) {
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
  // holds (32 per SM), down to one pass each.
  const int units = 1 << p.unit_log2, heads = a.num_heads + a.num_kv_heads;
  const int all = units > 32 ? heads : int((int64_t(heads) * units + 31) / 32);  // passes over a token
  int sms = 0, dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int want = (32 * sms + a.total_tokens - 1) / a.total_tokens;
  p.passes = (all + want - 1) / want;
  p.slices = (all + p.passes - 1) / p.passes;
  if (halves) {
    if constexpr (kMost >= 8)
      if (wide == 8) return launch_halves<T, 8>(p, s);
    return launch_halves<T, 4>(p, s);
  }
  switch (vp) {
    case 8: if constexpr (kMost >= 8) return launch_vp<T, 8>(p, interleaved, s);
    case 4: return launch_vp<T, 4>(p, interleaved, s);
    case 2: return launch_vp<T, 2>(p, interleaved, s);
    default: return launch_vp<T, 1>(p, interleaved, s);
  }
}

}  // namespace

attn_status launch_rope(const RopeArgs& a, const attn_rope_plan& plan, cudaStream_t s) {
  RopeParams p;
  p.a = a;
  p.rot = plan.rotary_dim;
  p.factor = plan.result_factor;
  for (int i = 0; i < ATTN_ROPE_MAX_PAIRS; ++i) p.turn[i] = plan.turn[i];
  const cudaError_t e = a.bf16 ? launch_t<__nv_bfloat16>(p, plan.interleaved != 0, s)
                               : launch_t<float>(p, plan.interleaved != 0, s);
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_rope launch");
}

}  // namespace attnmask
