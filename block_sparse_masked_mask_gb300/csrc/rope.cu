// Rotary positions: each pair of a head's leading rotary_dim dimensions is
// turned by position * theta_i, (x, y) -> (x cos a - y sin a, y cos a + x sin a);
// the gradient is the same with -a.
//
// One pass: every element is read and written once, so the memory bounds it.
// The angle's sine and cosine are computed once per token and pair and shared
// by all heads through shared memory.  A CTA takes one or a few whole tokens
// (all heads of q and k): its loads are issued before the angles are
// computed, so the two latencies overlap.
//
// The angle in turns is position * theta / (2 pi) modulo 1.  The plan holds
// theta / (2 pi) as a 64-bit fixed-point fraction, and an integer product
// modulo 2^64 drops the whole turns exactly, however far the position; the top
// 32 bits, read as signed, are the turn in [-1/2, 1/2) to 2^-33.
#include "cache.cuh"

namespace attnmask {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;      // units in flight per thread
constexpr int kRopeMaxTokens = 16;  // tokens per CTA

struct RopeParams {
  RopeArgs a;
  int rot;            // rotated dimensions
  int unit_log2;      // log2 of the units per head
  int tokens_per_cta;
  float factor;
  uint64_t turn[ATTN_ROPE_MAX_PAIRS];
};

// E elements of one memory access, E * sizeof(T) a power of two up to 16 bytes.
template <typename T, int E>
struct alignas(sizeof(T) * E) Vec {
  T x[E];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

// A unit is VP pairs: for the half layout VP elements of each half, for the
// interleaved one 2 VP consecutive elements.  Units behind rot are copied.
template <typename T, int VP, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 cs[kRopeMaxTokens][ATTN_ROPE_MAX_PAIRS];
  __shared__ int ok[kRopeMaxTokens];
  const RopeArgs& a = p.a;
  const int t0 = blockIdx.x * p.tokens_per_cta;
  const int nt = min(p.tokens_per_cta, a.total_tokens - t0);
  const int heads = a.num_heads + a.num_kv_heads;
  const int per_token = heads << p.unit_log2;
  const int total = nt * per_token;
  const int turned = p.rot / (2 * VP);  // units of a head that are rotated

  Vec<T, VP> lo[kRopeUnroll], hi[kRopeUnroll];
  auto locate = [&](int i, int& t, int& h, int& u) {
    t = nt == 1 ? 0 : i / per_token;
    const int r = i - t * per_token;
    h = r >> p.unit_log2;
    u = r & ((1 << p.unit_log2) - 1);
  };
  auto offsets = [&](int u, int& d0, int& d1) {
    if (u >= turned) {
      d0 = p.rot + (u - turned) * 2 * VP;
      d1 = d0 + VP;
    } else if (INTER) {
      d0 = u * 2 * VP;
      d1 = d0 + VP;
    } else {
      d0 = u * VP;
      d1 = p.rot / 2 + d0;
    }
  };
  for (int base = 0; base < total; base += kRopeThreads * kRopeUnroll) {
#pragma unroll
    for (int j = 0; j < kRopeUnroll; ++j) {
      const int i = base + j * kRopeThreads + threadIdx.x;
      if (i >= total) continue;
      int t, h, u, d0, d1;
      locate(i, t, h, u);
      offsets(u, d0, d1);
      const T* src = h < a.num_heads
                         ? static_cast<const T*>(a.q) + int64_t(t0 + t) * a.q_stride + h * a.head_dim
                         : static_cast<const T*>(a.k) + int64_t(t0 + t) * a.k_stride + (h - a.num_heads) * a.head_dim;
      lo[j] = *reinterpret_cast<const Vec<T, VP>*>(src + d0);
      hi[j] = *reinterpret_cast<const Vec<T, VP>*>(src + d1);
    }
    if (base == 0) {
      const int pairs = p.rot / 2;
      for (int i = threadIdx.x; i < nt * ATTN_ROPE_MAX_PAIRS; i += kRopeThreads) {
        const int t = i / ATTN_ROPE_MAX_PAIRS, c = i % ATTN_ROPE_MAX_PAIRS;
        int pos = 0;
        bool in = true;
        if (a.positions) {
          pos = a.positions[t0 + t];
        } else {
          // the last sequence that starts at or before the row
          int b0 = 0, b1 = a.batch;
          while (b0 + 1 < b1) {
            const int m = (b0 + b1) >> 1;
            if (a.cu[m] <= t0 + t) b0 = m; else b1 = m;
          }
          const int s0 = a.cu[b0], s1 = a.cu[b0 + 1];
          in = t0 + t >= s0 && t0 + t < s1;
          pos = t0 + t - s0 + (a.lens ? a.lens[b0] - (s1 - s0) : 0);
        }
        if (c == 0) ok[t] = in;
        if (c < pairs) {
          const int64_t turn = int64_t(uint64_t(int64_t(pos)) * p.turn[c]);
          float sn, cn;
          sincospif(float(int32_t(turn >> 32)) * 0x1p-31f, &sn, &cn);
          cs[t][c] = make_float2(cn * p.factor, (a.inverse ? -sn : sn) * p.factor);
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kRopeUnroll; ++j) {
      const int i = base + j * kRopeThreads + threadIdx.x;
      if (i >= total) continue;
      int t, h, u, d0, d1;
      locate(i, t, h, u);
      offsets(u, d0, d1);
      if (!ok[t]) continue;
      Vec<T, VP> x = lo[j], y = hi[j];
      if (u < turned) {
#pragma unroll
        for (int e = 0; e < VP; ++e) {
          // the half layout pairs lo with hi; the interleaved one neighbours
          T* px = INTER ? (2 * e < VP ? &x.x[2 * e] : &y.x[2 * e - VP]) : &x.x[e];
          T* py = INTER ? (2 * e + 1 < VP ? &x.x[2 * e + 1] : &y.x[2 * e + 1 - VP]) : &y.x[e];
          const float2 c = cs[t][u * VP + e];
          const float fx = to_f(*px), fy = to_f(*py);
          from_f(*px, fx * c.x - fy * c.y);
          from_f(*py, fy * c.x + fx * c.y);
        }
      }
      T* dst = h < a.num_heads
                   ? static_cast<T*>(a.q_out) + int64_t(t0 + t) * a.q_out_stride + h * a.head_dim
                   : static_cast<T*>(a.k_out) + int64_t(t0 + t) * a.k_out_stride + (h - a.num_heads) * a.head_dim;
      *reinterpret_cast<Vec<T, VP>*>(dst + d0) = x;
      *reinterpret_cast<Vec<T, VP>*>(dst + d1) = y;
    }
  }
}

template <typename T, int VP>
cudaError_t launch_vp(const RopeParams& p, bool interleaved, cudaStream_t s) {
  const unsigned grid = unsigned((p.a.total_tokens + p.tokens_per_cta - 1) / p.tokens_per_cta);
  if (interleaved)
    rope_kernel<T, VP, true><<<grid, kRopeThreads, 0, s>>>(p);
  else
    rope_kernel<T, VP, false><<<grid, kRopeThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(RopeParams& p, bool interleaved, cudaStream_t s) {
  const RopeArgs& a = p.a;
  // The widest access (up to 16 bytes) that pairs, addresses and strides allow.
  constexpr int kMost = 16 / sizeof(T);
  uint64_t bits = uint64_t(p.rot / 2) * sizeof(T);
  bits |= uint64_t(reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.q_out));
  bits |= uint64_t(a.q_stride | a.q_out_stride) * sizeof(T);
  if (a.num_kv_heads) {
    bits |= uint64_t(reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.k_out));
    bits |= uint64_t(a.k_stride | a.k_out_stride) * sizeof(T);
  }
  int vp = kMost;
  while (vp > 1 && (bits & (vp * sizeof(T) - 1))) vp >>= 1;
  p.unit_log2 = 0;
  while ((2 * vp << p.unit_log2) < a.head_dim) ++p.unit_log2;
  // Tokens per CTA: up to one unrolled pass of units, but enough CTAs for
  // four per SM while the tokens last.
  const int per_token = (a.num_heads + a.num_kv_heads) << p.unit_log2;
  int sms = 0, dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int tpc = kRopeThreads * kRopeUnroll / per_token;
  const int spread = a.total_tokens / (4 * sms);
  tpc = tpc < spread ? tpc : spread;
  p.tokens_per_cta = tpc < 1 ? 1 : (tpc > kRopeMaxTokens ? kRopeMaxTokens : tpc);
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
