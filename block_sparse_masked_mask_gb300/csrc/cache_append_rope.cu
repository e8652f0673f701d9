// Rotation and append in one launch: queries are turned (rope.cuh), new keys are turned
// and become e4m3 codes, new values become codes (cache_append.cu).
//
// The queries are most of the bytes, 4 per element against 3 of a key or value, and
// none of them waits for a page; so the launch has two kinds of CTAs, in turn: those that
// take pages have their lookups, one behind the other, under the stream of the rotated
// queries, the others' work.
// Pages: a team of threads owns the new tokens of one page and head, staged in shared
// memory, since a key's partner may be another thread's; the CTA's teams take different heads and
// share the sines and cosines of the page's tokens, a table in shared memory.  The turned
// elements stay in registers, 32 bits each, for their largest magnitude and their codes, so that
// a key goes from fp32 to its code without a rounding to bf16 between.
// Measured, 32 query and 8 key / value heads of 128: 64 single tokens 4.7 us, 32 trees of 17 to 64
// nodes 14 us (4.2 at the rate of a copy), 12 prompts of 257 to 2048 tokens, half of each head turned, pages of 32,
// 55 us (42); 5 prompts of 900 to 4001 in fp32, 16 and 16 heads of 64, 57 us (35).  One token each is lookups one
// behind the other.  The trees are 1024 CTAs for pages, of which 456 run at a time (and 224 find no page), each with that
// chain and its loads, turns, maximum and stores once, beside 160 for the queries; fewer CTAs of longer chains
// take longer (launch_t).  Prompts issue in half of their cycles (58%, fp32 47%): sines, roundings and the
// maximum beside the copies, with 24 warps per SM, where three CTAs fit its shared memory.  They do not with
// pages of 128 x 128 turned whole, whose angles take 64 KB beside 32 KB of elements (fp32 64): two CTAs per SM, or
// one, the queries' among them, and keys are turned twice (the 12 prompts turned whole, pages of 32 / 64 / 128:
// 59 / 61 / 86 us; 128 in fp32 163, 81 at the rate of a copy).
#include <type_traits>

#include "cache_rows.cuh"
#include "rope.cuh"

namespace attnmask {
namespace {

constexpr int kThreads = 32 * kRopeWarps;
constexpr int kPiece = 8;    // elements of a chunk, a thread's unit
constexpr int kPieces = 4;   // chunks of a thread, while a team has room to grow

struct AppendRopeParams {
  RopeParams rope;  // of the queries; the keys' too
  AppendArgs kv;
  bool interleaved;
  int team_log2, pieces;   // threads of a team, chunks of each
  int groups, key_groups;  // CTAs of a page: those of its keys, then of its values
  int loops;               // heads that a team takes in turn
  int page_ctas;
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// Eight elements in shared memory: 16-byte part p of a thread's j-th chunk at
// ((j * PARTS + p) * kThreads + thread) * 16.
template <typename T>
struct Staged {
  static constexpr int PARTS = sizeof(T) * kPiece / 16, PER = 16 / sizeof(T);
  __device__ static int at(int j, int thread, int e) {  // element e, in elements
    return ((j * PARTS + e / PER) * kThreads + thread) * PER + e % PER;
  }
  __device__ static void get(const T* staged, int j, int thread, float (&f)[kPiece]) {
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      const uint4 v = *reinterpret_cast<const uint4*>(staged + at(j, thread, p * PER));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        if constexpr (sizeof(T) == 4) f[p * PER + e] = __uint_as_float(w[e]);
        else f[p * PER + e] = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
      }
    }
  }
  // The same turned: dimensions d .. d + 7 of a token whose (cos, sin) are at `cs`.  A partner
  // half the rotated dimensions away lies in the chunk of another thread of the team.
  __device__ static void turned(const T* staged, int j, int d, int rot, bool interleaved, const float2* cs,
                                float (&f)[kPiece]) {
    get(staged, j, threadIdx.x, f);
    if (d >= rot) return;
    const int half = rot / 2;
    if (interleaved) {
#pragma unroll
      for (int e = 0; e < kPiece; e += 2) {
        if (d + e >= rot) continue;
        const float2 c = cs[(d + e) / 2];
        const float x = f[e], y = f[e + 1];
        f[e] = turned_x(x, y, c);
        f[e + 1] = turned_y(x, y, c);
      }
    } else if (half % kPiece == 0) {
      const bool low = d < half;
      float other[kPiece];
      get(staged, j, int(threadIdx.x) + (low ? half : -half) / kPiece, other);
      cs += low ? d : d - half;
#pragma unroll
      for (int e = 0; e < kPiece; ++e)
        f[e] = low ? turned_x(f[e], other[e], cs[e]) : turned_y(other[e], f[e], cs[e]);
    } else {
#pragma unroll
      for (int e = 0; e < kPiece; ++e) {
        if (d + e >= rot) continue;
        const bool low = d + e < half;
        const int to = d + e + (low ? half : -half);
        const float y = to_float(staged[at(j, int(threadIdx.x) + ((to & -kPiece) - d) / kPiece, to % kPiece)]);
        const float2 c = cs[low ? d + e : d + e - half];
        f[e] = low ? turned_x(f[e], y, c) : turned_y(y, f[e], c);
      }
    }
  }
};

// Pages that sequence b's new tokens touch; 0 where its numbers cannot be used.
__device__ __forceinline__ int new_pages(const AppendArgs& a, int b) {
  const CacheView& c = a.cache;
  if (b >= c.batch) return 0;
  const int q0 = a.cu[b], q1 = a.cu[b + 1], len = a.lens[b], n = q1 - q0;
  const bool good = q0 >= 0 && q1 > q0 && q1 <= a.total_tokens && (b > 0 || q0 == 0) && n <= a.max_new && len >= n &&
                    len <= c.max_pages << c.page_log2;
  return good ? ((len - 1) >> c.page_log2) - ((len - n) >> c.page_log2) + 1 : 0;
}

template <typename T>
__device__ __forceinline__ void append_pages(const AppendRopeParams& p, int block) {
  using S = Staged<T>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float warp_max[kRopeWarps];
  const AppendArgs& a = p.kv;
  const CacheView& c = a.cache;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ int found[2], place[128];  // place: the new tokens' positions
  const int pos = block / p.groups, group = block % p.groups;
  if (warp == 0) {
    // the sequence that this page of the line belongs to, 64 at a time, two neighbours per lane
    int b = 0, before = 0;
#pragma unroll 1
    for (; b < c.batch; b += 64) {
      const int n0 = new_pages(a, b + 2 * lane), n1 = new_pages(a, b + 2 * lane + 1);
      int sum = n0 + n1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, before + sum > pos);
      if (past) {
        const int at = __ffs(past) - 1;
        before += __shfl_sync(0xffffffffu, sum - n0 - n1, at);
        const int skip = __shfl_sync(0xffffffffu, n0, at);
        b += 2 * at;
        if (before + skip <= pos) {
          before += skip;
          ++b;
        }
        break;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) {
      found[0] = b;
      found[1] = pos - before;
    }
  } else if (block == p.page_ctas - 1 && warp == 1) {
    // what is wrong with the sequences is noted once
#pragma unroll 1
    for (int x = lane; x < c.batch; x += 32) {
      SeqRows r;
      if (load_rows(a.cu, a.lens, x, a.total_tokens, a.max_new, c.max_pages << c.page_log2, c.status, r) && r.len < r.n)
        atomicOr(c.status, kErrHeld);
    }
  }
  __syncthreads();
  const int b = found[0];
  if (b >= c.batch) return;
  const int q0 = a.cu[b], len = a.lens[b], held = len - (a.cu[b + 1] - q0);
  const int i = (held >> c.page_log2) + found[1];      // this CTA's page of the sequence
  const int start = i << c.page_log2;                  // its first token
  const int first = max(held - start, 0), last = min(len - start, 1 << c.page_log2);  // slots [first, last) are new
  const int number = __ldg(c.table + int64_t(b) * c.max_pages + i);  // needed only behind the loads
  const int row_log2 = 31 - __clz(c.head_dim / kPiece), mask = (1 << row_log2) - 1;  // chunks of a token
  const int team = threadIdx.x >> p.team_log2, tid = threadIdx.x & ((1 << p.team_log2) - 1), teams = kThreads >> p.team_log2;
  const bool keys = group < p.key_groups;
  const int head0 = (keys ? group : group - p.key_groups) * p.loops * teams + team;
  const int fill = ((last - first) << row_log2);                         // chunks of a head
  const int turns = (fill + (1 << p.team_log2) - 1) >> p.team_log2;      // of the team
  const T* src = static_cast<const T*>(keys ? a.k : a.v);
  const int64_t stride = keys ? a.k_stride : a.v_stride;
  T* const staged = reinterpret_cast<T*>(smem);
  float2* const cs = reinterpret_cast<float2*>(smem + p.pieces * S::PARTS * kThreads * 16);  // [new slot][pair]
  const int pairs = p.rope.rot / 2;
  const bool fine = in_pool(c, number);

  auto stage = [&](int l) {
    const int h = head0 + l * teams;
    const bool on = h < c.heads;
#pragma unroll 1
    for (int j = 0; j < turns; ++j) {
      const int ch = (j << p.team_log2) + tid;
      const bool here = on && ch < fill;
      const T* from = src + (here ? (q0 + start + first - held + (ch >> row_log2)) * stride + int64_t(h) * c.head_dim + (ch & mask) * kPiece : 0);
#pragma unroll
      for (int x = 0; x < S::PARTS; ++x)
        copy16_async(uint32_t(__cvta_generic_to_shared(staged + S::at(j, threadIdx.x, x * S::PER))), from + x * S::PER, here);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  stage(0);
#pragma unroll 1
  for (int l = 0; l < p.loops; ++l) {
    const int h = head0 + l * teams;
    const bool on = h < c.heads;
    if (l == 0 && keys) {
      if (int(threadIdx.x) < last - first)
        place[threadIdx.x] = p.rope.a.positions ? p.rope.a.positions[q0 + start + first - held + threadIdx.x] : start + first + int(threadIdx.x);
      __syncthreads();
      // 64 threads a token, four tokens at a time
      const int pair = threadIdx.x & 63;
      const uint64_t theta = p.rope.turn[min(pair, pairs - 1)];
      if (pair < pairs) {
#pragma unroll 2
        for (int x = threadIdx.x >> 6; x < last - first; x += kThreads / 64) {
          const int64_t turn = int64_t(uint64_t(int64_t(place[x])) * theta);
          float sn, cn;
          sincospif(float(int32_t(turn >> 32)) * 0x1p-31f, &sn, &cn);
          cs[x * pairs + pair] = make_float2(cn * p.rope.factor, sn * p.rope.factor);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();  // partners and angles are other threads'
    if (!fine) {
      if (threadIdx.x == 0) atomicOr(c.status, kErrBadPage);
      return;
    }
    const int64_t at = int64_t(number) * c.heads + (on ? h : 0);
    uint8_t* const codes = (keys ? c.k_pages : c.v_pages) + (at << c.page_log2) * c.head_dim;
    float* const scale = (keys ? c.k_scale : c.v_scale) + at;
    // The elements of kPieces turns from j0 on, turned.
    float f[kPieces][kPiece];
    auto get = [&](int j0) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        if (j0 + j >= turns) break;
        const int ch = ((j0 + j) << p.team_log2) + tid;
        if (keys && ch < fill) S::turned(staged, j0 + j, (ch & mask) * kPiece, p.rope.rot, p.interleaved, cs + (ch >> row_log2) * pairs, f[j]);
        else S::get(staged, j0 + j, threadIdx.x, f[j]);
      }
    };
    float amax = 0.f;
#pragma unroll 1
    for (int j0 = 0; j0 < turns; j0 += kPieces) {
      get(j0);
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        if (j0 + j >= turns) break;
#pragma unroll
        for (int e = 0; e < kPiece; ++e) {
          const float m = fabsf(f[j][e]);
          if (m < INFINITY) amax = fmaxf(amax, m);  // false for NaN too
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) warp_max[warp] = amax;
    const float was = first > 0 ? *scale : 0.f;  // read before the team's first thread replaces it
    __syncthreads();
    // the next head's elements, while this one's, held in registers, are rounded and stored
    if (turns <= kPieces && l + 1 < p.loops) stage(l + 1);
    const int warps = 1 << (p.team_log2 - 5);  // of the team
    for (int w = 0; w < warps; ++w) amax = fmaxf(amax, warp_max[team * warps + w]);
    int e = scale_exponent(amax);
    if (first > 0) {
      // a scale outside the range (the caller's memory) is taken into it
      const int e0 = max(kScaleExpMin, min(kScaleExpMax, exponent_of(was)));
      if (e0 < e && on) {
        const int bytes = first * c.head_dim;  // codes of the earlier tokens
#pragma unroll 1
        for (int x = tid * 8; x < bytes; x += 8 << p.team_log2) {
          uint2 w = *reinterpret_cast<uint2*>(codes + x);
          w.x = rescale4(w.x, e - e0);
          w.y = rescale4(w.y, e - e0);
          *reinterpret_cast<uint2*>(codes + x) = w;
        }
      }
      e = max(e, e0);
    }
    const float inv = pow2f(-e);
#pragma unroll 1
    for (int j0 = 0; j0 < turns; j0 += kPieces) {
      if (turns > kPieces) get(j0);  // (a page of 128 x 128: turned again)
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int ch = ((j0 + j) << p.team_log2) + tid;
        if (!on || ch >= fill) break;
        uint2 w;
        w.x = e4m3_pair(f[j][0] * inv, f[j][1] * inv) | (e4m3_pair(f[j][2] * inv, f[j][3] * inv) << 16);
        w.y = e4m3_pair(f[j][4] * inv, f[j][5] * inv) | (e4m3_pair(f[j][6] * inv, f[j][7] * inv) << 16);
        *reinterpret_cast<uint2*>(codes + int64_t((first << row_log2) + ch) * kPiece) = w;
      }
    }
    if (tid == 0 && on) *scale = pow2f(e);
    if (turns > kPieces && l + 1 < p.loops) {
      __syncthreads();  // this head's elements have been read
      stage(l + 1);
    }
  }
}

template <typename WAY>
__global__ void __launch_bounds__(kThreads, 3)  // (with 4 registers are spilled: prompts 54.9 us, 54.6)
    append_rope_kernel(const __grid_constant__ AppendRopeParams p) {
  // one of each kind in turn, then the rest of the longer kind
  const int x = blockIdx.x, pages = p.page_ctas, rows = int(gridDim.x) - pages, both = 2 * min(pages, rows);
  const bool page = x < both ? (x & 1) == 0 : pages > rows;
  const int mine = x < both ? x >> 1 : x - both / 2;
  if (page) append_pages<typename WAY::T>(p, mine);
  else WAY::run(p.rope, mine);
}

template <typename T>
cudaError_t launch_t(AppendRopeParams& p, cudaStream_t s) {
  const AppendArgs& a = p.kv;
  const CacheView& c = a.cache;
  const int page_size = 1 << c.page_log2, most = a.max_new < page_size ? a.max_new : page_size;  // new tokens of a page
  p.team_log2 = 5;
  while (p.team_log2 < 8 && (kPieces * kPiece << p.team_log2) < most * c.head_dim) ++p.team_log2;
  p.pieces = (most * c.head_dim / kPiece + (1 << p.team_log2) - 1) >> p.team_log2;
  const int teams = kThreads >> p.team_log2;
  // n tokens touch at most (n + page_size - 2) / page_size + 1 pages; all of them
  // together at most T / page_size whole ones and two more per sequence
  const int64_t each = (int64_t(a.max_new) + page_size - 2) / page_size + 1;
  const int64_t bound = a.total_tokens / page_size + 2ll * c.batch;
  const int64_t pages = each * c.batch < bound ? each * c.batch : bound;
  // Heads in turn share a table of angles, and one's elements are fetched while another's are stored; but few CTAs of
  // long chains begin and end unevenly.  As many as leave 608 CTAs for the pages (by 1 / 2 / 4 / 8: 32 trees
  // 14.3 / 15.3 / 18.6 / 26.4 us, 12 prompts 60.8 / 56.7 / 54.7 / 54.8, 5 in fp32 70.6 / 63.2 / 57.1 / 56.3).
  p.loops = 1;
  while (p.loops * teams < c.heads && pages * ((c.heads + 2 * p.loops * teams - 1) / (2 * p.loops * teams)) * 2 >= 4 * 152) p.loops *= 2;
  p.key_groups = (c.heads + p.loops * teams - 1) / (p.loops * teams);
  p.groups = 2 * p.key_groups;
  p.page_ctas = int(pages * p.groups);
  const int smem = p.pieces * Staged<T>::PARTS * kThreads * 16 + most * (p.rope.rot / 2) * int(sizeof(float2));
  // The limit is the kernel's, so every call sets the same one, the most that any asks for: by its own need, another host
  // thread could lower it between here and the launch.
  constexpr int kMostSmem = 128 * 128 * int(sizeof(T)) + 128 * ATTN_ROPE_MAX_PAIRS * int(sizeof(float2));
  auto launch = [&](auto way, int64_t ctas) {
    auto kernel = append_rope_kernel<decltype(way)>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e != cudaSuccess) return e;
    kernel<<<unsigned(p.page_ctas + ctas), kThreads, smem, s>>>(p);
    return cudaGetLastError();
  };
  if (p.rope.a.num_heads == 0) return launch(RopeWay<T, 0, 4, true>{}, 0);
  return with_way<T, true>(p.rope, p.interleaved, launch);
}

}  // namespace

attn_status launch_cache_append_rope(const AppendArgs& kv, const RopeArgs& q, const attn_rope_plan& plan, cudaStream_t s) {
  AppendRopeParams p;
  p.rope = rope_params(q, plan);
  p.rope.check = RopeCheck{kv.max_new, kv.cache.max_pages << kv.cache.page_log2, kv.cache.status};
  p.kv = kv;
  p.interleaved = plan.interleaved != 0;
  const cudaError_t e = kv.bf16 ? launch_t<__nv_bfloat16>(p, s) : launch_t<float>(p, s);
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_cache_append_rope launch");
}

}  // namespace attnmask
