// The launches of the rotation (rope.cuh).
#include "rope.cuh"

namespace attnmask {
namespace {

template <typename WAY>
__global__ void __launch_bounds__(32 * kRopeWarps, WAY::kPerSM) rope_kernel(const __grid_constant__ RopeParams p) {
  WAY::run(p, blockIdx.x);
}

template <typename T>
cudaError_t launch_t(RopeParams& p, bool interleaved, cudaStream_t s) {
  return with_way<T, false>(p, interleaved, [&](auto way, int64_t ctas) {
    rope_kernel<decltype(way)><<<unsigned(ctas), 32 * kRopeWarps, 0, s>>>(p);
    return cudaGetLastError();
  });
}

}  // namespace

attn_status launch_rope(const RopeArgs& a, const attn_rope_plan& plan, cudaStream_t s) {
  RopeParams p = rope_params(a, plan);
  const cudaError_t e = a.bf16 ? launch_t<__nv_bfloat16>(p, plan.interleaved != 0, s)
                               : launch_t<float>(p, plan.interleaved != 0, s);
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e, "attn_rope launch");
}

}  // namespace attnmask
