// kernel_gated_join.cu -- dx of the gated projections from the sums of its reduction's
// slices: added in their order in fp32 and rounded once.  A pass over memory (4 bytes per
// slice and element read, 2 written), the sums mostly still in L2.
#include <type_traits>

#include "ffn_common.cuh"
#include "gated.h"
#include "launch.h"

namespace dgb {

namespace {

constexpr int GJ_THREADS = 256;

// A thread takes 8 columns of a row at a time (K is a multiple of 8).
template <typename T>
__global__ void __launch_bounds__(GJ_THREADS) k_gated_join(const __grid_constant__ ffn_gated_grad_t a, int slices) {
  wait_for_prior_kernel();
  let_next_kernel_start();
  const int64_t groups = a.M * (a.K / 8), step = (int64_t)gridDim.x * GJ_THREADS;
  const float4* sums = static_cast<const float4*>(a.workspace);
  for (int64_t i = (int64_t)blockIdx.x * GJ_THREADS + threadIdx.x; i < groups; i += step) {
    float v[8] = {};
#pragma unroll 4
    for (int s = 0; s < slices; ++s) {
      const float4 lo = sums[2 * (s * groups + i)], hi = sums[2 * (s * groups + i) + 1];
      v[0] += lo.x, v[1] += lo.y, v[2] += lo.z, v[3] += lo.w;
      v[4] += hi.x, v[5] += hi.y, v[6] += hi.z, v[7] += hi.w;
    }
    const int64_t row = i / (a.K / 8);
    T* to = static_cast<T*>(a.dx) + row * a.ld_dx + (i - row * (a.K / 8)) * 8;
    alignas(16) T o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = from_f32<T>(v[e]);
    if ((reinterpret_cast<uintptr_t>(to) & 15u) == 0) {
      *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(o);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) to[e] = o[e];
    }
  }
}

}  // namespace

cudaError_t launch_gated_join(const ffn_gated_grad_t& a, int slices, int num_sms, cudaStream_t st) {
  LaunchSpec s;
  s.func = a.dtype == FFN_BF16 ? (const void*)k_gated_join<__nv_bfloat16> : (const void*)k_gated_join<__half>;
  const int64_t ctas = (a.M * (a.K / 8) + GJ_THREADS - 1) / GJ_THREADS;
  s.grid = dim3((unsigned)(ctas < 8 * num_sms ? ctas : 8 * num_sms), 1, 1);
  s.block = dim3(GJ_THREADS, 1, 1);
  s.pdl = true;
  ffn_gated_grad_t copy = a;
  void* args[] = {&copy, &slices};
  return launch_spec(s, args, st);
}

}  // namespace dgb
