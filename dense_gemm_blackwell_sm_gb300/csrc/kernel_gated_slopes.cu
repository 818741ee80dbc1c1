// kernel_gated_slopes.cu -- the gradient of the gated projections' pre-activations
// from kept ones: dgu = [dh * u * act'(g), dh * act(g)].
//
// dgu is rounded once to the inputs' type: it is the Tensor Core's operand next (see
// kernels_gated.cuh for what that costs in exactness).
//
// A pass over memory: 3 values read and 2 written per hidden feature and token.  A
// CTA takes a run of a row's columns, a thread 8 of them, with 16-byte accesses where
// they start on a boundary, else by element (a warp's elements are neighbours' then
// too, and L1 and L2 join them).  2048 x 14336 bf16: 50 us, 5.8 TB/s.
#include <type_traits>

#include "ffn_common.cuh"
#include "gated.h"
#include "launch.h"

namespace dgb {

namespace {

constexpr int GS_THREADS = 256;

__device__ __forceinline__ bool on_boundary(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// 8 columns from c on, those below F
template <typename T>
__device__ __forceinline__ void load8(float (&v)[8], const T* p, int n) {
  if (n >= 8 && on_boundary(p)) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      if constexpr (std::is_same<T, __half>::value) {
        f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      } else {
        f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      }
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e < n ? to_f32(p[e]) : 0.f;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8], int n) {
  if (n >= 8 && on_boundary(p)) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) p[e] = from_f32<T>(v[e]);
}

template <typename T, int ACT>
__global__ void __launch_bounds__(GS_THREADS) k_gated_slopes(const __grid_constant__ ffn_gated_grad_t a) {
  wait_for_prior_kernel();
  const int F = (int)a.F, c = ((int)blockIdx.x * GS_THREADS + (int)threadIdx.x) * 8, n = F - c;
  if (n <= 0) return;
  for (int64_t r = blockIdx.y; r < a.M; r += gridDim.y) {
    const T* gu = static_cast<const T*>(a.gu) + r * a.ld_gu + c;
    T* dgu = static_cast<T*>(a.dgu) + r * a.ld_dgu + c;
    float g[8], u[8], dh[8], dg[8];
    load8(g, gu, n);
    load8(u, gu + F, n);
    load8(dh, static_cast<const T*>(a.dh) + r * a.ld_dh + c, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float act, slope;
      act_and_slope<ACT>(g[e], act, slope);
      dg[e] = dh[e] * u[e] * slope;
      u[e] = dh[e] * act;
    }
    store8(dgu, dg, n);
    store8(dgu + F, u, n);
  }
  let_next_kernel_start();
}

template <typename T>
const void* slopes_kernel(int act) {
  switch (act) {
    case EPI_ACT_RELU: return (const void*)k_gated_slopes<T, EPI_ACT_RELU>;
    case EPI_ACT_SILU: return (const void*)k_gated_slopes<T, EPI_ACT_SILU>;
    case EPI_ACT_GELU_TANH: return (const void*)k_gated_slopes<T, EPI_ACT_GELU_TANH>;
    case EPI_ACT_GELU_ERF: return (const void*)k_gated_slopes<T, EPI_ACT_GELU_ERF>;
    default: return (const void*)k_gated_slopes<T, EPI_ACT_NONE>;
  }
}

}  // namespace

cudaError_t launch_gated_slopes(const ffn_gated_grad_t& a, int num_sms, cudaStream_t st) {
  LaunchSpec s;
  s.func = a.dtype == FFN_BF16 ? slopes_kernel<__nv_bfloat16>(a.activation) : slopes_kernel<__half>(a.activation);
  const int64_t columns = (a.F + GS_THREADS * 8 - 1) / (GS_THREADS * 8);
  // enough rows at once for 16 CTAs per SM
  const int64_t rows = ((int64_t)num_sms * 16 + columns - 1) / columns;
  s.grid = dim3((unsigned)columns, (unsigned)(a.M < rows ? a.M : rows < 65535 ? rows : 65535), 1);
  s.block = dim3(GS_THREADS, 1, 1);
  s.pdl = true;
  ffn_gated_grad_t copy = a;
  void* args[] = {&copy};
  return launch_spec(s, args, st);
}

}  // namespace dgb
