// kernel_gated_slopes.cu -- the gradient of the gated projections' pre-activations
// from kept ones: dgu = [dh * u * act'(g), dh * act(g)], a pass over memory.
#include "ffn_common.cuh"
#include "gated.h"

namespace dgb {

namespace {

template <typename T, int ACT>
__global__ void __launch_bounds__(256) k_gated_slopes(ffn_gated_grad_t a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.M * a.F) return;
  const int64_t r = i / a.F, c = i - r * a.F;
  const T* gu = static_cast<const T*>(a.gu) + r * a.ld_gu + c;
  T* dgu = static_cast<T*>(a.dgu) + r * a.ld_dgu + c;
  const float dh = to_f32(static_cast<const T*>(a.dh)[r * a.ld_dh + c]);
  float act, slope;
  act_and_slope<ACT>(to_f32(gu[0]), act, slope);
  dgu[0] = from_f32<T>(dh * to_f32(gu[a.F]) * slope);
  dgu[a.F] = from_f32<T>(dh * act);
}

template <typename T, int ACT>
cudaError_t slopes(const ffn_gated_grad_t& a, cudaStream_t st) {
  k_gated_slopes<T, ACT><<<(unsigned)((a.M * a.F + 255) / 256), 256, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t slopes_of(const ffn_gated_grad_t& a, cudaStream_t st) {
  switch (a.activation) {
    case EPI_ACT_RELU: return slopes<T, EPI_ACT_RELU>(a, st);
    case EPI_ACT_SILU: return slopes<T, EPI_ACT_SILU>(a, st);
    case EPI_ACT_GELU_TANH: return slopes<T, EPI_ACT_GELU_TANH>(a, st);
    case EPI_ACT_GELU_ERF: return slopes<T, EPI_ACT_GELU_ERF>(a, st);
    default: return slopes<T, EPI_ACT_NONE>(a, st);
  }
}

}  // namespace

cudaError_t launch_gated_slopes(const ffn_gated_grad_t& a, int, cudaStream_t st) {
  return a.dtype == FFN_BF16 ? slopes_of<__nv_bfloat16>(a, st) : slopes_of<__half>(a, st);
}

}  // namespace dgb
