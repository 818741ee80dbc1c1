// kernels_norm_f32.cu -- instances of the block norms' kernels for fp32 rows.
#include "kernels_norm.cuh"

namespace dgb {

cudaError_t norm_forward_f32(const ffn_norm_t& a, const NormShape& sh, cudaStream_t st) {
  return norm_forward<float, float>(a, sh, st);
}

cudaError_t norm_backward_f32(const ffn_norm_grad_t& a, const NormGradShape& sh, const NormSums& ws, cudaStream_t st) {
  return norm_backward<float, float>(a, sh, ws, st);
}

}  // namespace dgb
