// kernels_norm_f16.cu -- instances of the block norms' kernels for f16 rows.
#include "kernels_norm.cuh"

namespace dgb {

cudaError_t norm_forward_f16(const ffn_norm_t& a, const NormShape& sh, cudaStream_t st) {
  return a.param_dtype == FFN_F32 ? norm_forward<__half, float>(a, sh, st) : norm_forward<__half, __half>(a, sh, st);
}

cudaError_t norm_backward_f16(const ffn_norm_grad_t& a, const NormGradShape& sh, const NormSums& ws, cudaStream_t st) {
  return a.param_dtype == FFN_F32 ? norm_backward<__half, float>(a, sh, ws, st) : norm_backward<__half, __half>(a, sh, ws, st);
}

}  // namespace dgb
