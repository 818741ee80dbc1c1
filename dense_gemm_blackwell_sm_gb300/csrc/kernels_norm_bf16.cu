// kernels_norm_bf16.cu -- instances of the block norms' kernels for bf16 rows.
#include "kernels_norm.cuh"

namespace dgb {

cudaError_t norm_forward_bf16(const ffn_norm_t& a, const NormShape& sh, cudaStream_t st) {
  return a.param_dtype == FFN_F32 ? norm_forward<__nv_bfloat16, float>(a, sh, st) : norm_forward<__nv_bfloat16, __nv_bfloat16>(a, sh, st);
}

cudaError_t norm_backward_bf16(const ffn_norm_grad_t& a, const NormGradShape& sh, const NormSums& ws, cudaStream_t st) {
  return a.param_dtype == FFN_F32 ? norm_backward<__nv_bfloat16, float>(a, sh, ws, st) : norm_backward<__nv_bfloat16, __nv_bfloat16>(a, sh, ws, st);
}

}  // namespace dgb
