// kernels_norm_backward_bf16.cu -- instances of the block norms' backward kernels for bf16 rows.
#include "kernels_norm_launch.cuh"

namespace dgb {

cudaError_t norm_backward_bf16(const ffn_norm_grad_t& a, const NormGradShape& sh, const NormSums& ws,
                         const FfnDevice& dev, cudaStream_t st) {
  return a.param_dtype == FFN_F32 ? norm_backward<__nv_bfloat16, float>(a, sh, ws, dev, st) : norm_backward<__nv_bfloat16, __nv_bfloat16>(a, sh, ws, dev, st);
}

}  // namespace dgb
