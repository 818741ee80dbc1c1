// kernels_norm_backward_f16.cu -- instances of the block norms' backward kernels for f16 rows.
#include "kernels_norm_launch.cuh"

namespace dgb {

cudaError_t norm_backward_f16(const ffn_norm_grad_t& a, const NormGradShape& sh, const NormSums& ws,
                         const FfnDevice& dev, cudaStream_t st) {
  return a.param_dtype == FFN_F32 ? norm_backward<__half, float>(a, sh, ws, dev, st) : norm_backward<__half, __half>(a, sh, ws, dev, st);
}

}  // namespace dgb
