// kernels_norm_backward_f32.cu -- instances of the block norms' backward kernels for f32 rows.
#include "kernels_norm_launch.cuh"

namespace dgb {

cudaError_t norm_backward_f32(const ffn_norm_grad_t& a, const NormGradShape& sh, const NormSums& ws,
                         const FfnDevice& dev, cudaStream_t st) {
  return norm_backward<float, float>(a, sh, ws, dev, st);
}

}  // namespace dgb
