// kernels_norm_forward_f32.cu -- instances of the block norms' forward kernels for f32 rows.
#include "kernels_norm_launch.cuh"

namespace dgb {

cudaError_t norm_forward_f32(const ffn_norm_t& a, const NormShape& direct, const NormShape* ring,
                         const FfnDevice& dev, cudaStream_t st) {
  return norm_forward<float, float>(a, direct, ring, dev, st);
}

}  // namespace dgb
