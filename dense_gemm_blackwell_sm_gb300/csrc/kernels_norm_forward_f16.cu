// kernels_norm_forward_f16.cu -- instances of the block norms' forward kernels for f16 rows.
#include "kernels_norm_launch.cuh"

namespace dgb {

cudaError_t norm_forward_f16(const ffn_norm_t& a, const NormShape& direct, const NormShape* ring,
                         const FfnDevice& dev, cudaStream_t st) {
  return a.param_dtype == FFN_F32 ? norm_forward<__half, float>(a, direct, ring, dev, st)
                                    : norm_forward<__half, __half>(a, direct, ring, dev, st);
}

}  // namespace dgb
