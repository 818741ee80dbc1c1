// kernels_norm_forward_bf16.cu -- instances of the block norms' forward kernels for bf16 rows.
#include "kernels_norm_launch.cuh"

namespace dgb {

cudaError_t norm_forward_bf16(const ffn_norm_t& a, const NormShape& direct, const NormShape* ring,
                         const FfnDevice& dev, cudaStream_t st) {
  return a.param_dtype == FFN_F32 ? norm_forward<__nv_bfloat16, float>(a, direct, ring, dev, st)
                                    : norm_forward<__nv_bfloat16, __nv_bfloat16>(a, direct, ring, dev, st);
}

}  // namespace dgb
