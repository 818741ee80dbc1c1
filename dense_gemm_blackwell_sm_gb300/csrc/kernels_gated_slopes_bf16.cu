// kernels_gated_slopes_bf16.cu -- instances of the gated projections' products with
// the pre-activations' gradient as epilogue, for bf16.
#include "kernels_gated.cuh"

namespace dgb {

const void* gated_slopes_kernel_bf16(int consumers, int act) {
  return gated_kernel_of<__nv_bfloat16, GATED_SLOPES>(consumers, act);
}

}  // namespace dgb
