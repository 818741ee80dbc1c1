// kernels_gated_slopes_f16.cu -- instances of the gated projections' products with
// the pre-activations' gradient as epilogue, for f16.
#include "kernels_gated.cuh"

namespace dgb {

const void* gated_slopes_kernel_f16(int consumers, int act) {
  return gated_kernel_of<__half, GATED_SLOPES>(consumers, act);
}

}  // namespace dgb
