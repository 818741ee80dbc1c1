// kernels_gated_forward_f16.cu -- instances of the gated projections for f16.
#include "kernels_gated.cuh"

namespace dgb {

const void* gated_forward_kernel_f16(int consumers, int act) {
  return gated_kernel_of<__half, GATED_FORWARD>(consumers, act);
}

}  // namespace dgb
