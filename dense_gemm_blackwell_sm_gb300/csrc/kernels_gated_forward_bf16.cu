// kernels_gated_forward_bf16.cu -- instances of the gated projections for bf16.
#include "kernels_gated.cuh"

namespace dgb {

const void* gated_forward_kernel_bf16(int consumers, int act) {
  return gated_kernel_of<__nv_bfloat16, GATED_FORWARD>(consumers, act);
}

}  // namespace dgb
