// kernels_gated_products.cu -- instances of the two products of the gated
// projections' backward pass, and the choice among all instances.
#include "kernels_gated.cuh"

namespace dgb {

const void* gated_forward_kernel_f16(int consumers, int act);
const void* gated_forward_kernel_bf16(int consumers, int act);
const void* gated_slopes_kernel_f16(int consumers, int act);
const void* gated_slopes_kernel_bf16(int consumers, int act);

const void* gated_forward_kernel(bool bf16, int consumers, int act) {
  return bf16 ? gated_forward_kernel_bf16(consumers, act) : gated_forward_kernel_f16(consumers, act);
}

const void* gated_slopes_kernel(bool bf16, int consumers, int act) {
  return bf16 ? gated_slopes_kernel_bf16(consumers, act) : gated_slopes_kernel_f16(consumers, act);
}

const void* gated_products_kernel(bool bf16, int consumers) {
  return bf16 ? gated_kernel<__nv_bfloat16, GATED_PRODUCTS, 0>(consumers)
              : gated_kernel<__half, GATED_PRODUCTS, 0>(consumers);
}

size_t gated_smem_bytes(int consumers, int stages) {
  return 1024 + (size_t)stages * (consumers * GT_A_BYTES + GT_B_BYTES) + GT_STAGING + GT_CTRL;
}

static_assert(kGatedThreads == GT_THREADS, "launch shape");

}  // namespace dgb
