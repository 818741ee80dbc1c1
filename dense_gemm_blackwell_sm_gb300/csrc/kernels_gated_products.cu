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

int gated_stages(int consumers, int a_rows, int hw) {
  const size_t room = 232448 - 1024 - GT_STAGING - GT_CTRL;  // 227 KB per CTA
  const int n = (int)(room / ((size_t)(consumers * a_rows + hw) * 128));
  return n < GT_MAX_STAGES ? n : GT_MAX_STAGES;
}

size_t gated_smem_bytes(int consumers, int a_rows, int hw, int stages) {
  return 1024 + (size_t)stages * (size_t)(consumers * a_rows + hw) * 128 + GT_STAGING + GT_CTRL;
}

static_assert(kGatedThreads == GT_THREADS, "launch shape");
static_assert(GT_STAGING >= GT_A_BYTES, "an MMA on a short last stage reads into the staging space");
static_assert((2 * GT_MAX_STAGES + 5) * 8 + 12 <= GT_CTRL, "barriers");

}  // namespace dgb
