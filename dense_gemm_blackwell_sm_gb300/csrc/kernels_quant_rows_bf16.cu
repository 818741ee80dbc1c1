// kernels_quant_rows_bf16.cu -- the kernels of kernels_quant_rows.cuh for bf16 inputs
#include "kernels_quant_rows.cuh"

namespace dgb {

const void* quant_rows_bf16(int format, bool norm, int nv, bool bounded) {
  return norm ? rows_kernel_of<__nv_bfloat16, true>(format, nv, bounded)
              : rows_kernel_of<__nv_bfloat16, false>(format, nv, bounded);
}

}  // namespace dgb
