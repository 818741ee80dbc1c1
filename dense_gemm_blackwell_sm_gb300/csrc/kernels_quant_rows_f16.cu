// kernels_quant_rows_f16.cu -- the kernels of kernels_quant_rows.cuh for f16 inputs
#include "kernels_quant_rows.cuh"

namespace dgb {

const void* quant_rows_f16(int format, bool norm, int nv, bool bounded) {
  return norm ? rows_kernel_of<__half, true>(format, nv, bounded)
              : rows_kernel_of<__half, false>(format, nv, bounded);
}

}  // namespace dgb
