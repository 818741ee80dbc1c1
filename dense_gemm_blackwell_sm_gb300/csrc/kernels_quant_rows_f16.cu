// kernels_quant_rows_f16.cu -- the kernels of kernels_quant_rows.cuh for f16 inputs
#include "kernels_quant_rows.cuh"

namespace dgb {

const void* quant_rows_f16(int format, bool norm, int nv) {
  return norm ? rows_kernel_of<__half, true>(format, nv) : rows_kernel_of<__half, false>(format, nv);
}

}  // namespace dgb
