// kernels_quant_rows_f32.cu -- the kernels of kernels_quant_rows.cuh for f32 inputs
#include "kernels_quant_rows.cuh"

namespace dgb {

const void* quant_rows_f32(int format, bool norm, int nv, bool bounded) {
  return norm ? rows_kernel_of<float, true>(format, nv, bounded)
              : rows_kernel_of<float, false>(format, nv, bounded);
}

}  // namespace dgb
