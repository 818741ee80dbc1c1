// quant_launch.h -- internal interface between the C entry points of the low-precision
// operands (quant.cu) and their kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ffn_launch.h"
#include "quant.h"

namespace dgb {

// The pitches below are resolved (never 0).
cudaError_t launch_quant_rows(const quant_rows_t& a, const FfnDevice& dev, cudaStream_t st);
size_t quant_columns_workspace(const quant_rows_t& a);
// `count` arrays, at most kQuantColumnTasks, of one dtype and format
constexpr int kQuantColumnTasks = 4;
cudaError_t launch_quant_columns(const quant_rows_t* args, int count, cudaStream_t st);
cudaError_t launch_quant_norm(const quant_norm_t& a, const FfnDevice& dev, cudaStream_t st);
// whether a linear layer goes in one kernel; if so, its launch
bool fp4_linear_fused(const quant_linear_t& a);
cudaError_t launch_fp4_linear(const quant_linear_t& a, const FfnDevice& dev, cudaStream_t st);
cudaError_t launch_fp4_product(const quant_product_t& a, const FfnDevice& dev, cudaStream_t st);

// elements, scale columns and bytes of a quantised row
inline int64_t width_of(int64_t cols) { return cols < 32 ? 32 : (cols + 31) / 32 * 32; }
inline int64_t scales_of(int64_t width, int32_t format) {
  return format == QUANT_E4M3 ? 0 : format == QUANT_NVFP4 ? width / 16 : width / 32;
}
inline int64_t bytes_of(int64_t width, int32_t format) {
  return format == QUANT_MXFP4 || format == QUANT_NVFP4 ? width / 2 : width;
}

// The first byte past the last element of `rows` rows of `cols` elements, `ld` apart: where rows hold
// nothing, or there are none, the array's start, whatever the pitch.
inline const void* end_of_rows(const void* x, int64_t rows, int64_t ld, int64_t cols, int64_t elem) {
  if (rows <= 0 || cols <= 0) return x;
  return reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(x) + (uintptr_t)(((rows - 1) * ld + cols) * elem));
}
// Whether such rows end within 2^62 bytes, so that the sums above are those of 64 bits: a pitch and a
// number of rows that no memory has are refused.
inline bool rows_fit(int64_t rows, int64_t ld, int64_t cols, int64_t elem) {
  if (rows <= 1) return true;
  return ld <= (((int64_t)1 << 62) / elem - cols) / (rows - 1);
}

}  // namespace dgb
