// quant_rows.cu -- host side of the kernels in kernels_quant_rows.cuh: threads per row.
#include <algorithm>

#include "kernels_quant_rows.cuh"
#include "launch.h"
#include "quant_launch.h"

namespace dgb {

namespace {

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// 2: rows start on 32-byte boundaries, 1: on 16-byte ones, 0: neither
int alignment_of(const void* p, int64_t pitch_bytes) {
  const uintptr_t bits = p == nullptr ? 0 : reinterpret_cast<uintptr_t>(p) | (uintptr_t)pitch_bytes;
  return (bits & 31u) == 0 ? 2 : (bits & 15u) == 0 ? 1 : 0;
}

cudaError_t launch(QuantRowsParams& p, int32_t dtype, int32_t format, bool norm, int num_sms, cudaStream_t st) {
  const int64_t width = width_of(p.cols), scales = scales_of(width, format);
  p.chunks = (int32_t)(width / 16);
  p.blocks = (int32_t)up(scales, 4);
  p.all_chunks = scales == 0 ? p.chunks : (int32_t)(p.blocks * 4 * (format == QUANT_NVFP4 ? 1 : 2));
  p.all_rows = scales == 0 ? p.rows : (uint32_t)(up(p.rows, 128) * 128);
  // One run of 16 columns a thread up to 512 threads a row, then up to four.  4-bit rows that
  // fill the device take two from 64 runs on: half as many threads meet for the row's scale and
  // share a scale word (8192 x 4096 bf16 to NVFP4 20.5 -> 18.0 us, to MXFP4 16.9 -> 15.4; to
  // MXFP8 18.6 -> 20.0, a norm to NVFP4 43.5 -> 47.6, and rows off 16-byte boundaries, 8192 x 4095 to
  // MXFP4, 22.5 -> 25.1, so these keep one).
  int nv = 1;
  const bool four = format == QUANT_MXFP4 || format == QUANT_NVFP4;
  if (four && !norm && p.vec != 0 && p.chunks >= 64 && (int64_t)p.chunks * p.rows >= (int64_t)num_sms * 2048) nv = 2;
  // (a norm's longer rows take four: two CTAs of 256 threads fit an SM where one of 512 with two runs a
  // thread does, 2000 x 16384 bf16 45 us and 49)
  while (nv < 4 && up(p.chunks, nv) > 512) nv *= norm ? 4 : 2;
  const int threads = (int)std::min<int64_t>(512, up(up(p.chunks, nv), 32) * 32);
  const int rows = std::max(1, (nv == 2 ? 128 : 256) / threads);
  // NVFP4's two runs in 72 registers a thread or in the 99 they need: many rows of 160 to 448 threads take
  // the 72, which let a CTA more stand on an SM (two of 448 threads and not one), free and bounded, us:
  // 4096 x 5120 12.9 and 13.0, 8192 x 5120 23.2 and 22.3, 4096 x 6144 16.5 and 14.8, 8192 x 8192 34.7 and 33.0, 4096 x
  // 10240 28.8 and 23.1, 4096 x 14336 33.7 and 29.6.  Others lose by it: 8192 x 4096 19.1 and 19.7 (128
  // threads), 4096 x 15360 35.1 and 37.2 (480: one CTA either way), 1024 x 14336 10.3 and 10.5, 1024 x 8192 6.7 and
  // 7.0, while 1500 x 10240 gains (12.3 and 10.2).  With a linear layer's gradient around them, 8192 x 10240 x
  // 2048 289 and 268, 8192 x 12288 x 512 221 and 215, 4096 x 12288 x 4096 268 and 271, 4096 x 14336 x 4096 305 and 310.
  const bool bounded = threads >= 160 && threads <= 448 && p.rows >= 8u * (uint32_t)num_sms;
  LaunchSpec s;
  s.func = dtype == FFN_F32    ? quant_rows_f32(format, norm, nv, bounded)
           : dtype == FFN_BF16 ? quant_rows_bf16(format, norm, nv, bounded)
                               : quant_rows_f16(format, norm, nv, bounded);
  int resident = 0;
  const cudaError_t e = resident_ctas(s.func, threads * rows, 0, 0, &resident);
  if (e != cudaSuccess) return e;
  s.grid = dim3((unsigned)std::min<int64_t>(up(p.all_rows, rows), (int64_t)num_sms * std::max(1, resident)), 1, 1);
  s.block = dim3((unsigned)threads, (unsigned)rows, 1);
  s.pdl = true;
  void* args[] = {&p};
  return launch_spec(s, args, st);
}

}  // namespace

cudaError_t launch_quant_rows(const quant_rows_t& a, const FfnDevice& dev, cudaStream_t st) {
  const int e = a.dtype == FFN_F32 ? 4 : 2;
  QuantRowsParams p{};
  p.rows = (uint32_t)a.rows;
  p.cols = (int32_t)a.cols;
  p.vec = alignment_of(a.x, a.ld_x * e);
  p.x = a.x;
  p.x_end = end_of_rows(a.x, a.rows, a.ld_x, a.cols, e);
  p.data = static_cast<uint8_t*>(a.data);
  p.scales = static_cast<uint8_t*>(a.scales);
  p.row_scale = a.row_scale;
  p.ld_x = (uint32_t)a.ld_x;
  p.ld_data = (uint32_t)a.ld_data;
  return launch(p, a.dtype, a.format, false, dev.num_sms, st);
}

cudaError_t launch_quant_norm(const quant_norm_t& a, const FfnDevice& dev, cudaStream_t st) {
  const int e = a.dtype == FFN_F32 ? 4 : 2;
  QuantRowsParams p{};
  p.rows = (uint32_t)a.M;
  p.cols = (int32_t)a.D;
  p.vec = std::min({alignment_of(a.y, a.ld_y * e), alignment_of(a.residual, a.ld_residual * e),
                    alignment_of(a.s, a.ld_s * e)});
  p.x = a.y;
  p.residual = a.residual;
  p.x_end = end_of_rows(a.y, a.M, a.ld_y, a.D, e);
  if (a.residual) p.residual_end = end_of_rows(a.residual, a.M, a.ld_residual, a.D, e);
  if (a.weight) p.weight_end = end_of_rows(a.weight, 1, a.D, a.D, a.param_dtype == FFN_F32 ? 4 : 2);
  p.weight = a.weight;
  p.s = a.s;
  p.data = static_cast<uint8_t*>(a.data);
  p.scales = static_cast<uint8_t*>(a.scales);
  p.row_scale = a.row_scale;
  p.ld_x = (uint32_t)a.ld_y;
  p.ld_residual = (uint32_t)a.ld_residual;
  p.ld_s = (uint32_t)a.ld_s;
  p.ld_data = (uint32_t)a.ld_data;
  p.weight_f32 = a.param_dtype == FFN_F32;
  p.weight_vec = alignment_of(a.weight, 0);
  p.eps = a.eps;
  p.residual_scale = a.residual_scale;
  p.branch_scale = a.branch_scale;
  return launch(p, a.dtype, a.format, true, dev.num_sms, st);
}

}  // namespace dgb
