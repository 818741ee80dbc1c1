// fp4.h -- internal interface of the 4-bit product's kernels: what their host code (fp4.cu)
// and the kernel translation units share.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "quant.h"

namespace dgb {

// What happens to a sum: c = act(row_scale_a[i] row_scale_b[j] sum + bias[j]) + residual[i][j].
struct Fp4Epilogue {
  int32_t M, N, act;
  int32_t vec;              // c's and the residual's rows start on 16-byte boundaries
  const float* row_scale_a; // or null, as the next three
  const float* row_scale_b;
  const float* bias;
  const void* residual;
  void* c;
  int64_t ld_residual, ld_c;
};

struct Fp4Params {
  Fp4Epilogue e;
  int32_t steps;            // MMAs of 64 K-elements that a sum takes
  int32_t blocks;           // stages of 256 K-elements
  int32_t tiles_m, tiles_n, raster_group;
  uint32_t idesc;
  uint32_t debug_flags;
  uint32_t* status;
  uint64_t timeout_ns;
  // few tokens (kernel_fp4_few.cu)
  int32_t tokens;           // columns of an MMA: tokens of a tile
  int32_t split;            // CTAs of a cluster that share a sum
  int32_t static_b;
  int32_t stages;           // of the ring of copies
};

// Tokens that the kernel quantises itself (kernel_fp4_few.cu).
struct Fp4Tokens {
  const void* x;
  const void* x_end;        // the first byte past its last element
  int64_t ld_x;
  int32_t K;                // values of a token (the product's K is that padded)
  int32_t vec;              // rows start on boundaries of: 2 = 32 bytes, 1 = 16, 0 = neither
};

// Tiles of 64 x 128 with a sum shared by a cluster while they are no more than SMs, or two an SM with
// short sums; above that CTA pairs, but for M <= 64, where most of a pair's rows would be empty.
// (A pair's CTAs fill their SMs: they start when the kernel before has left.)  Few and pair, us, products
// behind one another:
//   up to one an SM: MXFP4 512 x 2048 x 4096 (128 tiles) 8.8 and 10.4, 256 x 4096 x 14336 (128) 17.2 and 24.9
//   two an SM, K < 1024: MXFP4 at 160, 162, 180, 192, 224, 250, 256 and 304 tiles (M of 100 to 1216) and K of 64
//     to 992 always less, 5.6 to 8.6 and 6.1 to 10.5 (512 x 2560 x 512 6.1 and 7.1, 1024 x 2048 x 256 6.1 and 6.7,
//     1216 x 2048 x 736 7.5 and 7.8); NVFP4 alone within 5 % either way up to 256 tiles (7.2 and 7.2,
//     7.2 and 6.9) and 9 % more at 304 (7.7 and 7.2), but less where other kernels stand around: gradients
//     of a linear layer, with the sums over M there of this kind, MXFP4 and NVFP4, 515 x 1097 x 1032 22.0 and
//     25.2, 25.4 and 27.8; 520 x 1200 x 1100 24.3 and 31.5, 29.2 and 35.2; 400 x 2000 x 1032 23.8 and 25.7, 28.7
//     and 29.2; 900 x 1097 x 1032 25.5 and 27.5, 30.8 and 32.0
//   two an SM, longer sums: gradients 1100 x 1100 x 1200 28.2 and 28.5, 32.8 and 32.3; 2048 x 1100 x 1200 31.7 and
//     29.7, 37.5 and 36.4; 4096 x 2048 x 1024 39.5 and 37.4, 50.8 and 47.8; NVFP4 alone 512 x 4096 x 2048 10.0 and
//     9.4, 768 x 2048 x 4096 12.5 and 11.7 (MXFP4 alone 8.5 and 9.2, 10.9 and 11.5, from K = 8192 on more)
//   more: MXFP4 2048 x 1200 (320 tiles) x 256 10.7 and 6.8, x 2048 15.2 and 9.3; NVFP4 12.7 and 6.9
inline bool fp4_on_pairs(int64_t M, int64_t N, int64_t K, int num_sms) {
  const int64_t few_tiles = ((M + 63) / 64) * ((N + 127) / 128);
  return M > 64 && few_tiles > (K < 1024 ? 2 : 1) * (int64_t)num_sms;
}

const void* fp4_pair_kernel(bool nv, bool out_f32);
size_t fp4_pair_smem(bool nv);
constexpr int kFp4PairThreads = 384;

const void* fp4_few_kernel(bool nv, bool out_f32);
size_t fp4_few_smem(bool nv, int tokens, int stages);
int fp4_few_stages(bool nv, int tokens);
constexpr int kFp4FewThreads = 256;

// the same with the tokens' quantisation; kb: the most stages of K a CTA takes
const void* fp4_linear_kernel(bool nv, bool out_f32, int dtype);
int fp4_linear_stages(bool nv, int kb);
size_t fp4_linear_smem(bool nv, int kb, int stages);

}  // namespace dgb
