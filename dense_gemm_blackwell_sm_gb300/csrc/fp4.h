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
