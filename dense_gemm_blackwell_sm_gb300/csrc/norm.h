// norm.h -- internal interface of the block norms' kernels: what their host code
// (norm.cu) and the kernel translation units (one per element type) share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ffn.h"
#include "ffn_launch.h"

namespace dgb {

// Forward: one row per warp (warp_rows) or per CTA, nv 16-byte vectors per thread.
struct NormShape {
  bool ring;       // rows through the shared-memory ring (kernels_norm_ring.cuh)
  bool aligned;    // rows and parameters on 16-byte boundaries, rows of whole 16-byte pieces
  bool warp_rows;
  int nv;
  int threads;     // per CTA
  int64_t grid;
  size_t smem;
};

// 16-byte vectors a thread can hold of a row: 32 elements
constexpr int norm_most_vectors(int element_bytes) { return 2 * element_bytes; }

// Backward: a part (a CTA, a cluster of CTAs sharing the columns, or a warp) takes a
// run of rows that lies in one of the gate's groups, or several whole groups.
struct NormGradShape {
  bool aligned;            // as in NormShape, with groups of 8 columns
  int stages;              // rows of the ring
  size_t smem;
  int cluster;             // CTAs that share a row's columns
  int threads;             // per row and CTA
  int lanes;               // rows a CTA takes at once (warps; 1 above 512 columns)
  int parts;               // grid = ceil(parts / lanes) * cluster
  int parts_per_group;     // > 0: a part is a slice of one group; 0: several whole groups
  int64_t columns;         // per CTA
  bool many;               // several whole groups per part (parts_per_group == 0)
  bool bias;               // sums of t and of dn are needed beside those with the unit rows
};

// The workspace of the column sums: `sums` arrays of parts x D fp32.
struct NormSums {
  float* a;  // sums of t * unit(y) (many: weighted with the gate)
  float* b;  // sums of t
  float* c;  // sums of dn * unit(s)
  float* e;  // sums of dn
};

cudaError_t norm_forward_f16(const ffn_norm_t& a, const NormShape& sh, const FfnDevice& dev, cudaStream_t st);
cudaError_t norm_forward_bf16(const ffn_norm_t& a, const NormShape& sh, const FfnDevice& dev, cudaStream_t st);
cudaError_t norm_forward_f32(const ffn_norm_t& a, const NormShape& sh, const FfnDevice& dev, cudaStream_t st);
cudaError_t norm_backward_f16(const ffn_norm_grad_t& a, const NormGradShape& sh, const NormSums& ws,
                              const FfnDevice& dev, cudaStream_t st);
cudaError_t norm_backward_bf16(const ffn_norm_grad_t& a, const NormGradShape& sh, const NormSums& ws,
                               const FfnDevice& dev, cudaStream_t st);
cudaError_t norm_backward_f32(const ffn_norm_grad_t& a, const NormGradShape& sh, const NormSums& ws,
                              const FfnDevice& dev, cudaStream_t st);

constexpr int kNormGradThreads = 256;  // most per CTA, 16 columns each
constexpr int kNormGradEach = 16;
constexpr int kNormStages = 3;                     // most rows of a ring
constexpr size_t kNormRingBytes = 200 * 1024;      // most of one CTA
// a slot holds a row at any offset, and the pieces a shifted read of its last group touches
inline size_t norm_slot_bytes(int64_t bytes) { return (size_t)(bytes + 31) / 32 * 32 + 32; }

}  // namespace dgb
