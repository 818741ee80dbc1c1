// norm.h -- internal interface of the block norms' kernels: what their host code
// (norm.cu) and the kernel translation units (one per element type) share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ffn.h"
#include "ffn_launch.h"

#if defined(__CUDACC__)
#define DGB_ROWS_FN __host__ __device__ __forceinline__
#else
#define DGB_ROWS_FN inline
#endif

namespace dgb {

// `n` things dealt to `parts` parts in order, the first ones one more.
struct NormShare {
  int each, more;
  static NormShare of(int64_t n, int64_t parts) { return {(int)(n / parts), (int)(n % parts)}; }
  DGB_ROWS_FN int begin(int part) const { return part * each + (part < more ? part : more); }
};

// A row slice that starts `shift` elements past a 16-byte boundary comes to shared
// memory in whole 16-byte pieces from that boundary on.  Where its first or last piece
// may hold memory outside the array it is copied by element instead (`head`: the array
// starts off a boundary, and this is one of its first rows; `tail`: one of its last),
// so nothing outside an array is read: another stream may own it.
struct RowPieces {
  int bytes;  // of all pieces
  int rest;   // elements of a partial last piece (0 where the slice ends before the row)
  DGB_ROWS_FN static RowPieces of(int shift, int cols, int per_piece, bool ends_row) {
    const int n = shift + cols;
    return {(n + per_piece - 1) / per_piece * 16, ends_row ? n % per_piece : 0};
  }
  // the bytes from the boundary on that come whole: from begin(head) to end(tail), if any
  DGB_ROWS_FN int begin(bool head) const { return head ? 16 : 0; }
  DGB_ROWS_FN int end(bool tail) const { return tail && rest != 0 ? bytes - 16 : bytes; }
};
// How many rows, `ld` elements apart, the piece over an end of the array can reach into:
// one but for rows shorter than a piece.  Of rows that start alike, pieces apart, only the
// first or the last is among them.
inline int rows_at_an_end(int64_t ld, int per_piece) { return (int)((per_piece - 2 + ld) / ld); }

// Forward, direct: one row per warp (warp_rows) or per CTA.  Ring: warps or CTAs walk
// rows of one class each (rows `period` apart start alike, see norm_walk).
struct NormShape {
  bool warp_rows;
  int nv;          // 16-byte vectors per thread
  int threads;     // per CTA
  int64_t grid;    // (ring: settled with the kernel's residency)
  size_t smem;
  int period;
  NormShare share; // blocks of `period` rows to slices of the grid
  int64_t head, tail;  // rows before `head` and from `tail` on: see RowPieces
};

// 16-byte vectors a thread can hold of a row: 32 elements
constexpr int norm_most_vectors(int element_bytes) { return 2 * element_bytes; }

// Backward: a part (a CTA, a cluster of CTAs sharing the columns, or a warp) takes
// rows of one of the gate's groups, or several whole groups.
struct NormGradShape {
  int stages;              // rows of the ring
  size_t smem;
  int cluster;             // CTAs that share a row's columns
  int each;                // columns per thread: 16, or 8
  int threads;             // per row and CTA
  int per_sm;              // CTAs that an SM is meant to hold
  int lanes;               // rows a CTA takes at once (warps; 1 where a row takes several)
  int parts;               // grid = ceil(parts / lanes) * cluster
  int parts_per_group;     // > 0: a part is in one group; 0: several whole groups
  int period;              // rows this far apart belong to one part
  int per;                 // rows of a gate's group
  NormShare share;         // blocks of `period` rows to the slices of a group; groups to parts (many)
  uint32_t slow;           // arrays off the walk's shift: s, dn, y, ds, dresidual, dy
  int64_t columns;         // per CTA
  bool many;               // several whole groups per part (parts_per_group == 0)
  bool full;               // both norms, and every row array given or asked for
  bool bias;               // sums of t and of dn are needed beside those with the unit rows
  int64_t tail;            // rows from here on: see RowPieces
};

// The workspace of the column sums: `sums` arrays of parts x D fp32.
struct NormSums {
  float* a;  // sums of t * unit(y) (many: weighted with the gate)
  float* b;  // sums of t
  float* c;  // sums of dn * unit(s)
  float* e;  // sums of dn
};

cudaError_t norm_forward_f16(const ffn_norm_t& a, const NormShape& direct, const NormShape* ring,
                             const FfnDevice& dev, cudaStream_t st);
cudaError_t norm_forward_bf16(const ffn_norm_t& a, const NormShape& direct, const NormShape* ring,
                             const FfnDevice& dev, cudaStream_t st);
cudaError_t norm_forward_f32(const ffn_norm_t& a, const NormShape& direct, const NormShape* ring,
                             const FfnDevice& dev, cudaStream_t st);
cudaError_t norm_backward_f16(const ffn_norm_grad_t& a, const NormGradShape& sh, const NormSums& ws,
                              const FfnDevice& dev, cudaStream_t st);
cudaError_t norm_backward_bf16(const ffn_norm_grad_t& a, const NormGradShape& sh, const NormSums& ws,
                               const FfnDevice& dev, cudaStream_t st);
cudaError_t norm_backward_f32(const ffn_norm_grad_t& a, const NormGradShape& sh, const NormSums& ws,
                              const FfnDevice& dev, cudaStream_t st);

constexpr int kNormGradThreads = 256;  // most per CTA
constexpr int kNormStages = 3;                     // most rows of a ring
constexpr size_t kNormRingBytes = 200 * 1024;      // most of one CTA

}  // namespace dgb
