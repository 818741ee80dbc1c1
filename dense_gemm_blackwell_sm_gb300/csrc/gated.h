// gated.h -- internal interface of the gated projections' kernels: what their
// host code (gated.cu) and the kernel translation units share.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "ffn.h"

#if defined(__CUDACC__)
#define DGB_BOTH __host__ __device__
#else
#define DGB_BOTH
#endif

namespace dgb {

enum GatedMode {
  GATED_FORWARD = 0,   // h (and the pre-activations) from x and w
  GATED_SLOPES = 1,    // the same products, the gradient of the pre-activations written
  GATED_PRODUCTS = 2,  // plain products of the backward pass, up to two in one launch
};

// One product and its tiles.
struct GatedTask {
  int32_t rows, cols;         // of the output (cols = F for the gated modes)
  int32_t kb;                 // 64-wide blocks of the reduction
  int32_t kb_slice;           // of one slice of it, where tiles take a slice each
  int32_t tiles_m, tiles_n, raster_group;
  int32_t a_mn;               // the first operand's rows run along the reduction
  uint32_t idesc;
  int32_t vec_out;            // alignment of the output's rows: 2 = 32 bytes, 1 = 16 bytes, 0 = neither
  void* out;
  int64_t ld_out;
  float* partial;             // slices x rows x cols, or null: the tiles' sums go to `out`
};

struct GatedParams {
  GatedTask task[2];
  int32_t n0, n1;             // tiles of the two tasks (n1 = 0: one task)
  int32_t fill;               // tiles of task 1 about as long as one of task 0
  int32_t hw;                 // MMA columns per CTA: half the tile's N
  int32_t a_rows;             // rows of the first operand a CTA brings per consumer (gated_a_rows)
  int32_t split;              // one consumer: threads that issue its MMAs (2: even and odd blocks)
  int32_t part_cols;          // TMEM columns between their accumulators
  int32_t two_slots;          // one consumer: accumulators for two tiles in turn
  int32_t stages;
  uint32_t debug_flags;
  uint32_t* status;
  uint64_t timeout_ns;
  void* gu;                   // GATED_FORWARD: pre-activations out, or null
  int64_t ld_gu;
  const void* dh;             // GATED_SLOPES
  int64_t ld_dh;
  int32_t vec_gate, vec_up, vec_dh;
};

// The i-th tile of cluster cid: task 0's tiles (the longer ones) in turn; then the
// clusters that got one fewer of them take `fill` tiles each of task 1, which last
// about as long; then the rest of task 1 in turn.  False after the last.
DGB_BOTH inline bool gated_tile(const GatedParams& p, int32_t cid, int32_t clusters, int32_t i, int32_t& task,
                                int32_t& tile) {
  const int32_t rem = p.n0 % clusters;
  const int32_t mine = p.n0 / clusters + (cid < rem ? 1 : 0);
  task = 0;
  tile = cid + i * clusters;
  if (i < mine) return true;
  i -= mine;
  task = 1;
  const int32_t idle = rem != 0 ? clusters - rem : 0;
  if (cid >= rem && idle != 0) {
    const int32_t first = cid - rem;
    int32_t filled = p.n1 > first ? (p.n1 - first + idle - 1) / idle : 0;
    if (filled > p.fill) filled = p.fill;
    tile = first + i * idle;
    if (i < filled) return true;
    i -= filled;
  }
  const int32_t base = p.fill * idle < p.n1 ? p.fill * idle : p.n1;
  tile = base + cid + i * clusters;
  return tile < p.n1;
}

// Rows of the first operand that a CTA brings per consumer.  With few tokens only their
// rows come to shared memory, which leaves it to the weights; two consumers' kernels count
// on whole operands, whatever the number of tokens.
inline int gated_a_rows(int consumers, int64_t tokens) {
  return consumers == 1 && tokens <= 120 ? (int)((tokens + 7) / 8 * 8) : 128;
}

const void* gated_forward_kernel(bool bf16, int consumers, int act);
const void* gated_slopes_kernel(bool bf16, int consumers, int act);
const void* gated_products_kernel(bool bf16, int consumers);
// stages that fit shared memory, and the bytes a CTA then takes
int gated_stages(int consumers, int a_rows, int hw);
size_t gated_smem_bytes(int consumers, int a_rows, int hw, int stages);
constexpr int kGatedThreads = 384;

// the gated projections for few tokens (kernel_gated_few.cu)
constexpr int64_t kGatedFewTokens = 32;
cudaError_t launch_gated_few(const ffn_gated_t& a, int num_sms, cudaStream_t st);

// adds the slices of dx
cudaError_t launch_gated_join(const ffn_gated_grad_t& a, int slices, int num_sms, cudaStream_t st);

// the pre-activations' gradient from kept ones (kernel_gated_slopes.cu)
cudaError_t launch_gated_slopes(const ffn_gated_grad_t& a, int num_sms, cudaStream_t st);

}  // namespace dgb
