// gated.cu -- host side of the gated projections: the choice of tile, TMA maps and
// launches of the kernels in kernels_gated.cuh and kernel_gated_slopes.cu.
#include <algorithm>

#include "ffn_launch.h"
#include "gated.h"
#include "idesc.h"
#include "launch.h"

namespace dgb {

namespace {

int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }

int alignment_of(const void* p, int64_t ld) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * 2);
  return (bits & 31u) == 0 ? 2 : (bits & 15u) == 0 ? 1 : 0;
}

struct Tiling {
  int consumers, hw;
};

// One consumer's MMAs are issued by two threads (see kernels_gated.cuh) where TMEM
// holds the accumulators: hw <= 64, or one tile per cluster.
bool split_of(int consumers, int hw, int64_t tiles, int clusters) {
  return consumers == 1 && (hw <= 64 || tiles <= clusters);
}

// Microseconds of x w^T for both projections on tiles of `consumers` x 256 rows and hw
// columns: a launch, and per wave of clusters the 64-wide blocks of the reduction and
// what a tile's end costs.  Fitted on 152 SMs to 14 shapes (M 40 - 8192, F 700 - 14336,
// K 464 - 4096) timed with every tile; wide tiles take the MMAs' own time (4.2 ns per
// block and column of h), narrow ones what issuing them costs, and two consumers have
// no second accumulator to fill while the first is read.
double pair_time(int64_t tiles, int clusters, int64_t kb, int consumers, int hw) {
  double block, end;
  if (consumers == 2) {
    block = std::max(0.32, 0.06 + 0.0039 * hw);
    end = 3.7;
  } else if (split_of(consumers, hw, tiles, clusters)) {
    block = std::max(0.21 + 0.0002 * hw, 0.0021 * hw);
    end = 0.7;
  } else {
    block = 0.27 + 0.0003 * hw;
    end = 0.7;
  }
  const double waves = (double)ceil_div64(tiles, clusters);
  return 6.0 + waves * (double)kb * block + (waves - 1) * end;
}

// The same for one tile of a product of the backward pass (its operands' rows run along
// the reduction), hw = 64 or 128 columns per CTA; fitted to eight shapes with long
// reductions, and to four with 1 to 10 blocks, where storing the tile takes longer than
// making the next one.
double product_tile_time(int64_t kb, int consumers, int hw) {
  const double n = (double)kb;
  if (consumers == 2) return hw == 128 ? std::max(0.63 * n + 3.0, 0.58 * n + 4.7) : 0.48 * n + 3.0;
  return hw == 128 ? std::max(0.42 * n + 0.7, 0.2 * n + 2.6) : std::max(0.36 * n + 0.7, 0.1 * n + 2.0);
}

// The tile that finishes soonest: one or two consumers (256 or 512 rows), hw = 16
// ... 128 columns of h.  Narrow tiles even out the last wave and spread a weight
// over more SMs when there are few rows.
Tiling gated_tiling(int64_t M, int64_t F, int64_t kb, int clusters) {
  Tiling best{1, 128};
  double least = 0;
  for (int consumers = 2; consumers >= 1; --consumers)
    for (int hw = 128; hw >= 16; hw -= 16) {
      const int64_t tiles = ceil_div64(M, 256 * consumers) * ceil_div64(F, hw);
      const double t = pair_time(tiles, clusters, kb, consumers, hw);
      if (least == 0 || t < least) {
        least = t;
        best = {consumers, hw};
      }
    }
  return best;
}

void fill_task(GatedTask* t, int64_t rows, int64_t cols, int64_t kb, int tile_m, int tile_n, bool bf16, int mma_n,
               uint32_t major, void* out, int64_t ld) {
  t->rows = (int32_t)rows;
  t->cols = (int32_t)cols;
  t->kb = (int32_t)kb;
  t->kb_slice = (int32_t)kb;
  t->tiles_m = (int32_t)ceil_div64(rows, tile_m);
  t->tiles_n = (int32_t)ceil_div64(cols, tile_n);
  t->raster_group = std::min(8, t->tiles_m);
  t->a_mn = (major & IDESC_A_MN_MAJOR) != 0;
  t->idesc = idesc_f16(bf16, 256, mma_n) | major;
  t->out = out;
  t->ld_out = ld;
  t->vec_out = alignment_of(out, ld);
}

cudaError_t launch_tiles(const void* func, int consumers, int64_t tiles, const FfnDevice& dev, CUtensorMap (&maps)[4],
                         GatedParams& p, cudaStream_t st) {
  p.stages = gated_stages(consumers, p.a_rows, p.hw);
  const size_t smem = gated_smem_bytes(consumers, p.a_rows, p.hw, p.stages);
  const cudaError_t e = allow_smem_once(func, 232448);
  if (e != cudaSuccess) return e;
  LaunchSpec s;
  s.func = func;
  s.grid = dim3(2u * (unsigned)std::min<int64_t>(tiles, std::max(1, dev.num_sms / 2)), 1, 1);
  s.block = dim3(kGatedThreads, 1, 1);
  s.smem = smem;
  s.cluster = 2;
  s.pdl = true;
  void* args[] = {&maps[0], &maps[1], &maps[2], &maps[3], &p};
  return launch_spec(s, args, st);
}

template <typename A>
GatedParams common_params(const A& a, const FfnDevice& dev) {
  GatedParams p{};
  p.status = dev.status;
  p.timeout_ns = a.timeout_ns ? (uint64_t)a.timeout_ns : 2000000000ull;
  p.debug_flags = (uint32_t)a.debug_flags;
  return p;
}

// x w^T for both projections, joined by the epilogue of `func_of`
template <typename A, typename F>
cudaError_t launch_pair(const A& a, const FfnDevice& dev, GatedParams& p, void* out, int64_t ld, F func_of,
                        cudaStream_t st) {
  const bool bf16 = a.dtype == FFN_BF16;
  const int clusters = std::max(1, dev.num_sms / 2);
  const int64_t kb = ceil_div64(a.K, 64);
  const Tiling t = gated_tiling(a.M, a.F, kb, clusters);
  fill_task(&p.task[0], a.M, a.F, kb, 256 * t.consumers, t.hw, bf16, 2 * t.hw, 0, out, ld);
  p.n0 = p.task[0].tiles_m * p.task[0].tiles_n;
  p.hw = t.hw;
  p.split = split_of(t.consumers, t.hw, p.n0, clusters) ? 2 : 1;
  p.part_cols = t.hw <= 64 ? 128 : 256;
  p.two_slots = p.split == 1 || t.hw <= 64;
  p.a_rows = gated_a_rows(t.consumers, a.M);
  CUtensorMap maps[4];
  if (!encode_rows16(&maps[0], bf16, a.x, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)a.ld_x, 64,
                     (uint32_t)p.a_rows) ||
      !encode_rows16(&maps[1], bf16, a.w, (uint64_t)a.K, (uint64_t)(2 * a.F), (uint64_t)a.ld_w, 64, (uint32_t)t.hw))
    return cudaErrorInvalidValue;
  maps[2] = maps[0];
  maps[3] = maps[1];
  return launch_tiles(func_of(bf16, t.consumers, a.activation), t.consumers, p.n0, dev, maps, p, st);
}

// How the products of the backward pass are cut: consumers and columns of a tile, and
// slices of dx's reduction.
struct ProductPlan {
  int consumers, hw, slices;
  int64_t kb_slice;
};

// The cut with the least time for both products' work spread over the clusters, whichever
// are wanted: a product's bits do not depend on the other's being asked for.  It takes
// the SM pairs of the device the library is for, so that it is known without a device.
// With few tokens and wide layers dx is a few tiles with a long reduction each; slices of
// it keep the other clusters busy, for a pass over their sums (a launch, and each sum
// written and read).
ProductPlan plan_products(int64_t M, int64_t F, int64_t K) {
  constexpr double kClusters = 76;
  const int64_t kb_dx = ceil_div64(2 * F, 64), kb_dw = ceil_div64(M, 64);
  ProductPlan best{1, 128, 1, kb_dx};
  double least = 0;
  for (int consumers = 2; consumers >= 1; --consumers)
    for (int hw = 128; hw >= 64; hw -= 64) {
      const int64_t tiles_k = ceil_div64(K, 2 * hw);
      const int64_t n_dx = ceil_div64(M, 256 * consumers) * tiles_k, n_dw = ceil_div64(2 * F, 256 * consumers) * tiles_k;
      for (const int64_t want : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
        const int64_t kb_slice = ceil_div64(kb_dx, want), slices = ceil_div64(kb_dx, kb_slice);
        const double sums = slices > 1 ? (double)slices * (double)M * (double)K * 4.0 : 0.0;
        if (want > 1 && (slices != want || kb_slice < 4 || sums > 64e6)) continue;
        const double dx = product_tile_time(kb_slice, consumers, hw), dw = product_tile_time(kb_dw, consumers, hw);
        const double t = std::max((dx * (double)(n_dx * slices) + dw * (double)n_dw) / kClusters, std::max(dx, dw)) +
                         (slices > 1 ? 3.0 + sums * 2 / 4e6 : 0.0);
        if (least == 0 || t < least) {
          least = t;
          best = {consumers, hw, (int)slices, kb_slice};
        }
      }
    }
  return best;
}

// dx = dgu w and dw = dgu^T x in one launch, the product with the longer reduction first
cudaError_t launch_products(const ffn_gated_grad_t& a, const FfnDevice& dev, cudaStream_t st) {
  if (!a.dx && !a.dw) return cudaSuccess;
  const bool bf16 = a.dtype == FFN_BF16;
  const int64_t kb_dx = ceil_div64(2 * a.F, 64), kb_dw = ceil_div64(a.M, 64);
  const ProductPlan best = plan_products(a.M, a.F, a.K);
  GatedParams p = common_params(a, dev);
  p.hw = best.hw;
  p.a_rows = 128;
  p.split = 1;  // (their operands' copies bound these, not the MMAs' issue)
  p.two_slots = 1;
  const int tile_m = 256 * best.consumers, tile_n = 2 * best.hw;
  const bool dx_first = a.dx && (!a.dw || best.kb_slice >= kb_dw);
  CUtensorMap maps[4];
  int32_t tiles[2] = {0, 0};
  int n = 0;
  bool ok = true;
  auto add_dx = [&] {
    fill_task(&p.task[n], a.M, a.K, kb_dx, tile_m, tile_n, bf16, tile_n, IDESC_B_MN_MAJOR, a.dx, a.ld_dx);
    p.task[n].kb_slice = (int32_t)best.kb_slice;
    if (best.slices > 1) p.task[n].partial = static_cast<float*>(a.workspace);
    tiles[n] = p.task[n].tiles_m * p.task[n].tiles_n * best.slices;
    ok = ok &&
         encode_rows16(&maps[2 * n], bf16, a.dgu, (uint64_t)(2 * a.F), (uint64_t)a.M, (uint64_t)a.ld_dgu, 64, 128) &&
         encode_rows16(&maps[2 * n + 1], bf16, a.w, (uint64_t)a.K, (uint64_t)(2 * a.F), (uint64_t)a.ld_w, 64, 64);
    ++n;
  };
  if (dx_first) add_dx();
  if (a.dw) {
    fill_task(&p.task[n], 2 * a.F, a.K, kb_dw, tile_m, tile_n, bf16, tile_n, IDESC_A_MN_MAJOR | IDESC_B_MN_MAJOR, a.dw,
              a.ld_dw);
    tiles[n] = p.task[n].tiles_m * p.task[n].tiles_n;
    ok = ok &&
         encode_rows16(&maps[2 * n], bf16, a.dgu, (uint64_t)(2 * a.F), (uint64_t)a.M, (uint64_t)a.ld_dgu, 64, 64) &&
         encode_rows16(&maps[2 * n + 1], bf16, a.x, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)a.ld_x, 64, 64);
    ++n;
  }
  if (a.dx && !dx_first) add_dx();
  if (!ok) return cudaErrorInvalidValue;
  p.n0 = tiles[0];
  p.n1 = tiles[1];
  if (n == 2) {
    p.fill = (int32_t)(product_tile_time(p.task[0].kb_slice, best.consumers, best.hw) /
                           product_tile_time(p.task[1].kb_slice, best.consumers, best.hw) +
                       0.5);
  } else {
    maps[2] = maps[0];
    maps[3] = maps[1];
  }
  const cudaError_t e = launch_tiles(gated_products_kernel(bf16, best.consumers), best.consumers,
                                     (int64_t)p.n0 + p.n1, dev, maps, p, st);
  if (e != cudaSuccess || !a.dx || best.slices == 1) return e;
  return launch_gated_join(a, best.slices, dev.num_sms, st);
}

}  // namespace

cudaError_t launch_gated(const ffn_gated_t& a, const FfnDevice& dev, cudaStream_t st) {
  if (a.M <= kGatedFewTokens) return launch_gated_few(a, dev.num_sms, st);
  GatedParams p = common_params(a, dev);
  p.gu = a.gu;
  p.ld_gu = a.ld_gu;
  p.vec_gate = alignment_of(a.gu, a.ld_gu);
  p.vec_up = alignment_of(static_cast<const char*>(a.gu) + 2 * a.F, a.ld_gu);
  return launch_pair(a, dev, p, a.h, a.ld_h, gated_forward_kernel, st);
}

size_t gated_backward_workspace(const ffn_gated_grad_t& a) {
  if (a.dx == nullptr || a.M == 0) return 0;
  const int slices = plan_products(a.M, a.F, a.K).slices;
  return slices > 1 ? (size_t)slices * (size_t)a.M * (size_t)a.K * 4 : 0;
}

cudaError_t launch_gated_backward(const ffn_gated_grad_t& a, const FfnDevice& dev, cudaStream_t st) {
  cudaError_t e;
  if (a.gu != nullptr) {
    e = launch_gated_slopes(a, dev.num_sms, st);
  } else {
    GatedParams p = common_params(a, dev);
    p.dh = a.dh;
    p.ld_dh = a.ld_dh;
    p.vec_dh = alignment_of(a.dh, a.ld_dh);
    p.vec_up = alignment_of(static_cast<const char*>(a.dgu) + 2 * a.F, a.ld_dgu);
    e = launch_pair(a, dev, p, a.dgu, a.ld_dgu, gated_slopes_kernel, st);
  }
  return e != cudaSuccess ? e : launch_products(a, dev, st);
}

}  // namespace dgb
