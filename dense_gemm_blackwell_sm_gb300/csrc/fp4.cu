// fp4.cu -- host side of the 4-bit product: the choice of kernel and split, TMA maps, launches.
#include "fp4.h"

#include <algorithm>

#include "idesc.h"
#include "launch.h"
#include "quant_launch.h"

namespace dgb {

namespace {

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool aligned_rows(const void* p, int64_t pitch_bytes) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)pitch_bytes) & 15u) == 0;
}

}  // namespace

cudaError_t launch_fp4_product(const quant_product_t& a, const FfnDevice& dev, cudaStream_t st) {
  const bool nv = a.format == QUANT_NVFP4, f32 = a.out_dtype == FFN_F32;
  const int64_t e = f32 ? 4 : 2;
  Fp4Params p{};
  p.e.M = (int32_t)a.M;
  p.e.N = (int32_t)a.N;
  p.e.act = a.activation;
  p.e.vec = aligned_rows(a.c, a.ld_c * e) && aligned_rows(a.residual, a.ld_residual * e);
  p.e.row_scale_a = a.row_scale_a;
  p.e.row_scale_b = a.row_scale_b;
  p.e.bias = a.bias;
  p.e.residual = a.residual;
  p.e.c = a.c;
  p.e.ld_residual = a.ld_residual;
  p.e.ld_c = a.ld_c;
  p.steps = (int32_t)up(a.K, 64);
  p.blocks = (int32_t)up(a.K, 256);
  p.debug_flags = (uint32_t)a.debug_flags;
  p.status = dev.status;
  p.timeout_ns = a.timeout_ns ? (uint64_t)a.timeout_ns : 2000000000ull;
  p.static_b = (a.flags & QUANT_STATIC_B) != 0;

  const uint32_t box_k = nv ? 4 : 2;  // scale blocks of a stage
  const uint64_t across = (uint64_t)up(scales_of(a.K, a.format), 4);
  CUtensorMap maps[5];
  LaunchSpec s;
  s.pdl = true;
  void* pair_args[] = {&maps[0], &maps[1], &maps[2], &maps[3], &maps[4], &p};
  void* few_args[] = {&maps[0], &maps[1], &maps[2], &maps[3], &p};
  void** args = few_args;
  if (!encode_scale_blocks(&maps[2], a.scales_a, across, (uint64_t)up(a.M, 128), box_k, 1)) return cudaErrorInvalidValue;

  const int64_t pair_tiles = up(a.M, 256) * up(a.N, 256);
  if (a.M > 128 && pair_tiles * 2 > dev.num_sms / 2) {
    p.tiles_m = (int32_t)up(a.M, 256);
    p.tiles_n = (int32_t)up(a.N, 256);
    // (both operands lie in L2 at sizes where that matters: 32 rows of tiles against 8 take 8192 x
    // 14336 x 4096 NVFP4 from 156 to 149 us, 8192^3 from 166 to 162)
    p.raster_group = std::min(32, p.tiles_m);
    p.stages = fp4_pair_stages(nv);
    p.idesc = idesc_fp4(!nv, 256, 256);
    if (!encode_byte_rows(&maps[0], a.a, (uint64_t)a.K / 2, (uint64_t)a.M, (uint64_t)a.ld_a, 128) ||
        !encode_byte_rows(&maps[1], a.b, (uint64_t)a.K / 2, (uint64_t)a.N, (uint64_t)a.ld_b, 128) ||
        !encode_scale_blocks(&maps[3], a.scales_b, across, (uint64_t)up(a.N, 128), box_k, 2))
      return cudaErrorInvalidValue;
    maps[4] = maps[0];  // (not used where c's rows are not aligned)
    if (p.e.vec && !encode_out_tiles(&maps[4], f32, a.c, (uint64_t)a.N, (uint64_t)a.M, (uint64_t)a.ld_c))
      return cudaErrorInvalidValue;
    args = pair_args;
    s.func = fp4_pair_kernel(nv, f32);
    s.grid = dim3(2u * (unsigned)std::min<int64_t>(pair_tiles, std::max(1, dev.num_sms / 2)), 1, 1);
    s.block = dim3(kFp4PairThreads, 1, 1);
    s.smem = fp4_pair_smem(nv);
    s.cluster = 2;
  } else {
    p.tokens = a.M <= 64 ? (int32_t)up(a.M, 16) * 16 : 64;
    p.tiles_m = (int32_t)up(a.M, p.tokens);
    p.tiles_n = (int32_t)up(a.N, 128);
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    // (all CTAs at once, two an SM)
    const int64_t slots = 2 * (int64_t)dev.num_sms;
    p.split = 1;
    while (p.split < 8 && p.split * 2 <= p.blocks && tiles * p.split * 2 <= slots) p.split *= 2;
    p.stages = fp4_few_stages(nv, p.tokens);
    p.idesc = idesc_fp4(!nv, 128, p.tokens);
    if (!encode_byte_rows(&maps[0], a.a, (uint64_t)a.K / 2, (uint64_t)a.M, (uint64_t)a.ld_a, (uint32_t)p.tokens) ||
        !encode_byte_rows(&maps[1], a.b, (uint64_t)a.K / 2, (uint64_t)a.N, (uint64_t)a.ld_b, 128) ||
        !encode_scale_blocks(&maps[3], a.scales_b, across, (uint64_t)up(a.N, 128), box_k, 1))
      return cudaErrorInvalidValue;
    s.func = fp4_few_kernel(nv, f32);
    s.grid = dim3((unsigned)(tiles * p.split), 1, 1);
    s.block = dim3(kFp4FewThreads, 1, 1);
    s.smem = fp4_few_smem(nv, p.tokens, p.stages);
    s.cluster = (unsigned)p.split;
  }
  const cudaError_t err = allow_smem_once(s.func, 232448);
  if (err != cudaSuccess) return err;
  return launch_spec(s, args, st);
}

}  // namespace dgb
