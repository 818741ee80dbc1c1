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

// What the kernels are told, from a product's or a linear layer's arguments.
template <typename Args>
Fp4Params params_of(const Args& a, int64_t K, const FfnDevice& dev) {
  const int64_t e = a.out_dtype == FFN_F32 ? 4 : 2;
  Fp4Params p{};
  p.e.M = (int32_t)a.M;
  p.e.N = (int32_t)a.N;
  p.e.act = a.activation;
  p.e.vec = aligned_rows(a.c, a.ld_c * e) && aligned_rows(a.residual, a.ld_residual * e);
  p.e.row_scale_b = a.row_scale_b;
  p.e.bias = a.bias;
  p.e.residual = a.residual;
  p.e.c = a.c;
  p.e.ld_residual = a.ld_residual;
  p.e.ld_c = a.ld_c;
  p.steps = (int32_t)up(K, 64);
  p.blocks = (int32_t)up(K, 256);
  p.debug_flags = (uint32_t)a.debug_flags;
  p.status = dev.status;
  p.timeout_ns = a.timeout_ns ? (uint64_t)a.timeout_ns : 2000000000ull;
  p.static_b = (a.flags & QUANT_STATIC_B) != 0;
  return p;
}

constexpr int kSplitSms = 152;

// CTAs that share a sum where there are few tiles: as many as let all CTAs be on the device at
// once, two an SM.
int split_of(int64_t tiles, int32_t blocks, int num_sms) {
  int split = 1;
  while (split < 8 && split * 2 <= blocks && tiles * split * 2 <= 2 * (int64_t)num_sms) split *= 2;
  return split;
}

}  // namespace

// Every CTA quantises its part of the tokens, and with a scale a token reads all of them for it:
// that work, in stages of K a token, is done for every 128 features again, where a launch of its
// own does it once.  MXFP4 in one kernel and in two: 1 x 14336 x 4096 (8 stages) 7.8 and 8.6 us, 4
// tokens (32) 8.3 and 8.7, 8 tokens (64) 9.9 and 8.8; 16 x 4096 x 4096 (32) 7.0 and 7.0.  NVFP4:
// 1 x 38400 x 2048 (16) 11.0 and 12.5, 1 x 14336 x 4096 (24) 10.0 and 9.6, 1 x 4096 x 14336 (63)
// 10.0 and 10.1, 4 x 4096 x 4096 (72) 8.2 and 7.0; the host makes one launch for two, 3 us less.  (That
// decides the cases beside the border: a graph's replay, which pays no launches, would take
// 1 x 14336 x 4096 NVFP4 in two.)
bool fp4_linear_fused(const quant_linear_t& a) {
  if (a.M > 16) return false;
  const int64_t blocks = up(width_of(a.K), 256), tiles = up(a.N, 128);
  // (the split as on the device the library is for, so that this is known without one)
  const int64_t kb = up(blocks, split_of(tiles, (int32_t)blocks, kSplitSms));
  if (kb > 8) return false;  // (a CTA holds its part of all tokens, 4 KB a stage)
  return a.M * (kb + (a.format == QUANT_NVFP4 ? blocks : 0)) <= 32;
}

cudaError_t launch_fp4_linear(const quant_linear_t& a, const FfnDevice& dev, cudaStream_t st) {
  const bool nv = a.format == QUANT_NVFP4, f32 = a.out_dtype == FFN_F32;
  const int64_t K = width_of(a.K), e = a.dtype == FFN_F32 ? 4 : 2;
  Fp4Params p = params_of(a, K, dev);
  p.tokens = 16;
  p.tiles_m = 1;
  p.tiles_n = (int32_t)up(a.N, 128);
  p.split = split_of(p.tiles_n, p.blocks, kSplitSms);
  const int kb = (int)up(p.blocks, p.split);
  p.stages = fp4_linear_stages(nv, kb);
  p.idesc = idesc_fp4(!nv, 128, 16);
  Fp4Tokens x{};
  x.x = a.x;
  x.x_end = end_of_rows(a.x, a.M, a.ld_x, a.K, e);
  x.ld_x = a.ld_x;
  x.K = (int32_t)a.K;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | (uintptr_t)(a.ld_x * e);
  x.vec = (bits & 31u) == 0 ? 2 : (bits & 15u) == 0 ? 1 : 0;
  CUtensorMap maps[2];
  if (!encode_byte_rows(&maps[0], a.b, (uint64_t)K / 2, (uint64_t)a.N, (uint64_t)a.ld_b, 128) ||
      !encode_scale_blocks(&maps[1], a.scales_b, (uint64_t)up(scales_of(K, a.format), 4), (uint64_t)up(a.N, 128),
                           nv ? 4 : 2, 1))
    return cudaErrorInvalidValue;
  LaunchSpec s;
  s.pdl = true;
  s.func = fp4_linear_kernel(nv, f32, a.dtype);
  s.grid = dim3((unsigned)(p.tiles_n * p.split), 1, 1);
  s.block = dim3(kFp4FewThreads, 1, 1);
  s.smem = fp4_linear_smem(nv, kb, p.stages);
  s.cluster = (unsigned)p.split;
  const cudaError_t err = allow_smem_once(s.func, 232448);
  if (err != cudaSuccess) return err;
  void* args[] = {&maps[0], &maps[1], &p, &x};
  return launch_spec(s, args, st);
}

cudaError_t launch_fp4_product(const quant_product_t& a, const FfnDevice& dev, cudaStream_t st) {
  const bool nv = a.format == QUANT_NVFP4, f32 = a.out_dtype == FFN_F32;
  Fp4Params p = params_of(a, a.K, dev);
  p.e.row_scale_a = a.row_scale_a;

  const uint32_t box_k = nv ? 4 : 2;  // scale blocks of a stage
  const uint64_t across = (uint64_t)up(scales_of(a.K, a.format), 4);
  CUtensorMap maps[5];
  LaunchSpec s;
  s.pdl = true;
  void* pair_args[] = {&maps[0], &maps[1], &maps[2], &maps[3], &maps[4], &p};
  void* few_args[] = {&maps[0], &maps[1], &maps[2], &maps[3], &p};
  void** args = few_args;
  if (!encode_scale_blocks(&maps[2], a.scales_a, across, (uint64_t)up(a.M, 128), box_k, 1)) return cudaErrorInvalidValue;

  if (fp4_on_pairs(a.M, a.N, a.K, dev.num_sms)) {
    const int64_t pair_tiles = up(a.M, 256) * up(a.N, 256);
    p.tiles_m = (int32_t)up(a.M, 256);
    p.tiles_n = (int32_t)up(a.N, 256);
    // (both operands lie in L2 at sizes where that matters: 32 rows of tiles against 8 take 8192 x
    // 14336 x 4096 NVFP4 from 156 to 149 us, 8192^3 from 166 to 162)
    p.raster_group = std::min(32, p.tiles_m);
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
    p.split = split_of(tiles, p.blocks, dev.num_sms);
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
