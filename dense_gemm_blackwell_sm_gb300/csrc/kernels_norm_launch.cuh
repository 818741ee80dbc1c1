// kernels_norm_launch.cuh -- launches of the block norms' kernels for one element
// type and one parameter type.
#pragma once

#include <algorithm>

#include "kernels_norm.cuh"
#include "kernels_norm_ring.cuh"
#include "launch.h"

namespace dgb {

namespace {

inline cudaError_t launch_dependent(const void* f, dim3 grid, int threads, int cluster, size_t smem, void** args,
                                    cudaStream_t st) {
  LaunchSpec s;
  s.func = f;
  s.grid = grid;
  s.block = dim3((unsigned)threads, 1, 1);
  s.cluster = (unsigned)cluster;
  s.smem = smem;
  s.pdl = true;
  if (smem > 0) {
    const cudaError_t e = allow_smem_once(f, kNormRingBytes);
    if (e != cudaSuccess) return e;
  }
  return launch_spec(s, args, st);
}

template <typename T, typename P, bool LAYER>
const void* norm_kernel(const NormShape& sh) {
  constexpr int MOST = norm_most_vectors((int)sizeof(T));
  if (sh.warp_rows) {
    switch (sh.nv) {
      case 1: return (const void*)k_norm<T, P, LAYER, true, 1, 256>;
      case 2: return (const void*)k_norm<T, P, LAYER, true, 2, 256>;
      default: return (const void*)k_norm<T, P, LAYER, true, 4, 256>;
    }
  }
  if (sh.threads > 512) return (const void*)k_norm<T, P, LAYER, false, MOST, 1024>;
  switch (sh.nv) {
    case 1: return (const void*)k_norm<T, P, LAYER, false, 1, 512>;
    case 2: return (const void*)k_norm<T, P, LAYER, false, 2, 512>;
    case 4: return (const void*)k_norm<T, P, LAYER, false, 4, 512>;
    default: return (const void*)k_norm<T, P, LAYER, false, MOST, 512>;
  }
}

template <typename T, typename P, bool LAYER>
const void* norm_ring_kernel(const NormShape& sh) {
  if (sh.warp_rows) {
    switch (sh.nv) {
      case 1: return (const void*)k_norm_ring<T, P, LAYER, true, 1>;
      case 2: return (const void*)k_norm_ring<T, P, LAYER, true, 2>;
      default: return (const void*)k_norm_ring<T, P, LAYER, true, 4>;
    }
  }
  if constexpr (!LAYER) {
    if (sh.nv == 4) return (const void*)k_norm_ring<T, P, false, false, 4>;
  }
  return (const void*)k_norm_ring<T, P, LAYER, false, 2>;
}

template <typename T, typename P>
cudaError_t norm_forward(const ffn_norm_t& a, const NormShape& direct, const NormShape* ring, const FfnDevice& dev,
                         cudaStream_t st) {
  const bool layer = a.kind == FFN_NORM_LAYER;
  ffn_norm_t args_a = a;
  uint32_t* status = dev.status;
  if (ring != nullptr) {
    NormShape sh = *ring;
    const void* k = layer ? norm_ring_kernel<T, P, true>(sh) : norm_ring_kernel<T, P, false>(sh);
    int per_sm = 0;
    const cudaError_t e = resident_ctas(k, sh.threads, sh.smem, kNormRingBytes, &per_sm);
    if (e != cudaSuccess) return e;
    // (a CTA of warps holds whole periods of parts: 8 is a multiple of every period)
    const int64_t unit = sh.warp_rows ? 1 : sh.period, groups = sh.warp_rows ? sh.threads / 32 : 1;
    sh.grid = std::max<int64_t>(unit, (int64_t)per_sm * dev.num_sms / unit * unit);
    if (a.M >= 2 * sh.grid * groups) {
      sh.share = NormShare::of((a.M + sh.period - 1) / sh.period, sh.grid * groups / sh.period);
      void* args[] = {&args_a, &sh, &status};
      return launch_dependent(k, dim3((unsigned)sh.grid), sh.threads, 1, sh.smem, args, st);
    }
  }
  void* args[] = {&args_a};
  return launch_dependent(layer ? norm_kernel<T, P, true>(direct) : norm_kernel<T, P, false>(direct),
                          dim3((unsigned)direct.grid), direct.threads, 1, 0, args, st);
}

template <typename T, typename P, bool LAYER, bool BIAS>
const void* norm_grad_kernel(const NormGradShape& sh) {
  if (sh.many) return (const void*)k_norm_grad<T, P, false, LAYER, BIAS, true, 2>;
  if (sh.each == 8)
    return sh.full ? (const void*)k_norm_grad<T, P, true, LAYER, BIAS, false, 1>
                   : (const void*)k_norm_grad<T, P, false, LAYER, BIAS, false, 1>;
  return sh.full ? (const void*)k_norm_grad<T, P, true, LAYER, BIAS, false, 2>
                 : (const void*)k_norm_grad<T, P, false, LAYER, BIAS, false, 2>;
}

template <typename T, typename P>
cudaError_t norm_backward(const ffn_norm_grad_t& a, const NormGradShape& sh, const NormSums& ws, const FfnDevice& dev,
                          cudaStream_t st) {
  const void* k = a.kind == FFN_NORM_LAYER
                      ? (sh.bias ? norm_grad_kernel<T, P, true, true>(sh) : norm_grad_kernel<T, P, true, false>(sh))
                      : (sh.bias ? norm_grad_kernel<T, P, false, true>(sh) : norm_grad_kernel<T, P, false, false>(sh));
  ffn_norm_grad_t args_a = a;
  NormGradShape args_sh = sh;
  NormSums args_ws = ws;
  uint32_t* status = dev.status;
  void* args[] = {&args_a, &args_sh, &args_ws, &status};
  const unsigned grid = (unsigned)((sh.parts + sh.lanes - 1) / sh.lanes * sh.cluster);
  cudaError_t e = launch_dependent(k, dim3(grid), sh.threads * sh.lanes, sh.cluster, sh.smem, args, st);
  if (e != cudaSuccess) return e;
  const bool totals = a.dpost_weight || a.dpost_bias || a.dpre_weight || a.dpre_bias;
  const bool gates = a.dgate != nullptr && !sh.many;
  if (!totals && !gates) return cudaSuccess;
  // one gate for all rows: its sum is the total; else a layer of CTAs per group.  Short
  // rows take 8 columns per CTA, so that there are CTAs for the parts
  const bool narrow = a.D <= 1024;
  const dim3 sums((unsigned)(narrow ? (a.D + 7) / 8 : (a.D + 31) / 32),
                  1u + (gates && a.groups > 1 ? (unsigned)a.groups : 0u));
  // four parts per lane where there are few; and no more threads than the device holds
  // while a lane's parts are at most 16 (1000 x 1001 fp32 with 8 gates 31.4 -> 22.7 us;
  // 4000 x 300 with 16 gates has 1520 parts: 27.3, with fewer threads 35.6)
  int threads = sh.parts <= 128 ? 256 : sh.parts <= 256 ? 512 : 1024;
  while (threads > 256 && (int64_t)sums.x * sums.y * threads > (int64_t)dev.num_sms * 2048 &&
         sh.parts * (narrow ? 8 : 32) <= 8 * threads)
    threads /= 2;
  int element_bytes = (int)sizeof(T);
  void* sums_args[] = {&args_a, &args_sh, &args_ws, &element_bytes};
  return launch_dependent(narrow ? (const void*)k_norm_column_sums<P, 8> : (const void*)k_norm_column_sums<P, 32>, sums,
                          threads, 1, 0, sums_args, st);
}

}  // namespace

}  // namespace dgb
