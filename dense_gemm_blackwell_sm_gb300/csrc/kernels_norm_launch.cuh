// kernels_norm_launch.cuh -- launches of the block norms' kernels for one element
// type and one parameter type.
#pragma once

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

template <typename T, typename P, bool ALIGNED, bool LAYER>
const void* norm_ring_kernel(const NormShape& sh) {
  if (sh.warp_rows) {
    switch (sh.nv) {
      case 1: return (const void*)k_norm_ring<T, P, ALIGNED, LAYER, true, 1>;
      case 2: return (const void*)k_norm_ring<T, P, ALIGNED, LAYER, true, 2>;
      default: return (const void*)k_norm_ring<T, P, ALIGNED, LAYER, true, 4>;
    }
  }
  switch (sh.nv) {
    case 1: return (const void*)k_norm_ring<T, P, ALIGNED, LAYER, false, 1>;
    case 2: return (const void*)k_norm_ring<T, P, ALIGNED, LAYER, false, 2>;
    default: return (const void*)k_norm_ring<T, P, ALIGNED, LAYER, false, 4>;
  }
}

template <typename T, typename P>
cudaError_t norm_forward(const ffn_norm_t& a, const NormShape& sh, const FfnDevice& dev, cudaStream_t st) {
  const bool layer = a.kind == FFN_NORM_LAYER;
  ffn_norm_t args_a = a;
  uint32_t* status = dev.status;
  void* args[] = {&args_a, &status};
  const void* k = sh.ring ? (sh.aligned ? (layer ? norm_ring_kernel<T, P, true, true>(sh) : norm_ring_kernel<T, P, true, false>(sh))
                                        : (layer ? norm_ring_kernel<T, P, false, true>(sh)
                                                 : norm_ring_kernel<T, P, false, false>(sh)))
                          : (layer ? norm_kernel<T, P, true>(sh) : norm_kernel<T, P, false>(sh));
  return launch_dependent(k, dim3((unsigned)sh.grid), sh.threads, 1, sh.smem, args, st);
}

template <typename T, typename P, bool LAYER, bool BIAS>
const void* norm_grad_kernel(const NormGradShape& sh) {
  if (sh.aligned)
    return sh.many ? (const void*)k_norm_grad<T, P, true, LAYER, BIAS, true>
                   : (const void*)k_norm_grad<T, P, true, LAYER, BIAS, false>;
  return sh.many ? (const void*)k_norm_grad<T, P, false, LAYER, BIAS, true>
                 : (const void*)k_norm_grad<T, P, false, LAYER, BIAS, false>;
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
  // one gate for all rows: its sum is the total; else a layer of CTAs per group
  const dim3 sums((unsigned)((a.D + 31) / 32), 1u + (gates && a.groups > 1 ? (unsigned)a.groups : 0u));
  return launch_dependent((const void*)k_norm_column_sums<P>, sums, 1024, 1, 0, args, st);
}

}  // namespace

}  // namespace dgb
