// fp4_common.cuh -- the epilogue of the 4-bit product's kernels.
#pragma once

#include "ffn_common.cuh"
#include "fp4.h"

namespace dgb {

// Scale blocks (128 rows x 4 scales, 512 bytes) of a stage of 256 K-elements: four with a scale
// per 16 elements, two with one per 32.
template <bool NV>
inline constexpr int kScaleBlocks = NV ? 4 : 2;

// The k-th MMA of a stage takes scale block k (NV), or block k / 2 and its bytes 0, 1 or 2, 3.
template <bool NV>
__device__ __forceinline__ uint32_t fp4_scale_block(int k) { return NV ? (uint32_t)k : (uint32_t)(k / 2); }
template <bool NV>
__device__ __forceinline__ uint32_t fp4_idesc(uint32_t idesc, int k) {
  if (NV) return idesc;
  const uint32_t id = 2u * (uint32_t)(k & 1);
  return idesc | (id << 4) | (id << 29);
}

// A bounded wait of a whole warp: one lane's answer for all.
template <bool CLUSTER_ACQ = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtl& w, uint32_t code) {
  if (__all_sync(0xffffffffu, CLUSTER_ACQ ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity))) return true;
  uint32_t ok = 1;
  if (lane_idx() == 0) ok = mbar_wait_slow<CLUSTER_ACQ>(bar, parity, w, code) ? 1u : 0u;
  // (every lane has to see the phase itself: the acquire is a thread's own)
  ok = __shfl_sync(0xffffffffu, ok, 0);
  if (ok) ok = CLUSTER_ACQ ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
  return __all_sync(0xffffffffu, ok != 0u);
}

template <int N>
__device__ __forceinline__ void fp4_act(float (&x)[N], int32_t act) {
  switch (act) {
    case EPI_ACT_RELU:
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = x[j] < 0.f ? 0.f : x[j];
      break;
    case EPI_ACT_SILU:
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = act_only<EPI_ACT_SILU>(x[j]);
      break;
    case EPI_ACT_GELU_TANH:
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = act_only<EPI_ACT_GELU_TANH>(x[j]);
      break;
    case EPI_ACT_GELU_ERF:
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = act_only<EPI_ACT_GELU_ERF>(x[j]);
      break;
    default: break;
  }
}

// 32 sums of row `row`, columns col .. col + 31 (fewer at the matrix' edge), to c.  A lane has a
// row; where rows are not aligned the values go through `staging` (32 x 33 floats of the
// warp's) so that lanes write neighbours.  Every lane of the warp calls it; rows past M are
// left out.
template <typename OutT>
__device__ __forceinline__ void fp4_store32(const Fp4Epilogue& e, const uint32_t (&v)[32], int32_t row0, int32_t col,
                                            float sa, float* staging, uint32_t lane) {
  const int32_t row = row0 + (int32_t)lane;
  const int32_t n = min(32, e.N - col);
  if (n <= 0 || row0 >= e.M) return;
  float x[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(v[j]) * sa;
  const bool whole = n == 32;
  auto columns = [&](const float* p, auto apply) {
    if (p == nullptr) return;
    if (whole && (reinterpret_cast<uintptr_t>(p + col) & 15u) == 0) {
      const float4* q = reinterpret_cast<const float4*>(p + col);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 f = __ldg(q + j);
        apply(x[4 * j], f.x);
        apply(x[4 * j + 1], f.y);
        apply(x[4 * j + 2], f.z);
        apply(x[4 * j + 3], f.w);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < n) apply(x[j], __ldg(p + col + j));
    }
  };
  columns(e.row_scale_b, [](float& a, float b) { a *= b; });
  columns(e.bias, [](float& a, float b) { a += b; });
  fp4_act(x, e.act);
  constexpr int per16 = 16 / (int)sizeof(OutT);
  if (e.vec != 0 && (whole || n % per16 == 0)) {
    if (row >= e.M) return;
    OutT* dst = reinterpret_cast<OutT*>(e.c) + (int64_t)row * e.ld_c + col;
    if (e.residual != nullptr) {
      const OutT* src = reinterpret_cast<const OutT*>(e.residual) + (int64_t)row * e.ld_residual + col;
#pragma unroll
      for (int q = 0; q < 32 / per16; ++q) {
        if (q * per16 >= n) break;
        const uint4 u = *reinterpret_cast<const uint4*>(src + q * per16);
        const OutT* w = reinterpret_cast<const OutT*>(&u);
#pragma unroll
        for (int j = 0; j < per16; ++j) x[q * per16 + j] += to_f32(w[j]);
      }
    }
    uint32_t o[8 * sizeof(OutT)];
    if constexpr (sizeof(OutT) == 4) {
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(x[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = pack_bf16x2(__float_as_uint(x[2 * j]), __float_as_uint(x[2 * j + 1]));
    }
    constexpr int words = (int)(8 * sizeof(OutT));
    if (e.vec == 2 && whole) {
#pragma unroll
      for (int j = 0; j < words / 8; ++j) st_global_v8(reinterpret_cast<uint32_t*>(dst) + 8 * j, o + 8 * j);
    } else {
#pragma unroll
      for (int j = 0; j < words / 4; ++j)
        if (j * per16 < n)
          reinterpret_cast<uint4*>(dst)[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
    }
    return;
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 32; ++j) staging[lane * 33 + j] = x[j];
  __syncwarp();
  if ((int32_t)lane < n) {
    const int32_t rows = min(32, e.M - row0);
    OutT* dst = reinterpret_cast<OutT*>(e.c) + (int64_t)row0 * e.ld_c + col + lane;
    const OutT* src = reinterpret_cast<const OutT*>(e.residual);
    if (src != nullptr) src += (int64_t)row0 * e.ld_residual + col + lane;
    for (int32_t r = 0; r < rows; ++r) {
      float y = staging[r * 33 + lane];
      if (src != nullptr) y += to_f32(src[(int64_t)r * e.ld_residual]);
      dst[(int64_t)r * e.ld_c] = from_f32<OutT>(y);
    }
  }
  __syncwarp();
}

}  // namespace dgb
