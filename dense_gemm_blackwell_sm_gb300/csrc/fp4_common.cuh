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

// A bounded wait of a whole warp: every lane looks for the phase itself (the acquire is a
// thread's own) and all leave together.  It calls nothing and no lane runs ahead: what the warp's
// loop keeps in uniform registers must not live across a call that one lane makes.  All of these
// kernels' loops wait like this, those that copy among them.
template <bool CLUSTER_ACQ = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtl& w, uint32_t code) {
  uint64_t since = 0;
  for (uint32_t spins = 1;; ++spins) {
    if (__all_sync(0xffffffffu, CLUSTER_ACQ ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity))) return true;
    if ((spins & 15u) != 0u) continue;
    const uint64_t now = globaltimer_ns();
    if (spins == 16u) since = now;
    const bool late = now - since > w.timeout_ns && now > since;
    if (late) raise_abort(w, code);  // (the first code stays)
    if (__any_sync(0xffffffffu, late || *w.abort_flag != 0u)) return false;
  }
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

// 16 bytes of residuals of a row from column col on, zeros behind the last column (rows are aligned)
template <typename OutT>
__device__ __forceinline__ uint4 residual16(const Fp4Epilogue& e, int32_t row, int32_t col) {
  constexpr int n = 16 / (int)sizeof(OutT);
  const OutT* src = reinterpret_cast<const OutT*>(e.residual) + (int64_t)row * e.ld_residual + col;
  if (col + n <= e.N) return *reinterpret_cast<const uint4*>(src);
  uint4 u = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int j = 0; j < n; ++j)
    if (col + j < e.N) reinterpret_cast<OutT*>(&u)[j] = src[j];
  return u;
}

// A lane's 32 residuals, of its row and of columns col .. col + 31: bf16 ones are loaded ahead of
// their use, 32 of fp32 leave no registers for that and are loaded where they are added.  (A tile's
// rows by neighbouring lanes, or fetched to L2 before, gain at most 5 %.)
template <typename OutT>
struct Residual32 {
  uint4 u[4];
  __device__ __forceinline__ void load(const Fp4Epilogue& e, int32_t row, int32_t col) {
    if constexpr (sizeof(OutT) == 2) {
      if (e.residual == nullptr || e.vec == 0 || row >= e.M) return;
#pragma unroll
      for (int q = 0; q < 4; ++q) u[q] = residual16<OutT>(e, row, col + 8 * q);
    }
  }
};

// 32 x 32 sums, a lane's row in v, of columns col .. col + 31, to c: scaled, finished, rounded
// into `staging` (4096 bytes of the warp's, 1024-byte aligned) and stored from there, by a TMA
// copy where c's rows are aligned to 16 bytes (tmC: boxes of 32 x 32, swizzled over 128 bytes for
// fp32 and 64 for bf16), else by the lanes, each a column, so that they write neighbours.
// A TMA store writes whole 16-byte pieces, also of a last one that C's columns end inside of; where
// rows lie in a wider array that is somebody else's memory, so such a run of columns goes by the lanes.
// `res`: the residuals; `scale` and `bias`: the columns' values in shared memory.  Every lane of
// the warp calls it; `buffer` counts the warp's copies: bf16 takes the halves of the staging space
// in turn.
template <typename OutT>
__device__ __forceinline__ void fp4_store32(const Fp4Epilogue& e, const CUtensorMap* tmC, const uint32_t (&v)[32],
                                            const Residual32<OutT>& res, int32_t row0, int32_t col, float sa,
                                            const float* scale, const float* bias, uint8_t* staging, uint32_t& buffer,
                                            uint32_t lane) {
  if (row0 >= e.M || col >= e.N) return;
  const int32_t row = row0 + (int32_t)lane;
  float x[32];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float4 s = reinterpret_cast<const float4*>(scale)[j], b = reinterpret_cast<const float4*>(bias)[j];
    x[4 * j] = fmaf(__uint_as_float(v[4 * j]) * sa, s.x, b.x);
    x[4 * j + 1] = fmaf(__uint_as_float(v[4 * j + 1]) * sa, s.y, b.y);
    x[4 * j + 2] = fmaf(__uint_as_float(v[4 * j + 2]) * sa, s.z, b.z);
    x[4 * j + 3] = fmaf(__uint_as_float(v[4 * j + 3]) * sa, s.w, b.w);
  }
  fp4_act(x, e.act);
  constexpr int per16 = 16 / (int)sizeof(OutT);
  if (e.vec != 0 && (col + 32 <= e.N || e.N % per16 == 0)) {
    if (e.residual != nullptr && row < e.M) {
#pragma unroll
      for (int q = 0; q < 32 / per16; ++q) {
        uint4 u;
        if constexpr (sizeof(OutT) == 2) u = res.u[q];
        else u = residual16<OutT>(e, row, col + q * per16);
        const OutT* w = reinterpret_cast<const OutT*>(&u);
#pragma unroll
        for (int j = 0; j < per16; ++j) x[q * per16 + j] += to_f32(w[j]);
      }
    }
    uint8_t* buf = staging + (sizeof(OutT) == 2 ? (buffer++ & 1u) * 2048u : 0u);
    // the copy issued from this buffer before has read it
    if (lane == 0) bulk_wait_group_read<sizeof(OutT) == 2 ? 1 : 0>();
    __syncwarp();
#pragma unroll
    for (uint32_t j = 0; j < 32 / per16; ++j) {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(OutT) == 4) o[i] = __float_as_uint(x[4 * j + i]);
        else o[i] = pack_bf16x2(__float_as_uint(x[8 * j + 2 * i]), __float_as_uint(x[8 * j + 2 * i + 1]));
      }
      // (64-byte rows swizzled: the 16-byte piece's index takes bits 1 and 2 of the row)
      const uint32_t at = sizeof(OutT) == 4 ? sw128_offset(lane, j) : lane * 64u + ((j ^ ((lane >> 1) & 3u)) << 4);
      *reinterpret_cast<uint4*>(buf + at) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(tmC, smem_u32(buf), col, row0);
      bulk_commit_group();
    }
    return;
  }
  float* rows = reinterpret_cast<float*>(staging);
  if (e.vec != 0 && lane == 0) bulk_wait_group_read<0>();  // (copies of other runs have read the space)
  __syncwarp();
#pragma unroll
  for (uint32_t j = 0; j < 32; ++j) rows[lane * 32u + (j ^ lane)] = x[j];
  __syncwarp();
  if (col + (int32_t)lane < e.N) {
    const int32_t n = min(32, e.M - row0);
    OutT* dst = reinterpret_cast<OutT*>(e.c) + (int64_t)row0 * e.ld_c + col + lane;
    const OutT* src = reinterpret_cast<const OutT*>(e.residual);
    if (src != nullptr) src += (int64_t)row0 * e.ld_residual + col + lane;
#pragma unroll 4
    for (int32_t r = 0; r < n; ++r) {
      float y = rows[r * 32 + (int32_t)(lane ^ (uint32_t)r)];
      if (src != nullptr) y += to_f32(src[(int64_t)r * e.ld_residual]);
      dst[(int64_t)r * e.ld_c] = from_f32<OutT>(y);
    }
  }
}

}  // namespace dgb
