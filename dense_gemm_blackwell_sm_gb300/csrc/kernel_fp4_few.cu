// kernel_fp4_few.cu -- the 4-bit product where there are few tiles for CTA pairs: few tokens, or
// small layers.
//
// The roles of the operands are exchanged: 128 rows of B (a layer's features) are the MMA's M,
// up to 128 rows of A (tokens) its N, so that a decoded token costs an MMA of 16 columns and
// B's rows stream through shared memory once.  A cluster of `split` CTAs shares a tile's sum:
// each takes a part of K, the partial sums meet in distributed shared memory, in a fixed order.
// Two CTAs fit an SM, so that one's copies run while the other ends.
//
// Warp 0 is the TMA producer, warp 1 copies the scales into TMEM and issues the MMAs, and all
// eight warps then add, scale and store.
#include <algorithm>
#include <type_traits>

#include "fp4_common.cuh"

namespace dgb {

namespace {

constexpr uint32_t kOperand = 128u * 128u;
constexpr int kMostStages = 6;

// TMEM columns of a CTA, the first of its scales, and the stages those and shared memory hold
struct FewShape {
  uint32_t columns, scale_col;
  int stages;
};

template <bool NV>
constexpr uint32_t kSlot = 8u * kScaleBlocks<NV>;  // TMEM columns of a stage's scales


// Sums [begin, end) of a tile's [token][feature] from the cluster's SPLIT CTAs, in the order of
// their ranks, to c: V neighbours a time.  What a thread reads from the CTAs is under way
// together (8 groups of 4 or 8 single values): one after the other, eight reads of distributed
// shared memory took 2 us.
__host__ __device__ inline uint32_t stage_bytes(int blocks, int tokens) {
  return kOperand + (uint32_t)tokens * 128u + 2u * 512u * (uint32_t)blocks;
}

__host__ __device__ inline FewShape few_shape(int blocks, int tokens) {
  // (227 KB for two CTAs, 1 KB of each the system's; for three with fewer stages 1 x 14336 x 4096
  // takes 9.4 us, for two 8.3)
  const uint32_t room = 111u * 1024u;
  FewShape f{256u, tokens <= 32 ? 32u : 64u, 0};
  const int in_tmem = (int)((f.columns - f.scale_col) / (8u * (uint32_t)blocks));
  const int in_room = (int)((room - 2048u) / stage_bytes(blocks, tokens));
  f.stages = in_tmem < in_room ? in_tmem : in_room;
  if (f.stages > kMostStages) f.stages = kMostStages;
  return f;
}

template <int V, int SPLIT, typename OutT>
__device__ __forceinline__ void few_finish(const Fp4Params& p, const float* partial, int32_t begin, int32_t end,
                                           int32_t row0, int32_t col0) {
  constexpr int U = (V == 4 ? 8 : 16) / SPLIT;
  using Word = typename std::conditional<V == 1, OutT, typename std::conditional<sizeof(OutT) == 4, uint4, uint2>::type>::type;
  constexpr int kStep = kFp4FewThreads * V;
  const Fp4Epilogue& e = p.e;
  uint32_t from[SPLIT];
#pragma unroll
  for (int r = 0; r < SPLIT; ++r) from[r] = SPLIT == 1 ? smem_u32(partial) : mapa_shared(smem_u32(partial), (uint32_t)r);
#pragma unroll 1
  for (int32_t i0 = begin + (int32_t)threadIdx.x * V; i0 < end; i0 += kStep * U) {
    float y[U][SPLIT][V];
    Word res[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t i = min(i0 + u * kStep, end - V);  // (a multiple of V)
      const int32_t col = col0 + i % 128;
      if (e.residual != nullptr && col + V <= e.N)
        res[u] = *reinterpret_cast<const Word*>(reinterpret_cast<const OutT*>(e.residual) +
                                                (int64_t)(row0 + i / 128) * e.ld_residual + col);
#pragma unroll
      for (int r = 0; r < SPLIT; ++r) {
        if constexpr (SPLIT == 1) {
#pragma unroll
          for (int j = 0; j < V; ++j) y[u][r][j] = partial[i + j];
        } else if constexpr (V == 4) {
          const float4 f = ld_cluster_f32x4(from[r] + 4u * (uint32_t)i);
          y[u][r][0] = f.x;
          y[u][r][1] = f.y;
          y[u][r][2] = f.z;
          y[u][r][3] = f.w;
        } else {
          y[u][r][0] = __uint_as_float(ld_cluster_u32(from[r] + 4u * (uint32_t)i));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t i = i0 + u * kStep;
      const int32_t row = row0 + i / 128, col = col0 + i % 128;
      if (i >= end || col >= e.N) continue;
      // (a group that the matrix' edge cuts goes by single values)
      const bool whole = col + V <= e.N;
      const float sa = e.row_scale_a != nullptr ? __ldg(e.row_scale_a + row) : 1.f;
      float x[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x[j] = y[u][0][j];
#pragma unroll
        for (int r = 1; r < SPLIT; ++r) x[j] += y[u][r][j];
        x[j] *= sa;
        const int32_t c = min(col + j, e.N - 1);
        if (e.row_scale_b != nullptr) x[j] *= __ldg(e.row_scale_b + c);
        if (e.bias != nullptr) x[j] += __ldg(e.bias + c);
      }
      fp4_act(x, e.act);
      OutT* dst = reinterpret_cast<OutT*>(e.c) + (int64_t)row * e.ld_c + col;
      if (whole) {
        OutT* t = reinterpret_cast<OutT*>(&res[u]);
#pragma unroll
        for (int j = 0; j < V; ++j) t[j] = from_f32<OutT>(e.residual != nullptr ? x[j] + to_f32(t[j]) : x[j]);
        *reinterpret_cast<Word*>(dst) = res[u];
      } else {
        const OutT* from_res = reinterpret_cast<const OutT*>(e.residual) + (int64_t)row * e.ld_residual + col;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (col + j >= e.N) break;
          dst[j] = from_f32<OutT>(e.residual != nullptr ? x[j] + to_f32(from_res[j]) : x[j]);
        }
      }
    }
  }
}

template <int V, typename OutT>
__device__ __forceinline__ void few_finish(const Fp4Params& p, const float* partial, int32_t begin, int32_t end,
                                           int32_t row0, int32_t col0) {
  switch (p.split) {
    case 1: return few_finish<V, 1, OutT>(p, partial, begin, end, row0, col0);
    case 2: return few_finish<V, 2, OutT>(p, partial, begin, end, row0, col0);
    case 4: return few_finish<V, 4, OutT>(p, partial, begin, end, row0, col0);
    default: return few_finish<V, 8, OutT>(p, partial, begin, end, row0, col0);
  }
}

template <bool NV, typename OutT>
__global__ void __launch_bounds__(kFp4FewThreads, 2)
    k_fp4_few(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
              const __grid_constant__ Fp4Params p) {
  constexpr uint32_t NB = (uint32_t)kScaleBlocks<NV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = align_1024(smem_raw);
  const uint32_t S = (uint32_t)p.stages, T = (uint32_t)p.tokens;
  const uint32_t STAGE = stage_bytes((int)NB, (int)T);
  const FewShape shape = few_shape((int)NB, (int)T);
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + S * STAGE);
  uint64_t* full = bars;
  uint64_t* empty = bars + kMostStages;
  uint64_t* done = bars + 2 * kMostStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  // (the stage: features, tokens, their scales)
  const uint32_t tokens_at = kOperand, fscales_at = kOperand + T * 128u, tscales_at = fscales_at + 512u * NB;

  const uint32_t warp = warp_idx(), lane = lane_idx();
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(smem_u32(full + s), 1);
      mbar_init(smem_u32(empty + s), 1);
    }
    mbar_init(smem_u32(done), 1);
    *abort_flag = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
  }
  if (warp == 0) {
    tmem_alloc<1>(smem_u32(tmem_slot), shape.columns);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);  // (the same in all lanes, for the compiler)
  const WaitCtl w{abort_flag, p.status, p.timeout_ns, 0};

  const int32_t rank = (int32_t)cluster_ctarank();
  const int32_t tile = (int32_t)(blockIdx.x / (uint32_t)p.split);
  const int32_t tm = tile % p.tiles_m, tn = tile / p.tiles_m;  // tokens, features
  const int32_t token0 = tm * (int32_t)T;
  // (64 tokens are half of a block of scales: the second half is its columns 2 and 3)
  const uint32_t token_col = (uint32_t)(token0 & 127) / 32u;
  const int32_t kb0 = (int32_t)((int64_t)p.blocks * rank / p.split);
  const int32_t nkb = (int32_t)((int64_t)p.blocks * (rank + 1) / p.split) - kb0;

  if (warp == 0 && lane == 0) {
    // -------------------------------------------------------------- producer
    bool skip = (p.debug_flags & QUANT_DEBUG_SKIP_ONE_LOAD) != 0;
    auto features = [&](int32_t j, uint32_t s) {
      const uint32_t st = smem_u32(ring + s * STAGE), fb = smem_u32(full + s);
      mbar_arrive_expect_tx(fb, STAGE);
      if (skip) {
        skip = false;  // test hook: this stage's bytes never all arrive
      } else {
        tma_load_2d(st, &tmB, fb, (kb0 + j) * 128, tn * 128);
      }
      tma_load_3d(st + fscales_at, &tmSB, fb, 0, (kb0 + j) * 4 * (int32_t)NB, tn);
    };
    auto token_rows = [&](int32_t j, uint32_t s) {
      const uint32_t st = smem_u32(ring + s * STAGE), fb = smem_u32(full + s);
      tma_load_2d(st + tokens_at, &tmA, fb, (kb0 + j) * 128, token0);
      tma_load_3d(st + tscales_at, &tmSA, fb, 0, (kb0 + j) * 4 * (int32_t)NB, token0 / 128);
    };
    const int32_t first = min(nkb, (int32_t)S);
    if (p.static_b)
      for (int32_t j = 0; j < first; ++j) features(j, (uint32_t)j);
    wait_for_prior_kernel();
    let_next_kernel_start();
    for (int32_t j = 0; j < nkb; ++j) {
      const uint32_t s = (uint32_t)j % S;
      if (j >= first && !mbar_wait(smem_u32(empty + s), ((uint32_t)j / S & 1u) ^ 1u, w, WAIT_PRODUCER_EMPTY)) break;
      if (j >= first || !p.static_b) features(j, s);
      token_rows(j, s);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------- scales and MMAs
    const uint32_t issue = elect_lane();
    for (int32_t j = 0; j < nkb; ++j) {
      const uint32_t s = (uint32_t)j % S;
      if (!warp_wait(smem_u32(full + s), (uint32_t)j / S & 1u, w, WAIT_MMA_FULL)) break;
      tc_fence_after();
      const uint32_t st = smem_u32(ring + s * STAGE);
      const uint32_t sf = tmem + shape.scale_col + s * kSlot<NV>;
#pragma unroll
      for (uint32_t i = 0; i < NB; ++i) {
        tmem_cp_32x128b_x4<1>(issue, sf + 4u * i, sdesc_rows16(st + fscales_at + 512u * i));
        tmem_cp_32x128b_x4<1>(issue, sf + 4u * NB + 4u * i, sdesc_rows16(st + tscales_at + 512u * i));
      }
      const uint64_t ad = sdesc_k_sw128(st), bd = sdesc_k_sw128(st + tokens_at);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t i = fp4_scale_block<NV>(k);
        if (4 * (kb0 + j) + k < p.steps)
          mma_fp4<1, NV>(issue, tmem, ad + 2 * k, bd + 2 * k, fp4_idesc<NV>(p.idesc, k), sf + 4u * i,
                         sf + 4u * NB + 4u * i + token_col, (uint32_t)(j | k));
      }
      if (issue) mma_commit(smem_u32(empty + s));
      __syncwarp();
    }
    if (issue) mma_commit(smem_u32(done));
  }
  __syncwarp();
  wait_for_prior_kernel();
  bool ok = warp_wait(smem_u32(done), 0, w, WAIT_LADDER_MMA);
  ok = __syncthreads_and(ok && *abort_flag == 0u) != 0;

  // The partial sums, [token][feature], where the stages were; each CTA of the cluster then
  // adds its share of them.
  float* partial = reinterpret_cast<float*>(ring);
  const int32_t tokens = min((int32_t)T, p.e.M - token0);
  if (ok) {
    tc_fence_after();
    // (warps 4-7 take every other 16 tokens)
    const uint32_t feature = (warp & 3u) * 32u + lane;
#pragma unroll 1
    for (int32_t t0 = 16 * (int32_t)(warp >> 2); t0 < tokens; t0 += 32) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(tmem + (((warp & 3u) * 32u) << 16) + (uint32_t)t0, v);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) partial[(t0 + j) * 128 + feature] = __uint_as_float(v[j]);
    }
  }
  if (p.split > 1) {
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  if (ok) {
    // (features of a tile that the matrix has; groups of four, or single ones where rows are not
    // aligned to groups)
    const int32_t total = tokens * 128;
    const int32_t share = ((total + p.split - 1) / p.split + 127) / 128 * 128;
    const int32_t begin = rank * share, end = min(total, begin + share);
    if (p.e.vec != 0) {
      few_finish<4, OutT>(p, partial, begin, end, token0, tn * 128);
    } else {
      few_finish<1, OutT>(p, partial, begin, end, token0, tn * 128);
    }
  }
  if (!ok && threadIdx.x == 0) {
    // copies in flight must land before shared memory is released
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {}
  }
  if (p.split > 1) cluster_sync_all();  // no partial sums go away before they are read
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, shape.columns);
  }
}

}  // namespace

const void* fp4_few_kernel(bool nv, bool out_f32) {
  if (nv)
    return out_f32 ? reinterpret_cast<const void*>(k_fp4_few<true, float>)
                   : reinterpret_cast<const void*>(k_fp4_few<true, __nv_bfloat16>);
  return out_f32 ? reinterpret_cast<const void*>(k_fp4_few<false, float>)
                 : reinterpret_cast<const void*>(k_fp4_few<false, __nv_bfloat16>);
}

int fp4_few_stages(bool nv, int tokens) { return few_shape(nv ? 4 : 2, tokens).stages; }

size_t fp4_few_smem(bool nv, int tokens, int stages) {
  return 1024 + (size_t)stages * stage_bytes(nv ? 4 : 2, tokens) + (2 * kMostStages + 1) * 8 + 16;
}

}  // namespace dgb
