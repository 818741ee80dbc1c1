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
// four warps then add, scale and store.
#include <algorithm>

#include "fp4_common.cuh"

namespace dgb {

namespace {

constexpr uint32_t kOperand = 128u * 128u;
constexpr uint32_t kTmemColumns = 256;
constexpr uint32_t kScaleCol = 128;
constexpr int kMostStages = 4;
constexpr uint32_t kRoom = 110u * 1024u;  // of shared memory, for two CTAs on an SM

template <bool NV>
constexpr uint32_t kSlot = 8u * kScaleBlocks<NV>;  // TMEM columns of a stage's scales
static_assert(kScaleCol + kMostStages * kSlot<true> <= kTmemColumns, "scales fit TMEM");

__host__ __device__ inline uint32_t stage_bytes(int blocks, int tokens) {
  return kOperand + (uint32_t)tokens * 128u + 2u * 512u * (uint32_t)blocks;
}

template <bool NV, typename OutT>
__global__ void __launch_bounds__(kFp4FewThreads)
    k_fp4_few(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
              const __grid_constant__ Fp4Params p) {
  constexpr uint32_t NB = (uint32_t)kScaleBlocks<NV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = align_1024(smem_raw);
  const uint32_t S = (uint32_t)p.stages, T = (uint32_t)p.tokens;
  const uint32_t STAGE = stage_bytes((int)NB, (int)T);
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
    tmem_alloc<1>(smem_u32(tmem_slot), kTmemColumns);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl w{abort_flag, p.status, p.timeout_ns, 0};

  const int32_t rank = (int32_t)cluster_ctarank();
  const int32_t tile = (int32_t)(blockIdx.x / (uint32_t)p.split);
  const int32_t tm = tile % p.tiles_m, tn = tile / p.tiles_m;  // tokens, features
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
      tma_load_2d(st + tokens_at, &tmA, fb, (kb0 + j) * 128, tm * 128);
      tma_load_3d(st + tscales_at, &tmSA, fb, 0, (kb0 + j) * 4 * (int32_t)NB, tm);
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
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------- scales and MMAs
    for (int32_t j = 0; j < nkb; ++j) {
      const uint32_t s = (uint32_t)j % S;
      if (!mbar_wait(smem_u32(full + s), (uint32_t)j / S & 1u, w, WAIT_MMA_FULL)) break;
      tc_fence_after();
      const uint32_t st = smem_u32(ring + s * STAGE);
      const uint32_t sf = tmem + kScaleCol + s * kSlot<NV>;
#pragma unroll
      for (uint32_t i = 0; i < NB; ++i) {
        tmem_cp_32x128b_x4<1>(sf + 4u * i, sdesc_rows16(st + fscales_at + 512u * i));
        tmem_cp_32x128b_x4<1>(sf + 4u * NB + 4u * i, sdesc_rows16(st + tscales_at + 512u * i));
      }
      const uint64_t ad = sdesc_k_sw128(st), bd = sdesc_k_sw128(st + tokens_at);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t i = fp4_scale_block<NV>(k);
        if (4 * (kb0 + j) + k < p.steps)
          mma_fp4<1, NV>(tmem, ad + 2 * k, bd + 2 * k, fp4_idesc<NV>(p.idesc, k), sf + 4u * i, sf + 4u * NB + 4u * i,
                         (uint32_t)(j | k));
      }
      mma_commit(smem_u32(empty + s));
    }
    mma_commit(smem_u32(done));
  }
  __syncwarp();
  wait_for_prior_kernel();
  bool ok = mbar_wait(smem_u32(done), 0, w, WAIT_LADDER_MMA);
  ok = __syncthreads_and(ok && *abort_flag == 0u) != 0;

  // The partial sums, [token][feature], where the stages were; each CTA of the cluster then
  // adds its share of them.
  float* partial = reinterpret_cast<float*>(ring);
  const int32_t tokens = min((int32_t)T, p.e.M - tm * 128);
  if (ok) {
    tc_fence_after();
    const uint32_t feature = warp * 32u + lane;
#pragma unroll 1
    for (int32_t t0 = 0; t0 < tokens; t0 += 16) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(tmem + ((warp * 32u) << 16) + (uint32_t)t0, v);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) partial[(t0 + j) * 128 + feature] = nkb > 0 ? __uint_as_float(v[j]) : 0.f;
    }
  }
  if (p.split > 1) {
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  if (ok) {
    const int32_t total = tokens * 128;
    const int32_t share = ((total + p.split - 1) / p.split + 31) / 32 * 32;
    const int32_t end = min(total, (rank + 1) * share);
    const uint32_t base = smem_u32(partial);
    for (int32_t i = rank * share + (int32_t)threadIdx.x; i < end; i += kFp4FewThreads) {
      float sum = 0.f;
      if (p.split > 1) {
        for (int32_t r = 0; r < p.split; ++r)
          sum += __uint_as_float(ld_cluster_u32(mapa_shared(base + 4u * (uint32_t)i, (uint32_t)r)));
      } else {
        sum = partial[i];
      }
      const int32_t row = tm * 128 + i / 128, col = tn * 128 + i % 128;
      if (col >= p.e.N) continue;
      if (p.e.row_scale_a != nullptr) sum *= __ldg(p.e.row_scale_a + row);
      if (p.e.row_scale_b != nullptr) sum *= __ldg(p.e.row_scale_b + col);
      if (p.e.bias != nullptr) sum += __ldg(p.e.bias + col);
      float x[1] = {sum};
      fp4_act(x, p.e.act);
      if (p.e.residual != nullptr)
        x[0] += to_f32(reinterpret_cast<const OutT*>(p.e.residual)[(int64_t)row * p.e.ld_residual + col]);
      reinterpret_cast<OutT*>(p.e.c)[(int64_t)row * p.e.ld_c + col] = fp4_out<OutT>(x[0]);
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
    tmem_dealloc<1>(tmem, kTmemColumns);
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

int fp4_few_stages(bool nv, int tokens) {
  return (int)std::min<uint32_t>(kMostStages, kRoom / stage_bytes(nv ? 4 : 2, tokens));
}

size_t fp4_few_smem(bool nv, int tokens, int stages) {
  return 1024 + (size_t)stages * stage_bytes(nv ? 4 : 2, tokens) + (2 * kMostStages + 1) * 8 + 16;
}

}  // namespace dgb
