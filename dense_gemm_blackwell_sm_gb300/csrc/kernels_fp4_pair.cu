// kernels_fp4_pair.cu -- the product of two microscaled 4-bit operands on CTA pairs.
//
// A pair (cta_group::2) computes a tile of 256 x 256: each CTA brings 128 rows of A and 128 of
// B, 256 K-elements a stage (128 bytes a row), and the block scales of its rows of A and of all
// 256 of B.  tcgen05.mma kind::mxf4 / mxf4nvf4 takes 64 K-elements at a time, with scales that
// tcgen05.cp has moved from shared memory into TMEM; the sums are one 256-column fp32
// accumulator, the scales take the other TMEM columns, a slot a stage.
//
// Roles (384 threads): warp 0 TMA producer, warp 1 MMA, warp 2 allocates TMEM, warp 3 copies the
// scales (one thread's issue rate bounds the MMAs, so the copies have a thread of their own),
// warps 4-11 the epilogue: each takes its part of the accumulator into registers, hands it back
// and then scales and stores it while the next tile's MMAs run.
//
// Every cluster takes the tiles cid, cid + clusters, ...: results depend on the sizes alone.
// Every wait is bounded (ptx.cuh); programmatic launches as in ffn_common.cuh.
#include <algorithm>

#include "fp4_common.cuh"

namespace dgb {

namespace {

constexpr uint32_t kOperand = 128u * 128u;  // 128 rows of 256 4-bit elements
constexpr uint32_t kStaging = 8u * 32u * 33u * 4u;
constexpr uint32_t kCtrl = 512;
constexpr int kMostStages = 8;
constexpr uint32_t kScaleCol = 256;  // first TMEM column of the scales

template <bool NV>
constexpr uint32_t kStage = 2u * kOperand + 3u * 512u * kScaleBlocks<NV>;
template <bool NV>
constexpr uint32_t kSlot = 12u * kScaleBlocks<NV>;  // TMEM columns of a stage's scales

template <bool NV>
__host__ __device__ constexpr int stages_of() {
  int s = kMostStages;
  while (1024u + (uint32_t)s * kStage<NV> + kStaging + kCtrl > 232448u || (uint32_t)s * kSlot<NV> > 256u) --s;
  return s;
}

template <bool NV, typename OutT>
__global__ void __launch_bounds__(kFp4PairThreads, 1)
    k_fp4_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
               const __grid_constant__ Fp4Params p) {
  constexpr uint32_t S = (uint32_t)stages_of<NV>();
  constexpr uint32_t NB = (uint32_t)kScaleBlocks<NV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = align_1024(smem_raw);
  float* staging = reinterpret_cast<float*>(ring + S * kStage<NV>);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(staging) + kStaging);
  uint64_t* full = bars;                     // TMA -> scale copies
  uint64_t* empty = bars + kMostStages;      // MMA -> TMA
  uint64_t* ready = bars + 2 * kMostStages;  // scale copies -> MMA
  uint64_t* acc_full = bars + 3 * kMostStages;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* drain_bar = acc_full + 2;
  uint64_t* copy_drain = acc_full + 3;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 4);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  volatile uint32_t* zero_word = tmem_slot + 2;
  // (the stage's scales follow its operands: A's blocks, B's blocks of rows 0-127, of 128-255)
  constexpr uint32_t kScalesAt = 2u * kOperand;

  const uint32_t warp = warp_idx(), lane = lane_idx();
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(smem_u32(full + s), 1);
      mbar_init(smem_u32(empty + s), 1);
      mbar_init(smem_u32(ready + s), 2);
    }
    mbar_init(smem_u32(acc_full), 1);
    mbar_init(smem_u32(acc_empty), 16);
    mbar_init(smem_u32(drain_bar), 1);
    mbar_init(smem_u32(copy_drain), 2);
    *abort_flag = 0u;
    *zero_word = 0u;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
  }
  if (warp == 2) {
    tmem_alloc<2>(smem_u32(tmem_slot), 512);
    tmem_relinquish<2>();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);  // (the same in all lanes, for the compiler)
  wait_for_prior_kernel();
  const WaitCtl w{abort_flag, p.status, p.timeout_ns, mapa_shared(smem_u32((const void*)abort_flag), rank ^ 1u)};
  const int32_t cid = (int32_t)(blockIdx.x / 2), clusters = (int32_t)(gridDim.x / 2);
  const int32_t tiles = p.tiles_m * p.tiles_n;

  if (warp == 0) {
    // -------------------------------------------------------------- producer
    if (lane == 0) {
      uint32_t stage = 0, sphase = 0, issued = 0;
      bool skip = (p.debug_flags & QUANT_DEBUG_SKIP_ONE_LOAD) != 0;
      bool ok = true;
      for (int32_t tile = cid; ok && tile < tiles; tile += clusters) {
        int32_t tm, tn;
        raster_tile(tile, p.tiles_m, p.tiles_n, p.raster_group, tm, tn);
        const int32_t rb = 2 * tm + (int32_t)rank;  // this CTA's 128 rows of A
        for (int32_t kb = 0; kb < p.blocks; ++kb) {
          if (!mbar_wait(smem_u32(empty + stage), sphase ^ 1u, w, WAIT_PRODUCER_EMPTY)) { ok = false; break; }
          const uint32_t own = smem_u32(full + stage);
          const uint32_t fb = mapa_shared(own, 0);
          if (leader) mbar_arrive_expect_tx(own, 2u * kStage<NV>);
          const uint32_t st = smem_u32(ring + stage * kStage<NV>);
          tma_load_2d_pair(st, &tmA, fb, kb * 128, rb * 128);
          if (skip) {
            skip = false;  // test hook: this stage's bytes never all arrive
          } else {
            tma_load_2d_pair(st + kOperand, &tmB, fb, kb * 128, (2 * tn + (int32_t)rank) * 128);
          }
          tma_load_3d_pair(st + kScalesAt, &tmSA, fb, 0, kb * 4 * (int32_t)NB, rb);
          tma_load_3d_pair(st + kScalesAt + 512u * NB, &tmSB, fb, 0, kb * 4 * (int32_t)NB, 2 * tn);
          ++issued;
          if (++stage == S) { stage = 0; sphase ^= 1u; }
        }
      }
      if (!ok) {
        // The copies in flight must land before shared memory is released: the leader
        // waits for its last issued stages (bounded), the other CTA, which cannot wait
        // on the leader's barriers, for the same bound in time.
        volatile uint32_t never = 0u;
        const WaitCtl wd{&never, nullptr, 2000000ull, 0};
        if (leader) {
          const uint32_t n = issued < S ? issued : S;
          for (uint32_t back = 1; back <= n; ++back) {
            const uint32_t sb = (stage + S - back) % S;
            mbar_wait(smem_u32(full + sb), back <= stage ? sphase : sphase ^ 1u, wd, 0u);
          }
        } else {
          const uint64_t t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < wd.timeout_ns) {}
        }
      }
    }
  } else if (warp == 1 && leader) {
    // ------------------------------------------------------------------ MMA
    // the whole warp walks the loop and one lane issues (see mma_fp4)
    const uint32_t issue = elect_lane();
    uint32_t stage = 0, sphase = 0, apar = 0;
    bool ok = true;
    for (int32_t tile = cid; ok && tile < tiles; tile += clusters, apar ^= 1u) {
      if (!warp_wait<true>(smem_u32(acc_empty), apar ^ 1u, w, WAIT_MMA_ACC_EMPTY)) break;
      tc_fence_after();
      for (int32_t kb = 0; kb < p.blocks; ++kb) {
        // (the copier saw the stage land, so this covers the operands too)
        if (!warp_wait(smem_u32(ready + stage), sphase, w, WAIT_MMA_FULL)) { ok = false; break; }
        tc_fence_after();
        const uint32_t st = smem_u32(ring + stage * kStage<NV>);
        const uint64_t ad = sdesc_k_sw128(st), bd = sdesc_k_sw128(st + kOperand);
        const uint32_t sf = tmem + kScaleCol + stage * kSlot<NV>;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t j = fp4_scale_block<NV>(k);
          if (4 * kb + k < p.steps)
            mma_fp4<2, NV>(issue, tmem, ad + 2 * k, bd + 2 * k, fp4_idesc<NV>(p.idesc, k), sf + 4u * j,
                           sf + 4u * NB + 8u * j, (uint32_t)(kb | k));
        }
        if (issue) mma_commit_pair(smem_u32(empty + stage), 3u);
        if (++stage == S) { stage = 0; sphase ^= 1u; }
      }
      if (!ok) break;
      if (issue) mma_commit_pair(smem_u32(acc_full), 3u);
    }
    if (issue) {
      // every MMA this thread issued must be complete before TMEM is released
      mma_commit_cg<2>(smem_u32(drain_bar));
      const WaitCtl wd{zero_word, p.status, p.timeout_ns, 0};
      mbar_wait(smem_u32(drain_bar), 0, wd, WAIT_DRAIN);
    }
  } else if ((warp == 2 || warp == 3) && leader) {
    // ---------------------------------------------------------- scale copies
    const uint32_t issue = elect_lane();
    const uint32_t part = warp - 2u;  // each of the two warps takes half of the blocks
    uint32_t stage = 0, sphase = 0;
    bool ok = true;
    for (int32_t tile = cid; ok && tile < tiles; tile += clusters) {
      for (int32_t kb = 0; kb < p.blocks; ++kb) {
        // the stage's slot was last read by MMAs that completed before the stage was
        // refilled, so it is free once the stage has landed
        if (!warp_wait(smem_u32(full + stage), sphase, w, WAIT_MMA_FULL)) { ok = false; break; }
        tc_fence_after();
        const uint32_t from = smem_u32(ring + stage * kStage<NV> + kScalesAt);
        const uint32_t to = tmem + kScaleCol + stage * kSlot<NV>;
#pragma unroll
        for (uint32_t i = 0; i < NB / 2; ++i) {
          const uint32_t j = i + part * (NB / 2);
          tmem_cp_32x128b_x4<2>(issue, to + 4u * j, sdesc_rows16(from + 512u * j));
          tmem_cp_32x128b_x4<2>(issue, to + 4u * NB + 8u * j, sdesc_rows16(from + 512u * (NB + j)));
          tmem_cp_32x128b_x4<2>(issue, to + 4u * NB + 8u * j + 4u, sdesc_rows16(from + 512u * (2u * NB + j)));
        }
        if (issue) mma_commit_cg<2>(smem_u32(ready + stage));
        if (++stage == S) { stage = 0; sphase ^= 1u; }
      }
    }
    if (issue) {
      // the copies this thread issued must be complete before TMEM is released
      mma_commit_cg<2>(smem_u32(copy_drain));
      const WaitCtl wd{zero_word, p.status, p.timeout_ns, 0};
      mbar_wait(smem_u32(copy_drain), 0, wd, WAIT_DRAIN);
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    const uint32_t q = warp & 3u;           // TMEM lane quarter
    const uint32_t half = (warp - 4u) >> 2;  // columns 0-127 or 128-255
    float* mine = staging + (warp - 4u) * 32u * 33u;
    uint32_t apar = 0;
    for (int32_t tile = cid; tile < tiles; tile += clusters, apar ^= 1u) {
      int32_t tm, tn;
      raster_tile(tile, p.tiles_m, p.tiles_n, p.raster_group, tm, tn);
      const int32_t row0 = tm * 256 + (int32_t)(rank * 128u + q * 32u), row = row0 + (int32_t)lane;
      const float sa = p.e.row_scale_a != nullptr && row < p.e.M ? __ldg(p.e.row_scale_a + row) : 1.f;
      uint32_t got = 1;
      if (lane == 0) got = mbar_wait(smem_u32(acc_full), apar, w, WAIT_EPI_ACC_FULL) ? 1u : 0u;
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) break;
      tc_fence_after();
      uint32_t v[4][32];
      const uint32_t at = tmem + ((q * 32u) << 16) + half * 128u;
#pragma unroll
      for (int s = 0; s < 4; ++s) tmem_ld_32x32b_x32(at + 32u * s, v[s]);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(acc_empty), 0));
#pragma unroll
      for (int s = 0; s < 4; ++s)
        fp4_store32<OutT>(p.e, v[s], row0, tn * 256 + (int32_t)half * 128 + 32 * s, sa, mine, lane);
    }
  }

  // ---------------------------------------------------------------- teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  let_next_kernel_start();
  cluster_sync_all();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc<2>(tmem, 512);
  }
}

}  // namespace

const void* fp4_pair_kernel(bool nv, bool out_f32) {
  if (nv)
    return out_f32 ? reinterpret_cast<const void*>(k_fp4_pair<true, float>)
                   : reinterpret_cast<const void*>(k_fp4_pair<true, __nv_bfloat16>);
  return out_f32 ? reinterpret_cast<const void*>(k_fp4_pair<false, float>)
                 : reinterpret_cast<const void*>(k_fp4_pair<false, __nv_bfloat16>);
}

int fp4_pair_stages(bool nv) { return nv ? stages_of<true>() : stages_of<false>(); }
size_t fp4_pair_smem(bool nv) {
  return 1024 + (size_t)fp4_pair_stages(nv) * (nv ? kStage<true> : kStage<false>) + kStaging + kCtrl;
}

}  // namespace dgb
