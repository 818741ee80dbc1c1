// kernels_fp4_pair.cu -- the product of two microscaled 4-bit operands on CTA pairs.
//
// A pair (cta_group::2) computes a tile of 256 x 256: each CTA brings 128 rows of A and 128 of
// B, 256 K-elements a stage (128 bytes a row), and the block scales of its rows of A and of all
// 256 of B.  tcgen05.mma kind::mxf4 / mxf4nvf4 takes 64 K-elements at a time, with scales that
// tcgen05.cp has moved from shared memory into TMEM, to one of a few slots in turn.
//
// The sums take 256 columns of TMEM, and the scales leave no room for two such accumulators.  So
// consecutive tiles overlap: even ones lie at columns 0-255, odd ones at 96-351.  The epilogue
// reads the 160 columns in common first and hands them back, and the next tile's MMAs start
// while it reads the other 96 and stores the tile.
//
// Roles (384 threads): warp 0 TMA producer, warp 1 MMA, warps 2 (which allocates TMEM) and 3 copy
// the scales, since one thread's issue rate bounds the MMAs (8192^3 NVFP4: 247 us with one copier,
// 206 with two), warps 4-11 the epilogue.  Issuing warps walk their loops as a whole and one lane's
// predicate lets an instruction go (8192^3: 176 us).
//
// Bound by the tensor pipe and, with all SMs at it, by the operands' way from L2: a stage (38 KB an SM
// with a scale per 16, 35 with one per 32) takes 590 cycles where its MMAs take 512, a tile's start
// 1000 more.  8192^3 MXFP4 150 us (7.3 PFLOP/s), NVFP4 160 (6.9); 8192 x 14336 x 4096 138 and 147 (7.0, 6.5),
// with fp32 C 180 and 187, with a bf16 residual 209 and 212, rows off 16-byte boundaries 230 and 239;
// 4096^3 29 and 30 (4.6: 256 tiles are 3.4 rounds of the pairs).
//
// Every cluster takes the tiles cid, cid + clusters, ...: results depend on the sizes alone.
// Every wait is bounded (ptx.cuh); programmatic launches as in ffn_common.cuh.
#include <algorithm>

#include "fp4_common.cuh"
#include "fp4_turns.h"

namespace dgb {

namespace {

constexpr uint32_t kOperand = 128u * 128u;  // 128 rows of 256 4-bit elements
constexpr uint32_t kStaging = 8u * 4096u;
constexpr uint32_t kColumns = 2u * 256u * 4u;  // a tile's column scales and biases
constexpr uint32_t kCtrl = 512;
constexpr int kMostStages = 8;
constexpr int32_t kOwn = 96;          // columns of an accumulator that the next tile's does not take
constexpr uint32_t kScaleCol = 256u + kOwn;  // first TMEM column of the scales

template <bool NV>
constexpr uint32_t kStage = 2u * kOperand + 3u * 512u * kScaleBlocks<NV>;
template <bool NV>
constexpr uint32_t kSlot = 12u * kScaleBlocks<NV>;  // TMEM columns of a stage's scales

template <bool NV>
constexpr uint32_t kSlots = (512u - kScaleCol) / kSlot<NV>;  // 3 with a scale per 16, 6 with one per 32

template <bool NV>
__host__ __device__ constexpr size_t smem_of(int stages) {
  return 1024u + (size_t)stages * kStage<NV> + kStaging + kColumns + kCtrl;
}
template <bool NV>
__host__ __device__ constexpr int stages_of() {
  int s = kMostStages;
  while (smem_of<NV>(s) > 232448u) --s;
  return s;
}

// the eight warps of the epilogue
__device__ __forceinline__ void epilogue_sync() { asm volatile("barrier.sync 1, 256;" ::: "memory"); }

template <bool NV, typename OutT>
__global__ void __launch_bounds__(kFp4PairThreads, 1)
    k_fp4_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
               const __grid_constant__ CUtensorMap tmC, const __grid_constant__ Fp4Params p) {
  constexpr uint32_t S = (uint32_t)stages_of<NV>();
  constexpr uint32_t NB = (uint32_t)kScaleBlocks<NV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = align_1024(smem_raw);
  uint8_t* staging = ring + S * kStage<NV>;
  float* columns = reinterpret_cast<float*>(staging + kStaging);
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kStaging + kColumns);
  uint64_t* full = bars;                     // TMA -> scale copies
  uint64_t* empty = bars + kMostStages;      // MMA -> TMA
  uint64_t* ready = bars + 2 * kMostStages;  // scale copies -> MMA
  uint64_t* acc_full = bars + 3 * kMostStages;
  uint64_t* acc_empty = acc_full + 1;  // the common columns are read, and all of the tile before
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
    if (p.e.vec != 0) tma_prefetch_desc(&tmC);
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
    // the whole warp walks the loop and one lane copies (see warp_wait)
    uint32_t stage = 0, sphase = 0;
    bool skip = (p.debug_flags & QUANT_DEBUG_SKIP_ONE_LOAD) != 0;
    bool ok = true;
    for (int32_t tile = cid; ok && tile < tiles; tile += clusters) {
      int32_t tm, tn;
      raster_tile(tile, p.tiles_m, p.tiles_n, p.raster_group, tm, tn);
      const int32_t rb = 2 * tm + (int32_t)rank;  // this CTA's 128 rows of A
      for (int32_t kb = 0; kb < p.blocks; ++kb) {
        if (!warp_wait(smem_u32(empty + stage), sphase ^ 1u, w, WAIT_PRODUCER_EMPTY)) { ok = false; break; }
        if (lane == 0) {
          const uint32_t own = smem_u32(full + stage);
          const uint32_t fb = mapa_shared(own, 0);
          if (leader) mbar_arrive_expect_tx(own, 2u * kStage<NV>);
          const uint32_t st = smem_u32(ring + stage * kStage<NV>);
          tma_load_2d_pair(st, &tmA, fb, kb * 128, rb * 128);
          // (test hook: with skip this stage's bytes never all arrive)
          if (!skip) tma_load_2d_pair(st + kOperand, &tmB, fb, kb * 128, (2 * tn + (int32_t)rank) * 128);
          tma_load_3d_pair(st + kScalesAt, &tmSA, fb, 0, kb * 4 * (int32_t)NB, rb);
          tma_load_3d_pair(st + kScalesAt + 512u * NB, &tmSB, fb, 0, kb * 4 * (int32_t)NB, 2 * tn);
        }
        __syncwarp();
        skip = false;
        if (++stage == S) { stage = 0; sphase ^= 1u; }
      }
    }
    if (!ok) {
      // The copies in flight must land before shared memory is released: a bound in time, since the
      // other CTA cannot wait on the leader's barriers and a stage that was skipped never fills.
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) {}
    }
  } else if (warp == 1 && leader) {
    // ------------------------------------------------------------------ MMA
    // the whole warp walks the loop and one lane issues (see mma_fp4)
    const uint32_t issue = elect_lane();
    uint32_t stage = 0, sphase = 0, n = 0, slot = 0;
    bool ok = true;
    for (int32_t tile = cid; ok && tile < tiles; tile += clusters, ++n) {
      // the tile before has handed the common columns back, which no warp does before it has read the
      // own columns of the tile before that (fp4_turns.h)
      if (!warp_wait<true>(smem_u32(acc_empty), fp4_empty_parity(n), w, WAIT_MMA_ACC_EMPTY)) break;
      tc_fence_after();
      const uint32_t d = tmem + (fp4_turn(n) != 0u ? (uint32_t)kOwn : 0u);
      for (int32_t kb = 0; kb < p.blocks; ++kb) {
        // (the copier saw the stage land, so this covers the operands too)
        if (!warp_wait(smem_u32(ready + stage), sphase, w, WAIT_MMA_FULL)) { ok = false; break; }
        tc_fence_after();
        const uint32_t st = smem_u32(ring + stage * kStage<NV>);
        const uint64_t ad = sdesc_k_sw128(st), bd = sdesc_k_sw128(st + kOperand);
        const uint32_t sf = tmem + kScaleCol + slot * kSlot<NV>;
        if (++slot == kSlots<NV>) slot = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t j = fp4_scale_block<NV>(k);
          if (4 * kb + k < p.steps)
            mma_fp4<2, NV>(issue, d, ad + 2 * k, bd + 2 * k, fp4_idesc<NV>(p.idesc, k), sf + 4u * j,
                           sf + 4u * NB + 8u * j, (uint32_t)(kb | k));
        }
        if (issue) mma_commit_pair(smem_u32(empty + stage), 3u);
        __syncwarp();
        if (++stage == S) { stage = 0; sphase ^= 1u; }
      }
      if (!ok) break;
      if (issue) mma_commit_pair(smem_u32(acc_full), 3u);
      __syncwarp();
    }
    // every MMA this warp issued must be complete before TMEM is released
    if (issue) mma_commit_cg<2>(smem_u32(drain_bar));
    const WaitCtl wd{zero_word, p.status, p.timeout_ns, 0};
    warp_wait(smem_u32(drain_bar), 0, wd, WAIT_DRAIN);
  } else if ((warp == 2 || warp == 3) && leader) {
    // ---------------------------------------------------------- scale copies
    const uint32_t issue = elect_lane();
    const uint32_t part = warp - 2u;  // each of the two warps takes half of the blocks
    uint32_t stage = 0, sphase = 0, slot = 0, behind = 0, bphase = 0;
    int64_t copied = 0;
    bool ok = true;
    for (int32_t tile = cid; ok && tile < tiles; tile += clusters) {
      for (int32_t kb = 0; kb < p.blocks; ++kb) {
        if (!warp_wait(smem_u32(full + stage), sphase, w, WAIT_MMA_FULL)) { ok = false; break; }
        // The slot was last read by the MMAs of the stage kSlots before this one.  With more slots
        // than stages those completed before this stage was refilled.
        if (kSlots<NV> < S && copied >= (int64_t)kSlots<NV>) {
          if (!warp_wait(smem_u32(empty + behind), bphase, w, WAIT_PRODUCER_EMPTY)) { ok = false; break; }
          if (++behind == S) { behind = 0; bphase ^= 1u; }
        }
        ++copied;
        tc_fence_after();
        const uint32_t from = smem_u32(ring + stage * kStage<NV> + kScalesAt);
        const uint32_t to = tmem + kScaleCol + slot * kSlot<NV>;
        if (++slot == kSlots<NV>) slot = 0;
#pragma unroll
        for (uint32_t i = 0; i < NB / 2; ++i) {
          const uint32_t j = i + part * (NB / 2);
          tmem_cp_32x128b_x4<2>(issue, to + 4u * j, sdesc_rows16(from + 512u * j));
          tmem_cp_32x128b_x4<2>(issue, to + 4u * NB + 8u * j, sdesc_rows16(from + 512u * (NB + j)));
          tmem_cp_32x128b_x4<2>(issue, to + 4u * NB + 8u * j + 4u, sdesc_rows16(from + 512u * (2u * NB + j)));
        }
        if (issue) mma_commit_cg<2>(smem_u32(ready + stage));
        __syncwarp();
        if (++stage == S) { stage = 0; sphase ^= 1u; }
      }
    }
    // the copies both warps issued must be complete before TMEM is released
    if (issue) mma_commit_cg<2>(smem_u32(copy_drain));
    const WaitCtl wd{zero_word, p.status, p.timeout_ns, 0};
    warp_wait(smem_u32(copy_drain), 0, wd, WAIT_DRAIN);
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    // Four of the eight runs of 32 columns a warp: of the five in common with the next tile (first
    // `common`, which lie at the tile's end in even tiles, at its start in odd ones) group 0 takes
    // three, of the three others one.
    const uint32_t q = warp & 3u;  // TMEM lane quarter
    const uint32_t group = (warp - 4u) >> 2;
    uint8_t* mine = staging + (warp - 4u) * 4096u;
    const int32_t thread = (int32_t)threadIdx.x - 128;
    uint32_t n = 0, buffer = 0;
    bool dead = false;
    for (int32_t tile = cid; tile < tiles; tile += clusters, ++n) {
      const uint32_t apar = fp4_turn(n);
      int32_t tm, tn;
      raster_tile(tile, p.tiles_m, p.tiles_n, p.raster_group, tm, tn);
      const int32_t row0 = tm * 256 + (int32_t)(rank * 128u + q * 32u), row = row0 + (int32_t)lane;
      const int32_t col0 = tn * 256;
      const float sa = p.e.row_scale_a != nullptr && row < p.e.M ? __ldg(p.e.row_scale_a + row) : 1.f;
      const bool in = col0 + thread < p.e.N;
      const float cs = in && p.e.row_scale_b != nullptr ? __ldg(p.e.row_scale_b + col0 + thread) : 1.f;
      const float cb = in && p.e.bias != nullptr ? __ldg(p.e.bias + col0 + thread) : 0.f;
      const int32_t common = (apar != 0u ? 0 : kOwn) + 96 * (int32_t)group;
      const int32_t own = (apar != 0u ? 256 - kOwn : 0) + 32 * (int32_t)group;
      // Residuals come a run ahead, the tile's first ones while its sums are made (8192 x 14336 x
      // 4096 NVFP4 takes 212 us with them, 147 without; read when they are added, 18 us more).
      Residual32<OutT> ra, rb;
      auto fetch = [&](Residual32<OutT>& r, int32_t c) { r.load(p.e, row, col0 + c); };
      fetch(ra, common);
      epilogue_sync();  // (the tile before is done with the columns)
      columns[thread] = cs;
      columns[256 + thread] = cb;
      epilogue_sync();
      // (a warp that gave up still meets the others at every tile's barriers)
      dead = dead || !warp_wait(smem_u32(acc_full), apar, w, WAIT_EPI_ACC_FULL);
      if (dead) continue;
      tc_fence_after();
      const uint32_t acc = tmem + ((q * 32u) << 16) + (apar != 0u ? (uint32_t)kOwn : 0u);
      auto hand_back = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_light(mapa_shared(smem_u32(acc_empty), 0));
      };
      auto store = [&](const uint32_t(&v)[32], int32_t c, const Residual32<OutT>& r) {
        fp4_store32<OutT>(p.e, &tmC, v, r, row0, col0 + c, sa, columns + c, columns + 256 + c, mine, buffer, lane);
      };
      uint32_t v0[32], v1[32];
      tmem_ld_32x32b_x32(acc + (uint32_t)common, v0);
      tmem_ld_32x32b_x32(acc + (uint32_t)common + 32u, v1);
      if (group == 0) {
        uint32_t v2[32];
        tmem_ld_32x32b_x32(acc + (uint32_t)common + 64u, v2);
        tmem_wait_ld();
        hand_back();
        fetch(rb, common + 32);
        store(v0, common, ra);
        fetch(ra, common + 64);
        store(v1, common + 32, rb);
        fetch(rb, own);
        store(v2, common + 64, ra);
        tmem_ld_32x32b_x32(acc + (uint32_t)own, v0);
        tmem_wait_ld();
        store(v0, own, rb);
      } else {
        tmem_wait_ld();
        hand_back();
        fetch(rb, common + 32);
        store(v0, common, ra);
        fetch(ra, own);
        store(v1, common + 32, rb);
        tmem_ld_32x32b_x32(acc + (uint32_t)own, v0);
        tmem_ld_32x32b_x32(acc + (uint32_t)own + 32u, v1);
        tmem_wait_ld();
        fetch(rb, own + 32);
        store(v0, own, ra);
        store(v1, own + 32, rb);
      }
    }
    if (lane == 0) bulk_wait_group<0>();
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

size_t fp4_pair_smem(bool nv) {
  return nv ? smem_of<true>(stages_of<true>()) : smem_of<false>(stages_of<false>());
}

}  // namespace dgb
