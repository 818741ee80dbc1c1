// kernels_gated.cuh -- the gated projections h = act(x Wg^T) * (x Wu^T) on the
// tcgen05 Tensor Core, the same products with the gradient of the pre-activations
// as their epilogue, and the two products of the backward pass in one launch.
//
// A CTA pair (cta_group::2) computes a tile of 256 rows per MMA consumer.  For the
// gated forms the MMA's N columns are hw rows of Wg and the same hw rows of Wu: in
// a pair the second operand is split between the CTAs along N, so CTA 0 simply
// loads the gate's rows and CTA 1 the up projection's, and a thread of the epilogue
// finds g and u of one element of h in the same TMEM lane, hw columns apart.  The
// activation, the product and the one rounding to the output's type happen there;
// neither g nor u goes through memory (unless the caller keeps them).
//
// Roles (384 threads): warp 0 TMA producer, warps 1 and 3 one MMA consumer each
// (NCONS = 2: 512-row tiles, both consumers share the stage's weight rows, one
// 256-column accumulator each; NCONS = 1: one consumer, two accumulators in turn),
// warp 2 allocates TMEM, warps 4-11 the epilogue.  With two consumers warps 4-7
// serve the first and 8-11 the second; with one they share its columns.
//
// One thread hands the tensor pipe its MMAs at about 75 clocks each (300 per 64-wide
// block), more than a narrow tile's MMAs take, so with one consumer two threads take
// the blocks in turn (`split`), each into an accumulator of its own; the epilogue adds
// the two.  64 x 4096 x 4096: 24.7 -> 20.3 us.  Two accumulators per tile leave TMEM
// room for two tiles up to hw = 64; wider tiles are split only where a cluster takes
// one.
//
// Bound by the tensor pipe once there are tiles for every SM pair: 8192 x 14336 x 4096
// bf16 takes 960 to 980 us (1960 to 2000 TFLOP/s; 1050 to 1150 when the pre-activations
// are written too; replayed in a graph: under the power cap of longer runs 1120), the
// pipe is active 89% of 2048 x 14336 x 4096.  Two consumers share a weight stage, so
// that a 512-row tile reads 3/4 of the bytes of two 256-row ones; the price is that
// nothing hides the end of a tile (3.7 us).  The backward products take 1065 to 1095 us
// with the pass that makes their operand at 4096 x 14336 x 4096 (1760 to 1810 TFLOP/s): their
// operands' rows run along the reduction, so a stage is more and smaller copies.
//
// The gradient of the pre-activations is rounded to the inputs' 16 bits, since it is an
// operand of the two products (one type for both operands): dx and dw are sqrt 2 as far
// from the exact values as one rounding.  Two 16-bit parts would double the products' time.
//
// Where F is no multiple of 8 the epilogue's rows go through shared memory and 2-byte
// stores: 8192 x 14335 x 4096 takes 1056 us, 1218 with the pre-activations.
//
// Every cluster walks its own list of tiles (no scheduler, no atomics): which
// tiles a cluster takes depends on the sizes alone, so results do too.
//
// Every wait is bounded (ptx.cuh).  The kernels launch as programmatic dependents:
// barriers, TMEM and the cluster are set up while the previous kernel drains, and
// every thread waits for that kernel before it touches global memory.  The next kernel
// may be placed when a CTA's tiles are done (ffn_common.cuh).
#pragma once

#include <type_traits>

#include "ffn_common.cuh"
#include "gated.h"
#include "idesc.h"

namespace dgb {

namespace {

constexpr int GT_THREADS = 384;
constexpr uint32_t GT_A_BYTES = 128u * 128u;  // 128 rows of 64 16-bit elements
constexpr int GT_STAGE_ROW = 34;              // 16-bit elements of a staged epilogue row (32 + 2: no bank conflicts)
constexpr uint32_t GT_STAGING = 8u * 32u * GT_STAGE_ROW * 2u;
constexpr uint32_t GT_CTRL = 384;
constexpr int GT_MAX_STAGES = 16;

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (std::is_same<T, __half>::value) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  } else {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  }
}

__device__ __forceinline__ uint16_t half_of(uint32_t w, int e) { return (uint16_t)(e ? w >> 16 : w); }

// A warp's 32 rows x 32 columns of 16-bit results: lane r holds row r in w.  `vec`
// says how the rows are aligned (uniform): 2 and 1, 32 and 16 bytes: each lane
// stores its own row; 0: the rows go through the warp's staging space so that the
// lanes store neighbouring elements (an odd pitch: 32 sectors per store otherwise).
__device__ __forceinline__ void store_rows32(uint16_t* first_row, int64_t ld, int rows, int n, const uint32_t (&w)[16],
                                             int vec, uint16_t* staging, uint32_t lane) {
  if (vec != 0) {
    if ((int)lane >= rows) return;
    uint16_t* dst = first_row + (int64_t)lane * ld;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (vec == 2 && 16 * j + 16 <= n) {
        st_global_v8(dst + 16 * j, w + 8 * j);
        continue;
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int c = 16 * j + 8 * q;
        if (c + 8 <= n) {
          *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[c / 2], w[c / 2 + 1], w[c / 2 + 2], w[c / 2 + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < n) dst[c + e] = half_of(w[(c + e) / 2], e & 1);
        }
      }
    }
    return;
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 16; ++j) *reinterpret_cast<uint32_t*>(staging + lane * GT_STAGE_ROW + 2 * j) = w[j];
  __syncwarp();
  if ((int)lane < n)
    for (int r = 0; r < rows; ++r) first_row[(int64_t)r * ld + lane] = staging[r * GT_STAGE_ROW + lane];
}

// the same way in: lane r's 32 columns of row r, 0 outside rows x n
__device__ __forceinline__ void load_rows32(const uint16_t* first_row, int64_t ld, int rows, int n, uint32_t (&w)[16],
                                            int vec, uint16_t* staging, uint32_t lane) {
  if (vec != 0) {
    const uint16_t* src = first_row + (int64_t)lane * ld;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if ((int)lane < rows && 8 * q + 8 <= n) {
        v = __ldg(reinterpret_cast<const uint4*>(src + 8 * q));
      } else if ((int)lane < rows && 8 * q < n) {
        uint32_t t[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (8 * q + e < n) t[e / 2] |= (uint32_t)src[8 * q + e] << (16 * (e & 1));
        v = make_uint4(t[0], t[1], t[2], t[3]);
      }
      w[4 * q] = v.x;
      w[4 * q + 1] = v.y;
      w[4 * q + 2] = v.z;
      w[4 * q + 3] = v.w;
    }
    return;
  }
  __syncwarp();
  for (int r = 0; r < 32; ++r)
    staging[r * GT_STAGE_ROW + lane] = (r < rows && (int)lane < n) ? first_row[(int64_t)r * ld + lane] : (uint16_t)0;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = *reinterpret_cast<const uint32_t*>(staging + lane * GT_STAGE_ROW + 2 * j);
  __syncwarp();
}

template <typename T, int NCONS, int MODE, int ACT>
__global__ void __launch_bounds__(GT_THREADS, 1)
    k_gated(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmB0,
            const __grid_constant__ CUtensorMap tmA1, const __grid_constant__ CUtensorMap tmB1,
            const __grid_constant__ GatedParams p) {
  constexpr int TILE_M = 256 * NCONS;
  constexpr uint32_t EPI_WARPS = NCONS == 2 ? 4 : 8;  // per accumulator and CTA
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = align_1024(smem_raw);
  const uint32_t S = (uint32_t)p.stages;
  // A stage holds a_rows rows of the first operand per consumer and hw of the second.
  // With fewer rows than the MMA's 128 (few tokens) the MMA reads on into what follows;
  // those rows of the accumulator are never stored.
  const uint32_t A_BYTES = NCONS == 2 ? GT_A_BYTES : (uint32_t)p.a_rows * 128u;
  const uint32_t STAGE = NCONS * A_BYTES + (uint32_t)p.hw * 128u;
  uint16_t* staging = reinterpret_cast<uint16_t*>(ring + (size_t)S * STAGE);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(staging) + GT_STAGING);
  uint64_t* full = bars;                         // [16] TMA -> MMA
  uint64_t* empty = bars + GT_MAX_STAGES;        // [16] MMA -> TMA
  uint64_t* acc_full = bars + 2 * GT_MAX_STAGES;  // [2] MMA -> epilogue
  uint64_t* acc_empty = acc_full + 2;            // [2] epilogue -> MMA
  uint64_t* drain_bar = acc_full + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 5);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  volatile uint32_t* zero_word = tmem_slot + 2;

  const uint32_t warp = warp_idx(), lane = lane_idx();
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(smem_u32(full + s), 1);
      mbar_init(smem_u32(empty + s), NCONS);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(acc_full + i), NCONS == 2 ? 1u : (uint32_t)p.split);
      mbar_init(smem_u32(acc_empty + i), 2 * EPI_WARPS);
    }
    mbar_init(smem_u32(drain_bar), NCONS == 2 ? 2u : (uint32_t)p.split);
    *abort_flag = 0u;
    *zero_word = 0u;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA0);
    tma_prefetch_desc(&tmB0);
    if constexpr (MODE == GATED_PRODUCTS) {
      tma_prefetch_desc(&tmA1);
      tma_prefetch_desc(&tmB1);
    }
  }
  if (warp == 2) {
    tmem_alloc<2>(smem_u32(tmem_slot), 512);
    tmem_relinquish<2>();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_for_prior_kernel();
  const WaitCtl w{abort_flag, p.status, p.timeout_ns, mapa_shared(smem_u32((const void*)abort_flag), rank ^ 1u)};
  const int32_t cid = (int32_t)(blockIdx.x / 2), clusters = (int32_t)(gridDim.x / 2);

  // the slice of the reduction a tile takes (products; `tile` is then the tile in it), and
  // its blocks
  auto slice_of = [&](const GatedTask& t, int32_t& tile) {
    if (MODE != GATED_PRODUCTS || t.partial == nullptr) return 0;
    const int32_t tiles = t.tiles_m * t.tiles_n, slice = tile / tiles;
    tile -= slice * tiles;
    return slice;
  };
  auto blocks_of = [&](const GatedTask& t, int32_t slice) {
    return MODE == GATED_PRODUCTS ? min(t.kb_slice, t.kb - slice * t.kb_slice) : t.kb;
  };

  // the accumulator of a cluster's i-th tile: two take turns where TMEM holds them
  auto slot_of = [&](int32_t i, uint32_t cons) {
    return NCONS == 2 ? cons : p.two_slots ? (uint32_t)(i & 1) : 0u;
  };
  auto parity_of = [&](int32_t i) {
    return NCONS == 1 && p.two_slots ? (uint32_t)((i >> 1) & 1) : (uint32_t)(i & 1);
  };

  if (warp == 0) {
    // -------------------------------------------------------------- producer
    if (lane == 0) {
      uint32_t stage = 0, sphase = 0, issued = 0;
      bool skip = (p.debug_flags & FFN_DEBUG_SKIP_ONE_LOAD) != 0;
      bool ok = true;
      int32_t task, tile;
      for (int32_t i = 0; ok && gated_tile(p, cid, clusters, i, task, tile); ++i) {
        const GatedTask& t = p.task[task];
        const CUtensorMap* tmA = (MODE == GATED_PRODUCTS && task) ? &tmA1 : &tmA0;
        const CUtensorMap* tmB = (MODE == GATED_PRODUCTS && task) ? &tmB1 : &tmB0;
        int32_t tm, tn;
        const int32_t slice = slice_of(t, tile);
        raster_tile(tile, t.tiles_m, t.tiles_n, t.raster_group, tm, tn);
        const int32_t row0 = tm * TILE_M + (int32_t)rank * 128;
        const int32_t first = slice * t.kb_slice, blocks = blocks_of(t, slice);
        for (int32_t it = 0; it < blocks; ++it) {
          const int32_t k0 = (first + it) * 64;
          if (!mbar_wait(smem_u32(empty + stage), sphase ^ 1u, w, WAIT_PRODUCER_EMPTY)) { ok = false; break; }
          const uint32_t own = smem_u32(full + stage);
          const uint32_t fb = mapa_shared(own, 0);
          if (leader) mbar_arrive_expect_tx(own, 2u * STAGE);
          uint8_t* st = ring + (size_t)stage * STAGE;
          for (int c = 0; c < NCONS; ++c) {
            const uint32_t dst = smem_u32(st + c * A_BYTES);
            const int32_t row = row0 + c * 256;
            if (MODE == GATED_PRODUCTS && t.a_mn) {
              tma_load_2d_pair(dst, tmA, fb, row, k0);
              tma_load_2d_pair(dst + 8192, tmA, fb, row + 64, k0);
            } else {
              tma_load_2d_pair(dst, tmA, fb, k0, row);
            }
          }
          const uint32_t dst = smem_u32(st + NCONS * A_BYTES);
          if (skip) {
            skip = false;  // test hook: this stage's bytes never all arrive
          } else if constexpr (MODE == GATED_PRODUCTS) {
            // columns along the rows in memory: boxes of 64 columns x 64 reduction rows
            for (int32_t h = 0; h < p.hw; h += 64)
              tma_load_2d_pair(dst + (uint32_t)h * 128u, tmB, fb, (2 * tn + (int32_t)rank) * p.hw + h, k0);
          } else {
            // hw rows of Wg (CTA 0) or of Wu (CTA 1)
            tma_load_2d_pair(dst, tmB, fb, k0, tn * p.hw + (rank ? t.cols : 0));
          }
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
  } else if ((warp == 1 || (warp == 3 && (NCONS == 2 || p.split == 2))) && leader) {
    // ------------------------------------------------------------------ MMA
    if (lane == 0) {
      const uint32_t me = warp == 1 ? 0u : 1u;
      // two consumers: each its own rows of every block; one, split: the two threads take
      // the blocks in turn, each into its own accumulator
      const uint32_t cons = NCONS == 2 ? me : 0u, first = NCONS == 2 ? 0u : me,
                     step = NCONS == 2 ? 1u : (uint32_t)p.split;
      uint32_t stage = 0, sphase = 0;
      int32_t task, tile;
      bool ok = true;
      for (int32_t i = 0; ok && gated_tile(p, cid, clusters, i, task, tile); ++i) {
        const GatedTask& t = p.task[task];
        const int32_t blocks = blocks_of(t, slice_of(t, tile));
        const uint32_t slot = slot_of(i, cons), apar = parity_of(i);
        if (!mbar_wait<true>(smem_u32(acc_empty + slot), apar ^ 1u, w, WAIT_MMA_ACC_EMPTY)) break;
        tc_fence_after();
        const uint32_t d = tmem + (NCONS == 2 ? cons * 256u : slot * 256u + me * (uint32_t)p.part_cols);
        const bool a_mn = MODE == GATED_PRODUCTS && t.a_mn;
        auto advance = [&](uint32_t n) {
          stage += n;
          if (stage >= S) { stage -= S; sphase ^= 1u; }
        };
        advance(first);
        int32_t it = (int32_t)first;
        for (; it < blocks; it += (int32_t)step) {
          if (!mbar_wait(smem_u32(full + stage), sphase, w, WAIT_MMA_FULL)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(ring + (size_t)stage * STAGE + cons * A_BYTES);
          const uint32_t sb = smem_u32(ring + (size_t)stage * STAGE + NCONS * A_BYTES);
          const uint64_t ad = a_mn ? sdesc_mn_sw128(sa, 8192) : sdesc_k_sw128(sa);
          const uint64_t bd = MODE == GATED_PRODUCTS ? sdesc_mn_sw128(sb, 8192) : sdesc_k_sw128(sb);
          const uint64_t astep = a_mn ? 128 : 2, bstep = MODE == GATED_PRODUCTS ? 128 : 2;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16<2>(d, ad + astep * k, bd + bstep * k, t.idesc, (uint32_t)(it - (int32_t)first) | (uint32_t)k);
          mma_commit_pair(smem_u32(empty + stage), 3u);
          advance(step);
        }
        if (!ok) break;
        // (the ring goes on behind the last block: step back where this thread went past it)
        if (it > blocks) {
          if (stage == 0) { stage = S - 1u; sphase ^= 1u; } else { --stage; }
        }
        mma_commit_pair(smem_u32(acc_full + slot), 3u);
      }
      // every MMA this thread issued must be complete before TMEM is released
      mma_commit_cg<2>(smem_u32(drain_bar));
      const WaitCtl wd{zero_word, p.status, p.timeout_ns, 0};
      mbar_wait(smem_u32(drain_bar), 0, wd, WAIT_DRAIN);
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    const uint32_t q = warp & 3u;            // TMEM lane quarter
    const uint32_t grp = (warp - 4u) >> 2;   // two consumers: which; one: which half of the steps
    uint16_t* my_staging = staging + (warp - 4u) * 32u * GT_STAGE_ROW;
    const int32_t width = MODE == GATED_PRODUCTS ? 2 * p.hw : p.hw;  // output columns of a tile
    int32_t task, tile;
    for (int32_t i = 0; gated_tile(p, cid, clusters, i, task, tile); ++i) {
      const GatedTask& t = p.task[task];
      int32_t tm, tn;
      const int32_t slice = slice_of(t, tile);
      raster_tile(tile, t.tiles_m, t.tiles_n, t.raster_group, tm, tn);
      const uint32_t slot = slot_of(i, grp), apar = parity_of(i);
      const int32_t row0 =
          tm * TILE_M + (NCONS == 2 ? (int32_t)grp * 256 : 0) + (int32_t)rank * 128 + (int32_t)q * 32;
      const int32_t rows = min(32, t.rows - row0);  // may be negative
      const int32_t col_end = min(t.cols, (tn + 1) * width);
      const int32_t step0 = NCONS == 2 ? 0 : (int32_t)grp, dstep = NCONS == 2 ? 1 : 2;
      const int32_t steps = (width + 31) / 32;
      uint32_t got = 1;
      if (lane == 0) got = mbar_wait(smem_u32(acc_full + slot), apar, w, WAIT_EPI_ACC_FULL) ? 1u : 0u;
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) break;
      tc_fence_after();
      const uint32_t tbase = tmem + ((q * 32u) << 16) + slot * 256u;
      auto hand_back = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(acc_empty + slot), 0));
      };
      // 32 columns of the accumulator; one consumer: of the even blocks', plus the odd ones'
      auto load_sums = [&](uint32_t at, uint32_t (&v)[32]) {
        tmem_ld_32x32b_x32(at, v);
        if (NCONS == 1 && p.split == 2 && t.kb > 1) {
          uint32_t more[32];
          tmem_ld_32x32b_x32(at + (uint32_t)p.part_cols, more);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(more[j]));
        } else {
          tmem_wait_ld();
        }
      };
      if (step0 >= steps) hand_back();
#pragma unroll 1
      for (int32_t s = step0; s < steps; s += dstep) {
        const int32_t col = tn * width + 32 * s;
        const int32_t n = min(32, col_end - col);  // may be negative
        uint16_t* out = reinterpret_cast<uint16_t*>(t.out) + (int64_t)row0 * t.ld_out + col;
        if constexpr (MODE == GATED_PRODUCTS) {
          uint32_t v[32];
          load_sums(tbase + 32u * (uint32_t)s, v);
          if (s + dstep >= steps) hand_back();
          if (t.partial != nullptr) {  // (rows of cols fp32: a multiple of 32 bytes)
            float* dst = t.partial + ((int64_t)slice * t.rows + row0 + (int32_t)lane) * t.cols + col;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if ((int)lane < rows && 8 * j + 8 <= n) st_global_v8(dst + 8 * j, v + 8 * j);
            continue;
          }
          uint32_t o[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = pack2<T>(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
          if (rows > 0 && n > 0) store_rows32(out, t.ld_out, rows, n, o, t.vec_out, my_staging, lane);
        } else {
          uint32_t dh[MODE == GATED_SLOPES ? 16 : 1];
          if constexpr (MODE == GATED_SLOPES) {
            if (rows > 0 && n > 0)
              load_rows32(reinterpret_cast<const uint16_t*>(p.dh) + (int64_t)row0 * p.ld_dh + col, p.ld_dh, rows, n, dh,
                          p.vec_dh, my_staging, lane);
          }
          uint32_t gr[32], ur[32];
          if constexpr (NCONS == 2) {
            tmem_ld_32x32b_x32(tbase + 32u * (uint32_t)s, gr);
            tmem_ld_32x32b_x32(tbase + (uint32_t)p.hw + 32u * (uint32_t)s, ur);
            tmem_wait_ld();
          } else {
            load_sums(tbase + 32u * (uint32_t)s, gr);
            load_sums(tbase + (uint32_t)p.hw + 32u * (uint32_t)s, ur);
          }
          if (s + dstep >= steps) hand_back();
          auto g = [&](int j) { return __uint_as_float(gr[j]); };
          auto u = [&](int j) { return __uint_as_float(ur[j]); };
          if (rows <= 0 || n <= 0) continue;
          uint32_t o[16];
          if constexpr (MODE == GATED_FORWARD) {
            if (p.gu != nullptr) {
              uint16_t* gu = reinterpret_cast<uint16_t*>(p.gu) + (int64_t)row0 * p.ld_gu + col;
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = pack2<T>(g(2 * j), g(2 * j + 1));
              store_rows32(gu, p.ld_gu, rows, n, o, p.vec_gate, my_staging, lane);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = pack2<T>(u(2 * j), u(2 * j + 1));
              store_rows32(gu + t.cols, p.ld_gu, rows, n, o, p.vec_up, my_staging, lane);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
              o[j] = pack2<T>(act_only<ACT>(g(2 * j)) * u(2 * j), act_only<ACT>(g(2 * j + 1)) * u(2 * j + 1));
            store_rows32(out, t.ld_out, rows, n, o, t.vec_out, my_staging, lane);
          } else {
            uint32_t o2[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 d = unpack2<T>(dh[j]);
              float a0, a1, s0, s1;
              act_and_slope<ACT>(g(2 * j), a0, s0);
              act_and_slope<ACT>(g(2 * j + 1), a1, s1);
              o[j] = pack2<T>(d.x * u(2 * j) * s0, d.y * u(2 * j + 1) * s1);
              o2[j] = pack2<T>(d.x * a0, d.y * a1);
            }
            store_rows32(out, t.ld_out, rows, n, o, t.vec_out, my_staging, lane);
            store_rows32(out + t.cols, t.ld_out, rows, n, o2, p.vec_up, my_staging, lane);
          }
        }
      }
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

template <typename T, int MODE, int ACT>
const void* gated_kernel(int consumers) {
  return consumers == 2 ? reinterpret_cast<const void*>(k_gated<T, 2, MODE, ACT>)
                        : reinterpret_cast<const void*>(k_gated<T, 1, MODE, ACT>);
}

template <typename T, int MODE>
const void* gated_kernel_of(int consumers, int act) {
  switch (act) {
    case EPI_ACT_RELU: return gated_kernel<T, MODE, EPI_ACT_RELU>(consumers);
    case EPI_ACT_SILU: return gated_kernel<T, MODE, EPI_ACT_SILU>(consumers);
    case EPI_ACT_GELU_TANH: return gated_kernel<T, MODE, EPI_ACT_GELU_TANH>(consumers);
    case EPI_ACT_GELU_ERF: return gated_kernel<T, MODE, EPI_ACT_GELU_ERF>(consumers);
    default: return gated_kernel<T, MODE, EPI_ACT_NONE>(consumers);
  }
}

}  // namespace

}  // namespace dgb
