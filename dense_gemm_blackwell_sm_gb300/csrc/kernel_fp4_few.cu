// kernel_fp4_few.cu -- the 4-bit product where there are few tiles for CTA pairs: few tokens, or
// small layers.
//
// The roles of the operands are exchanged: 128 rows of B (a layer's features) are the MMA's M,
// up to 64 rows of A (tokens) its N, so that a decoded token costs an MMA of 16 columns and
// B's rows stream through shared memory once.  A cluster of `split` CTAs shares a tile's sum:
// each takes a part of K, the partial sums meet in distributed shared memory, in a fixed order.
// Two CTAs fit an SM, so that one's copies run while the other ends.
//
// The same body takes up to 16 tokens as they are (k_fp4_linear): while the features are on their
// way warps 2-7 quantise the CTA's part of the tokens into shared memory, where the MMAs read it.
// One launch instead of two: 8 x 4096 x 4096 bf16 to MXFP4 7.0 -> 6.5 us on the device (6.2 over weights
// in turn), and with calls made one at a time 11.9 -> 6.6; 1 x 14336 x 4096 to NVFP4 12.9 -> 9.7.
//
// Bound by the weights' bytes, at 3.6 to 3.8 TB/s: 1 x 14336 x 4096 8.2 us (MXFP4) and 9.3 (NVFP4), 16 tokens
// 8.7 and 9.8, 64 tokens 10.5 and 11.9; below that by a launch, one CTA's chain of copies and MMAs and the
// cluster's exchange (1 x 4096 x 4096 5.2 us, 1 x 1024 x 1024 3.1).  1024 x 1024 x 4096 8.7 us.  (Launches of
// one graph over weights in turn, none of which L2 still holds.)
//
// Warp 0 is the TMA producer, warp 1 copies the scales into TMEM and issues the MMAs, and all
// eight warps then add, scale and store.
#include <algorithm>
#include <type_traits>

#include "fp4_common.cuh"
#include "kernels_quant_rows.cuh"

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

__host__ __device__ inline uint32_t stage_bytes(int blocks, int tokens) {
  return kOperand + (uint32_t)tokens * 128u + 2u * 512u * (uint32_t)blocks;
}

// Tokens quantised in the kernel: 16 at most, all of a CTA's K at once (`kb` stages of it)
constexpr uint32_t kLinearTokens = 16;
__host__ __device__ inline uint32_t token_bytes(int blocks, int kb) {
  return (uint32_t)kb * (kLinearTokens * 128u + 512u * (uint32_t)blocks);
}
__host__ __device__ inline FewShape linear_shape(int blocks, int kb) {
  const uint32_t room = 111u * 1024u - 2048u, taken = token_bytes(blocks, kb);
  FewShape f{256u, 32u, 0};
  const int in_tmem = (int)((f.columns - f.scale_col) / (8u * (uint32_t)blocks));
  const int in_room = taken > room ? 0 : (int)((room - taken) / (kOperand + 512u * (uint32_t)blocks));
  f.stages = in_tmem < in_room ? in_tmem : in_room;
  if (f.stages > kMostStages) f.stages = kMostStages;
  return f;
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

// Sums [begin, end) of a tile's [token][feature] from the cluster's SPLIT CTAs, in the order of
// their ranks, to c: four neighbours a time, which go out together where rows are ALIGNED to that,
// else one by one.  What a thread reads from the CTAs is under way together (8 groups): one after
// the other, eight reads of distributed shared memory took 2 us.
template <bool ALIGNED, int SPLIT, typename OutT>
__device__ __forceinline__ void few_finish(const Fp4Params& p, const float* token_scale, const float* partial,
                                           int32_t begin, int32_t end, int32_t row0, int32_t col0) {
  constexpr int U = 8 / SPLIT;
  union Four {
    typename std::conditional<sizeof(OutT) == 4, uint4, uint2>::type all;
    OutT one[4];
    __device__ __forceinline__ Four() {}
  };
  constexpr int kStep = kFp4FewThreads * 4;
  const Fp4Epilogue& e = p.e;
  uint32_t from[SPLIT];
#pragma unroll
  for (int r = 0; r < SPLIT; ++r) from[r] = mapa_shared(smem_u32(partial), (uint32_t)r);
#pragma unroll 1
  for (int32_t i0 = begin + (int32_t)threadIdx.x * 4; i0 < end; i0 += kStep * U) {
    float4 y[U][SPLIT];
    Four res[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t i = min(i0 + u * kStep, end - 4);  // (a multiple of 4)
      const int32_t col = col0 + i % 128;
      if (e.residual != nullptr) {
        const OutT* src = reinterpret_cast<const OutT*>(e.residual) + (int64_t)(row0 + i / 128) * e.ld_residual + col;
        // (a group that the matrix' edge cuts goes by single values)
        if (ALIGNED && col + 4 <= e.N) {
          res[u].all = *reinterpret_cast<const decltype(res[u].all)*>(src);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (col + j < e.N) res[u].one[j] = src[j];
        }
      }
#pragma unroll
      for (int r = 0; r < SPLIT; ++r)
        y[u][r] = SPLIT == 1 ? *reinterpret_cast<const float4*>(partial + i) : ld_cluster_f32x4(from[r] + 4u * (uint32_t)i);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t i = i0 + u * kStep;
      const int32_t row = row0 + i / 128, col = col0 + i % 128;
      if (i >= end || col >= e.N) continue;
      const float sa = token_scale != nullptr ? token_scale[row] : 1.f;
      float x[4] = {y[u][0].x, y[u][0].y, y[u][0].z, y[u][0].w};
#pragma unroll
      for (int r = 1; r < SPLIT; ++r) {
        x[0] += y[u][r].x;
        x[1] += y[u][r].y;
        x[2] += y[u][r].z;
        x[3] += y[u][r].w;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] *= sa;
        const int32_t c = min(col + j, e.N - 1);
        if (e.row_scale_b != nullptr) x[j] *= __ldg(e.row_scale_b + c);
        if (e.bias != nullptr) x[j] += __ldg(e.bias + c);
      }
      fp4_act(x, e.act);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        res[u].one[j] = from_f32<OutT>(e.residual != nullptr ? x[j] + to_f32(res[u].one[j]) : x[j]);
      OutT* dst = reinterpret_cast<OutT*>(e.c) + (int64_t)row * e.ld_c + col;
      if (ALIGNED && col + 4 <= e.N) {
        *reinterpret_cast<decltype(res[u].all)*>(dst) = res[u].all;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col + j < e.N) dst[j] = res[u].one[j];
      }
    }
  }
}

template <bool ALIGNED, typename OutT>
__device__ __forceinline__ void few_finish(const Fp4Params& p, const float* token_scale, const float* partial,
                                           int32_t begin, int32_t end, int32_t row0, int32_t col0) {
  switch (p.split) {
    case 1: return few_finish<ALIGNED, 1, OutT>(p, token_scale, partial, begin, end, row0, col0);
    case 2: return few_finish<ALIGNED, 2, OutT>(p, token_scale, partial, begin, end, row0, col0);
    case 4: return few_finish<ALIGNED, 4, OutT>(p, token_scale, partial, begin, end, row0, col0);
    default: return few_finish<ALIGNED, 8, OutT>(p, token_scale, partial, begin, end, row0, col0);
  }
}

// the threads that quantise
constexpr uint32_t kQuantThreads = kFp4FewThreads - 64;
__device__ __forceinline__ void quantisers_sync() { asm volatile("barrier.sync 1, %0;" ::"n"(kQuantThreads) : "memory"); }

// the tokens' largest magnitudes, as bits, and what comes of them
struct TokenScales {
  uint32_t most[kLinearTokens];
  float scale[kLinearTokens], inv[kLinearTokens];
};

// Tokens 0 .. M - 1, K-elements [256 kb0, 256 (kb0 + nkb)), into the places of the MMAs' second
// operand and of its scales.  The threads of warps 2-7 call it together.  Where a token has a
// scale of its own every CTA finds the largest magnitude of all the token by itself: the tokens
// are few and in L2, and to tell one another takes the CTAs of a cluster longer (1 x 14336 x 4096
// 10.5 us where this takes 10.0).
template <bool NV, typename XT>
__device__ __forceinline__ void quantise_tokens(const Fp4Params& p, const Fp4Tokens& x, uint8_t* tokens, uint8_t* scales,
                                                TokenScales* ts, int32_t kb0, int32_t nkb) {
  constexpr int F = NV ? QUANT_NVFP4 : QUANT_MXFP4;
  constexpr uint32_t NB = (uint32_t)kScaleBlocks<NV>;
  constexpr bool EXACT = sizeof(XT) == 4;
  constexpr int AHEAD = EXACT ? 2 : 4;  // runs of 16 values a thread has on their way
  const int32_t thread = (int32_t)threadIdx.x - 64;
  const int32_t runs = nkb * 16, total = runs * p.e.M;
  const XT* values = reinterpret_cast<const XT*>(x.x);
  Run<XT> run[AHEAD];
  auto load = [&](int32_t u) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int32_t at = u + i * (int32_t)kQuantThreads, row = at / runs;
      if (at < total) {
        load16<XT>(run[i], values + row * x.ld_x, kb0 * 256 + (at - row * runs) * 16, x.K, x.vec, x.x, x.x_end);
      } else {
        run[i].clear();
      }
    }
  };
  load(thread);
  if constexpr (NV) {
    // a warp takes runs of one token at a time
    const int32_t chunks = (x.K + 511) / 512, tasks = chunks * p.e.M;
#pragma unroll 1
    for (int32_t t = thread / 32; t < tasks; t += AHEAD * (int32_t)(kQuantThreads / 32)) {
      Run<XT> r[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int32_t task = t + i * (int32_t)(kQuantThreads / 32), row = task / chunks;
        r[i].clear();
        if (task < tasks)
          load16<XT>(r[i], values + row * x.ld_x, (task - row * chunks) * 512 + (thread & 31) * 16, x.K, x.vec, x.x, x.x_end);
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int32_t task = t + i * (int32_t)(kQuantThreads / 32);
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = r[i][j];
        // (magnitudes as bits are in order, a NaN's above all)
        const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(largest16(v)));
        if (task < tasks && (thread & 31) == 0) atomicMax(&ts->most[task / chunks], most);
      }
    }
    quantisers_sync();
    if (thread < p.e.M) {
      const RowUnit unit = row_unit<F>(__uint_as_float(ts->most[thread]));
      ts->scale[thread] = unit.scale;
      ts->inv[thread] = unit.inv;
    }
    quantisers_sync();
  }
#pragma unroll 1
  for (int32_t u = thread; u < total + (thread & 31); u += AHEAD * (int32_t)kQuantThreads) {
    if (u != thread) load(u);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int32_t at = u + i * (int32_t)kQuantThreads, row = min(at / runs, p.e.M - 1), c = at - row * runs;
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = run[i][j];
      float most = largest16(v);
      // (32 values are two lanes'; all lanes of a warp are here, those behind the end with zeros)
      if (!NV) most = larger(most, __shfl_xor_sync(0xffffffffu, most, 1));
      if (at >= total) continue;
      const RowUnit unit = NV ? RowUnit{ts->scale[row], ts->inv[row]} : row_unit<F>(0.f);
      const BlockUnit b = block_unit<F, EXACT>(most, unit);
      uint32_t codes[2];
      codes16<F, EXACT>(codes, v, unit, b);
      const uint32_t j = (uint32_t)c / 16u, q = (uint32_t)c % 16u;  // the stage, and its 16 elements
      *reinterpret_cast<uint2*>(tokens + j * (kLinearTokens * 128u) + sw128_offset((uint32_t)row, q / 2u) + (q & 1u) * 8u) =
          make_uint2(codes[0], codes[1]);
      uint8_t* to = scales + j * (512u * NB) + (uint32_t)row * 16u;
      if constexpr (NV) {
        to[(q / 4u) * 512u + q % 4u] = (uint8_t)b.byte;
      } else if ((q & 1u) == 0u) {
        to[(q / 8u) * 512u + q / 2u % 4u] = (uint8_t)b.byte;
      }
    }
  }
  fence_proxy_async_smem();  // (the MMAs and the copies into TMEM read them)
  quantisers_sync();
}

// XT: the tokens' type where they are quantised here, void where tmA and tmSA bring them.
template <bool NV, typename OutT, typename XT>
__device__ __forceinline__ void few_body(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmSA,
                                         const CUtensorMap& tmSB, const Fp4Params& p, const Fp4Tokens& x) {
  constexpr bool LINEAR = !std::is_void<XT>::value;
  constexpr uint32_t NB = (uint32_t)kScaleBlocks<NV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = align_1024(smem_raw);
  const uint32_t S = (uint32_t)p.stages, T = LINEAR ? kLinearTokens : (uint32_t)p.tokens;
  const int32_t most_kb = (p.blocks + p.split - 1) / p.split;
  const uint32_t STAGE = LINEAR ? kOperand + 512u * NB : stage_bytes((int)NB, (int)T);
  const FewShape shape = LINEAR ? linear_shape((int)NB, most_kb) : few_shape((int)NB, (int)T);
  uint8_t* tokens_here = ring + S * STAGE;  // LINEAR: the tokens' codes, then their scales
  uint8_t* token_scales = tokens_here + (uint32_t)most_kb * kLinearTokens * 128u;
  TokenScales* ts = reinterpret_cast<TokenScales*>(ring + S * STAGE + (LINEAR ? token_bytes((int)NB, most_kb) : 0u));
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(ts) + (LINEAR ? sizeof(TokenScales) : 0));
  uint64_t* full = bars;
  uint64_t* empty = bars + kMostStages;
  uint64_t* done = bars + 2 * kMostStages;
  uint64_t* quantised = done + 1;  // LINEAR: the tokens are in place
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 2);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  // (the stage: features, tokens, their scales)
  const uint32_t tokens_at = kOperand, fscales_at = LINEAR ? kOperand : kOperand + T * 128u,
                 tscales_at = fscales_at + 512u * NB;

  const uint32_t warp = warp_idx(), lane = lane_idx();
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(smem_u32(full + s), 1);
      mbar_init(smem_u32(empty + s), 1);
    }
    mbar_init(smem_u32(done), 1);
    mbar_init(smem_u32(quantised), 1);
    *abort_flag = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSB);
    if constexpr (!LINEAR) {
      tma_prefetch_desc(&tmA);
      tma_prefetch_desc(&tmSA);
    }
  }
  if (LINEAR && threadIdx.x >= 64u && threadIdx.x < 64u + kLinearTokens) ts->most[threadIdx.x - 64u] = 0u;
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

  if (warp == 0) {
    // -------------------------------------------------------------- producer
    // the whole warp walks the loop and one lane copies (see warp_wait)
    const bool skip = (p.debug_flags & QUANT_DEBUG_SKIP_ONE_LOAD) != 0;
    auto features = [&](int32_t j, uint32_t s) {
      const uint32_t st = smem_u32(ring + s * STAGE), fb = smem_u32(full + s);
      mbar_arrive_expect_tx(fb, STAGE);
      // (test hook: with skip the first stage's bytes never all arrive)
      if (!skip || j != 0) tma_load_2d(st, &tmB, fb, (kb0 + j) * 128, tn * 128);
      tma_load_3d(st + fscales_at, &tmSB, fb, 0, (kb0 + j) * 4 * (int32_t)NB, tn);
    };
    auto token_rows = [&](int32_t j, uint32_t s) {
      const uint32_t st = smem_u32(ring + s * STAGE), fb = smem_u32(full + s);
      tma_load_2d(st + tokens_at, &tmA, fb, (kb0 + j) * 128, token0);
      tma_load_3d(st + tscales_at, &tmSA, fb, 0, (kb0 + j) * 4 * (int32_t)NB, token0 / 128);
    };
    const int32_t first = min(nkb, (int32_t)S);
    if (p.static_b && lane == 0)
      for (int32_t j = 0; j < first; ++j) features(j, (uint32_t)j);
    __syncwarp();
    wait_for_prior_kernel();
    let_next_kernel_start();
    for (int32_t j = 0; j < nkb; ++j) {
      const uint32_t s = (uint32_t)j % S;
      if (j >= first && !warp_wait(smem_u32(empty + s), ((uint32_t)j / S & 1u) ^ 1u, w, WAIT_PRODUCER_EMPTY)) break;
      if (lane == 0) {
        if (j >= first || !p.static_b) features(j, s);
        if constexpr (!LINEAR) token_rows(j, s);
      }
      __syncwarp();
    }
  } else if (LINEAR && warp >= 2) {
    // ----------------------------------------------------------- the tokens
    wait_for_prior_kernel();
    if constexpr (LINEAR) quantise_tokens<NV, XT>(p, x, tokens_here, token_scales, ts, kb0, nkb);
    if (threadIdx.x == 64u) mbar_arrive(smem_u32(quantised));
  } else if (warp == 1) {
    // ------------------------------------------------------- scales and MMAs
    // (no wait below begins while the kernel before still runs: its time is not theirs)
    wait_for_prior_kernel();
    const uint32_t issue = elect_lane();
    const bool there = !LINEAR || warp_wait(smem_u32(quantised), 0, w, WAIT_MMA_FULL);
    for (int32_t j = 0; there && j < nkb; ++j) {
      const uint32_t s = (uint32_t)j % S;
      if (!warp_wait(smem_u32(full + s), (uint32_t)j / S & 1u, w, WAIT_MMA_FULL)) break;
      tc_fence_after();
      const uint32_t st = smem_u32(ring + s * STAGE);
      const uint32_t tk = LINEAR ? smem_u32(tokens_here) + (uint32_t)j * kLinearTokens * 128u : st + tokens_at;
      const uint32_t tsc = LINEAR ? smem_u32(token_scales) + (uint32_t)j * 512u * NB : st + tscales_at;
      const uint32_t sf = tmem + shape.scale_col + s * kSlot<NV>;
#pragma unroll
      for (uint32_t i = 0; i < NB; ++i) {
        tmem_cp_32x128b_x4<1>(issue, sf + 4u * i, sdesc_rows16(st + fscales_at + 512u * i));
        tmem_cp_32x128b_x4<1>(issue, sf + 4u * NB + 4u * i, sdesc_rows16(tsc + 512u * i));
      }
      const uint64_t ad = sdesc_k_sw128(st), bd = sdesc_k_sw128(tk);
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
  __syncwarp();
  if (p.split > 1) {
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  if (ok) {
    const float* token_scale = LINEAR ? (NV ? ts->scale : nullptr) : p.e.row_scale_a;
    // (features of a tile that the matrix has; groups of four, or single ones where rows are not
    // aligned to groups)
    const int32_t total = tokens * 128;
    const int32_t share = ((total + p.split - 1) / p.split + 127) / 128 * 128;
    const int32_t begin = rank * share, end = min(total, begin + share);
    if (p.e.vec != 0) {
      few_finish<true, OutT>(p, token_scale, partial, begin, end, token0, tn * 128);
    } else {
      few_finish<false, OutT>(p, token_scale, partial, begin, end, token0, tn * 128);
    }
  }
  if (!ok && threadIdx.x == 0) {
    // copies in flight must land before shared memory is released
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {}
  }
  __syncwarp();
  if (p.split > 1) cluster_sync_all();  // no partial sums go away before they are read
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, shape.columns);
  }
}

template <bool NV, typename OutT>
__global__ void __launch_bounds__(kFp4FewThreads, 2)
    k_fp4_few(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
              const __grid_constant__ Fp4Params p) {
  few_body<NV, OutT, void>(tmA, tmB, tmSA, tmSB, p, Fp4Tokens{});
}

template <bool NV, typename OutT, typename XT>
__global__ void __launch_bounds__(kFp4FewThreads, 2)
    k_fp4_linear(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmSB,
                 const __grid_constant__ Fp4Params p, const __grid_constant__ Fp4Tokens x) {
  few_body<NV, OutT, XT>(tmB, tmB, tmSB, tmSB, p, x);
}

template <bool NV, typename OutT>
const void* linear_kernel(int dtype) {
  switch (dtype) {
    case FFN_F16: return reinterpret_cast<const void*>(k_fp4_linear<NV, OutT, __half>);
    case FFN_BF16: return reinterpret_cast<const void*>(k_fp4_linear<NV, OutT, __nv_bfloat16>);
    default: return reinterpret_cast<const void*>(k_fp4_linear<NV, OutT, float>);
  }
}

constexpr size_t kBarriers = (2 * kMostStages + 2) * 8 + 16;

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
  return 1024 + (size_t)stages * stage_bytes(nv ? 4 : 2, tokens) + kBarriers;
}

const void* fp4_linear_kernel(bool nv, bool out_f32, int dtype) {
  if (nv) return out_f32 ? linear_kernel<true, float>(dtype) : linear_kernel<true, __nv_bfloat16>(dtype);
  return out_f32 ? linear_kernel<false, float>(dtype) : linear_kernel<false, __nv_bfloat16>(dtype);
}

int fp4_linear_stages(bool nv, int kb) { return linear_shape(nv ? 4 : 2, kb).stages; }

size_t fp4_linear_smem(bool nv, int kb, int stages) {
  const int blocks = nv ? 4 : 2;
  return 1024 + (size_t)stages * (kOperand + 512u * (uint32_t)blocks) + token_bytes(blocks, kb) + sizeof(TokenScales) +
         kBarriers;
}

}  // namespace dgb
