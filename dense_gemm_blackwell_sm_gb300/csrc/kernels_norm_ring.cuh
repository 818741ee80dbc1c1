// kernels_norm_ring.cuh -- the block norms with rows that come through a ring in
// shared memory filled by bulk copies (cp.async.bulk), so an SM has tens of KB on
// their way whatever its threads do, and the backward kernel can read a row's values
// again instead of holding them in registers.
//
// A group (a warp, a CTA, or in the backward kernel a cluster of CTAs that share
// the columns) walks rows that start at the same offset to 16-byte boundaries, a few
// rows ahead in the ring.  Every wait is bounded; a wait that runs out is recorded in
// the device's status word.
#pragma once

#include "kernels_norm.cuh"

namespace dgb {

namespace {

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// (arguments by value: a ring whose address escapes would live in local memory, and
// every access to it would go there)
static __device__ __noinline__ bool ring_wait_slow(uint32_t full, uint32_t stage, uint32_t phase, uint32_t stages,
                                                   volatile uint32_t* abort_flag, uint32_t* status, uint32_t left) {
  const WaitCtl w{abort_flag, status, 2000000000ull, 0};
  if (mbar_wait(full + 8u * stage, phase, w, WAIT_MMA_FULL)) return true;
  volatile uint32_t never = 0u;
  const WaitCtl wd{&never, nullptr, 2000000ull, 0};
  for (; left > 0; --left) {
    mbar_wait(full + 8u * stage, phase, wd, 0u);
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  return false;
}

// Test hook: one arrival more than will come, on the first stage of the first group.
__device__ __forceinline__ uint32_t missing_arrival(int32_t debug_flags, int group, uint32_t stage) {
  return (debug_flags & FFN_DEBUG_SKIP_ONE_LOAD) != 0 && blockIdx.x == 0 && group == 0 && stage == 0 ? 1u : 0u;
}

// The ring of one group: `arrays` rows (or column slices of rows) per stage.
struct Ring {
  uint8_t* slots;      // [stages][arrays][pitch]
  uint64_t* full;      // [stages]
  volatile uint32_t* abort_flag;
  uint32_t* status;
  uint32_t stages, arrays, pitch;  // bytes of a slot
  uint32_t stage = 0, phase = 0;   // of the row being read
  uint32_t filled = 0;             // (the lanes that fill) the stage to fill next

  __device__ __forceinline__ uint8_t* slot(uint32_t st, uint32_t array) const {
    return slots + (size_t)((st * arrays + array) * pitch);
  }
  // all threads: the row at `stage` has landed.  False where the wait ran out; `left`
  // rows are then in flight, and a lane that filled sees them land before shared memory
  // goes.
  __device__ __forceinline__ bool wait(uint32_t left) const {
    if (mbar_try_wait(smem_u32(full + stage), phase)) return true;
    return ring_wait_slow(smem_u32(full), stage, phase, stages, abort_flag, status, left);
  }
  __device__ __forceinline__ void advance() {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// Brings row slices to slots, which keep their offset to a boundary (see RowPieces).
template <typename T>
struct RowCopies {
  static constexpr int N = 16 / (int)sizeof(T);
  RowPieces pieces;
  int shift;
  __device__ __forceinline__ RowCopies(int shift_, int cols, bool ends_row)
      : pieces(RowPieces::of(shift_, cols, N, ends_row)), shift(shift_) {}
  __device__ __forceinline__ static void by_element(const T* row, uint8_t* slot, int shift, int begin, int end) {
    T* to = reinterpret_cast<T*>(slot);
#pragma unroll 1
    for (int e = begin; e < end; ++e)
      if (e >= shift) to[e] = row[e - shift];
  }
  // One array's row: one arrival on the stage's barrier (which counts the arrays).  A
  // null row (an array that its readers fetch themselves) only arrives.
  __device__ __forceinline__ void issue(const T* row, uint8_t* slot, uint32_t bar, bool tail) const {
    uint32_t n = row != nullptr ? (uint32_t)pieces.bytes : 0u;
    if (tail && pieces.rest != 0 && n != 0u) {
      n -= 16u;
      const int first = (int)(n / sizeof(T));
      by_element(row, slot, shift, first, first + pieces.rest);
    }
    mbar_arrive_expect_tx(bar, n);  // (after the elements copied one by one)
    if (n != 0u) bulk_load(smem_u32(slot), row - shift, n, bar);
  }
};

// The same for one of the first rows of an array that starts off a boundary.
template <typename T>
static __device__ __noinline__ void issue_head(const T* row, uint8_t* slot, uint32_t bar, int shift, int cols, bool tail) {
  constexpr int N = 16 / (int)sizeof(T);
  const RowPieces p = RowPieces::of(shift, cols, N, true);
  const int begin = p.begin(true), end = p.end(tail);
  RowCopies<T>::by_element(row, slot, shift, 0, min(N, shift + cols));
  RowCopies<T>::by_element(row, slot, shift, max(N, end / (int)sizeof(T)), shift + cols);
  const uint32_t n = begin < end ? (uint32_t)(end - begin) : 0u;
  mbar_arrive_expect_tx(bar, n);
  if (n != 0u) bulk_load(smem_u32(slot) + (uint32_t)begin, row - shift + N, n, bar);
}

// A group's E elements from a slot; `piece` is the thread's first 16-byte piece there.
template <typename T, int E>
__device__ __forceinline__ void from_slot(float (&v)[E], const uint8_t* slot, int piece) {
  const uint4* from = reinterpret_cast<const uint4*>(slot) + piece;
  Pack<T, E> p;
#pragma unroll
  for (int k = 0; k < Pack<T, E>::W / 4; ++k) {
    const uint4 q = from[k];
    p.w[4 * k] = q.x;
    p.w[4 * k + 1] = q.y;
    p.w[4 * k + 2] = q.z;
    p.w[4 * k + 3] = q.w;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = element(p, e);
}

// A row's first and last group (and those past it) hold elements of other rows or
// nothing: the thread that reads them makes them 0 in its own piece of the slot, so
// that no reader has to look.  (Ordered before the bulk copy that refills the slot.)
template <typename T, int E>
__device__ __forceinline__ void clean_slot(uint8_t* slot, int piece, const Places& at) {
  T* to = reinterpret_cast<T*>(slot + (size_t)piece * 16);
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (!at.inside(e)) to[e] = from_f32<T>(0.f);
  fence_proxy_async_smem();
}

// A group's E elements to a row that starts at the shift its places were made for; a
// group that is not whole 16-byte pieces there goes by element.
template <typename T, int E>
__device__ __forceinline__ void to_row(T* row, const float (&f)[E], const Places& at, bool whole) {
  const Pack<T, E> p = packed<T>(f);
  row += at.first;
  if (whole) {
#pragma unroll
    for (int k = 0; k < Pack<T, E>::W / 4; ++k)
      reinterpret_cast<uint4*>(row)[k] = make_uint4(p.w[4 * k], p.w[4 * k + 1], p.w[4 * k + 2], p.w[4 * k + 3]);
  } else if (at.first < at.end) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (at.inside(e)) {
        const uint32_t w = p.w[e * (int)sizeof(T) / 4];
        if constexpr (sizeof(T) == 4) {
          reinterpret_cast<uint32_t*>(row)[e] = w;
        } else {
          reinterpret_cast<uint16_t*>(row)[e] = (uint16_t)((e & 1) ? w >> 16 : w);
        }
      }
  }
}

// ------------------------------------------------------------------- forward

// A thread keeps its columns' factors in registers where it can (HOLD): with 32-bit
// parameters they are more bytes than a 16-bit row, and with most of the SM's memory
// given to the ring they would come from L2 for every row (8192 x 4096: 63 us so, 45
// held).
//   z -> s:  post_weight * gate * branch_scale, post_bias * gate * branch_scale
//   s -> n:  pre_weight, pre_bias
template <typename P, bool LAYER, int NV, int E>
struct RowFactors {
  static constexpr int NB = LAYER ? NV : 1, EB = LAYER ? E : 1;  // biases are held for the layer norm
  float branch[NV][E], branch_bias[NB][EB], pre[NV][E], pre_bias[NB][EB];

  __device__ __forceinline__ void for_gate(const ffn_norm_t& a, const P* gate, const Places (&at)[NV]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float g[E];
      parameters<P>(g, gate, 1.f, at[j]);
      parameters<P>(branch[j], a.post_weight, 1.f, at[j]);
#pragma unroll
      for (int e = 0; e < E; ++e) branch[j][e] *= a.branch_scale * g[e];
      zero_outside(branch[j], at[j]);
      if constexpr (LAYER) {
        parameters<P>(branch_bias[j], a.post_bias, 0.f, at[j]);
        if (a.post_bias != nullptr) {  // (an absent bias stays 0 whatever the gate)
#pragma unroll
          for (int e = 0; e < E; ++e) branch_bias[j][e] *= a.branch_scale * g[e];
        }
      }
    }
  }
  __device__ __forceinline__ RowFactors(const ffn_norm_t& a, const Places (&at)[NV]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      parameters<P>(pre[j], a.pre_weight, 1.f, at[j]);
      if constexpr (LAYER) parameters<P>(pre_bias[j], a.pre_bias, 0.f, at[j]);
    }
  }
};

// Bound by memory: 8192 x 4096 bf16, RMS twice, 45 us (6.0 TB/s of the four arrays'
// bytes); as a layer norm 73, where the sums around the warps' means and their joining
// take as long as the copies.  (An RMS norm with biases takes the direct form.)
template <typename T, typename P, bool LAYER, bool WARP, int NV>
__global__ void __launch_bounds__(WARP ? 256 : 512, WARP && !(LAYER && NV == 4) ? 2 : 1)
    k_norm_ring(const __grid_constant__ ffn_norm_t a, const __grid_constant__ NormShape sh, uint32_t* status) {
  constexpr int E = 16 / (int)sizeof(T);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[8 * kNormStages];
  __shared__ __align__(16) float parts[2 * RowSums::kFloats];
  __shared__ volatile uint32_t abort_flag;
  const int tid = WARP ? (int)lane_idx() : (int)threadIdx.x, per_row = WARP ? 32 : (int)blockDim.x;
  const int lane_group = WARP ? (int)(threadIdx.x >> 5) : 0, groups = WARP ? (int)(blockDim.x / 32) : 1;
  const int D = (int)a.D;
  Ring ring;
  ring.stages = kNormStages;
  ring.arrays = a.residual != nullptr ? 2u : 1u;
  ring.pitch = (uint32_t)(NV * per_row * 16);
  ring.slots = smem + (size_t)lane_group * ring.stages * ring.arrays * ring.pitch;
  ring.full = bars + lane_group * kNormStages;
  ring.abort_flag = &abort_flag;
  ring.status = status;
  RowSums sum{parts, WARP ? 1 : (int)(blockDim.x / 32), 1, 0, 0};
  if constexpr (!WARP) sum.clear();
  if (tid == 0) {
    for (uint32_t s = 0; s < ring.stages; ++s)
      mbar_init(smem_u32(ring.full + s), ring.arrays + missing_arrival(a.debug_flags, lane_group, s));
    fence_mbar_init();
  }
  if (threadIdx.x == 0) abort_flag = 0u;
  __syncthreads();
  wait_for_prior_kernel();
  let_next_kernel_start();
  // this group's rows: a slice, and in it the rows of one class (see norm_walk)
  const int part = (int)blockIdx.x * groups + lane_group, slice = part / sh.period;
  const int64_t step = sh.period;
  const int64_t r0 = (int64_t)sh.share.begin(slice) * step + (part - slice * sh.period);
  const int64_t r1 = min(a.M, (int64_t)sh.share.begin(slice + 1) * step);
  if (r0 >= r1) return;  // (a whole group)
  const int shift = row_shift(static_cast<const T*>(a.y) + r0 * a.ld_y);
  // the first lanes fill, an array each, so that the rows' copies cost one array's code
  const bool fills = tid < (int)ring.arrays;
  const T* in = static_cast<const T*>(tid == 0 ? a.y : a.residual);
  const int64_t in_ld = tid == 0 ? a.ld_y : a.ld_residual;
  int64_t ahead = r0;  // (the lanes that fill) the row to fetch next
  uint32_t in_flight = 0;
  const RowCopies<T> copies(shift, D, true);
  auto next_stage = [&]() {
    if (++ring.filled == ring.stages) ring.filled = 0;
    ahead += step;
    ++in_flight;
  };
  auto issue = [&]() {
    if (ahead >= r1) return;
    copies.issue(in + ahead * in_ld, ring.slot(ring.filled, (uint32_t)tid), smem_u32(ring.full + ring.filled),
                 ahead >= sh.tail);
    next_stage();
  };
  if (fills) {
    if (r0 < sh.head && shift != 0) {
      issue_head(in + r0 * in_ld, ring.slot(0, (uint32_t)tid), smem_u32(ring.full), shift, D, r0 >= sh.tail);
      next_stage();
    }
#pragma unroll 1
    while (in_flight < ring.stages && ahead < r1) issue();
  }

  const bool post = (a.flags & FFN_NORM_POST) != 0, pre = (a.flags & FFN_NORM_PRE) != 0;
  Places at[NV];
  bool whole[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    at[j] = Places{(j * per_row + tid) * E - shift, D};
    whole[j] = at[j].template whole<E>();
  }
  const float n_w = LAYER ? warp_elements<NV, E>(at) : 0.f;
  RowFactors<P, LAYER, NV, E> f(a, at);
  const uint32_t per = (uint32_t)a.M / (uint32_t)(a.gate != nullptr ? a.groups : 1);
  int64_t gate_end = 0;  // the first row with another gate
  for (int64_t r = r0; r < r1; r += step) {
    if (r >= gate_end) {
      const P* gate = gate_row<P>(a.gate, a.ld_gate, a.M, a.groups, r);
      gate_end = (int64_t)((uint32_t)r / per + 1u) * per;
      f.for_gate(a, gate, at);
    }
    if (!ring.wait(in_flight)) return;
    float v[NV][E];
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (!whole[j]) {
        clean_slot<T, E>(ring.slot(ring.stage, 0), j * per_row + tid, at[j]);
        if (a.residual != nullptr) clean_slot<T, E>(ring.slot(ring.stage, 1), j * per_row + tid, at[j]);
      }
#pragma unroll
    for (int j = 0; j < NV; ++j) from_slot<T>(v[j], ring.slot(ring.stage, 0), j * per_row + tid);
    float2 st = make_float2(0.f, 1.f);
    if (post) st = unit_of<LAYER>(v, at, D, n_w, a.eps, sum);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (post) {
        if constexpr (LAYER) add_to(v[j], v[j], -st.x);
        mul_to(v[j], v[j], st.y);
      }
      if constexpr (LAYER) {
        fma_to(v[j], v[j], f.branch[j], f.branch_bias[j]);
      } else {
        mul_to(v[j], v[j], f.branch[j]);
      }
      if (a.residual != nullptr) {
        float q[E];
        from_slot<T>(q, ring.slot(ring.stage, 1), j * per_row + tid);
        fma_to(v[j], q, a.residual_scale, v[j]);
      }
      if (LAYER && !whole[j]) {  // (past the row: a mean)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (!at[j].inside(e)) v[j][e] = 0.f;
      }
      if (a.s != nullptr) to_row(static_cast<T*>(a.s) + r * a.ld_s, v[j], at[j], whole[j]);
    }
    // the group has read the row's slots once it meets at the next barrier
    if (pre) st = unit_of<LAYER>(v, at, D, n_w, a.eps, sum);
    if constexpr (WARP) {
      __syncwarp();
    } else {
      if (!pre || per_row == 32) __syncthreads();
    }
    if (fills) {
      --in_flight;
      issue();
    }
    ring.advance();
    if (pre) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if constexpr (LAYER) add_to(v[j], v[j], -st.x);
        mul_to(v[j], v[j], st.y);
        if constexpr (LAYER) {
          fma_to(v[j], v[j], f.pre[j], f.pre_bias[j]);
        } else {
          mul_to(v[j], v[j], f.pre[j]);
        }
        to_row(static_cast<T*>(a.n) + r * a.ld_n, v[j], at[j], whole[j]);
      }
    }
  }
}

// ------------------------------------------------------------------ backward

// Rows of the backward kernel through a ring: s and dn, y, ds, those that are given.
// Arrays whose rows do not start at the walk's shift (odd pitches; a walk over whole
// groups) are brought to their slots by the threads that read them.
// The factors of a thread's columns stay in shared memory too, in places only that
// thread reads and writes: from global memory they came from L2 for every row, since
// the ring leaves little of the SM's memory to L1 (8192 x 4096: 238 us so, 78 now).
template <typename T, typename P, bool FULL, int G>
struct RowsRing {
  const ffn_norm_grad_t& a;
  const NormGradShape& sh;
  const Places (&at)[G];
  const RowCopies<T> copies;
  Ring ring;
  int64_t ahead, end, step;
  uint32_t y_at, ds_at;
  uint32_t slow;   // bits of the arrays off the walk's shift: s, dn, y, ds, dresidual, dy
  float* factors;  // [pre_weight, branch][G] groups of 8, `stride` floats apart
  int stride, col0, piece[G], clusters, rank, threads, tid;
  const T* in;     // (the lanes that fill, an array each) its row 0 here, null where it is slow
  int64_t in_ld;
  // (the lanes that fill) where a row's slot is free again: at the barrier of its second
  // round of sums, or, where it is read after that, at the next row's first barrier
  bool whole[G], fills, alone, first_row, early, late;

  __device__ __forceinline__ void issue() {
    if (ahead >= end) return;
    // (arrays that come this way start on a boundary)
    copies.issue(in != nullptr ? in + ahead * in_ld : nullptr, ring.slot(ring.filled, (uint32_t)lane_idx()),
                 smem_u32(ring.full + ring.filled), ahead >= sh.tail);
    if (++ring.filled == ring.stages) ring.filled = 0;
    ahead += step;
  }
  __device__ __forceinline__ void begin(const NormWalk& w) {
    ahead = w.first;
    end = w.end;
    step = w.step;
    first_row = true;
    if (fills) {
#pragma unroll 1
      for (uint32_t s = 0; s < ring.stages; ++s) issue();
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
      float f[8];
      parameters<P>(f, from_column<P>(a.pre_weight, col0), 1.f, at[j]);
      zero_outside(f, at[j]);
      keep(f, j);
    }
  }
  __device__ __forceinline__ void set_group(int64_t g) {
#pragma unroll
    for (int j = 0; j < G; ++j) {
      float f[8], w[8];
      parameters<P>(f, from_column<P>(a.gate, g * a.ld_gate + col0), 1.f, at[j]);
      parameters<P>(w, from_column<P>(a.post_weight, col0), 1.f, at[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= a.branch_scale * w[e];
      zero_outside(f, at[j]);
      keep(f, G + j);
    }
  }
  __device__ __forceinline__ void fetch(const void* p, int64_t ld, int64_t r, uint32_t array) {
    const T* row = static_cast<const T*>(p) + r * ld + col0;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      T* to = reinterpret_cast<T*>(ring.slot(ring.stage, array) + (size_t)piece[j] * 16);
#pragma unroll 4
      for (int e = 0; e < 8; ++e)
        if (at[j].inside(e)) to[e] = row[at[j].first + e];
    }
  }
  static constexpr int64_t kStopped = INT64_MAX;
  // The row's values are there; false where the wait for them ran out.  A CTA of a cluster
  // goes on then, on values that are void and without fetching more: its peers meet it at
  // every sum and write to its shared memory there.
  __device__ __forceinline__ bool next(int64_t r) {
    if (!ring.wait(fills && ahead != kStopped ? ring.stages : 0u)) {
      if (clusters == 1) return false;
      ahead = kStopped;
    }
    if (slow & 15u) {  // (a thread's own places: no one else reads them)
      if (a.dn != nullptr && (slow & 1u)) fetch(a.s, a.ld_s, r, 0);
      if (a.dn != nullptr && (slow & 2u)) fetch(a.dn, a.ld_dn, r, 1);
      if (a.y != nullptr && (slow & 4u)) fetch(a.y, a.ld_y, r, y_at);
      if (a.ds != nullptr && (slow & 8u)) fetch(a.ds, a.ld_ds, r, ds_at);
    }
#pragma unroll
    for (int j = 0; j < G; ++j)
      if (!whole[j]) {
#pragma unroll 1
        for (uint32_t k = 0; k < ring.arrays; ++k) clean_slot<T, 8>(ring.slot(ring.stage, k), piece[j], at[j]);
      }
    return true;
  }
  // every thread of the group has come to this row: the slots of the one before are free
  __device__ __forceinline__ void met() {
    if (late && !first_row) issue();
    first_row = false;
  }
  // every thread has this row's second sums: all but y has been read
  __device__ __forceinline__ void met_again() {
    if (early) issue();
  }
  __device__ __forceinline__ void done() {
    ring.advance();
    if (!alone) return;  // a lone warp meets no one at the next row's barrier
    __syncwarp();
    if (fills) issue();
  }
  __device__ __forceinline__ void values(float (&v)[8], uint32_t array, int j) const {
    from_slot<T>(v, ring.slots + ((FULL ? 4u : ring.arrays) * ring.stage + array) * ring.pitch, piece[j]);
  }
  __device__ __forceinline__ void s(float (&v)[8], int j) const { values(v, 0, j); }
  __device__ __forceinline__ void dn(float (&v)[8], int j) const { values(v, 1, j); }
  __device__ __forceinline__ void y(float (&v)[8], int j) const { values(v, FULL ? 2u : y_at, j); }
  __device__ __forceinline__ void ds(float (&v)[8], int j) const { values(v, FULL ? 3u : ds_at, j); }
  __device__ __forceinline__ void keep(const float (&v)[8], int k) {
    float4* to = reinterpret_cast<float4*>(factors + k * stride);
    to[0] = make_float4(v[0], v[1], v[2], v[3]);
    to[stride / 8] = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void factors_of(float (&f)[8], int k) const {
    const float4* from = reinterpret_cast<const float4*>(factors + k * stride);
    const float4 lo = from[0], hi = from[stride / 8];
    f[0] = lo.x, f[1] = lo.y, f[2] = lo.z, f[3] = lo.w;
    f[4] = hi.x, f[5] = hi.y, f[6] = hi.z, f[7] = hi.w;
  }
  __device__ __forceinline__ void pre_factors(float (&f)[8], int j) const { factors_of(f, j); }
  __device__ __forceinline__ void scale_pre(float (&v)[8], int j) const {
    float f[8];
    factors_of(f, j);
    mul_to(v, v, f);
  }
  __device__ __forceinline__ void scale_branch(float (&v)[8], int j) const {
    float f[8];
    factors_of(f, G + j);
    mul_to(v, v, f);
  }
  // where the part's sums of this thread's first group go in a sums array
  __device__ __forceinline__ int64_t sums_at(int part) const {
    return ((int64_t)part * clusters + rank) * threads * 8 * G + tid * 8;
  }
  // output 0: dresidual, 1: dy
  template <int OUTPUT>
  __device__ __forceinline__ void put(T* row, const float (&v)[8], int j) const {
    to_row(row, v, at[j], whole[j] && !(slow & (16u << OUTPUT)));
  }
};

// 8192 x 4096 bf16, RMS twice: 78 us with the columns' sums, 5.1 TB/s of the six arrays'
// bytes.  128 registers hold a thread's parameter sums and one row's values, so 16 warps
// share an SM, and what a row's two rounds of sums leave idle is what is missing: about
// half the issue slots are used.  As a layer norm 136 us: one more pass over the row.
template <typename T, typename P, bool FULL, bool LAYER, bool BIAS, bool MANY, int G>
__global__ void __launch_bounds__(kNormGradThreads, MANY || (sizeof(T) == 4 && G == 2) ? 1 : 2)
    k_norm_grad(const __grid_constant__ ffn_norm_grad_t a, const __grid_constant__ NormGradShape sh,
                const __grid_constant__ NormSums ws, uint32_t* status) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[8 * kNormStages];
  __shared__ __align__(16) float parts[2 * RowSums::kFloats];
  __shared__ volatile uint32_t abort_flag;
  const int rank = sh.cluster > 1 ? (int)cluster_ctarank() : 0;
  const int tid = sh.lanes > 1 ? (int)lane_idx() : (int)threadIdx.x;
  const int lane_group = sh.lanes > 1 ? (int)(threadIdx.x >> 5) : 0;
  const int part = sh.lanes > 1 ? (int)blockIdx.x * sh.lanes + lane_group : (int)blockIdx.x / sh.cluster;
  RowSums sum{parts, sh.threads / 32, sh.cluster, rank, 0};
  if (sh.cluster == 1) sum.clear();
  // The walk's shift is that of rows without gaps from a 16-byte boundary on, whatever
  // the arrays' pitches: which elements a thread adds up, and so the results' last
  // bits, depend on the sizes alone.
  const NormWalk walk = norm_walk<MANY>(a, sh, min(part, sh.parts - 1));
  const int col0 = (int)(rank * sh.columns), cols = min((int)a.D - col0, (int)sh.columns);
  const int shift = norm_part_shift(a, sh, min(part, sh.parts - 1), sizeof(T));
  Places at[G];
#pragma unroll
  for (int j = 0; j < G; ++j) at[j] = Places{(j * sh.threads + tid) * 8 - shift, cols};
  RowsRing<T, P, FULL, G> rows{a, sh, at, RowCopies<T>(shift, cols, rank == sh.cluster - 1)};
  rows.y_at = a.dn != nullptr ? 2u : 0u;
  rows.ds_at = rows.y_at + (a.y != nullptr ? 1u : 0u);
  rows.alone = sum.warps == 1 && sum.cluster == 1;
  rows.col0 = col0;
  rows.clusters = sh.cluster;
  rows.rank = rank;
  rows.threads = sh.threads;
  rows.tid = tid;
  rows.slow = sh.slow;
#pragma unroll
  for (int j = 0; j < G; ++j) {
    rows.piece[j] = (j * sh.threads + tid) * (int)sizeof(T) / 2;
    rows.whole[j] = at[j].template whole<8>();
  }
  // thread i's 16-byte pieces of the factors, i pieces in: no bank conflicts
  rows.stride = 8 * (int)blockDim.x;
  rows.factors = reinterpret_cast<float*>(smem) + 4 * threadIdx.x;
  rows.ring.stages = (uint32_t)sh.stages;
  rows.ring.arrays = rows.ds_at + (a.ds != nullptr ? 1u : 0u);
  rows.ring.pitch = (uint32_t)(8 * G * sh.threads * (int)sizeof(T));
  rows.fills = tid < (int)rows.ring.arrays;
  {
    // lane k fills the k-th array given: s and dn, then y, then ds
    const bool s = a.dn != nullptr && tid == 0, dn = a.dn != nullptr && tid == 1;
    const bool y = !s && !dn && a.y != nullptr && tid == (int)rows.y_at;
    const void* p = s ? a.s : dn ? a.dn : y ? a.y : a.ds;
    rows.in_ld = s ? a.ld_s : dn ? a.ld_dn : y ? a.ld_y : a.ld_ds;
    const uint32_t bit = s ? 1u : dn ? 2u : y ? 4u : 8u;
    rows.in = (p == nullptr || (sh.slow & bit)) ? nullptr : static_cast<const T*>(p) + col0;
    // (8192 x 4096 82.4 -> 78.0 us; the layer norm's kernel has no registers left for it:
    // 142 -> 149)
    const bool again = !LAYER && (FULL || (a.dy != nullptr && (a.flags & FFN_NORM_POST) != 0));
    rows.early = rows.fills && !rows.alone && again && !y;
    rows.late = rows.fills && !rows.alone && !rows.early;
  }
  rows.ring.slots = smem + (size_t)2 * G * rows.stride * sizeof(float) +
                    (size_t)lane_group * sh.stages * rows.ring.arrays * rows.ring.pitch;
  rows.ring.full = bars + lane_group * kNormStages;
  rows.ring.abort_flag = &abort_flag;
  rows.ring.status = status;
  if (tid == 0) {
    for (int s = 0; s < sh.stages; ++s)
      mbar_init(smem_u32(rows.ring.full + s), rows.ring.arrays + missing_arrival(a.debug_flags, lane_group, (uint32_t)s));
    fence_mbar_init();
  }
  if (threadIdx.x == 0) abort_flag = 0u;
  if (sh.cluster > 1) {
    cluster_sync_all();  // (the peers' shared memory may be written from here on)
  } else {
    __syncthreads();
  }
  wait_for_prior_kernel();
  let_next_kernel_start();
  if (part >= sh.parts) return;  // (whole warps only)
  // from here on columns count from the slice's first, in every array
  norm_grad_rows<FULL, LAYER, BIAS, MANY, G, T, P>(a, sh, ws, rows, sum, part, walk, at, col0);
}

}  // namespace

}  // namespace dgb
