// kernels_norm_ring.cuh -- the block norms with rows that come through a ring in
// shared memory filled by bulk copies (cp.async.bulk), so an SM has tens of KB on
// their way whatever its threads do, and the backward kernel can read a row's values
// again instead of holding them in registers.  Rows may start anywhere: a copy
// brings the whole 16-byte pieces a row lies in, and reads shift by its offset.
//
// A group (a warp, a CTA, or in the backward kernel a cluster of CTAs that share
// the columns) walks its rows with `stages` rows ahead.  Every wait is bounded; a
// wait that runs out is recorded in the device's status word.
#pragma once

#include "kernels_norm.cuh"

namespace dgb {

namespace {

// raise the transaction bytes a phase expects, without arriving
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

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

// The ring of one group: `arrays` rows (or column slices of rows) per stage.
struct Ring {
  uint8_t* slots;      // [stages][arrays][pitch]
  uint64_t* full;      // [stages]
  volatile uint32_t* abort_flag;
  uint32_t* status;
  uint32_t stages, arrays, bytes, pitch;  // bytes of a row (slice); of a slot
  uint32_t stage = 0, phase = 0;          // of the row being read
  uint32_t filled = 0;                    // (the group's first thread) the stage to fill next

  __device__ __forceinline__ uint8_t* slot(uint32_t st, uint32_t array) const {
    return slots + (size_t)((st * arrays + array) * pitch);
  }
  // all threads: the row at `stage` has landed.  False where the wait ran out; `left`
  // copies of this thread's are then in flight, and it sees them land before shared
  // memory goes.
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

// One array of a call: where its rows are, and where they may be read.
template <typename T, bool ALIGNED>
struct RingArray {
  const T* base;  // row 0, from this group's first column on
  int64_t ld;
  uintptr_t lo, hi;  // the array's first byte and the end of its last row

  __device__ __forceinline__ RingArray(const void* p, int64_t pitch, int64_t rows, int64_t D, int col0)
      : base(static_cast<const T*>(p) + col0), ld(pitch), lo(reinterpret_cast<uintptr_t>(p)) {
    hi = lo + (uintptr_t)(((rows - 1) * pitch + D) * (int64_t)sizeof(T));
  }
  // how far row r starts past a 16-byte boundary
  __device__ __forceinline__ uint32_t off(int64_t r) const {
    if constexpr (ALIGNED) return 0u;
    return ((uint32_t)reinterpret_cast<uintptr_t>(base) + (uint32_t)r * (uint32_t)(ld * (int64_t)sizeof(T))) & 15u;
  }
  // The 16-byte pieces row r's `bytes` lie in, [from, to); where the first or last of
  // them reaches outside the array, only the pieces inside.
  __device__ __forceinline__ void span(int64_t r, uint32_t bytes, uintptr_t& from, uintptr_t& to) const {
    const uintptr_t begin = reinterpret_cast<uintptr_t>(base + r * ld), end = begin + bytes;
    from = begin & ~(uintptr_t)15;
    to = (end + 15) & ~(uintptr_t)15;
    if (from < lo) from += 16;
    if (to > hi) to -= 16;
    if (to < from) to = from;
  }
  // Brings row r to `slot`, which keeps its offset to 16-byte boundaries: whole pieces
  // by a bulk copy, elements of pieces that reach outside the array one by one.
  __device__ __forceinline__ void copy(int64_t r, uint32_t bytes, uint8_t* slot, uint32_t bar) const {
    if constexpr (ALIGNED) {
      bulk_load(smem_u32(slot), base + r * ld, bytes, bar);
      return;
    }
    uintptr_t from, to;
    span(r, bytes, from, to);
    const uintptr_t begin = reinterpret_cast<uintptr_t>(base + r * ld), end = begin + bytes;
    const uintptr_t origin = begin & ~(uintptr_t)15;
    for (uintptr_t q = begin; q < end && q < from; q += sizeof(T))
      *reinterpret_cast<T*>(slot + (q - origin)) = *reinterpret_cast<const T*>(q);
    for (uintptr_t q = to > begin ? to : begin; q < end; q += sizeof(T))
      if (q >= from) *reinterpret_cast<T*>(slot + (q - origin)) = *reinterpret_cast<const T*>(q);
    if (to > from) bulk_load(smem_u32(slot + (from - origin)), reinterpret_cast<const void*>(from), (uint32_t)(to - from), bar);
  }
  __device__ __forceinline__ uint32_t copied(int64_t r, uint32_t bytes) const {
    if constexpr (ALIGNED) return bytes;
    uintptr_t from, to;
    span(r, bytes, from, to);
    return (uint32_t)(to - from);
  }
};

// bytes of a slot: a row at any offset, and the piece after it that a shifted read touches
__host__ __device__ constexpr uint32_t ring_pitch(uint32_t bytes) { return (bytes + 31u) / 32u * 32u + 32u; }

// E elements from element `i` on of the row at offset m of a slot; 0 from element
// `end` on
template <typename T, bool ALIGNED, int E>
__device__ __forceinline__ void from_slot(float (&v)[E], const uint8_t* slot, uint32_t m, int i, int end) {
  constexpr int W = Pack<T, E>::W;
  Pack<T, E> p;
  const uint4* from = reinterpret_cast<const uint4*>(slot + (size_t)i * sizeof(T));
  if constexpr (ALIGNED) {
    const bool live = i < end;
#pragma unroll
    for (int k = 0; k < W / 4; ++k) {
      const uint4 q = live ? from[k] : make_uint4(0u, 0u, 0u, 0u);
      p.w[4 * k] = q.x;
      p.w[4 * k + 1] = q.y;
      p.w[4 * k + 2] = q.z;
      p.w[4 * k + 3] = q.w;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = element(p, e);
  } else {
    uint32_t w[W + 4];
#pragma unroll
    for (int k = 0; k < W / 4 + 1; ++k) {
      const uint4 q = i < end ? from[k] : make_uint4(0u, 0u, 0u, 0u);
      w[4 * k] = q.x;
      w[4 * k + 1] = q.y;
      w[4 * k + 2] = q.z;
      w[4 * k + 3] = q.w;
    }
    shift_down(w, m);
#pragma unroll
    for (int k = 0; k < W; ++k) p.w[k] = w[k];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = i + e < end ? element(p, e) : 0.f;
  }
}

// a parameter vector's elements; the vectors of an ALIGNED call start on 16-byte boundaries
template <typename P, bool ALIGNED, int E>
__device__ __forceinline__ void row_parameters(float (&v)[E], const void* p, float absent, const Places& at) {
  if constexpr (!ALIGNED) {
    parameters<P>(v, p, absent, at);
  } else {
    if (p == nullptr) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = absent;
      return;
    }
    Pack<P, E> raw;
#pragma unroll
    for (int k = 0; k < Pack<P, E>::W / 4; ++k) {
      const uint4 q = at.inside(0) ? __ldg(reinterpret_cast<const uint4*>(static_cast<const P*>(p) + at.first) + k)
                                   : make_uint4(0u, 0u, 0u, 0u);
      raw.w[4 * k] = q.x;
      raw.w[4 * k + 1] = q.y;
      raw.w[4 * k + 2] = q.z;
      raw.w[4 * k + 3] = q.w;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = element(raw, e);
  }
}

template <typename T, bool ALIGNED, int E>
__device__ __forceinline__ void row_store(T* row, const float (&f)[E], const Places& at) {
  if constexpr (!ALIGNED) {
    store(row, f, at);
  } else {
    if (!at.inside(0)) return;
    const Pack<T, E> w = packed<T>(f);
#pragma unroll
    for (int k = 0; k < Pack<T, E>::W / 4; ++k)
      reinterpret_cast<uint4*>(row + at.first)[k] =
          make_uint4(w.w[4 * k], w.w[4 * k + 1], w.w[4 * k + 2], w.w[4 * k + 3]);
  }
}

// ------------------------------------------------------------------- forward

// A thread keeps its columns' parameters in registers where it has at most two
// vectors (HOLD): with 32-bit parameters they are more bytes than a 16-bit row, and
// with most of the SM's memory given to the ring they would come from L2 for every
// row (8192 x 4096: 63 us read per row).
template <typename P, bool ALIGNED, int NV, int E, bool HOLD>
struct RowFactors {
  const P* p;
  float held[HOLD ? NV : 1][HOLD ? E : 1];
  __device__ __forceinline__ RowFactors(const void* from, const Places (&at)[NV]) : p(static_cast<const P*>(from)) {
    if constexpr (HOLD) {
      if (p != nullptr) {
#pragma unroll
        for (int j = 0; j < NV; ++j) row_parameters<P, ALIGNED>(held[j], p, 1.f, at[j]);
      }
    }
  }
  __device__ __forceinline__ void times(float (&v)[E], int j, const Places& at) const {
    if (p == nullptr) return;
    float f[E];
    get(f, j, at);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] *= f[e];
  }
  __device__ __forceinline__ void plus(float (&v)[E], int j, const Places& at) const {
    if (p == nullptr) return;
    float f[E];
    get(f, j, at);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] += f[e];
  }
  __device__ __forceinline__ void get(float (&f)[E], int j, const Places& at) const {
    if constexpr (HOLD) {
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = held[j][e];
    } else {
      row_parameters<P, ALIGNED>(f, p, 1.f, at);
    }
  }
};

template <typename T, typename P, bool ALIGNED, bool LAYER, bool WARP, int NV>
__global__ void __launch_bounds__(WARP ? 256 : 512, WARP ? 2 : 1) k_norm_ring(const __grid_constant__ ffn_norm_t a, uint32_t* status) {
  constexpr int E = 16 / (int)sizeof(T);
  constexpr bool HOLD = !WARP && NV <= 2;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[8 * kNormStages];
  __shared__ float parts[2 * RowSums::kFloats];
  __shared__ volatile uint32_t abort_flag;
  const int tid = WARP ? (int)lane_idx() : (int)threadIdx.x, per_row = WARP ? 32 : (int)blockDim.x;
  const int group = WARP ? (int)(threadIdx.x >> 5) : 0, groups = WARP ? (int)(blockDim.x / 32) : 1;
  const int D = (int)a.D;
  Ring ring;
  ring.stages = kNormStages;
  ring.arrays = a.residual != nullptr ? 2u : 1u;
  ring.bytes = (uint32_t)(D * (int)sizeof(T));
  ring.pitch = ring_pitch(ring.bytes);
  ring.slots = smem + (size_t)group * ring.stages * ring.arrays * ring.pitch;
  ring.full = bars + group * kNormStages;
  ring.abort_flag = &abort_flag;
  ring.status = status;
  RowSums sum{parts, WARP ? 1 : (int)(blockDim.x / 32), 1, 0, 0};
  if (tid == 0) {
    for (uint32_t s = 0; s < ring.stages; ++s) mbar_init(smem_u32(ring.full + s), 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) abort_flag = 0u;
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t step = (int64_t)gridDim.x * groups, r0 = (int64_t)blockIdx.x * groups + group;
  int64_t ahead = r0;  // (the group's first thread) the row to fetch next
  uint32_t in_flight = 0;
  const RingArray<T, ALIGNED> in_y(a.y, a.ld_y, a.M, D, 0), in_res(a.residual, a.ld_residual, a.M, D, 0);
  auto issue = [&]() {
    if (ahead >= a.M) return;
    const uint32_t bar = smem_u32(ring.full + ring.filled);
    const bool two = a.residual != nullptr;
    // (the elements a copy brings one by one are ordered by this arrival: they come first)
    const uint32_t bytes = in_y.copied(ahead, ring.bytes) + (two ? in_res.copied(ahead, ring.bytes) : 0u);
    mbar_expect_tx(bar, bytes);
    in_y.copy(ahead, ring.bytes, ring.slot(ring.filled, 0), bar);
    if (two) in_res.copy(ahead, ring.bytes, ring.slot(ring.filled, 1), bar);
    mbar_arrive(bar);
    if (++ring.filled == ring.stages) ring.filled = 0;
    ahead += step;
    ++in_flight;
  };
  if (tid == 0)
    for (uint32_t s = 0; s < ring.stages; ++s) issue();

  const bool post = (a.flags & FFN_NORM_POST) != 0, pre = (a.flags & FFN_NORM_PRE) != 0;
  Places at[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) at[j] = Places{(j * per_row + tid) * E, D};
  const float n_w = LAYER ? warp_elements<NV, E>(at) : 0.f;
  const bool one_gate = a.groups == 1;
  const RowFactors<P, ALIGNED, NV, E, HOLD> post_weight(a.post_weight, at), pre_weight(a.pre_weight, at),
      shared_gate(one_gate ? a.gate : nullptr, at);
  const RowFactors<P, ALIGNED, NV, E, HOLD && LAYER> post_bias(a.post_bias, at), pre_bias(a.pre_bias, at);
  for (int64_t r = r0; r < a.M; r += step) {
    float own_gate[NV][E];  // (asked for early: it comes from L2)
    if (a.gate != nullptr && !one_gate) {
      const P* gate = gate_row<P>(a.gate, a.ld_gate, a.M, a.groups, r);
#pragma unroll
      for (int j = 0; j < NV; ++j) row_parameters<P, ALIGNED>(own_gate[j], gate, 1.f, at[j]);
    }
    if (!ring.wait(in_flight)) return;
    const uint32_t off_y = in_y.off(r), off_res = in_res.off(r);
    float v[NV][E];
#pragma unroll
    for (int j = 0; j < NV; ++j) from_slot<T, ALIGNED>(v[j], ring.slot(ring.stage, 0), off_y, at[j].first, D);
    if (post) {
      const float2 st = unit_of<LAYER, ALIGNED>(v, at, D, n_w, a.eps, sum);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[j][e] = (v[j][e] - st.x) * st.y;
        post_weight.times(v[j], j, at[j]);
        post_bias.plus(v[j], j, at[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[j][e] *= a.branch_scale;
      if (a.gate != nullptr) {
        if (one_gate) {
          shared_gate.times(v[j], j, at[j]);
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) v[j][e] *= own_gate[j][e];
        }
      }
      if (a.residual != nullptr) {
        float q[E];
        from_slot<T, ALIGNED>(q, ring.slot(ring.stage, 1), off_res, at[j].first, D);
#pragma unroll
        for (int e = 0; e < E; ++e) v[j][e] = fmaf(a.residual_scale, q[e], v[j][e]);
      }
      if (!ALIGNED || LAYER) {  // (past the end: a mean or a bias of the post norm)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (!at[j].inside(ALIGNED ? 0 : e)) v[j][e] = 0.f;
      }
      if (a.s != nullptr) row_store<T, ALIGNED>(static_cast<T*>(a.s) + r * a.ld_s, v[j], at[j]);
    }
    // the group has read the row's slots once it meets at the next barrier
    float2 st = make_float2(0.f, 1.f);
    if (pre) st = unit_of<LAYER, ALIGNED>(v, at, D, n_w, a.eps, sum);
    if constexpr (WARP) {
      __syncwarp();
    } else {
      if (!pre || per_row == 32) __syncthreads();
    }
    if (tid == 0) {
      --in_flight;
      issue();
    }
    ring.advance();
    if (pre) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[j][e] = (v[j][e] - st.x) * st.y;
        pre_weight.times(v[j], j, at[j]);
        pre_bias.plus(v[j], j, at[j]);
        row_store<T, ALIGNED>(static_cast<T*>(a.n) + r * a.ld_n, v[j], at[j]);
      }
    }
  }
}

// ------------------------------------------------------------------ backward

// Rows of the backward kernel through a ring: s and dn, y, ds, those that are given.
// The factors of a thread's columns stay in shared memory too, in places only that
// thread reads and writes: from global memory they came from L2 for every row, since
// the ring leaves little of the SM's memory to L1 (8192 x 4096: 238 us).
template <typename T, typename P, bool ALIGNED>
struct RowsRing {
  static constexpr bool kWhole = ALIGNED;  // groups of 8 columns lie wholly in or out of a row
  const ffn_norm_grad_t& a;
  const Places (&at)[2];
  RingArray<T, ALIGNED> in_s, in_dn, in_y, in_ds;
  Ring ring;
  int64_t ahead, r1;
  uint32_t y_at, ds_at;
  float* factors;  // [pre_weight, branch][2] groups of 8, `stride` floats apart
  int stride;
  int local[2], cols;  // this thread's columns in a slot, and how many a slot has
  uint32_t off_s, off_dn, off_y, off_ds;  // the row's offsets
  bool first_thread, alone;

  __device__ __forceinline__ void issue() {
    if (ahead >= r1) return;
    const uint32_t bar = smem_u32(ring.full + ring.filled), n = ring.bytes;
    uint32_t bytes = 0;
    if (a.dn != nullptr) bytes += in_s.copied(ahead, n) + in_dn.copied(ahead, n);
    if (a.y != nullptr) bytes += in_y.copied(ahead, n);
    if (a.ds != nullptr) bytes += in_ds.copied(ahead, n);
    mbar_expect_tx(bar, bytes);
    if (a.dn != nullptr) {
      in_s.copy(ahead, n, ring.slot(ring.filled, 0), bar);
      in_dn.copy(ahead, n, ring.slot(ring.filled, 1), bar);
    }
    if (a.y != nullptr) in_y.copy(ahead, n, ring.slot(ring.filled, y_at), bar);
    if (a.ds != nullptr) in_ds.copy(ahead, n, ring.slot(ring.filled, ds_at), bar);
    mbar_arrive(bar);  // (after the elements that were copied one by one)
    if (++ring.filled == ring.stages) ring.filled = 0;
    ++ahead;
  }
  __device__ __forceinline__ void begin(int64_t from, int64_t to) {
    ahead = from;
    r1 = to;
    if (first_thread)
      for (uint32_t s = 0; s < ring.stages; ++s) issue();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float w[8];
      row_parameters<P, ALIGNED>(w, a.pre_weight, 1.f, at[j]);
      keep(w, j);
    }
  }
  __device__ __forceinline__ void set_group(int64_t g) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float f[8];
      float w[8];
      row_parameters<P, ALIGNED>(f, a.gate != nullptr ? static_cast<const P*>(a.gate) + g * a.ld_gate : nullptr, 1.f,
                                 at[j]);
      row_parameters<P, ALIGNED>(w, a.post_weight, 1.f, at[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __fmul_rn(__fmul_rn(a.branch_scale, f[e]), w[e]);
      keep(f, 2 + j);
    }
  }
  __device__ __forceinline__ bool next(int64_t r) {
    if (!ring.wait(first_thread ? (uint32_t)(ahead - r) : 0u)) return false;
    off_s = in_s.off(r);
    off_dn = in_dn.off(r);
    off_y = in_y.off(r);
    off_ds = in_ds.off(r);
    return true;
  }
  // every thread of the group has come to this row: the slots of the one before are free
  __device__ __forceinline__ void met() {
    if (first_thread && !alone && !first_row) issue();
    first_row = false;
  }
  bool first_row = true;
  __device__ __forceinline__ void done() {
    ring.advance();
    if (!alone) return;  // a lone warp meets no one at the next row's barrier
    __syncwarp();
    if (first_thread) issue();
  }
  __device__ __forceinline__ void values(float (&v)[8], uint32_t array, uint32_t off, int j) const {
    from_slot<T, ALIGNED>(v, ring.slot(ring.stage, array), off, local[j], cols);
  }
  __device__ __forceinline__ void s(float (&v)[8], int j) const { values(v, 0, off_s, j); }
  __device__ __forceinline__ void dn(float (&v)[8], int j) const { values(v, 1, off_dn, j); }
  __device__ __forceinline__ void y(float (&v)[8], int j) const { values(v, y_at, off_y, j); }
  __device__ __forceinline__ void ds(float (&v)[8], int j) const { values(v, ds_at, off_ds, j); }
  __device__ __forceinline__ void keep(const float (&v)[8], int k) {
    float4* to = reinterpret_cast<float4*>(factors + k * stride);
    to[0] = make_float4(v[0], v[1], v[2], v[3]);
    to[stride / 8] = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void scale(float (&v)[8], int k) const {
    const float4* from = reinterpret_cast<const float4*>(factors + k * stride);
    const float4 lo = from[0], hi = from[stride / 8];
    const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], f[e]);
  }
  __device__ __forceinline__ void scale_pre(float (&v)[8], int j) const { scale(v, j); }
  __device__ __forceinline__ void scale_branch(float (&v)[8], int j) const { scale(v, 2 + j); }
  __device__ __forceinline__ void put(T* to, const float (&v)[8], const Places& w) const {
    row_store<T, ALIGNED>(to, v, w);
  }
};

template <typename T, typename P, bool ALIGNED, bool LAYER, bool BIAS, bool MANY>
__global__ void __launch_bounds__(kNormGradThreads, MANY || sizeof(T) == 4 ? 1 : 2)
    k_norm_grad(const __grid_constant__ ffn_norm_grad_t a, const __grid_constant__ NormGradShape sh,
                const __grid_constant__ NormSums ws, uint32_t* status) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[8 * kNormStages];
  __shared__ float parts[2 * RowSums::kFloats];
  __shared__ volatile uint32_t abort_flag;
  const NormGradPlace w(a, sh);
  RowSums sum{parts, sh.threads / 32, sh.cluster, w.rank, 0};
  RowsRing<T, P, ALIGNED> rows{a,
                      w.at,
                      RingArray<T, ALIGNED>(a.s, a.ld_s, a.M, a.D, w.col0),
                      RingArray<T, ALIGNED>(a.dn, a.ld_dn, a.M, a.D, w.col0),
                      RingArray<T, ALIGNED>(a.y, a.ld_y, a.M, a.D, w.col0),
                      RingArray<T, ALIGNED>(a.ds, a.ld_ds, a.M, a.D, w.col0)};
  rows.y_at = a.dn != nullptr ? 2u : 0u;
  rows.ds_at = rows.y_at + (a.y != nullptr ? 1u : 0u);
  rows.first_thread = w.tid == 0;
  rows.alone = sum.warps == 1 && sum.cluster == 1;
  rows.cols = w.cols;
#pragma unroll
  for (int j = 0; j < 2; ++j) rows.local[j] = w.at[j].first - w.col0;
  // thread i's 16-byte pieces of the factors, i pieces in: no bank conflicts
  rows.stride = 8 * (int)blockDim.x;
  rows.factors = reinterpret_cast<float*>(smem) + 4 * threadIdx.x;
  rows.ring.stages = (uint32_t)sh.stages;
  rows.ring.arrays = rows.ds_at + (a.ds != nullptr ? 1u : 0u);
  rows.ring.bytes = (uint32_t)(w.cols * (int)sizeof(T));
  rows.ring.pitch = ring_pitch((uint32_t)(sh.columns * (int64_t)sizeof(T)));
  rows.ring.slots = smem + (size_t)4 * rows.stride * sizeof(float) +
                    (size_t)w.group * sh.stages * rows.ring.arrays * rows.ring.pitch;
  rows.ring.full = bars + w.group * kNormStages;
  rows.ring.abort_flag = &abort_flag;
  rows.ring.status = status;
  if (rows.first_thread) {
    for (int s = 0; s < sh.stages; ++s) mbar_init(smem_u32(rows.ring.full + s), 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) abort_flag = 0u;
  if (sh.cluster > 1) {
    cluster_sync_all();  // (the peers' shared memory may be written from here on)
  } else {
    __syncthreads();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (w.part >= sh.parts) return;  // (whole warps only)
  norm_grad_rows<LAYER, BIAS, MANY, T, P>(a, sh, ws, rows, sum, w.part, w.at);
}

}  // namespace

}  // namespace dgb
