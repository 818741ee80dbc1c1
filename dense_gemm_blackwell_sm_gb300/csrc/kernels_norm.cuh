// kernels_norm.cuh -- the norms around a block fused with its gate, its scales and
// the residual stream, one pass over the rows, and their gradients, one pass too.
//
// Bound by memory: 4 row reads and writes forward (y, residual, s, n), 6 backward
// (ds, dn, y, s, dresidual, dy).  Every row is read once and written once.
#pragma once

#include <type_traits>

#include "ffn_common.cuh"
#include "norm.h"

namespace dgb {

namespace {

// E consecutive elements of T as loaded: E = 16 bytes' worth, or twice that for
// fp32 in the backward kernel
template <typename T, int E>
struct Pack {
  static constexpr int W = E * (int)sizeof(T) / 4;
  uint32_t w[W];
};

template <typename T, int E>
__device__ __forceinline__ float element(const Pack<T, E>& p, int e) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(p.w[e]);
  } else {
    const uint16_t h = (uint16_t)((e & 1) ? p.w[e / 2] >> 16 : p.w[e / 2]);
    if constexpr (std::is_same<T, __half>::value) {
      return __half2float(__ushort_as_half(h));
    } else {
      return __uint_as_float((uint32_t)h << 16);
    }
  }
}

// A thread's elements of a row: E adjacent ones from `first` on, those of 0 .. end - 1
// (`first` may lie before the row: see the shift below); the lanes of a warp hold
// neighbouring groups.
//
// A row that starts `shift` elements past a 16-byte boundary is split over the
// threads from that boundary on, so every group but the row's first and last is
// whole 16-byte pieces in memory: odd row lengths cost no more than even ones.
struct Places {
  int first, end;
  __device__ __forceinline__ bool inside(int e) const { return first + e >= 0 && first + e < end; }
  template <int E>
  __device__ __forceinline__ bool whole() const { return first >= 0 && first + E <= end; }
};

// 16 bytes of a row from element i on; elements outside the row read as 0 and are not
// touched, pieces off their boundary are read by element
template <typename T>
__device__ __forceinline__ void load_piece(uint32_t* w, const T* row, int i, int end) {
  constexpr int N = 16 / (int)sizeof(T);
  if (i >= 0 && i + N <= end && (reinterpret_cast<uintptr_t>(row + i) & 15u) == 0) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + i);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = 0u;
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (i + e >= 0 && i + e < end) {
      if constexpr (sizeof(T) == 4) {
        w[e] = reinterpret_cast<const uint32_t*>(row)[i + e];
      } else {
        w[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[i + e] << (16 * (e & 1));
      }
    }
}

template <typename T, int E>
__device__ __forceinline__ void load(Pack<T, E>& p, const T* row, const Places& at) {
  constexpr int N = 16 / (int)sizeof(T);
#pragma unroll
  for (int j = 0; j < E / N; ++j) load_piece(p.w + 4 * j, row, at.first + j * N, at.end);
}

template <typename T, int E>
__device__ __forceinline__ Pack<T, E> packed(const float (&f)[E]) {
  Pack<T, E> p;
#pragma unroll
  for (int i = 0; i < Pack<T, E>::W; ++i) {
    if constexpr (sizeof(T) == 4) {
      p.w[i] = __float_as_uint(f[i]);
    } else if constexpr (std::is_same<T, __half>::value) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      p.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      p.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return p;
}

template <typename T, int E>
__device__ __forceinline__ void store(T* row, const float (&f)[E], const Places& at) {
  constexpr int N = 16 / (int)sizeof(T), PER = 4 / (int)sizeof(T);
  const Pack<T, E> p = packed<T>(f);
#pragma unroll
  for (int j = 0; j < E / N; ++j) {
    const int i = at.first + j * N;
    if (i >= 0 && i + N <= at.end && (reinterpret_cast<uintptr_t>(row + i) & 15u) == 0) {
      *reinterpret_cast<uint4*>(row + i) = make_uint4(p.w[4 * j], p.w[4 * j + 1], p.w[4 * j + 2], p.w[4 * j + 3]);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint32_t w = p.w[4 * j + e / PER];
        if (i + e < 0 || i + e >= at.end) continue;
        if constexpr (sizeof(T) == 4) {
          reinterpret_cast<uint32_t*>(row)[i + e] = w;
        } else {
          reinterpret_cast<uint16_t*>(row)[i + e] = (uint16_t)((e & 1) ? w >> 16 : w);
        }
      }
    }
  }
}

// A parameter vector's elements, `absent` where there is none.  Places outside the row
// get the nearest element inside (they meet values that are 0 or not stored), so that
// the unaligned form needs no predicates: a call's code is fetched cold for few rows.
template <typename P, int E>
__device__ __forceinline__ void parameters(float (&v)[E], const void* p, float absent, const Places& at) {
  const P* from = static_cast<const P*>(p) + at.first;
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = absent;
  } else if (at.template whole<E>() && (reinterpret_cast<uintptr_t>(from) & 15u) == 0) {
    Pack<P, E> raw;
#pragma unroll
    for (int k = 0; k < Pack<P, E>::W / 4; ++k) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(from) + k);
      raw.w[4 * k] = q.x;
      raw.w[4 * k + 1] = q.y;
      raw.w[4 * k + 2] = q.z;
      raw.w[4 * k + 3] = q.w;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = element(raw, e);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      v[e] = to_f32(static_cast<const P*>(p)[min(max(at.first + e, 0), at.end - 1)]);
  }
}

// Zeros at the places outside the row: a factor that meets a 0 there and is
// infinite would make it a NaN, which a sum over the row takes in.
template <int E>
__device__ __forceinline__ void zero_outside(float (&v)[E], const Places& at) {
  if (at.template whole<E>()) return;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (!at.inside(e)) v[e] = 0.f;
}

// a parameter array from element i on, or null
template <typename P>
__device__ __forceinline__ const P* from_column(const void* p, int64_t i) {
  return p == nullptr ? nullptr : static_cast<const P*>(p) + i;
}

// Arithmetic on a thread's elements in pairs: one instruction for two fp32 operations,
// each rounded as by itself.  An operand is an array or one value for all elements.
template <typename V>
__device__ __forceinline__ float2 pair_of(const V& v, int i) {
  if constexpr (std::is_array<V>::value) {
    return make_float2(v[2 * i], v[2 * i + 1]);
  } else {
    return make_float2(v, v);
  }
}
template <int E, typename A, typename B, typename C>
__device__ __forceinline__ void fma_to(float (&to)[E], const A& a, const B& b, const C& c) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const float2 r = __ffma2_rn(pair_of(a, i), pair_of(b, i), pair_of(c, i));
    to[2 * i] = r.x;
    to[2 * i + 1] = r.y;
  }
}
template <int E, typename A, typename B>
__device__ __forceinline__ void mul_to(float (&to)[E], const A& a, const B& b) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const float2 r = __fmul2_rn(pair_of(a, i), pair_of(b, i));
    to[2 * i] = r.x;
    to[2 * i + 1] = r.y;
  }
}
template <int E, typename A, typename B>
__device__ __forceinline__ void add_to(float (&to)[E], const A& a, const B& b) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const float2 r = __fadd2_rn(pair_of(a, i), pair_of(b, i));
    to[2 * i] = r.x;
    to[2 * i + 1] = r.y;
  }
}
template <int E>
__device__ __forceinline__ void dot_to(float2& sum, const float (&a)[E], const float (&b)[E]) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) sum = __ffma2_rn(pair_of(a, i), pair_of(b, i), sum);
}
template <int E>
__device__ __forceinline__ void sum_to(float2& sum, const float (&a)[E]) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) sum = __fadd2_rn(pair_of(a, i), sum);
}

// Sums of N values (1 to 4) over a warp: lanes 32 / N k (8 k for three) and the next
// hold value k's.  The values are added by halves: each exchange step adds one half of
// the values in one half of the lanes, so four values take 6 shuffles instead of 20.
template <int N>
__device__ __forceinline__ float warp_sums_apart(const float (&v)[N]) {
  const uint32_t lane = lane_idx();
  float x;
  if constexpr (N > 2) {
    const bool hi = (lane & 16u) != 0, odd = (lane & 8u) != 0;
    const float v3 = N == 4 ? v[N - 1] : 0.f;
    float k0 = hi ? v[2] : v[0], k1 = hi ? v3 : v[1];
    k0 += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
    k1 += __shfl_xor_sync(0xffffffffu, hi ? v[1] : v3, 16);
    x = (odd ? k1 : k0) + __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 8);
  } else if constexpr (N == 2) {
    const bool hi = (lane & 16u) != 0;
    x = (hi ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[1], 16);
  } else {
    x = v[0];
  }
#pragma unroll
  for (int o = (N > 2 ? 4 : 16 / N); o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
template <int N>
constexpr int kLanesPerSum = N > 2 ? 8 : 32 / N;

// the same in every lane
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {
  const float x = warp_sums_apart(v);
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = N == 1 ? x : __shfl_sync(0xffffffffu, x, k * kLanesPerSum<N>);
}

// What the warps of a row tell one another: one warp; a CTA's warps; or, in a
// cluster, the warps of all its CTAs.  The buffers alternate, so one barrier per
// exchange suffices: a buffer is written again only after the barrier of the
// exchange in between.
struct RowSums {
  float* parts;  // [2][8 values][kMost warps] in shared memory
  int warps;     // per row and CTA
  int cluster, rank, turn;
  static constexpr int kMost = 64, kFloats = 8 * kMost;

  __device__ __forceinline__ bool alone() const { return warps * cluster == 1; }

  // Before the first sums: places behind the warps that are read with theirs.
  __device__ __forceinline__ void clear() {
    for (int i = (int)threadIdx.x; i < 64; i += (int)blockDim.x) {
      const int w = (warps & ~3) + (i & 3);
      if (w >= warps) parts[(i >> 2) * kMost + w] = 0.f;
    }
  }

  // every warp's N values (the same in all its lanes), value k of warp w at
  // [k * kMost + w] of the answer
  template <int N>
  __device__ __forceinline__ const float* exchange(const float (&v)[N]) {
    float* buf = parts + turn * kFloats;
    turn ^= 1;
    const uint32_t warp = threadIdx.x >> 5, lane = lane_idx();
    if (cluster == 1) {
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) buf[k * kMost + warp] = v[k];
      }
      __syncthreads();
    } else {
      if (lane < (uint32_t)cluster) {
        const uint32_t to = mapa_shared(smem_u32(buf + rank * warps + warp), lane);
#pragma unroll
        for (int k = 0; k < N; ++k) st_cluster_u32(to + 4u * kMost * k, __float_as_uint(v[k]));
      }
      cluster_sync_all();
    }
    return buf;
  }

  // Sums over all the row's threads, in every thread.  A CTA's warps' sums are read
  // four at a time by every thread, which takes less than a second round of shuffles.
  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    if (alone()) {
      warp_sums(v);
    } else if (cluster == 1) {
      const float x = warp_sums_apart(v);
      float* buf = parts + turn * kFloats;
      turn ^= 1;
      const int lane = (int)lane_idx(), k = lane / kLanesPerSum<N>;
      if (lane % kLanesPerSum<N> == 0 && k < N) buf[k * kMost + (int)(threadIdx.x >> 5)] = x;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = 0.f;
      for (int w = 0; w < warps; w += 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float4 q = *reinterpret_cast<const float4*>(buf + i * kMost + w);
          v[i] += (q.x + q.y) + (q.z + q.w);
        }
      }
    } else {
      warp_sums(v);
      const float* buf = exchange(v);
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = 0.f;
      for (int w = (int)lane_idx(); w < warps * cluster; w += 32) {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += buf[k * kMost + w];
      }
      warp_sums(v);
    }
  }
};

// elements from the 16-byte boundary at or before a row to its start
template <typename T>
__device__ __forceinline__ int row_shift(const T* row) {
  return (int)((uint32_t)reinterpret_cast<uintptr_t>(row) & 15u) / (int)sizeof(T);
}

// ------------------------------------------------------------------- forward

// the gate of row r, or null
template <typename P>
__device__ __forceinline__ const P* gate_row(const void* gate, int64_t ld, int64_t M, int64_t groups, int64_t r) {
  if (gate == nullptr || groups == 1) return static_cast<const P*>(gate);
  return static_cast<const P*>(gate) + (int64_t)((uint32_t)r / ((uint32_t)M / (uint32_t)groups)) * ld;
}

// Mean (layer norm) and reciprocal deviation of a row held as v[NV][E]; elements past
// the row's end are 0.  The layer norm's variance is taken around the warp's own
// mean, and the warps' means and variances are then joined exactly,
//   sum (v - mean)^2 = sum over warps of (its own sum + n_w (mean_w - mean)^2),
// so one exchange serves both and nothing cancels.  n_w: the warp's elements.
template <bool LAYER, int NV, int E>
__device__ __forceinline__ float2 unit_of(const float (&v)[NV][E], const Places (&at)[NV], int D, float n_w, float eps,
                                          RowSums& sum) {
  const float inv = 1.f / (float)D;
  float2 pairs = make_float2(0.f, 0.f);
  float s[1];
  if constexpr (!LAYER) {
#pragma unroll
    for (int j = 0; j < NV; ++j) dot_to(pairs, v[j], v[j]);
    s[0] = pairs.x + pairs.y;
    sum(s);
    return make_float2(0.f, rsqrtf(s[0] * inv + eps));
  } else {
    const float inv_w = n_w > 0.f ? 1.f / n_w : 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) sum_to(pairs, v[j]);
    s[0] = pairs.x + pairs.y;
    warp_sums(s);
    float mean = s[0] * inv_w;
    pairs = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float c[E];
      add_to(c, v[j], -mean);
      if (!at[j].template whole<E>()) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (!at[j].inside(e)) c[e] = 0.f;
      }
      dot_to(pairs, c, c);
    }
    s[0] = pairs.x + pairs.y;
    warp_sums(s);
    if (!sum.alone()) {  // (one CTA per row here)
      const float mine[3] = {n_w, mean, s[0]};
      const float* all = sum.exchange(mine);
      constexpr int M = RowSums::kMost;
      auto four = [&](int i) { return *reinterpret_cast<const float4*>(all + i); };
      mean = 0.f;
      for (int w = 0; w < sum.warps; w += 4) {
        const float4 n = four(w), m = four(M + w);
        mean += fmaf(n.x, m.x, n.y * m.y) + fmaf(n.z, m.z, n.w * m.w);
      }
      mean *= inv;
      s[0] = 0.f;
      for (int w = 0; w < sum.warps; w += 4) {
        const float4 n = four(w), m = four(M + w), q = four(2 * M + w);
        const float4 c = make_float4(m.x - mean, m.y - mean, m.z - mean, m.w - mean);
        s[0] += (fmaf(n.x * c.x, c.x, q.x) + fmaf(n.y * c.y, c.y, q.y)) +
                (fmaf(n.z * c.z, c.z, q.z) + fmaf(n.w * c.w, c.w, q.w));
      }
    }
    return make_float2(mean, rsqrtf(s[0] * inv + eps));
  }
}

// the elements a warp holds of a row
template <int NV, int E>
__device__ __forceinline__ float warp_elements(const Places (&at)[NV]) {
  float n[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j) n[0] += (float)(max(0, min(at[j].end, at[j].first + E)) - max(0, min(at[j].end, at[j].first)));
  warp_sums(n);
  return n[0];
}

// A row per warp or CTA straight from global memory, for calls with too few rows to
// keep a ring busy: bound by the launch and one row's latency (1 x 4096 bf16 2.7 us).
template <typename T, typename P, bool LAYER, bool WARP, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) k_norm(const __grid_constant__ ffn_norm_t a) {
  constexpr int E = 16 / (int)sizeof(T);
  __shared__ __align__(16) float parts[2 * RowSums::kFloats];
  const int tid = WARP ? (int)lane_idx() : (int)threadIdx.x, per_row = WARP ? 32 : (int)blockDim.x;
  const int64_t r = WARP ? (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  const int D = (int)a.D;
  RowSums sum{parts, WARP ? 1 : (int)(blockDim.x / 32), 1, 0, 0};
  if constexpr (!WARP) sum.clear();
  Places at[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    at[j].end = D;
    // (shifted as rows without gaps from a 16-byte boundary on: which elements a thread
    // adds up depends on the sizes alone)
    at[j].first = (j * per_row + tid) * E - (int)(((uint32_t)r * (uint32_t)D * (uint32_t)sizeof(T)) & 15u) / (int)sizeof(T);
    // the widest rows leave no thread for the shift
    if (THREADS == 1024 && NV * per_row * E < D + E - 1) at[j].first = (j * per_row + tid) * E;
  }
  wait_for_prior_kernel();
  let_next_kernel_start();
  if (r >= a.M) return;  // (whole warps only: with a CTA per row every r is a row)
  const float n_w = LAYER ? warp_elements<NV, E>(at) : 0.f;
  Pack<T, E> y[NV], res[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) load(y[j], static_cast<const T*>(a.y) + r * a.ld_y, at[j]);
  if (a.residual != nullptr) {
#pragma unroll
    for (int j = 0; j < NV; ++j) load(res[j], static_cast<const T*>(a.residual) + r * a.ld_residual, at[j]);
  }
  float v[NV][E];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) v[j][e] = element(y[j], e);
  if (a.flags & FFN_NORM_POST) {
    const float2 st = unit_of<LAYER>(v, at, D, n_w, a.eps, sum);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[E], b[E];
      parameters<P>(w, a.post_weight, 1.f, at[j]);
      parameters<P>(b, a.post_bias, 0.f, at[j]);
#pragma unroll
      for (int e = 0; e < E; ++e) v[j][e] = fmaf((v[j][e] - st.x) * st.y, w[e], b[e]);
    }
  }
  const P* gate = gate_row<P>(a.gate, a.ld_gate, a.M, a.groups, r);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float g[E];
    parameters<P>(g, gate, 1.f, at[j]);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      v[j][e] *= a.branch_scale * g[e];
      if (a.residual != nullptr) v[j][e] = fmaf(a.residual_scale, element(res[j], e), v[j][e]);
      if (!at[j].inside(e)) v[j][e] = 0.f;  // (a post bias reaches past the end)
    }
    if (a.s != nullptr) store(static_cast<T*>(a.s) + r * a.ld_s, v[j], at[j]);
  }
  if (a.flags & FFN_NORM_PRE) {
    const float2 st = unit_of<LAYER>(v, at, D, n_w, a.eps, sum);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[E], b[E];
      parameters<P>(w, a.pre_weight, 1.f, at[j]);
      parameters<P>(b, a.pre_bias, 0.f, at[j]);
#pragma unroll
      for (int e = 0; e < E; ++e) v[j][e] = fmaf((v[j][e] - st.x) * st.y, w[e], b[e]);
      store(static_cast<T*>(a.n) + r * a.ld_n, v[j], at[j]);
    }
  }
}

// ------------------------------------------------------------------ backward

// The rows of one part.  Rows `period` apart start at the same offset to 16-byte
// boundaries (period = 1 where all do), and a part takes rows of one such class, so
// that its threads' columns stay the same: parts are numbered slice by slice, and
// within a slice of a group's rows class by class.
struct NormWalk {
  int64_t first, end, step, group;
};
template <bool MANY>
__device__ __forceinline__ NormWalk norm_walk(const ffn_norm_grad_t& a, const NormGradShape& sh, int part) {
  NormWalk w;
  if constexpr (MANY) {
    const int next = part + 1;
    w.group = sh.share.begin(part);
    w.first = w.group * sh.per;
    w.end = (int64_t)sh.share.begin(next) * sh.per;
    w.step = 1;
  } else {
    const int g = part / sh.parts_per_group, i = part - g * sh.parts_per_group;
    const int slice = i / sh.period, kind = i - slice * sh.period;
    w.group = g;
    const int64_t row0 = (int64_t)g * sh.per;
    w.first = row0 + (int64_t)sh.share.begin(slice) * sh.period + kind;
    w.end = row0 + min((int64_t)sh.per, (int64_t)sh.share.begin(slice + 1) * sh.period);
    w.step = sh.period;
  }
  return w;
}

// The shift a part's columns have (see k_norm_grad).
__device__ __forceinline__ int norm_part_shift(const ffn_norm_grad_t& a, const NormGradShape& sh, int part,
                                               int element_bytes) {
  if (sh.period == 1) return 0;
  const int g = part / sh.parts_per_group, kind = (part - g * sh.parts_per_group) % sh.period;
  const uint32_t row = (uint32_t)g * (uint32_t)sh.per + (uint32_t)kind;
  return (int)((row * (uint32_t)a.D * (uint32_t)element_bytes) & 15u) / element_bytes;
}

// v - mean for the layer norm; elements outside the row stay 0
template <bool LAYER, int E>
__device__ __forceinline__ void centre(float (&v)[E], float mean, const Places& at, bool whole) {
  if constexpr (LAYER) {
    if (whole) {
      add_to(v, v, -mean);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] -= at.inside(e) ? mean : 0.f;
    }
  }
}

// With u = unit(s), v = unit(y), a = dn * pre_weight, t = ds + r_s (a - u mean(a u)
// [- mean a]) and b = branch_scale * gate * t * post_weight, a thread holds G
// groups of 8 columns of each of the rows its part takes, and over those rows the sums
//   A = sum t v,  B = sum t,  C = sum dn u,  Eo = sum dn,
// from which every parameter's gradient follows, since gate and post_weight are
// constant over a group's rows:
//   dgate = branch_scale (post_weight A + post_bias B),
//   dpost_weight = branch_scale sum over groups of gate A, dpost_bias the same of B.
// A row takes two rounds of sums over its columns (RMS: of s^2, a s and y^2; of
// b v).
//
// Rows come through RowsIn, a ring in shared memory (kernels_norm_ring.cuh).  FULL:
// both norms and every array are there, known to the compiler.
template <bool FULL, bool LAYER, bool BIAS, bool MANY, int G, typename T, typename P, typename RowsIn>
__device__ __forceinline__ void norm_grad_rows(const ffn_norm_grad_t& a, const NormGradShape& sh, const NormSums& ws,
                                               RowsIn& rows, RowSums& sum, int part, const NormWalk& walk,
                                               const Places (&at)[G], int col0) {
  constexpr int E = 8;
  const bool post = FULL || (a.flags & FFN_NORM_POST) != 0, pre = FULL || (a.flags & FFN_NORM_PRE) != 0;
  const bool has_ds = FULL || a.ds != nullptr, has_y = FULL || a.y != nullptr;
  const bool has_dres = FULL || a.dresidual != nullptr, has_dy = FULL || a.dy != nullptr;
  const float inv = 1.f / (float)a.D, n_w = LAYER ? warp_elements<G, E>(at) : 0.f;
  const float inv_w = n_w > 0.f ? 1.f / n_w : 0.f;
  const int64_t per = sh.per;
  int64_t g = walk.group, group_end = (g + 1) * per;
  bool whole[G];
#pragma unroll
  for (int j = 0; j < G; ++j) whole[j] = at[j].template whole<E>();
  float A[G][E] = {}, C[G][E] = {}, B[G][BIAS ? E : 1] = {}, Eo[G][BIAS ? E : 1] = {};
  float GA[G][MANY ? E : 1] = {}, GB[G][(MANY && BIAS) ? E : 1] = {};
  rows.begin(walk);
  rows.set_group(g);
  for (int64_t r = walk.first; r < walk.end; r += walk.step) {
    if (!rows.next(r)) break;
    float mean_s = 0.f, mean_y = 0.f, mean_a = 0.f, k[3];
    float2 k2[3];  // sums of the even and of the odd elements
    auto zero = [&] { k2[0] = k2[1] = k2[2] = make_float2(0.f, 0.f); };
    auto join = [&] {
#pragma unroll
      for (int i = 0; i < 3; ++i) k[i] = k2[i].x + k2[i].y;
    };
    zero();
    if constexpr (LAYER) {
#pragma unroll
      for (int j = 0; j < G; ++j) {
        if (pre) {
          float s[E], dn[E];
          rows.s(s, j);
          rows.dn(dn, j);
          rows.scale_pre(dn, j);
          sum_to(k2[0], s);
          sum_to(k2[2], dn);
        }
        if (post) {
          float y[E];
          rows.y(y, j);
          sum_to(k2[1], y);
        }
      }
      join();
      zero();
      warp_sums(k);
      mean_s = k[0] * inv_w;  // the warp's own for now
      mean_y = k[1] * inv_w;
      mean_a = k[2];
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
      if (pre) {
        float s[E], dn[E];
        rows.s(s, j);
        rows.dn(dn, j);
        rows.scale_pre(dn, j);
        centre<LAYER>(s, mean_s, at[j], whole[j]);
        dot_to(k2[0], s, s);
        dot_to(k2[1], s, dn);
      }
      if (post) {
        float y[E];
        rows.y(y, j);
        centre<LAYER>(y, mean_y, at[j], whole[j]);
        dot_to(k2[2], y, y);
      }
    }
    join();
    if constexpr (!LAYER) {
      sum(k);
    } else {
      // the warps' means, squares and products around them, joined exactly (unit_of)
      warp_sums(k);
      if (!sum.alone()) {
        const float mine[7] = {n_w, mean_s, mean_y, mean_a, k[0], k[1], k[2]};
        const float* all = sum.exchange(mine);
        const int l = (int)lane_idx(), n = sum.warps * sum.cluster;
        constexpr int M = RowSums::kMost;
        k[0] = k[1] = k[2] = 0.f;
        for (int w = l; w < n; w += 32) {
          const float* q = all + w;
          k[0] = fmaf(q[0], q[M], k[0]);
          k[1] = fmaf(q[0], q[2 * M], k[1]);
          k[2] += q[3 * M];
        }
        warp_sums(k);
        mean_s = k[0] * inv;
        mean_y = k[1] * inv;
        mean_a = k[2];
        k[0] = k[1] = k[2] = 0.f;
        for (int w = l; w < n; w += 32) {
          const float* q = all + w;
          const float cs = q[M] - mean_s, cy = q[2 * M] - mean_y;
          k[0] += fmaf(q[0] * cs, cs, q[4 * M]);
          k[1] += fmaf(q[3 * M], cs, q[5 * M]);
          k[2] += fmaf(q[0] * cy, cy, q[6 * M]);
        }
        warp_sums(k);
      }
      mean_a *= inv;
    }
    rows.met();
    // With c = s - mean_s and d = y - mean_y, u = c r_s and v = d r_y, in as few
    // operations per element (the kernel is bound by their number):
    //   t  = ds - r_s mean(a) + c (-r_s^3 mean(a c)) + (dn r_s) pre_weight
    //   dy = b r_y - r_y mean(b) + d (-r_y^3 mean(b d))
    const float r_s = rsqrtf(k[0] * inv + a.eps), k_c = -(k[1] * inv) * r_s * r_s * r_s, k_s = r_s * mean_a;
    const float r_y = post ? rsqrtf(k[2] * inv + a.eps) : 1.f;
    float t[G][E];
    float2 two2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int j = 0; j < G; ++j) {
      if (has_ds) {
        rows.ds(t[j], j);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) t[j][e] = 0.f;
      }
      if (pre) {
        float s[E], dn[E], w[E];
        rows.s(s, j);
        rows.dn(dn, j);
        rows.pre_factors(w, j);
        if constexpr (LAYER) {
          add_to(s, s, -mean_s);
          add_to(t[j], t[j], -k_s);
        }
        if constexpr (BIAS) add_to(Eo[j], Eo[j], dn);
        mul_to(dn, dn, r_s);
        fma_to(C[j], dn, s, C[j]);
        fma_to(t[j], s, k_c, t[j]);
        fma_to(t[j], dn, w, t[j]);
      }
      if (LAYER && !whole[j]) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (!at[j].inside(e)) t[j][e] = 0.f;  // (0 - mean)
      }
      if (has_dres) {
        T* to = static_cast<T*>(a.dresidual) + r * a.ld_dresidual + col0;
        if (a.residual_scale == 1.f) {
          rows.template put<0>(to, t[j], j);
        } else {
          float o[E];
          mul_to(o, t[j], a.residual_scale);
          rows.template put<0>(to, o, j);
        }
      }
      float y[E];
      if (has_y) {
        rows.y(y, j);
        if constexpr (LAYER) add_to(y, y, -mean_y);
        float tr[E];
        mul_to(tr, t[j], r_y);
        fma_to(A[j], tr, y, A[j]);
        if constexpr (BIAS) add_to(B[j], B[j], t[j]);
      }
      if (has_dy) {
        rows.scale_branch(t[j], j);
        if (post) {
          dot_to(two2[0], t[j], y);
          if constexpr (LAYER) sum_to(two2[1], t[j]);
        }
      }
    }
    if (has_dy) {
      if (post) {
        float two[2] = {two2[0].x + two2[0].y, two2[1].x + two2[1].y};
        if constexpr (LAYER) {
          sum(two);
        } else {
          float one[1] = {two[0]};
          sum(one);
          two[0] = one[0];
        }
        if constexpr (!LAYER) rows.met_again();
        const float k_d = -(two[0] * inv) * r_y * r_y * r_y, k_b = two[1] * inv * r_y;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          float y[E];
          rows.y(y, j);
          if constexpr (LAYER) {
            add_to(y, y, -mean_y);
            fma_to(t[j], t[j], r_y, -k_b);
          } else {
            mul_to(t[j], t[j], r_y);
          }
          fma_to(t[j], y, k_d, t[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < G; ++j) rows.template put<1>(static_cast<T*>(a.dy) + r * a.ld_dy + col0, t[j], j);
    }
    rows.done();
    if constexpr (MANY) {
      if (r + 1 == group_end) {  // the group's last row: its gate's gradient is complete
#pragma unroll
        for (int j = 0; j < G; ++j) {
          if (a.dgate != nullptr) {
            float o[E];
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = a.branch_scale * A[j][e];
            float pw[E];
            parameters<P>(pw, from_column<P>(a.post_weight, col0), 1.f, at[j]);
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = __fmul_rn(o[e], pw[e]);
            if constexpr (BIAS) {
              float pb[E];
              parameters<P>(pb, from_column<P>(a.post_bias, col0), 0.f, at[j]);
#pragma unroll
              for (int e = 0; e < E; ++e) o[e] = fmaf(a.branch_scale * B[j][e], pb[e], o[e]);
            }
            store(a.dgate + g * a.D + col0, o, at[j]);
          }
          float gate[E];
          parameters<P>(gate, from_column<P>(a.gate, g * a.ld_gate + col0), 1.f, at[j]);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            GA[j][e] = fmaf(gate[e], A[j][e], GA[j][e]);
            A[j][e] = 0.f;
            if constexpr (BIAS) {
              GB[j][BIAS ? e : 0] = fmaf(gate[e], B[j][e], GB[j][BIAS ? e : 0]);
              B[j][e] = 0.f;
            }
          }
        }
        ++g;
        group_end += per;
        if (r + 1 < walk.end) rows.set_group(g);
      }
    }
  }
  // the sums of this part's rows, for k_norm_column_sums: at the threads' places, whole
  const int64_t out = rows.sums_at(part);
#pragma unroll
  for (int j = 0; j < G; ++j) {
    auto put = [&](float* to, const auto& v) {
      if (to == nullptr) return;
      float4* q = reinterpret_cast<float4*>(to + out + j * sh.threads * 8);
      q[0] = make_float4(v[0], v[1], v[2], v[3]);
      q[1] = make_float4(v[4], v[5], v[6], v[7]);
    };
    if constexpr (MANY) {
      put(ws.a, GA[j]);
      if constexpr (BIAS) put(ws.b, GB[j]);
    } else {
      put(ws.a, A[j]);
      if constexpr (BIAS) put(ws.b, B[j]);
    }
    put(ws.c, C[j]);
    if constexpr (BIAS) put(ws.e, Eo[j]);
  }
}

template <typename P>
__device__ __forceinline__ float parameter(const void* p, int64_t i, float absent) {
  return p == nullptr ? absent : to_f32(static_cast<const P*>(p)[i]);
}

// Adds the parts' sums, COLS columns and blockDim / COLS lanes of parts per CTA, always
// in the same order.  blockIdx.y = 0: the sums over all rows (and a single gate's); 1 + g:
// the gate of group g.
template <typename P, int COLS>
__global__ void __launch_bounds__(1024)
    k_norm_column_sums(const __grid_constant__ ffn_norm_grad_t a, const __grid_constant__ NormGradShape sh,
                       const __grid_constant__ NormSums ws, int element_bytes) {
  const int LANES = (int)blockDim.x / COLS, warps = (int)blockDim.x / 32;
  __shared__ float sums[32][COLS * 4 + 1];
  const int c = (int)threadIdx.x % COLS, l = (int)threadIdx.x / COLS, D = (int)a.D;
  const int i = (int)blockIdx.x * COLS + c;
  const int g = (int)blockIdx.y - 1;
  wait_for_prior_kernel();
  let_next_kernel_start();
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  const bool weighted = g < 0 && !sh.many && a.groups > 1;  // sums over groups: each part with its gate
  if (i < D) {
    // the column's place: its slice's, and in it the part's shift
    const int rank = i / (int)sh.columns, place = rank * sh.threads * sh.each + i - rank * (int)sh.columns;
    const int64_t pitch = (int64_t)sh.cluster * sh.threads * sh.each;
    const int p0 = g < 0 ? 0 : g * sh.parts_per_group, p1 = g < 0 ? sh.parts : p0 + sh.parts_per_group;
    // (parts come in whole periods and so do lanes: a lane's parts are of one kind)
    const uint32_t row_bytes = (uint32_t)D * (uint32_t)element_bytes;
    const uint32_t kind_bytes = sh.period > 1 ? (uint32_t)(l % sh.period) * row_bytes : 0u;
    const float per_group = sh.many ? 0.f : 1.f / (float)sh.parts_per_group;
#pragma unroll 4
    for (int p = p0 + l; p < p1; p += LANES) {
      const int pg = (int)(((float)p + 0.5f) * per_group);  // the part's group: exact below 2^22
      const uint32_t off =
          sh.period > 1 ? (((uint32_t)pg * (uint32_t)sh.per * row_bytes + kind_bytes) & 15u) / (uint32_t)element_bytes : 0u;
      const int64_t at = p * pitch + place + off;
      const float f = weighted ? parameter<P>(a.gate, (int64_t)pg * a.ld_gate + i, 1.f) : 1.f;
      if (ws.a != nullptr) v[0] = fmaf(f, ws.a[at], v[0]);
      if (ws.b != nullptr) v[1] = fmaf(f, ws.b[at], v[1]);
      if (g < 0 && ws.c != nullptr) v[2] += ws.c[at];
      if (g < 0 && ws.e != nullptr) v[3] += ws.e[at];
    }
  }
#pragma unroll
  for (int o = COLS; o < 32; o *= 2)
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  const int lane = (int)lane_idx(), warp = (int)(threadIdx.x >> 5);
  if (lane < COLS) {
#pragma unroll
    for (int k = 0; k < 4; ++k) sums[warp][lane * 4 + k] = v[k];
  }
  __syncthreads();
  // a warp adds the warps' values of one column and sum at a time
#pragma unroll 1
  for (int q = warp; q < COLS * 4; q += warps) {
    float s[1] = {lane < warps ? sums[lane][q] : 0.f};
    warp_sums(s);
    __syncwarp();
    if (lane == 0) sums[0][q] = s[0];
  }
  __syncthreads();
  if (threadIdx.x >= COLS || i >= D) return;
  const float A = sums[0][c * 4] * a.branch_scale, B = sums[0][c * 4 + 1] * a.branch_scale;
  if (a.dgate != nullptr && !sh.many && (g >= 0 || a.groups == 1))
    a.dgate[(int64_t)max(g, 0) * D + i] = parameter<P>(a.post_weight, i, 1.f) * A +
                                          (ws.b != nullptr ? parameter<P>(a.post_bias, i, 0.f) * B : 0.f);
  if (g >= 0) return;
  const float f = !sh.many && a.groups == 1 ? parameter<P>(a.gate, i, 1.f) : 1.f;
  if (a.dpost_weight != nullptr) a.dpost_weight[i] = f * A;
  if (a.dpost_bias != nullptr) a.dpost_bias[i] = f * B;
  if (a.dpre_weight != nullptr) a.dpre_weight[i] = sums[0][c * 4 + 2];
  if (a.dpre_bias != nullptr) a.dpre_bias[i] = sums[0][c * 4 + 3];
}

}  // namespace

}  // namespace dgb
