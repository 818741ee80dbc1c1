// kernels_norm.cuh -- the norms around a block fused with its gate, its scales and
// the residual stream, one pass over the rows, and their gradients, one pass too.
//
// Bound by memory: 4 row reads and writes forward (y, residual, s, n), 6 backward
// (ds, dn, y, s, dresidual, dy).  A row stays in registers from its load to its
// stores, all loads of a row are issued before the first sum over it, and sums use
// the values in registers (the variance is taken around the mean, not from the
// sum of squares).
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

// A thread's elements of a row: E adjacent ones from `first` on, those below `end`;
// the lanes of a warp hold neighbouring groups.
struct Places {
  int first, end;
  __device__ __forceinline__ bool inside(int e) const { return first + e < end; }
};

// 16 aligned bytes, elements i .. of a row; those outside 0 .. end - 1 read as 0 and
// are not touched
template <typename T>
__device__ __forceinline__ void load_chunk(uint32_t* w, const T* row, int i, int end) {
  constexpr int N = 16 / (int)sizeof(T);
  if (i >= 0 && i + N <= end) {
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

// word i of `v` moved down by `bytes` (1 .. 15, of an element's size): v is shifted in
// place, its last four words are consumed
template <int W>
__device__ __forceinline__ void shift_down(uint32_t (&v)[W], uint32_t bytes) {
  if (bytes & 8u) {
#pragma unroll
    for (int i = 0; i + 2 < W; ++i) v[i] = v[i + 2];
  }
  if (bytes & 4u) {
#pragma unroll
    for (int i = 0; i + 1 < W; ++i) v[i] = v[i + 1];
  }
  if (bytes & 2u) {
#pragma unroll
    for (int i = 0; i + 1 < W; ++i) v[i] = __funnelshift_r(v[i], v[i + 1], 16);
  }
}

// Loads a warp's groups of a row that may start anywhere: where the row is off a
// 16-byte boundary by m bytes, every lane loads the aligned chunks that its first
// elements lie in, takes the chunk after them from the next lane, and shifts.  All
// lanes of the warp call.
template <typename T, int E>
__device__ __forceinline__ void load(Pack<T, E>& p, const T* row, const Places& at) {
  constexpr int N = 16 / (int)sizeof(T), W = Pack<T, E>::W;
  const uint32_t m = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
  if (m == 0) {
#pragma unroll
    for (int j = 0; j < W / 4; ++j) load_chunk(p.w + 4 * j, row, at.first + j * N, at.end);
    return;
  }
  uint32_t v[W + 4];
  const int start = at.first - (int)(m / sizeof(T));
#pragma unroll
  for (int j = 0; j < W / 4; ++j) load_chunk(v + 4 * j, row, start + j * N, at.end);
#pragma unroll
  for (int k = 0; k < 4; ++k) v[W + k] = __shfl_down_sync(0xffffffffu, v[k], 1);
  if (lane_idx() == 31) load_chunk(v + W, row, start + E, at.end);
  shift_down(v, m);
#pragma unroll
  for (int i = 0; i < W; ++i) p.w[i] = v[i];
  // (what follows `end` is 0 already: load_chunk reads nothing there)
}

template <typename T>
__device__ __forceinline__ void store_one(T* p, uint32_t word, int odd) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<uint32_t*>(p) = word;
  } else {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)(odd ? word >> 16 : word);
  }
}

// The same way out: aligned chunks hold the end of a lane's group and the start of
// the next lane's; the warp's first and last pieces are stored by element.
template <typename T, int E>
__device__ __forceinline__ void store(T* row, const float (&f)[E], const Places& at) {
  constexpr int N = 16 / (int)sizeof(T), W = Pack<T, E>::W, PER = 4 / (int)sizeof(T);
  uint32_t w[W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(f[i]);
    } else if constexpr (std::is_same<T, __half>::value) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  const uint32_t m = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
  if (m == 0) {
#pragma unroll
    for (int j = 0; j < W / 4; ++j) {
      const int i = at.first + j * N;
      if (i + N <= at.end) {
        *reinterpret_cast<uint4*>(row + i) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (i + e < at.end) store_one(row + i + e, w[4 * j + e / PER], e % PER);
      }
    }
    return;
  }
  // the chunks from the first boundary inside this lane's group on: `head` elements in
  const int head = N - (int)(m / sizeof(T));
  uint32_t v[W + 4];
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = w[i];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[W + k] = __shfl_down_sync(0xffffffffu, w[k], 1);
  shift_down(v, 16u - m);
  const bool last = lane_idx() == 31;
#pragma unroll
  for (int j = 0; j < W / 4; ++j) {
    const int i = at.first + head + j * N;
    // (the last lane has no next one: its last chunk ends with its group)
    const int end = last ? min(at.end, at.first + E) : at.end;
    if (i + N <= end) {
      *reinterpret_cast<uint4*>(row + i) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (i + e < end) store_one(row + i + e, v[4 * j + e / PER], e % PER);
    }
  }
  if (lane_idx() == 0) {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < head && at.inside(e)) store_one(row + at.first + e, w[e / PER], e % PER);
  }
}

// a parameter vector's elements, `absent` where there is none
template <typename P, int E>
__device__ __forceinline__ void parameters(float (&v)[E], const void* p, float absent, const Places& at) {
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = absent;
    return;
  }
  Pack<P, E> raw;
  load(raw, static_cast<const P*>(p), at);
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = element(raw, e);
}

// Sums of K values over the threads of a row: one warp; a CTA's warps; or, in a
// cluster, the warps of all its CTAs.  Every thread gets the same values.  The
// buffers alternate, so one barrier per sum suffices: a buffer is written again
// only after the barrier of the sum in between.
template <int K>
struct RowSums {
  float* parts;  // [2][128][K] in shared memory
  int warps;     // per row and CTA; 1 and cluster 1: the warp alone
  int cluster, rank, turn;

  __device__ __forceinline__ void operator()(float (&v)[K]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (warps == 1 && cluster == 1) return;
    float* buf = parts + turn * 128 * K;
    turn ^= 1;
    const int lane = (int)lane_idx(), warp = (int)(threadIdx.x >> 5);
    if (cluster == 1) {
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) buf[warp * K + k] = v[k];
      }
      __syncthreads();
    } else {
      if (lane < cluster) {
        const uint32_t there = mapa_shared(smem_u32(buf + (rank * warps + warp) * K), (uint32_t)lane);
#pragma unroll
        for (int k = 0; k < K; ++k) st_cluster_u32(there + 4u * k, __float_as_uint(v[k]));
      }
      cluster_sync_all();
    }
    const int n = warps * cluster;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
    for (int i = lane; i < n; i += 32) {
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += buf[i * K + k];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
};

// ------------------------------------------------------------------- forward

// mean (layer norm) and reciprocal deviation of a row held as v[NV][E]; elements
// past the row's end are excluded by `at` (WHOLE: vectors lie wholly in or out)
template <bool LAYER, bool WHOLE = false, int NV, int E>
__device__ __forceinline__ float2 unit_of(const float (&v)[NV][E], const Places (&at)[NV], int D, float eps,
                                          RowSums<1>& sum) {
  const float inv = 1.f / (float)D;
  float mean = 0.f, s[1];
  if constexpr (LAYER) {
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) s[0] += v[j][e];  // elements past the end are 0
    sum(s);
    mean = s[0] * inv;
  }
  s[0] = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float c = v[j][e] - mean;
      if (!LAYER || at[j].inside(WHOLE ? 0 : e)) s[0] = fmaf(c, c, s[0]);
    }
  sum(s);
  return make_float2(mean, rsqrtf(s[0] * inv + eps));
}

template <typename T, typename P, bool LAYER, bool WARP, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) k_norm(const ffn_norm_t a) {
  constexpr int E = 16 / (int)sizeof(T);
  __shared__ float parts[2 * 128];
  const int tid = WARP ? (int)lane_idx() : (int)threadIdx.x, per_row = WARP ? 32 : (int)blockDim.x;
  const int64_t r = WARP ? (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  const int D = (int)a.D;
  RowSums<1> sum{parts, WARP ? 1 : (int)(blockDim.x / 32), 1, 0, 0};
  Places at[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    at[j].end = D;
    at[j].first = (j * per_row + tid) * E;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (r >= a.M) return;  // (whole warps only: with a CTA per row every r is a row)
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
    const float2 st = unit_of<LAYER>(v, at, D, a.eps, sum);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[E], b[E];
      parameters<P>(w, a.post_weight, 1.f, at[j]);
      parameters<P>(b, a.post_bias, 0.f, at[j]);
#pragma unroll
      for (int e = 0; e < E; ++e) v[j][e] = fmaf((v[j][e] - st.x) * st.y, w[e], b[e]);
    }
  }
  const P* gate =
      a.gate != nullptr ? static_cast<const P*>(a.gate) + (r / (a.M / a.groups)) * a.ld_gate : nullptr;
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
    const float2 st = unit_of<LAYER>(v, at, D, a.eps, sum);
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

// the rows of one part
template <bool MANY>
__device__ __forceinline__ void norm_part_rows(const ffn_norm_grad_t& a, const NormGradShape& sh, int part, int64_t& r0,
                                               int64_t& r1) {
  const int64_t per = a.M / a.groups;
  if constexpr (MANY) {
    r0 = a.groups * part / sh.parts * per;
    r1 = a.groups * (part + 1) / sh.parts * per;
  } else {
    const int64_t g = part / sh.parts_per_group, i = part % sh.parts_per_group;
    r0 = g * per + per * i / sh.parts_per_group;
    r1 = g * per + per * (i + 1) / sh.parts_per_group;
  }
}

// The arithmetic of a row's elements, in one place with every rounding spelt out, so
// that both forms of the kernel give the same bits.
__device__ __forceinline__ float unit_value(float v, float mean, float r) { return __fmul_rn(v - mean, r); }
// r (a - u mean(a u) - mean(a)), added to t
__device__ __forceinline__ float unit_slope(float t, float r, float a, float u, float mean_au, float mean_a) {
  return fmaf(r, __fsub_rn(fmaf(-u, mean_au, a), mean_a), t);
}

// With u = unit(s), v = unit(y), a = dn * pre_weight, t = ds + r_s (a - u mean(a u)
// [- mean a]) and b = branch_scale * gate * t * post_weight, a thread holds 8
// columns of each of the rows its part takes, and over those rows the sums
//   A = sum t v,  B = sum t,  C = sum dn u,  Eo = sum dn,
// from which every parameter's gradient follows, since gate and post_weight are
// constant over a group's rows:
//   dgate = branch_scale (post_weight A + post_bias B),
//   dpost_weight = branch_scale sum over groups of gate A, dpost_bias the same of B.
// A row takes two rounds of sums over its columns (RMS: of s^2, a s and y^2; of
// b y), three for the layer norm (means first).  (This form takes rows that start
// anywhere; kernels_norm_ring.cuh has the one for aligned rows.)
template <typename T, typename P, bool LAYER, bool BIAS, bool MANY>
__global__ void __launch_bounds__(kNormGradThreads, (MANY || sizeof(T) == 4) ? 1 : 2)
    k_norm_grad(const ffn_norm_grad_t a, const NormGradShape sh, const NormSums ws) {
  constexpr int E = kNormGradEach;
  constexpr int K = LAYER ? 4 : 3;
  __shared__ float parts_smem[2 * 128 * K];
  const int D = (int)a.D;
  const int rank = sh.cluster > 1 ? (int)cluster_ctarank() : 0;
  const int tid = sh.lanes > 1 ? (int)lane_idx() : (int)threadIdx.x;
  const int part = sh.lanes > 1 ? (int)blockIdx.x * sh.lanes + (int)(threadIdx.x >> 5) : (int)blockIdx.x / sh.cluster;
  RowSums<K> sum{parts_smem, sh.threads / 32, sh.cluster, rank, 0};
  Places at;
  at.end = min(D, (int)((rank + 1) * sh.columns));
  at.first = (int)(rank * sh.columns) + tid * E;
  const bool post = (a.flags & FFN_NORM_POST) != 0, pre = (a.flags & FFN_NORM_PRE) != 0;
  const float inv = 1.f / (float)D;
  const int64_t per = a.M / a.groups;
  int64_t r0, r1;
  norm_part_rows<MANY>(a, sh, part, r0, r1);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (part >= sh.parts) return;          // (whole warps only)
  if (sh.cluster > 1) cluster_sync_all();  // the cluster's CTAs have started: their shared memory may be written

  struct Row {
    Pack<T, E> ds, dn, y, s;
  };
  auto fetch = [&](Row& q, int64_t r) {
    if (pre) {
      load(q.s, static_cast<const T*>(a.s) + r * a.ld_s, at);
      load(q.dn, static_cast<const T*>(a.dn) + r * a.ld_dn, at);
    }
    if (a.y != nullptr) load(q.y, static_cast<const T*>(a.y) + r * a.ld_y, at);
    if (a.ds != nullptr) load(q.ds, static_cast<const T*>(a.ds) + r * a.ld_ds, at);
  };
  float A[E] = {}, C[E] = {}, B[BIAS ? E : 1] = {}, Eo[BIAS ? E : 1] = {};
  float GA[MANY ? E : 1] = {}, GB[(MANY && BIAS) ? E : 1] = {};
  for (int64_t r = r0; r < r1; ++r) {
    Row q;
    fetch(q, r);
    float mean_s = 0.f, mean_y = 0.f;
    float k[K];
    float w[E];
    parameters<P>(w, a.pre_weight, 1.f, at);
    if constexpr (LAYER) {
#pragma unroll
      for (int i = 0; i < K; ++i) k[i] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (pre) {
          k[0] += element(q.s, e);
          k[2] += __fmul_rn(element(q.dn, e), w[e]);
        }
        if (post) k[1] += element(q.y, e);
      }
      sum(k);
      mean_s = k[0] * inv;
      mean_y = k[1] * inv;
    }
    const float mean_a = LAYER ? k[LAYER ? 2 : 0] * inv : 0.f;
#pragma unroll
    for (int i = 0; i < K; ++i) k[i] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (!LAYER || at.inside(e)) {
        if (pre) {
          const float c = element(q.s, e) - mean_s;
          k[0] = fmaf(c, c, k[0]);
          k[1] = fmaf(c, __fmul_rn(element(q.dn, e), w[e]), k[1]);
        }
        if (post) {
          const float c = element(q.y, e) - mean_y;
          k[2] = fmaf(c, c, k[2]);
        }
      }
    sum(k);
    const float r_s = rsqrtf(k[0] * inv + a.eps), mean_au = k[1] * inv * r_s;
    const float r_y = post ? rsqrtf(k[2] * inv + a.eps) : 1.f;
    float t[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      t[e] = a.ds != nullptr ? element(q.ds, e) : 0.f;
      if (pre) {
        const float u = unit_value(element(q.s, e), mean_s, r_s), dn = element(q.dn, e);
        t[e] = unit_slope(t[e], r_s, __fmul_rn(dn, w[e]), u, mean_au, mean_a);
        if (at.inside(e)) {
          C[e] = fmaf(dn, u, C[e]);
          if constexpr (BIAS) Eo[e] += dn;
        }
      }
      if (!at.inside(e)) t[e] = 0.f;
    }
    if (a.dresidual != nullptr) {
      float o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = a.residual_scale * t[e];
      store(static_cast<T*>(a.dresidual) + r * a.ld_dresidual, o, at);
    }
    if (a.y != nullptr) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        A[e] = fmaf(t[e], unit_value(element(q.y, e), mean_y, r_y), A[e]);
        if constexpr (BIAS) B[e] += t[e];
      }
    }
    const int64_t g = r / per;
    float gate[E];
    if (a.dy != nullptr || MANY)
      parameters<P>(gate, a.gate != nullptr ? static_cast<const P*>(a.gate) + g * a.ld_gate : nullptr, 1.f, at);
    if (a.dy != nullptr) {
      float o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = __fmul_rn(t[e], __fmul_rn(a.branch_scale, gate[e]));
      if (post) {
        float pw[E];
        parameters<P>(pw, a.post_weight, 1.f, at);
#pragma unroll
        for (int i = 0; i < K; ++i) k[i] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          o[e] = __fmul_rn(o[e], pw[e]);
          k[0] = fmaf(o[e], unit_value(element(q.y, e), mean_y, r_y), k[0]);
          if constexpr (LAYER) k[1] += o[e];
        }
        sum(k);
        const float mean_bv = k[0] * inv, mean_b = LAYER ? k[1] * inv : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
          o[e] = unit_slope(0.f, r_y, o[e], unit_value(element(q.y, e), mean_y, r_y), mean_bv, mean_b);
      }
      store(static_cast<T*>(a.dy) + r * a.ld_dy, o, at);
    }
    if constexpr (MANY) {
      if (r + 1 == (g + 1) * per) {  // the group's last row: its gate's gradient is complete
        if (a.dgate != nullptr) {
          float pw[E], pb[E], o[E];
          parameters<P>(pw, a.post_weight, 1.f, at);
          parameters<P>(pb, a.post_bias, 0.f, at);
#pragma unroll
          for (int e = 0; e < E; ++e)
            o[e] = a.branch_scale * (pw[e] * A[e] + (BIAS ? pb[e] * B[BIAS ? e : 0] : 0.f));
          store(a.dgate + g * (int64_t)D, o, at);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
          GA[e] = fmaf(gate[e], A[e], GA[e]);
          A[e] = 0.f;
          if constexpr (BIAS) {
            GB[BIAS ? e : 0] = fmaf(gate[e], B[e], GB[BIAS ? e : 0]);
            B[e] = 0.f;
          }
        }
      }
    }
  }
  // the sums of this part's rows, for k_norm_column_sums
  const int64_t row = (int64_t)part * D;
  if constexpr (MANY) {
    if (ws.a != nullptr) store(ws.a + row, GA, at);
    if constexpr (BIAS) {
      if (ws.b != nullptr) store(ws.b + row, GB, at);
    }
  } else {
    if (ws.a != nullptr) store(ws.a + row, A, at);
    if constexpr (BIAS) {
      if (ws.b != nullptr) store(ws.b + row, B, at);
    }
  }
  if (ws.c != nullptr) store(ws.c + row, C, at);
  if constexpr (BIAS) {
    if (ws.e != nullptr) store(ws.e + row, Eo, at);
  }
}

template <typename P>
__device__ __forceinline__ float parameter(const void* p, int64_t i, float absent) {
  return p == nullptr ? absent : to_f32(static_cast<const P*>(p)[i]);
}

// Adds the parts' sums, 32 columns and 32 parts' lanes per CTA, always in the same
// order.  blockIdx.y = 0: the sums over all rows (and a single gate's); 1 + g: the gate
// of group g.
template <typename P>
__global__ void __launch_bounds__(1024) k_norm_column_sums(const ffn_norm_grad_t a, const NormGradShape sh,
                                                           const NormSums ws) {
  __shared__ float sums[4][32][33];
  const int c = (int)lane_idx(), l = (int)(threadIdx.x >> 5), D = (int)a.D;
  const int i = (int)blockIdx.x * 32 + c;
  const int g = (int)blockIdx.y - 1;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  const bool weighted = g < 0 && !sh.many && a.groups > 1;  // sums over groups: each part with its gate
  if (i < D) {
    const int p0 = g < 0 ? 0 : g * sh.parts_per_group, p1 = g < 0 ? sh.parts : p0 + sh.parts_per_group;
#pragma unroll 4
    for (int p = p0 + l; p < p1; p += 32) {
      const int64_t at = (int64_t)p * D + i;
      float f = 1.f;
      if (weighted) f = parameter<P>(a.gate, (int64_t)(p / sh.parts_per_group) * a.ld_gate + i, 1.f);
      if (ws.a != nullptr) v[0] = fmaf(f, ws.a[at], v[0]);
      if (ws.b != nullptr) v[1] = fmaf(f, ws.b[at], v[1]);
      if (g < 0) {
        if (ws.c != nullptr) v[2] += ws.c[at];
        if (ws.e != nullptr) v[3] += ws.e[at];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) sums[k][l][c] = v[k];
  __syncthreads();
  // warp l adds the 32 lanes of sum l & 3 for 4 columns
  const int k = l & 3;
  for (int j = 0; j < 4; ++j) {
    const int col = (l >> 2) * 4 + j;
    float s = sums[k][c][col];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncwarp();
    if (c == 0) sums[k][0][col] = s;
  }
  __syncthreads();
  if (l != 0 || i >= D) return;
  const float A = sums[0][0][c] * a.branch_scale, B = sums[1][0][c] * a.branch_scale;
  if (a.dgate != nullptr && !sh.many && (g >= 0 || a.groups == 1))
    a.dgate[(int64_t)max(g, 0) * D + i] = parameter<P>(a.post_weight, i, 1.f) * A +
                                          (ws.b != nullptr ? parameter<P>(a.post_bias, i, 0.f) * B : 0.f);
  if (g >= 0) return;
  const float f = !sh.many && a.groups == 1 ? parameter<P>(a.gate, i, 1.f) : 1.f;
  if (a.dpost_weight != nullptr) a.dpost_weight[i] = f * A;
  if (a.dpost_bias != nullptr) a.dpost_bias[i] = f * B;
  if (a.dpre_weight != nullptr) a.dpre_weight[i] = sums[2][0][c];
  if (a.dpre_bias != nullptr) a.dpre_bias[i] = sums[3][0][c];
}

}  // namespace

}  // namespace dgb
