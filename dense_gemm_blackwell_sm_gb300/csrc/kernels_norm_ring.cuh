// kernels_norm_ring.cuh -- the block norms for rows that start on 16-byte
// boundaries and have whole 16-byte vectors: rows come through a ring in shared
// memory filled by bulk copies (cp.async.bulk), so an SM has tens of KB on their
// way whatever its threads do, and the backward kernel can read a row's values
// again instead of holding them in registers.
//
// A group (a warp, a CTA, or in the backward kernel a cluster of CTAs that share
// the columns) walks its rows with `stages` rows ahead.  Every wait is bounded; a
// wait that runs out is recorded in the device's status word.
#pragma once

#include "kernels_norm.cuh"

namespace dgb {

namespace {

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// The ring of one group: `arrays` rows (or column slices of rows) per stage.
struct Ring {
  uint8_t* slots;      // [stages][arrays][bytes]
  uint64_t* full;      // [stages]
  volatile uint32_t* abort_flag;
  uint32_t* status;
  uint32_t stages, arrays, bytes, pitch;  // bytes of a row (slice); of a slot

  __device__ __forceinline__ uint8_t* slot(uint32_t stage, uint32_t array) const {
    return slots + (size_t)(stage * arrays + array) * pitch;
  }
  __device__ __forceinline__ WaitCtl ctl() const { return WaitCtl{abort_flag, status, 2000000000ull, 0}; }
  // all threads: the i-th row of the group has landed
  __device__ __forceinline__ bool wait(uint32_t i) const {
    return mbar_wait(smem_u32(full + i % stages), (i / stages) & 1u, ctl(), WAIT_MMA_FULL);
  }
  // after a wait that ran out: the copies still in flight land before shared memory goes
  __device__ __noinline__ void settle(uint32_t issued, uint32_t from) const {
    volatile uint32_t never = 0u;
    const WaitCtl w{&never, nullptr, 2000000ull, 0};
    for (uint32_t i = from; i < issued; ++i) mbar_wait(smem_u32(full + i % stages), (i / stages) & 1u, w, 0u);
  }
};

template <typename T, int E>
__device__ __forceinline__ void from_slot(float (&v)[E], const uint8_t* slot, int first, bool live) {
  Pack<T, E> p;
#pragma unroll
  for (int i = 0; i < Pack<T, E>::W / 4; ++i) {
    const uint4 q = live ? reinterpret_cast<const uint4*>(slot + (size_t)first * sizeof(T))[i] : make_uint4(0, 0, 0, 0);
    p.w[4 * i] = q.x;
    p.w[4 * i + 1] = q.y;
    p.w[4 * i + 2] = q.z;
    p.w[4 * i + 3] = q.w;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = element(p, e);
}

template <typename P, int E>
__device__ __forceinline__ void aligned_parameters(float (&v)[E], const P* p, int first, bool live) {
  Pack<P, E> raw;
#pragma unroll
  for (int i = 0; i < Pack<P, E>::W / 4; ++i) {
    const uint4 q = live ? __ldg(reinterpret_cast<const uint4*>(p + first) + i) : make_uint4(0, 0, 0, 0);
    raw.w[4 * i] = q.x;
    raw.w[4 * i + 1] = q.y;
    raw.w[4 * i + 2] = q.z;
    raw.w[4 * i + 3] = q.w;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = element(raw, e);
}

template <typename T, int E>
__device__ __forceinline__ void aligned_store(T* p, const float (&f)[E], bool live) {
  if (!live) return;
  uint32_t w[Pack<T, E>::W];
#pragma unroll
  for (int i = 0; i < Pack<T, E>::W; ++i) {
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
#pragma unroll
  for (int i = 0; i < Pack<T, E>::W / 4; ++i)
    reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// ------------------------------------------------------------------- forward

template <typename T, typename P, bool LAYER, bool WARP, int NV>
__global__ void __launch_bounds__(WARP ? 256 : 512, WARP ? 4 : 2)
    k_norm_ring(const ffn_norm_t a, uint32_t* status) {
  constexpr int E = 16 / (int)sizeof(T);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[8 * kNormStages];
  __shared__ float parts[2 * 128];
  __shared__ volatile uint32_t abort_flag;
  const int tid = WARP ? (int)lane_idx() : (int)threadIdx.x, per_row = WARP ? 32 : (int)blockDim.x;
  const int group = WARP ? (int)(threadIdx.x >> 5) : 0, groups = WARP ? (int)(blockDim.x / 32) : 1;
  const int D = (int)a.D;
  Ring ring;
  ring.stages = kNormStages;
  ring.arrays = a.residual != nullptr ? 2u : 1u;
  ring.bytes = (uint32_t)(D * (int)sizeof(T));
  ring.pitch = ring.bytes;
  ring.slots = smem + (size_t)group * ring.stages * ring.arrays * ring.pitch;
  ring.full = bars + group * kNormStages;
  ring.abort_flag = &abort_flag;
  ring.status = status;
  RowSums<1> sum{parts, WARP ? 1 : (int)(blockDim.x / 32), 1, 0, 0};
  if (tid == 0) {
    for (uint32_t s = 0; s < ring.stages; ++s) mbar_init(smem_u32(ring.full + s), 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) abort_flag = 0u;
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t step = (int64_t)gridDim.x * groups, r0 = (int64_t)blockIdx.x * groups + group;
  uint32_t issued = 0;  // (the group's first thread)
  auto issue = [&]() {
    const int64_t r = r0 + (int64_t)issued * step;
    if (r >= a.M) return;
    const uint32_t stage = issued % ring.stages, bar = smem_u32(ring.full + stage);
    mbar_arrive_expect_tx(bar, ring.arrays * ring.bytes);
    bulk_load(smem_u32(ring.slot(stage, 0)), static_cast<const T*>(a.y) + r * a.ld_y, ring.bytes, bar);
    if (a.residual != nullptr)
      bulk_load(smem_u32(ring.slot(stage, 1)), static_cast<const T*>(a.residual) + r * a.ld_residual, ring.bytes, bar);
    ++issued;
  };
  if (tid == 0)
    for (uint32_t s = 0; s < ring.stages; ++s) issue();

  const bool post = (a.flags & FFN_NORM_POST) != 0, pre = (a.flags & FFN_NORM_PRE) != 0;
  Places at[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) at[j] = Places{(j * per_row + tid) * E, D};
  uint32_t i = 0;
  for (int64_t r = r0; r < a.M; r += step, ++i) {
    if (!ring.wait(i)) {
      if (tid == 0) ring.settle(issued, i);
      return;
    }
    const uint32_t stage = i % ring.stages;
    float v[NV][E];
#pragma unroll
    for (int j = 0; j < NV; ++j) from_slot<T>(v[j], ring.slot(stage, 0), at[j].first, at[j].inside(0));
    if (post) {
      const float2 st = unit_of<LAYER, true>(v, at, D, a.eps, sum);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const bool live = at[j].inside(0);
#pragma unroll
        for (int e = 0; e < E; ++e) v[j][e] = (v[j][e] - st.x) * st.y;
        if (a.post_weight != nullptr) {
          float w[E];
          aligned_parameters(w, static_cast<const P*>(a.post_weight), at[j].first, live);
#pragma unroll
          for (int e = 0; e < E; ++e) v[j][e] *= w[e];
        }
        if (a.post_bias != nullptr) {
          float b[E];
          aligned_parameters(b, static_cast<const P*>(a.post_bias), at[j].first, live);
#pragma unroll
          for (int e = 0; e < E; ++e) v[j][e] += b[e];
        }
      }
    }
    const P* gate =
        a.gate != nullptr ? static_cast<const P*>(a.gate) + (r / (a.M / a.groups)) * a.ld_gate : nullptr;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool live = at[j].inside(0);
      if (gate != nullptr) {
        float g[E];
        aligned_parameters(g, gate, at[j].first, live);
#pragma unroll
        for (int e = 0; e < E; ++e) v[j][e] *= a.branch_scale * g[e];
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[j][e] *= a.branch_scale;
      }
      if (a.residual != nullptr) {
        float q[E];
        from_slot<T>(q, ring.slot(stage, 1), at[j].first, live);
#pragma unroll
        for (int e = 0; e < E; ++e) v[j][e] = fmaf(a.residual_scale, q[e], v[j][e]);
      }
      if (LAYER && !live) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[j][e] = 0.f;  // (0 - mean of the post norm)
      }
      if (a.s != nullptr) aligned_store(static_cast<T*>(a.s) + r * a.ld_s + at[j].first, v[j], live);
    }
    // the group has read the row's slots once it meets at the next barrier
    float2 st = make_float2(0.f, 1.f);
    if (pre) st = unit_of<LAYER, true>(v, at, D, a.eps, sum);
    if constexpr (WARP) {
      __syncwarp();
    } else {
      if (!pre || per_row == 32) __syncthreads();
    }
    if (tid == 0) issue();
    if (pre) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const bool live = at[j].inside(0);
#pragma unroll
        for (int e = 0; e < E; ++e) v[j][e] = (v[j][e] - st.x) * st.y;
        if (a.pre_weight != nullptr) {
          float w[E];
          aligned_parameters(w, static_cast<const P*>(a.pre_weight), at[j].first, live);
#pragma unroll
          for (int e = 0; e < E; ++e) v[j][e] *= w[e];
        }
        if (a.pre_bias != nullptr) {
          float b[E];
          aligned_parameters(b, static_cast<const P*>(a.pre_bias), at[j].first, live);
#pragma unroll
          for (int e = 0; e < E; ++e) v[j][e] += b[e];
        }
        aligned_store(static_cast<T*>(a.n) + r * a.ld_n + at[j].first, v[j], live);
      }
    }
  }
}

// ------------------------------------------------------------------ backward

// k_norm_grad on rows that come through a ring: the same sums (see there), the
// values read from shared memory where they are used.
template <typename T, typename P, bool LAYER, bool BIAS, bool MANY>
__global__ void __launch_bounds__(kNormGradThreads, (MANY || sizeof(T) == 4) ? 1 : 2)
    k_norm_grad_ring(const ffn_norm_grad_t a, const NormGradShape sh, const NormSums ws, uint32_t* status) {
  constexpr int E = kNormGradEach;
  constexpr int K = LAYER ? 4 : 3;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[8 * kNormStages];
  __shared__ float parts_smem[2 * 128 * K];
  __shared__ volatile uint32_t abort_flag;
  const int D = (int)a.D;
  const int rank = sh.cluster > 1 ? (int)cluster_ctarank() : 0;
  const bool lone = sh.lanes > 1;  // a warp per part
  const int tid = lone ? (int)lane_idx() : (int)threadIdx.x;
  const int group = lone ? (int)(threadIdx.x >> 5) : 0;
  const int part = lone ? (int)blockIdx.x * sh.lanes + group : (int)blockIdx.x / sh.cluster;
  RowSums<K> sum{parts_smem, sh.threads / 32, sh.cluster, rank, 0};
  const bool post = (a.flags & FFN_NORM_POST) != 0, pre = (a.flags & FFN_NORM_PRE) != 0;
  const int col0 = (int)(rank * sh.columns), cols = min(D - col0, (int)sh.columns);
  const int first = col0 + tid * E;  // this thread's columns
  const bool live = tid * E < cols;
  Ring ring;
  ring.stages = kNormStages;
  const uint32_t y_at = pre ? 2u : 0u, ds_at = y_at + (a.y != nullptr ? 1u : 0u);
  ring.arrays = ds_at + (a.ds != nullptr ? 1u : 0u);
  ring.bytes = (uint32_t)(cols * (int)sizeof(T));
  ring.pitch = (uint32_t)(sh.columns * (int64_t)sizeof(T));
  ring.slots = smem + (size_t)group * ring.stages * ring.arrays * ring.pitch;
  ring.full = bars + group * kNormStages;
  ring.abort_flag = &abort_flag;
  ring.status = status;
  if (tid == 0) {
    for (uint32_t s = 0; s < ring.stages; ++s) mbar_init(smem_u32(ring.full + s), 1);
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
  if (part >= sh.parts) return;  // (whole warps only)
  int64_t r0, r1;
  const int64_t per = a.M / a.groups;
  norm_part_rows<MANY>(a, sh, part, r0, r1);
  uint32_t issued = 0;  // (the group's first thread)
  auto issue = [&]() {
    const int64_t r = r0 + issued;
    if (r >= r1) return;
    const uint32_t stage = issued % ring.stages, bar = smem_u32(ring.full + stage);
    mbar_arrive_expect_tx(bar, ring.arrays * ring.bytes);
    auto copy = [&](uint32_t array, const void* base, int64_t ld) {
      bulk_load(smem_u32(ring.slot(stage, array)), static_cast<const T*>(base) + r * ld + col0, ring.bytes, bar);
    };
    if (pre) {
      copy(0, a.s, a.ld_s);
      copy(1, a.dn, a.ld_dn);
    }
    if (a.y != nullptr) copy(y_at, a.y, a.ld_y);
    if (a.ds != nullptr) copy(ds_at, a.ds, a.ld_ds);
    ++issued;
  };
  if (tid == 0)
    for (uint32_t s = 0; s < ring.stages; ++s) issue();

  const float inv = 1.f / (float)D;
  const int local = tid * E;  // in a slot
  const bool alone = sum.warps == 1 && sum.cluster == 1;
  float A[E] = {}, C[E] = {}, B[BIAS ? E : 1] = {}, Eo[BIAS ? E : 1] = {};
  float GA[MANY ? E : 1] = {}, GB[(MANY && BIAS) ? E : 1] = {};
  uint32_t i = 0;
  for (int64_t r = r0; r < r1; ++r, ++i) {
    if (!ring.wait(i)) {
      if (tid == 0) ring.settle(issued, i);
      break;
    }
    const uint32_t stage = i % ring.stages;
    float mean_s = 0.f, mean_y = 0.f, mean_a = 0.f, k[K];
    if constexpr (LAYER) {
#pragma unroll
      for (int q = 0; q < K; ++q) k[q] = 0.f;
      if (pre) {
        float s[E], dn[E];
        from_slot<T>(s, ring.slot(stage, 0), local, live);
        from_slot<T>(dn, ring.slot(stage, 1), local, live);
        if (a.pre_weight != nullptr) {
          float w[E];
          aligned_parameters(w, static_cast<const P*>(a.pre_weight), first, live);
#pragma unroll
          for (int e = 0; e < E; ++e) dn[e] = __fmul_rn(dn[e], w[e]);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
          k[0] += s[e];
          k[2] += dn[e];
        }
      }
      if (post) {
        float y[E];
        from_slot<T>(y, ring.slot(stage, y_at), local, live);
#pragma unroll
        for (int e = 0; e < E; ++e) k[1] += y[e];
      }
      sum(k);
      if (i > 0 && tid == 0 && !alone) issue();  // (every thread is past the row before: its slots are free)
      mean_s = k[0] * inv;
      mean_y = k[1] * inv;
      mean_a = k[2] * inv;
    }
#pragma unroll
    for (int q = 0; q < K; ++q) k[q] = 0.f;
    if (live && pre) {
      float s[E], dn[E];
      from_slot<T>(s, ring.slot(stage, 0), local, true);
      from_slot<T>(dn, ring.slot(stage, 1), local, true);
      if (a.pre_weight != nullptr) {
        float w[E];
        aligned_parameters(w, static_cast<const P*>(a.pre_weight), first, true);
#pragma unroll
        for (int e = 0; e < E; ++e) dn[e] = __fmul_rn(dn[e], w[e]);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float c = s[e] - mean_s;
        k[0] = fmaf(c, c, k[0]);
        k[1] = fmaf(c, dn[e], k[1]);
      }
    }
    if (live && post) {
      float y[E];
      from_slot<T>(y, ring.slot(stage, y_at), local, true);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float c = y[e] - mean_y;
        k[2] = fmaf(c, c, k[2]);
      }
    }
    __syncwarp();
    sum(k);
    if constexpr (!LAYER) {
      if (i > 0 && tid == 0 && !alone) issue();
    }
    const float r_s = rsqrtf(k[0] * inv + a.eps), mean_au = k[1] * inv * r_s;
    const float r_y = post ? rsqrtf(k[2] * inv + a.eps) : 1.f;
    float t[E];
    if (a.ds != nullptr) {
      from_slot<T>(t, ring.slot(stage, ds_at), local, live);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) t[e] = 0.f;
    }
    if (pre && live) {
      float s[E], dn[E];
      from_slot<T>(s, ring.slot(stage, 0), local, true);
      from_slot<T>(dn, ring.slot(stage, 1), local, true);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        s[e] = unit_value(s[e], mean_s, r_s);
        C[e] = fmaf(dn[e], s[e], C[e]);
        if constexpr (BIAS) Eo[e] += dn[e];
      }
      if (a.pre_weight != nullptr) {
        float w[E];
        aligned_parameters(w, static_cast<const P*>(a.pre_weight), first, true);
#pragma unroll
        for (int e = 0; e < E; ++e) dn[e] = __fmul_rn(dn[e], w[e]);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) t[e] = unit_slope(t[e], r_s, dn[e], s[e], mean_au, mean_a);
    }
    if (a.dresidual != nullptr) {
      float o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = a.residual_scale * t[e];
      aligned_store(static_cast<T*>(a.dresidual) + r * a.ld_dresidual + first, o, live);
    }
    float y[E];
    if (a.y != nullptr) {
      from_slot<T>(y, ring.slot(stage, y_at), local, live);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        y[e] = unit_value(y[e], mean_y, r_y);
        A[e] = fmaf(t[e], y[e], A[e]);
        if constexpr (BIAS) B[e] += t[e];
      }
    }
    const int64_t g = r / per;
    float gate[E];
    if (a.gate != nullptr) {
      aligned_parameters(gate, static_cast<const P*>(a.gate) + g * a.ld_gate, first, live);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) gate[e] = 1.f;
    }
    if (a.dy != nullptr) {
#pragma unroll
      for (int e = 0; e < E; ++e) t[e] = __fmul_rn(t[e], __fmul_rn(a.branch_scale, gate[e]));
      if (post) {
        if (a.post_weight != nullptr) {
          float w[E];
          aligned_parameters(w, static_cast<const P*>(a.post_weight), first, live);
#pragma unroll
          for (int e = 0; e < E; ++e) t[e] = __fmul_rn(t[e], w[e]);
        }
#pragma unroll
        for (int q = 0; q < K; ++q) k[q] = 0.f;
        if (live) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            k[0] = fmaf(t[e], y[e], k[0]);
            if constexpr (LAYER) k[1] += t[e];
          }
        }
        __syncwarp();
        sum(k);
        const float mean_bv = k[0] * inv, mean_b = LAYER ? k[1] * inv : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) t[e] = unit_slope(0.f, r_y, t[e], y[e], mean_bv, mean_b);
      }
      aligned_store(static_cast<T*>(a.dy) + r * a.ld_dy + first, t, live);
    }
    if (alone) {  // no barrier of the next row to wait for
      __syncwarp();
      if (tid == 0) issue();
    }
    if constexpr (MANY) {
      if (r + 1 == (g + 1) * per) {  // the group's last row: its gate's gradient is complete
        if (a.dgate != nullptr) {
          float o[E], pw[E], pb[E];
          parameters<P>(pw, a.post_weight, 1.f, Places{first, col0 + cols});
          parameters<P>(pb, a.post_bias, 0.f, Places{first, col0 + cols});
#pragma unroll
          for (int e = 0; e < E; ++e)
            o[e] = a.branch_scale * (pw[e] * A[e] + (BIAS ? pb[e] * B[BIAS ? e : 0] : 0.f));
          store(a.dgate + g * (int64_t)D, o, Places{first, col0 + cols});
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
  const int64_t out = (int64_t)part * D + first;
  if constexpr (MANY) {
    if (ws.a != nullptr) aligned_store(ws.a + out, GA, live);
    if constexpr (BIAS) {
      if (ws.b != nullptr) aligned_store(ws.b + out, GB, live);
    }
  } else {
    if (ws.a != nullptr) aligned_store(ws.a + out, A, live);
    if constexpr (BIAS) {
      if (ws.b != nullptr) aligned_store(ws.b + out, B, live);
    }
  }
  if (ws.c != nullptr) aligned_store(ws.c + out, C, live);
  if constexpr (BIAS) {
    if (ws.e != nullptr) aligned_store(ws.e + out, Eo, live);
  }
}

}  // namespace

}  // namespace dgb
