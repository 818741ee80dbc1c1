// kernel_norm.cu -- the norms around a block fused with its gate, its scales and
// the residual stream, and their gradients.
//
// Forward: one CTA per row, the row staged in shared memory as fp32.  Backward:
// one CTA per row writes the inputs' gradients and the row's statistics, then a
// second kernel sums the parameters' gradients over the rows, one thread per
// column and group of rows.
#include <type_traits>

#include "ffn_common.cuh"
#include "ffn_launch.h"

namespace dgb {

namespace {

constexpr int NT = 256;

// sum over the CTA, the same value in every thread
__device__ __forceinline__ float cta_sum(float v) {
  __shared__ float part[NT / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();  // the last sum's values have been read
  if (lane_idx() == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) v += part[i];
  return v;
}

// mean (layer norm) and reciprocal deviation of a row of fp32 values, two passes
template <bool LAYER>
__device__ __forceinline__ float2 row_stats(const float* row, int D, float eps) {
  float mean = 0.f;
  if constexpr (LAYER) {
    float s = 0.f;
    for (int i = threadIdx.x; i < D; i += NT) s += row[i];
    mean = cta_sum(s) / (float)D;
  }
  float q = 0.f;
  for (int i = threadIdx.x; i < D; i += NT) q += (row[i] - mean) * (row[i] - mean);
  return make_float2(mean, rsqrtf(cta_sum(q) / (float)D + eps));
}

template <typename P>
__device__ __forceinline__ float param(const void* p, int64_t i, float absent) {
  return p == nullptr ? absent : to_f32(static_cast<const P*>(p)[i]);
}

template <typename T, typename P, bool LAYER>
__global__ void __launch_bounds__(NT) k_norm(ffn_norm_t a) {
  extern __shared__ float row[];
  const int64_t r = blockIdx.x;
  const int D = (int)a.D;
  const int64_t g = a.gate ? r / (a.M / a.groups) : 0;
  const T* y = static_cast<const T*>(a.y) + r * a.ld_y;
  for (int i = threadIdx.x; i < D; i += NT) row[i] = to_f32(y[i]);
  float2 st = make_float2(0.f, 1.f);
  const bool post = (a.flags & FFN_NORM_POST) != 0;
  if (post) st = row_stats<LAYER>(row, D, a.eps);
  for (int i = threadIdx.x; i < D; i += NT) {
    float z = row[i];
    if (post) z = (z - st.x) * st.y * param<P>(a.post_weight, i, 1.f) + param<P>(a.post_bias, i, 0.f);
    z *= a.branch_scale * param<P>(a.gate, g * a.ld_gate + i, 1.f);
    if (a.residual) z += a.residual_scale * to_f32(static_cast<const T*>(a.residual)[r * a.ld_residual + i]);
    row[i] = z;
    if (a.s) static_cast<T*>(a.s)[r * a.ld_s + i] = from_f32<T>(z);
  }
  if (a.flags & FFN_NORM_PRE) {
    st = row_stats<LAYER>(row, D, a.eps);
    for (int i = threadIdx.x; i < D; i += NT)
      static_cast<T*>(a.n)[r * a.ld_n + i] = from_f32<T>(
          (row[i] - st.x) * st.y * param<P>(a.pre_weight, i, 1.f) + param<P>(a.pre_bias, i, 0.f));
  }
}

// a row's numbers the column sums need: statistics of s and y, and the two means
// of the pre-norm's gradient
struct RowNumbers {
  float mean_s, r_s, mean_y, r_y, mean_a, mean_au;
};

template <typename T, typename P>
struct GradRow {
  const ffn_norm_grad_t& a;
  int64_t r, g;
  __device__ GradRow(const ffn_norm_grad_t& args, int64_t row) : a(args), r(row) {
    g = (a.gate || a.dgate) ? r / (a.M / a.groups) : 0;
  }
  __device__ float y(int i) const { return to_f32(static_cast<const T*>(a.y)[r * a.ld_y + i]); }
  __device__ float s(int i) const { return to_f32(static_cast<const T*>(a.s)[r * a.ld_s + i]); }
  __device__ float dn(int i) const { return to_f32(static_cast<const T*>(a.dn)[r * a.ld_dn + i]); }
  // gradient of the stream
  __device__ float t(int i, const RowNumbers& q) const {
    float v = a.ds ? to_f32(static_cast<const T*>(a.ds)[r * a.ld_ds + i]) : 0.f;
    if (a.flags & FFN_NORM_PRE)
      v += q.r_s * (dn(i) * param<P>(a.pre_weight, i, 1.f) - (s(i) - q.mean_s) * q.r_s * q.mean_au - q.mean_a);
    return v;
  }
  __device__ float dz(int i, float t) const {
    return t * a.branch_scale * param<P>(a.gate, g * a.ld_gate + i, 1.f);
  }
};

template <typename T, typename P, bool LAYER>
__global__ void __launch_bounds__(NT) k_norm_grad(ffn_norm_grad_t a) {
  extern __shared__ float row[];
  const int D = (int)a.D;
  const GradRow<T, P> R(a, blockIdx.x);
  RowNumbers q{0.f, 1.f, 0.f, 1.f, 0.f, 0.f};
  if (a.flags & FFN_NORM_PRE) {
    for (int i = threadIdx.x; i < D; i += NT) row[i] = R.s(i);
    const float2 st = row_stats<LAYER>(row, D, a.eps);
    q.mean_s = st.x;
    q.r_s = st.y;
    float sa = 0.f, sau = 0.f;
    for (int i = threadIdx.x; i < D; i += NT) {
      const float v = R.dn(i) * param<P>(a.pre_weight, i, 1.f);
      sa += v;
      sau += v * (row[i] - q.mean_s) * q.r_s;
    }
    q.mean_au = cta_sum(sau) / (float)D;
    if constexpr (LAYER) q.mean_a = cta_sum(sa) / (float)D;
  }
  float mean_b = 0.f, mean_bu = 0.f;
  const bool post = (a.flags & FFN_NORM_POST) != 0;
  if (post) {
    for (int i = threadIdx.x; i < D; i += NT) row[i] = R.y(i);
    const float2 st = row_stats<LAYER>(row, D, a.eps);
    q.mean_y = st.x;
    q.r_y = st.y;
    float sb = 0.f, sbu = 0.f;
    for (int i = threadIdx.x; i < D; i += NT) {
      const float v = R.dz(i, R.t(i, q)) * param<P>(a.post_weight, i, 1.f);
      sb += v;
      sbu += v * (row[i] - q.mean_y) * q.r_y;
    }
    mean_bu = cta_sum(sbu) / (float)D;
    if constexpr (LAYER) mean_b = cta_sum(sb) / (float)D;
  }
  for (int i = threadIdx.x; i < D; i += NT) {
    const float t = R.t(i, q);
    if (a.dresidual) static_cast<T*>(a.dresidual)[R.r * a.ld_dresidual + i] = from_f32<T>(a.residual_scale * t);
    if (a.dy) {
      float v = R.dz(i, t);
      if (post)
        v = q.r_y * (v * param<P>(a.post_weight, i, 1.f) - (row[i] - q.mean_y) * q.r_y * mean_bu - mean_b);
      static_cast<T*>(a.dy)[R.r * a.ld_dy + i] = from_f32<T>(v);
    }
  }
  if (threadIdx.x == 0 && a.workspace) static_cast<RowNumbers*>(a.workspace)[R.r] = q;
}

// sums over the rows: 32 columns x 8 row lanes per CTA; blockIdx.y is the gate's
// group for dgate (which = 0) or 0 for the sums over all rows
template <typename T, typename P>
__global__ void __launch_bounds__(256) k_norm_column_sums(ffn_norm_grad_t a, bool gates) {
  __shared__ float part[4][8][33];
  const int c = threadIdx.x & 31, lane = threadIdx.x >> 5, D = (int)a.D;
  const int i = blockIdx.x * 32 + c;
  const int64_t per = gates ? a.M / a.groups : a.M, r0 = (int64_t)blockIdx.y * per;
  const RowNumbers* rows = static_cast<const RowNumbers*>(a.workspace);
  float sums[4] = {};
  if (i < D)
    for (int64_t r = r0 + lane; r < r0 + per; r += 8) {
      const GradRow<T, P> R(a, r);
      const RowNumbers q = rows[r];
      const float t = R.t(i, q);
      const float uy = a.y ? (R.y(i) - q.mean_y) * q.r_y : 0.f;
      if (gates) {
        const float z =
            (a.flags & FFN_NORM_POST) ? uy * param<P>(a.post_weight, i, 1.f) + param<P>(a.post_bias, i, 0.f) : uy;
        sums[0] += t * z * a.branch_scale;
      } else {
        const float dz = R.dz(i, t);
        sums[0] += dz * uy;
        sums[1] += dz;
        if (a.flags & FFN_NORM_PRE) {
          sums[2] += R.dn(i) * (R.s(i) - q.mean_s) * q.r_s;
          sums[3] += R.dn(i);
        }
      }
    }
#pragma unroll
  for (int k = 0; k < 4; ++k) part[k][lane][c] = sums[k];
  __syncthreads();
  if (lane < 4 && i < D) {
    float v = 0.f;
#pragma unroll
    for (int l = 0; l < 8; ++l) v += part[lane][l][c];
    float* const out[4] = {gates ? a.dgate + (int64_t)blockIdx.y * D : a.dpost_weight, a.dpost_bias, a.dpre_weight,
                           a.dpre_bias};
    if ((!gates || lane == 0) && out[lane]) out[lane][i] = v;
  }
}

template <typename F>
cudaError_t by_types(int32_t dtype, int32_t param_dtype, int32_t kind, F f) {
  auto with = [&](auto t, auto p) {
    return kind == FFN_NORM_LAYER ? f(t, p, std::true_type{}) : f(t, p, std::false_type{});
  };
  if (dtype == FFN_F32) return with(float{}, float{});
  if (dtype == FFN_BF16)
    return param_dtype == FFN_F32 ? with(__nv_bfloat16{}, float{}) : with(__nv_bfloat16{}, __nv_bfloat16{});
  return param_dtype == FFN_F32 ? with(__half{}, float{}) : with(__half{}, __half{});
}

cudaError_t row_smem(const void* f, size_t bytes) {
  return bytes > 32 * 1024 ? cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)
                           : cudaSuccess;
}

}  // namespace

cudaError_t launch_norm(const ffn_norm_t& a, const FfnDevice&, cudaStream_t st) {
  const size_t smem = (size_t)a.D * 4;
  return by_types(a.dtype, a.param_dtype, a.kind, [&](auto t, auto p, auto layer) -> cudaError_t {
    auto* k = k_norm<decltype(t), decltype(p), decltype(layer)::value>;
    const cudaError_t e = row_smem((const void*)k, smem);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)a.M, NT, smem, st>>>(a);
    return cudaGetLastError();
  });
}

size_t norm_backward_workspace(const ffn_norm_grad_t& a) {
  return (a.dgate || a.dpost_weight || a.dpost_bias || a.dpre_weight || a.dpre_bias)
             ? (size_t)a.M * sizeof(RowNumbers)
             : 0;
}

cudaError_t launch_norm_backward(const ffn_norm_grad_t& a, const FfnDevice&, cudaStream_t st) {
  const size_t smem = (size_t)a.D * 4;
  return by_types(a.dtype, a.param_dtype, a.kind, [&](auto t, auto p, auto layer) -> cudaError_t {
    using T = decltype(t);
    using P = decltype(p);
    auto* k = k_norm_grad<T, P, decltype(layer)::value>;
    cudaError_t e = row_smem((const void*)k, smem);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)a.M, NT, smem, st>>>(a);
    e = cudaGetLastError();
    const unsigned cols = (unsigned)((a.D + 31) / 32);
    if (e == cudaSuccess && (a.dpost_weight || a.dpost_bias || a.dpre_weight || a.dpre_bias)) {
      k_norm_column_sums<T, P><<<dim3(cols, 1), 256, 0, st>>>(a, false);
      e = cudaGetLastError();
    }
    if (e == cudaSuccess && a.dgate) {
      if (a.groups > 65535) return cudaErrorInvalidConfiguration;
      k_norm_column_sums<T, P><<<dim3(cols, (unsigned)a.groups), 256, 0, st>>>(a, true);
      e = cudaGetLastError();
    }
    return e;
  });
}

}  // namespace dgb
