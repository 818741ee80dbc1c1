// kernels_gated.cu -- the gated projections h = act(x Wg^T) * (x Wu^T) and their
// gradients: one tiled product kernel on the CUDA cores, whose epilogue joins the
// gate's and the up projection's sums.
//
// A CTA of 256 threads owns a 64 x 64 output tile and walks the reduction in
// steps of 16 staged in shared memory as fp32; a thread owns 4 x 4 outputs.
// Operands are read through two strides each, so the one kernel also does the
// products of the backward pass.
#include "ffn_common.cuh"
#include "ffn_launch.h"

namespace dgb {

namespace {

struct Product {
  int64_t rows, cols, depth;
  const void* a;
  int64_t a_row, a_k;  // strides of A(row, k)
  const void* b;
  int64_t b_col, b_k;  // strides of B(col, k)
  int64_t b_up;        // offset of the up projection's operand (two-product form)
  void* c;
  int64_t ld_c;
  void* gu;
  int64_t ld_gu;
  const void* dh;
  int64_t ld_dh;
};

enum Join { JOIN_NONE = 0, JOIN_FORWARD = 1, JOIN_GRAD = 2 };

template <typename T, int JOIN, int ACT>
__global__ void __launch_bounds__(256) k_product(Product p) {
  constexpr int N_B = JOIN == JOIN_NONE ? 1 : 2;
  __shared__ float as[16][65], bs[N_B][16][65];
  const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
  const T* A = static_cast<const T*>(p.a);
  const T* B = static_cast<const T*>(p.b);
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float acc[N_B][4][4] = {};
  for (int64_t k0 = 0; k0 < p.depth; k0 += 16) {
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
      const int r = i / 16, k = i % 16;
      as[k][r] = (r0 + r < p.rows && k0 + k < p.depth) ? to_f32(A[(r0 + r) * p.a_row + (k0 + k) * p.a_k]) : 0.f;
#pragma unroll
      for (int b = 0; b < N_B; ++b)
        bs[b][k][r] = (c0 + r < p.cols && k0 + k < p.depth)
                          ? to_f32(B[b * p.b_up + (c0 + r) * p.b_col + (k0 + k) * p.b_k])
                          : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int b = 0; b < N_B; ++b) acc[b][i][j] = fmaf(as[k][ty + 16 * i], bs[b][k][tx + 16 * j], acc[b][i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = r0 + ty + 16 * i, c = c0 + tx + 16 * j;
      if (r >= p.rows || c >= p.cols) continue;
      T* out = static_cast<T*>(p.c) + r * p.ld_c + c;
      if constexpr (JOIN == JOIN_NONE) {
        *out = from_f32<T>(acc[0][i][j]);
      } else {
        const float g = acc[0][i][j], u = acc[1][i][j];
        float a, d;
        act_and_slope<ACT>(g, a, d);
        if constexpr (JOIN == JOIN_FORWARD) {
          *out = from_f32<T>(a * u);
          if (p.gu != nullptr) {
            T* gu = static_cast<T*>(p.gu) + r * p.ld_gu + c;
            gu[0] = from_f32<T>(g);
            gu[p.cols] = from_f32<T>(u);
          }
        } else {
          const float dh = to_f32(static_cast<const T*>(p.dh)[r * p.ld_dh + c]);
          out[0] = from_f32<T>(dh * u * d);
          out[p.cols] = from_f32<T>(dh * a);
        }
      }
    }
}

// dgu from kept pre-activations: one element pair per thread
template <typename T, int ACT>
__global__ void __launch_bounds__(256) k_gated_slopes(ffn_gated_grad_t a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.M * a.F) return;
  const int64_t r = i / a.F, c = i - r * a.F;
  const T* gu = static_cast<const T*>(a.gu) + r * a.ld_gu + c;
  T* dgu = static_cast<T*>(a.dgu) + r * a.ld_dgu + c;
  const float dh = to_f32(static_cast<const T*>(a.dh)[r * a.ld_dh + c]);
  float act, slope;
  act_and_slope<ACT>(to_f32(gu[0]), act, slope);
  dgu[0] = from_f32<T>(dh * to_f32(gu[a.F]) * slope);
  dgu[a.F] = from_f32<T>(dh * act);
}

template <typename T, int JOIN, int ACT>
cudaError_t product(const Product& p, cudaStream_t st) {
  const dim3 grid((unsigned)((p.cols + 63) / 64), (unsigned)((p.rows + 63) / 64));
  if (grid.y > 65535) return cudaErrorInvalidConfiguration;
  k_product<T, JOIN, ACT><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int ACT>
cudaError_t forward(const ffn_gated_t& a, cudaStream_t st) {
  Product p{a.M, a.F, a.K, a.x, a.ld_x, 1, a.w, a.ld_w, 1, a.F * a.ld_w, a.h, a.ld_h, a.gu, a.ld_gu, nullptr, 0};
  return product<T, JOIN_FORWARD, ACT>(p, st);
}

template <typename T, int ACT>
cudaError_t backward(const ffn_gated_grad_t& a, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (a.gu != nullptr) {
    k_gated_slopes<T, ACT><<<(unsigned)((a.M * a.F + 255) / 256), 256, 0, st>>>(a);
    e = cudaGetLastError();
  } else {
    e = product<T, JOIN_GRAD, ACT>(Product{a.M, a.F, a.K, a.x, a.ld_x, 1, a.w, a.ld_w, 1, a.F * a.ld_w, a.dgu,
                                           a.ld_dgu, nullptr, 0, a.dh, a.ld_dh}, st);
  }
  if (e == cudaSuccess && a.dx != nullptr)
    e = product<T, JOIN_NONE, 0>(Product{a.M, a.K, 2 * a.F, a.dgu, a.ld_dgu, 1, a.w, 1, a.ld_w, 0, a.dx, a.ld_dx,
                                         nullptr, 0, nullptr, 0}, st);
  if (e == cudaSuccess && a.dw != nullptr)
    e = product<T, JOIN_NONE, 0>(Product{2 * a.F, a.K, a.M, a.dgu, 1, a.ld_dgu, a.x, 1, a.ld_x, 0, a.dw, a.ld_dw,
                                         nullptr, 0, nullptr, 0}, st);
  return e;
}

template <typename T, typename A>
cudaError_t by_activation(const A& a, cudaStream_t st) {
  auto go = [&](auto act) -> cudaError_t {
    constexpr int ACT = decltype(act)::value;
    if constexpr (std::is_same<A, ffn_gated_t>::value) {
      return forward<T, ACT>(a, st);
    } else {
      return backward<T, ACT>(a, st);
    }
  };
  switch (a.activation) {
    case GEMM_ACT_RELU: return go(std::integral_constant<int, EPI_ACT_RELU>{});
    case GEMM_ACT_SILU: return go(std::integral_constant<int, EPI_ACT_SILU>{});
    case GEMM_ACT_GELU_TANH: return go(std::integral_constant<int, EPI_ACT_GELU_TANH>{});
    case GEMM_ACT_GELU_ERF: return go(std::integral_constant<int, EPI_ACT_GELU_ERF>{});
    default: return go(std::integral_constant<int, EPI_ACT_NONE>{});
  }
}

}  // namespace

cudaError_t launch_gated(const ffn_gated_t& a, const FfnDevice&, cudaStream_t st) {
  return a.dtype == FFN_BF16 ? by_activation<__nv_bfloat16>(a, st) : by_activation<__half>(a, st);
}

cudaError_t launch_gated_backward(const ffn_gated_grad_t& a, const FfnDevice&, cudaStream_t st) {
  return a.dtype == FFN_BF16 ? by_activation<__nv_bfloat16>(a, st) : by_activation<__half>(a, st);
}

}  // namespace dgb
