// kernel_gated_few.cu -- the gated projections for few tokens (M <= 16): both weight
// streams read once, the activation and the product in the same kernel.
//
// Bound by the weights, 2F x K of 2 bytes: at one to sixteen operations per byte the
// work is to keep enough of them on their way.  Every lane loads 16-byte pieces of
// its rows straight into registers, a group of pieces ahead of the one in use, and
// the arithmetic is warp-level mma.sync m16n8k16: the fragment's rows 0-7 are eight
// rows of Wg and its rows 8-15 the same rows of Wu, so the lane that ends up with g
// of a token also ends up with u, and each 16-byte piece of x serves both.  The order
// of K inside the fragments is free because weights and tokens use the same one.
//
// A CTA owns 8 hidden features; its 8 warps split K and add their sums in shared
// memory, where one thread per feature and token joins g and u.  The launch is a
// programmatic dependent of the previous kernel; while it waits, L2 fetches the
// first weights (a prefetch returns no data, so it may run ahead of the wait even if
// the previous kernel writes them).  1 x 14336 x 4096: 33.4 us, 7.0 TB/s; the weights
// are read exactly once (235 MB).
#include <type_traits>

#include "ffn_common.cuh"
#include "gated.h"
#include "launch.h"

namespace dgb {

namespace {

constexpr int GF_THREADS = 256;
constexpr int GF_ROWS = 8;  // hidden features per CTA
constexpr int GF_PIECES = 2;  // 16-byte pieces of each of the two rows in a group
constexpr int GF_GROUPS = 2;  // groups on their way

__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <typename T>
__device__ __forceinline__ void mma_rows16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                           uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// NT: token tiles of 8 (1 for M <= 8, 2 for M <= 16)
template <typename T, int NT, int ACT>
__global__ void __launch_bounds__(GF_THREADS, 4) k_gated_few(const __grid_constant__ ffn_gated_t a) {
  constexpr int W = GF_THREADS / 32;
  __shared__ float red[W][2 * GF_ROWS][8 * NT + 1];
  const int K8 = (int)(a.K / 8);               // 16-byte pieces of a row
  const int S = (K8 + W - 1) / W;              // of this warp's slice of K
  const int w = (int)warp_idx(), lane = (int)lane_idx();
  const int gr = lane >> 2, c = lane & 3;      // fragment row, piece within 32 elements
  const int64_t f = (int64_t)blockIdx.x * GF_ROWS + gr;
  const bool row_in = f < a.F;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const int k0 = w * S, k1 = min(K8, k0 + S);  // this warp's pieces
  const uint4* gate = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.w) + f * a.ld_w);
  const uint4* up = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.w) + (a.F + f) * a.ld_w);
  const int NG = (max(0, k1 - k0) + 4 * GF_PIECES - 1) / (4 * GF_PIECES);
  uint4 bw[GF_GROUPS][2][GF_PIECES];
  auto load_group = [&](int q, uint4 (&b)[2][GF_PIECES]) {
#pragma unroll
    for (int v = 0; v < GF_PIECES; ++v) {
      const int k = k0 + (q * GF_PIECES + v) * 4 + c;
      const bool in = row_in && k < k1;
      b[0][v] = in ? load_once(gate + k) : zero;
      b[1][v] = in ? load_once(up + k) : zero;
    }
  };
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (row_in && c < 2 && k0 + 8 * c < k1) {
    prefetch_l2_line(gate + k0 + 8 * c);
    prefetch_l2_line(up + k0 + 8 * c);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
  for (int i = 0; i < GF_GROUPS; ++i) load_group(i, bw[i]);
  float d[NT][4] = {};
  for (int q0 = 0; q0 < NG; q0 += GF_GROUPS) {
#pragma unroll
    for (int i = 0; i < GF_GROUPS; ++i) {
      const int q = q0 + i;
      if (q < NG) {
#pragma unroll
        for (int v = 0; v < GF_PIECES; ++v) {
          const int k = k0 + (q * GF_PIECES + v) * 4 + c;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const int m = 8 * t + gr;
            const uint4 x = (m < a.M && k < k1)
                                ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + m * a.ld_x) + k)
                                : zero;
            mma_rows16<T>(d[t], bw[i][0][v].x, bw[i][1][v].x, bw[i][0][v].y, bw[i][1][v].y, x.x, x.y);
            mma_rows16<T>(d[t], bw[i][0][v].z, bw[i][1][v].z, bw[i][0][v].w, bw[i][1][v].w, x.z, x.w);
          }
        }
        load_group(q + GF_GROUPS, bw[i]);
      }
    }
  }
  // d[t][0..1]: gate row gr, tokens 8 t + 2 c and the next; d[t][2..3]: up row gr
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[w][gr + 8 * (e >> 1)][8 * t + 2 * c + (e & 1)] = d[t][e];
  __syncthreads();
  const int i = (int)threadIdx.x, r = i & 7, m = i >> 3;  // neighbouring threads store neighbouring features
  const int64_t fo = (int64_t)blockIdx.x * GF_ROWS + r;
  if (m >= 8 * NT || m >= a.M || fo >= a.F) return;
  float g = 0.f, u = 0.f;
#pragma unroll
  for (int q = 0; q < W; ++q) {
    g += red[q][r][m];
    u += red[q][r + 8][m];
  }
  static_cast<T*>(a.h)[m * a.ld_h + fo] = from_f32<T>(act_only<ACT>(g) * u);
  if (a.gu != nullptr) {
    T* gu = static_cast<T*>(a.gu) + m * a.ld_gu + fo;
    gu[0] = from_f32<T>(g);
    gu[a.F] = from_f32<T>(u);
  }
}

template <typename T, int NT>
const void* few_kernel(int act) {
  switch (act) {
    case EPI_ACT_RELU: return (const void*)k_gated_few<T, NT, EPI_ACT_RELU>;
    case EPI_ACT_SILU: return (const void*)k_gated_few<T, NT, EPI_ACT_SILU>;
    case EPI_ACT_GELU_TANH: return (const void*)k_gated_few<T, NT, EPI_ACT_GELU_TANH>;
    case EPI_ACT_GELU_ERF: return (const void*)k_gated_few<T, NT, EPI_ACT_GELU_ERF>;
    default: return (const void*)k_gated_few<T, NT, EPI_ACT_NONE>;
  }
}

}  // namespace

cudaError_t launch_gated_few(const ffn_gated_t& a, cudaStream_t st) {
  LaunchSpec s;
  s.func = a.dtype == FFN_BF16
               ? (a.M <= 8 ? few_kernel<__nv_bfloat16, 1>(a.activation) : few_kernel<__nv_bfloat16, 2>(a.activation))
               : (a.M <= 8 ? few_kernel<__half, 1>(a.activation) : few_kernel<__half, 2>(a.activation));
  s.grid = dim3((unsigned)((a.F + GF_ROWS - 1) / GF_ROWS), 1, 1);
  s.block = dim3(GF_THREADS, 1, 1);
  s.pdl = true;
  ffn_gated_t copy = a;
  void* args[] = {&copy};
  return launch_spec(s, args, st);
}

}  // namespace dgb
