// kernel_gated_few.cu -- the gated projections for few tokens (M <= kGatedFewTokens):
// both weight streams read once, the activation and the product in the same kernel.
//
// Bound by the weights, 2F x K of 2 bytes: at one to 32 operations per byte the work
// is to keep enough of them on their way.  Every lane loads 16-byte pieces of its rows
// straight into registers, a group of pieces ahead of the one in use, and the
// arithmetic is warp-level mma.sync m16n8k16: the fragment's rows 0-7 are eight rows
// of Wg and its rows 8-15 the same rows of Wu, so the lane that ends up with g of a
// token also ends up with u, and each 16-byte piece of x serves both.  The order of K
// inside the fragments is free because weights and tokens use the same one.
//
// A CTA owns 8 hidden features; its 8 warps split K and add their sums in shared
// memory, where one thread per feature and token joins g and u.  Above 8 tokens, x
// (which comes through L1, a piece per 8 tokens) would be as many loads as the weights,
// so a CTA owns 16 features and each piece of x serves four weight rows.  Where that
// leaves the SMs half empty, 16 warps split K (up to 16 tokens: their sums fit shared
// memory).  The launch is a programmatic dependent of the previous kernel; while it
// waits, L2 fetches the first weights (a prefetch returns no data, so it may run ahead
// of the wait even if the previous kernel writes them).
//
// us for F x K = 14336 x 4096, 4096 x 4096 and 1024 x 1024 (bf16):
//    1 token    33.4 (7.0 TB/s)  10.9   1.6     the weights are read exactly once
//   16 tokens   37.9             13.2   2.4     with 8 features per CTA 45.4, 15.2, 3.2
//   32 tokens   45.0             15.8   3.7     on tensor-memory tiles 46.2, 20.3, 8.1
//   48 tokens   76.7             28.3   6.9     the same, 46.6, 20.3, 8.1: hence the limit
// 16 and 8 warps at one token: 2048 x 4096 5.9 and 8.2, 700 x 4096 4.3 and 6.9,
// 4096 x 4096 (512 CTAs) 12.8 and 11.0.
#include <type_traits>

#include "ffn_common.cuh"
#include "gated.h"
#include "launch.h"

namespace dgb {

namespace {

constexpr int GF_ROWS = 8;  // hidden features of a fragment

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

// NT: token tiles of 8.  FR: fragments of 8 features (with their gate and up rows) a warp
// takes at once, which share the tokens' pieces.  W: warps that split K.
template <typename T, int NT, int FR, int W, int ACT>
__global__ void __launch_bounds__(32 * W, (FR == 1 ? 32 : 16) / W)
    k_gated_few(const __grid_constant__ ffn_gated_t a) {
  constexpr int ROWS = GF_ROWS * FR;
  constexpr int PIECES = 3 - FR;  // 16-byte pieces of each row in a group
  constexpr int GROUPS = 2;       // groups on their way
  __shared__ float red[W][2 * ROWS][8 * NT + 1];
  const int K8 = (int)(a.K / 8);               // 16-byte pieces of a row
  const int S = (K8 + W - 1) / W;              // of this warp's slice of K
  const int w = (int)warp_idx(), lane = (int)lane_idx();
  const int gr = lane >> 2, c = lane & 3;      // fragment row, piece within 32 elements
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const int k0 = w * S, k1 = min(K8, k0 + S);  // this warp's pieces
  bool row_in[FR];
  const uint4* row[FR][2];  // gate and up
#pragma unroll
  for (int r = 0; r < FR; ++r) {
    const int64_t f = (int64_t)blockIdx.x * ROWS + r * GF_ROWS + gr;
    row_in[r] = f < a.F;
    row[r][0] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.w) + f * a.ld_w);
    row[r][1] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.w) + (a.F + f) * a.ld_w);
  }
  const int NG = (max(0, k1 - k0) + 4 * PIECES - 1) / (4 * PIECES);
  uint4 bw[GROUPS][FR][2][PIECES];
  auto token = [&](int k, int t) {
    const int m = 8 * t + gr;
    return m < a.M && k < k1 ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + m * a.ld_x) + k)
                             : zero;
  };
  auto load_group = [&](int q, uint4 (&b)[FR][2][PIECES]) {
#pragma unroll
    for (int v = 0; v < PIECES; ++v) {
      const int k = k0 + (q * PIECES + v) * 4 + c;
#pragma unroll
      for (int r = 0; r < FR; ++r) {
        const bool in = row_in[r] && k < k1;
        b[r][0][v] = in ? load_once(row[r][0] + k) : zero;
        b[r][1][v] = in ? load_once(row[r][1] + k) : zero;
      }
    }
  };
#pragma unroll
  for (int r = 0; r < FR; ++r)
    if (row_in[r] && c < 2 && k0 + 8 * c < k1) {
      prefetch_l2_line(row[r][0] + k0 + 8 * c);
      prefetch_l2_line(row[r][1] + k0 + 8 * c);
    }
  wait_for_prior_kernel();
  let_next_kernel_start();
#pragma unroll
  for (int i = 0; i < GROUPS; ++i) load_group(i, bw[i]);
  float d[FR][NT][4] = {};
  for (int q0 = 0; q0 < NG; q0 += GROUPS) {
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      const int q = q0 + i;
      if (q < NG) {
#pragma unroll
        for (int v = 0; v < PIECES; ++v) {
          const int k = k0 + (q * PIECES + v) * 4 + c;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint4 x = token(k, t);
#pragma unroll
            for (int r = 0; r < FR; ++r) {
              const uint4 g = bw[i][r][0][v], u = bw[i][r][1][v];
              mma_rows16<T>(d[r][t], g.x, u.x, g.y, u.y, x.x, x.y);
              mma_rows16<T>(d[r][t], g.z, u.z, g.w, u.w, x.z, x.w);
            }
          }
        }
        load_group(q + GROUPS, bw[i]);
      }
    }
  }
  // d[r][t][0..1]: gate row gr of fragment r, tokens 8 t + 2 c and the next; [2..3]: up row gr
#pragma unroll
  for (int r = 0; r < FR; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        red[w][GF_ROWS * r + gr + ROWS * (e >> 1)][8 * t + 2 * c + (e & 1)] = d[r][t][e];
  __syncthreads();
  // neighbouring threads store neighbouring features
#pragma unroll
  for (int i = (int)threadIdx.x; i < 8 * NT * ROWS; i += 32 * W) {
    const int r = i % ROWS, m = i / ROWS;
    const int64_t fo = (int64_t)blockIdx.x * ROWS + r;
    if (m >= a.M || fo >= a.F) continue;
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int q = 0; q < W; ++q) {
      g += red[q][r][m];
      u += red[q][r + ROWS][m];
    }
    static_cast<T*>(a.h)[m * a.ld_h + fo] = from_f32<T>(act_only<ACT>(g) * u);
    if (a.gu != nullptr) {
      T* gu = static_cast<T*>(a.gu) + m * a.ld_gu + fo;
      gu[0] = from_f32<T>(g);
      gu[a.F] = from_f32<T>(u);
    }
  }
}

template <typename T, int NT, int FR, int W>
const void* few_kernel(int act) {
  switch (act) {
    case EPI_ACT_RELU: return (const void*)k_gated_few<T, NT, FR, W, EPI_ACT_RELU>;
    case EPI_ACT_SILU: return (const void*)k_gated_few<T, NT, FR, W, EPI_ACT_SILU>;
    case EPI_ACT_GELU_TANH: return (const void*)k_gated_few<T, NT, FR, W, EPI_ACT_GELU_TANH>;
    case EPI_ACT_GELU_ERF: return (const void*)k_gated_few<T, NT, FR, W, EPI_ACT_GELU_ERF>;
    default: return (const void*)k_gated_few<T, NT, FR, W, EPI_ACT_NONE>;
  }
}

template <typename T>
const void* few_kernel(int64_t M, int act, bool wide) {
  if (M <= 8) return wide ? few_kernel<T, 1, 1, 16>(act) : few_kernel<T, 1, 1, 8>(act);
  if (M <= 16) return wide ? few_kernel<T, 2, 2, 16>(act) : few_kernel<T, 2, 2, 8>(act);
  return M <= 24 ? few_kernel<T, 3, 2, 8>(act) : few_kernel<T, 4, 2, 8>(act);
}

}  // namespace

cudaError_t launch_gated_few(const ffn_gated_t& a, int num_sms, cudaStream_t st) {
  const int rows = a.M <= 8 ? GF_ROWS : 2 * GF_ROWS;
  const int64_t ctas = (a.F + rows - 1) / rows;
  const bool wide = a.M <= 16 && ctas <= (a.M <= 8 ? 2 : 1) * (int64_t)num_sms;
  LaunchSpec s;
  s.func = a.dtype == FFN_BF16 ? few_kernel<__nv_bfloat16>(a.M, a.activation, wide)
                               : few_kernel<__half>(a.M, a.activation, wide);
  s.grid = dim3((unsigned)ctas, 1, 1);
  s.block = dim3(wide ? 512 : 256, 1, 1);
  s.pdl = true;
  ffn_gated_t copy = a;
  void* args[] = {&copy};
  return launch_spec(s, args, st);
}

}  // namespace dgb
