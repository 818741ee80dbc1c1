// kernel_quant_columns.cu -- quantisation by columns: the operand of x^T, whose rows are x's
// columns.
//
// A CTA takes 256 rows x 64 columns of x through shared memory; a warp then takes 32 of the
// rows, which is one block of 32 or two of 16 of every column, and a lane two columns.
// Where a column has a scale of its own, a first kernel finds the largest magnitudes of
// parts of the columns (x is then read twice, the second time from L2 as far as it holds it).
//
// Bound by memory: 2 bytes read per element, 0.56 to 1.03 written.
#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "quant_format.cuh"
#include "quant_launch.h"

namespace dgb {

namespace {

constexpr int kTileRows = 256, kTileCols = 64, kThreads = 256;
constexpr int kMostParts = 32;  // parts of a column whose largest magnitudes are found apart

struct QuantColumnsParams {
  int64_t rows, cols;       // of x
  int64_t width;            // elements of the operand's rows (rows of x, padded)
  int32_t blocks;           // 512-byte scale blocks across one of them
  int32_t vec;              // x's rows start on 16-byte boundaries
  int32_t parts;
  int32_t row_tiles;
  int64_t part_rows;
  const void* x;
  uint8_t* data;
  uint8_t* scales;
  float* row_scale;
  float* most;              // parts x cols
  int64_t ld_x, ld_data;
};

// 16 bytes of row r from column `col` on, zeros outside the array
template <typename T>
__device__ __forceinline__ uint4 load_piece(const QuantColumnsParams& p, int64_t r, int64_t col) {
  constexpr int n = 16 / (int)sizeof(T);
  const T* row = reinterpret_cast<const T*>(p.x) + r * p.ld_x;
  if (r < p.rows && p.vec && col + n <= p.cols) return __ldg(reinterpret_cast<const uint4*>(row + col));
  union {
    T e[n];
    uint4 u;
  } piece;
  piece.u = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int j = 0; j < n; ++j)
    if (r < p.rows && col + j < p.cols) piece.e[j] = row[col + j];
  return piece.u;
}

// Whether rows r0 .. r0 + n and columns c0 .. c0 + 63 are whole and aligned
__device__ __forceinline__ bool inside(const QuantColumnsParams& p, int64_t r0, int64_t n, int64_t c0) {
  return p.vec != 0 && r0 + n <= p.rows && c0 + kTileCols <= p.cols;
}

// largest magnitudes of 16 bytes of values, pairs at a time for 16-bit types
template <typename T>
struct Most {
  static constexpr int n = 16 / (int)sizeof(T);
  float v[n];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < n; ++j) v[j] = 0.f;
  }
  __device__ __forceinline__ void take(const uint4& u) {
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int j = 0; j < n; ++j) v[j] = larger(v[j], to_f32(e[j]));
  }
  __device__ __forceinline__ float at(int j) const { return v[j]; }
};
template <typename T, typename T2>
struct MostPairs {
  static constexpr int n = 8;
  T2 v[4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t zero = 0u;
      v[j] = *reinterpret_cast<const T2*>(&zero);
    }
  }
  __device__ __forceinline__ void take(const uint4& u) {
    const T2* e = reinterpret_cast<const T2*>(&u);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __hmax2_nan(v[j], __habs2(e[j]));
  }
  __device__ __forceinline__ float at(int j) const { return to_f32(reinterpret_cast<const T*>(v)[j]); }
};
template <>
struct Most<__half> : MostPairs<__half, __half2> {};
template <>
struct Most<__nv_bfloat16> : MostPairs<__nv_bfloat16, __nv_bfloat162> {};

// the largest magnitudes of part blockIdx.y of 64 columns
template <typename T>
__global__ void __launch_bounds__(kThreads) k_quant_column_most(const QuantColumnsParams p) {
  constexpr int n = 16 / (int)sizeof(T), across = kTileCols / n, down = kThreads / across, U = 8;
  __shared__ float found[down][kTileCols + 1];
  wait_for_prior_kernel();
  let_next_kernel_start();
  const int tx = (int)threadIdx.x % across, ty = (int)threadIdx.x / across;
  const int64_t c0 = (int64_t)blockIdx.x * kTileCols;
  const int64_t r0 = blockIdx.y * p.part_rows, r1 = min(p.rows, r0 + p.part_rows);
  Most<T> most;
  most.clear();
  int64_t r = r0 + ty;
  if (inside(p, 0, 0, c0)) {
    // eight rows of a thread on their way at once
    const uint4* from = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.x) + r * p.ld_x + c0 + tx * n);
    const int64_t step = (int64_t)down * p.ld_x / n;
    for (; r + (U - 1) * down < r1; r += U * down, from += U * step) {
      uint4 u[U];
#pragma unroll
      for (int i = 0; i < U; ++i) u[i] = __ldg(from + i * step);
#pragma unroll
      for (int i = 0; i < U; ++i) most.take(u[i]);
    }
  }
  for (; r < r1; r += down) most.take(load_piece<T>(p, r, c0 + tx * n));
#pragma unroll
  for (int j = 0; j < n; ++j) found[ty][tx * n + j] = most.at(j);
  __syncthreads();
  const int64_t c = c0 + threadIdx.x;
  if (threadIdx.x < kTileCols && c < p.cols) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < down; ++i) m = larger(m, found[i][threadIdx.x]);
    p.most[blockIdx.y * p.cols + c] = m;
  }
}

template <typename T>
constexpr int kPitch = kTileCols + (sizeof(T) == 2 ? 8 : 4);  // elements: 16-byte pieces, lanes on different banks

template <typename T, int F>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) k_quant_columns(const QuantColumnsParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  T* tile = reinterpret_cast<T*>(smem);
  __shared__ uint8_t bytes[kTileCols][16];
  __shared__ RowUnit units[kTileCols];
  wait_for_prior_kernel();
  let_next_kernel_start();
  constexpr int n = 16 / (int)sizeof(T), across = kTileCols / n, down = kThreads / across;
  const int64_t strip = blockIdx.x / p.row_tiles, row_tile = blockIdx.x - strip * p.row_tiles;
  const int64_t c0 = strip * kTileCols, r0 = row_tile * kTileRows;
  {
    const int tx = (int)threadIdx.x % across, ty = (int)threadIdx.x / across;
    if (inside(p, r0, kTileRows, c0)) {
      constexpr int U = 8;
      const uint4* from = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.x) + (r0 + ty) * p.ld_x + c0 + tx * n);
      const int64_t step = (int64_t)down * p.ld_x / n;
#pragma unroll 1
      for (int r = ty; r < kTileRows; r += U * down, from += U * step) {
        uint4 u[U];
#pragma unroll
        for (int i = 0; i < U; ++i) u[i] = __ldg(from + i * step);
#pragma unroll
        for (int i = 0; i < U; ++i) *reinterpret_cast<uint4*>(tile + (r + i * down) * kPitch<T> + tx * n) = u[i];
      }
    } else {
      for (int r = ty; r < kTileRows; r += down)
        *reinterpret_cast<uint4*>(tile + r * kPitch<T> + tx * n) = load_piece<T>(p, r0 + r, c0 + tx * n);
    }
  }
  if (threadIdx.x < kTileCols) {
    float most = 0.f;
    if constexpr (kRowScaled<F>) {
      const int64_t c = c0 + threadIdx.x;
      if (c < p.cols)
#pragma unroll 8
        for (int i = 0; i < p.parts; ++i) most = larger(most, p.most[i * p.cols + c]);
      units[threadIdx.x] = row_unit<F>(most);
      if (row_tile == 0 && c < p.cols) p.row_scale[c] = units[threadIdx.x].scale;
    } else {
      units[threadIdx.x] = row_unit<F>(0.f);
    }
  }
  __syncthreads();
  const int warp = (int)threadIdx.x / 32, lane = (int)threadIdx.x % 32;
  const int64_t k0 = r0 + warp * 32;  // the operand's first column of this warp
  using Two = typename std::conditional<sizeof(T) == 2, uint32_t, float2>::type;
  Two both[32];  // two columns of a lane
#pragma unroll
  for (int j = 0; j < 32; ++j) both[j] = *reinterpret_cast<const Two*>(tile + (warp * 32 + j) * kPitch<T> + 2 * lane);
  float most[2][2];  // of either 16 rows, of either column
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (sizeof(T) == 2) {
      using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
      T2 m = __habs2(reinterpret_cast<const T2&>(both[16 * i]));
#pragma unroll
      for (int j = 1; j < 16; ++j) m = __hmax2_nan(m, __habs2(reinterpret_cast<const T2&>(both[16 * i + j])));
      most[i][0] = to_f32(m.x);
      most[i][1] = to_f32(m.y);
    } else {
      most[i][0] = most[i][1] = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        most[i][0] = larger(most[i][0], both[16 * i + j].x);
        most[i][1] = larger(most[i][1], both[16 * i + j].y);
      }
    }
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int col = 2 * lane + half;
    const int64_t c = c0 + col;
    const RowUnit row = units[col];
    const bool in = c < p.cols && k0 < p.width;
    if constexpr (kBlock<F> == 32) most[0][half] = most[1][half] = larger(most[0][half], most[1][half]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      BlockUnit b{0u, row.inv, 1.f};
      if constexpr (kBlock<F> != 0) {
        b = block_unit<F, sizeof(T) == 4>(most[i][half], row);
        if constexpr (kBlock<F> == 16) bytes[col][2 * warp + i] = (uint8_t)(in ? b.byte : 0u);
        if (kBlock<F> == 32 && i == 0) bytes[col][warp] = (uint8_t)(in ? b.byte : 0u);
      }
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = to_f32(reinterpret_cast<const T*>(&both[16 * i + j])[half]);
      if (in)
        store_codes<F, sizeof(T) == 4>(p.data + c * p.ld_data + (kFourBit<F> ? (k0 + 16 * i) / 2 : k0 + 16 * i), v, row, b);
    }
  }
  if constexpr (kBlock<F> != 0) {
    __syncthreads();
    constexpr int words = kTileRows / kBlock<F> / 4;  // scale words of a column
    const int64_t scale0 = r0 / kBlock<F>;
    for (int i = (int)threadIdx.x; i < kTileCols * words; i += kThreads) {
      const int col = i % kTileCols, word = i / kTileCols;
      if (scale0 / 4 + word < p.blocks)
        *reinterpret_cast<uint32_t*>(p.scales + scale_offset(c0 + col, scale0 + 4 * word, p.blocks)) =
            *reinterpret_cast<const uint32_t*>(&bytes[col][4 * word]);
    }
  }
}

template <typename T>
const void* columns_kernel(int format) {
  switch (format) {
    case QUANT_E4M3: return reinterpret_cast<const void*>(k_quant_columns<T, QUANT_E4M3>);
    case QUANT_MXE4M3: return reinterpret_cast<const void*>(k_quant_columns<T, QUANT_MXE4M3>);
    case QUANT_MXFP4: return reinterpret_cast<const void*>(k_quant_columns<T, QUANT_MXFP4>);
    default: return reinterpret_cast<const void*>(k_quant_columns<T, QUANT_NVFP4>);
  }
}

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Parts of the columns: enough CTAs for the device, of 64 rows at least.
int parts_of(int64_t rows, int64_t cols) {
  const int64_t strips = std::max<int64_t>(1, up(cols, kTileCols));
  return (int)std::max<int64_t>(1, std::min({up(4 * 152, strips), up(rows, 64), (int64_t)kMostParts}));
}

}  // namespace

size_t quant_columns_workspace(const quant_rows_t& a) {
  if (a.format != QUANT_E4M3 && a.format != QUANT_NVFP4) return 0;
  return (size_t)parts_of(a.rows, a.cols) * (size_t)a.cols * sizeof(float);
}

cudaError_t launch_quant_columns(const quant_rows_t& a, const FfnDevice&, cudaStream_t st) {
  const int e = a.dtype == FFN_F32 ? 4 : 2;
  QuantColumnsParams p{};
  p.rows = a.rows;
  p.cols = a.cols;
  p.width = width_of(a.rows);
  const int64_t scales = scales_of(p.width, a.format);
  p.blocks = (int32_t)up(scales, 4);
  p.vec = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.ld_x * e % 16 == 0;
  p.parts = parts_of(a.rows, a.cols);
  p.part_rows = up(a.rows, p.parts);
  p.x = a.x;
  p.data = static_cast<uint8_t*>(a.data);
  p.scales = static_cast<uint8_t*>(a.scales);
  p.row_scale = a.row_scale;
  p.most = static_cast<float*>(a.workspace);
  p.ld_x = a.ld_x;
  p.ld_data = a.ld_data;
  LaunchSpec s;
  s.block = dim3(kThreads, 1, 1);
  s.pdl = true;
  void* args[] = {&p};
  if (a.format == QUANT_E4M3 || a.format == QUANT_NVFP4) {
    s.func = a.dtype == FFN_F32    ? reinterpret_cast<const void*>(k_quant_column_most<float>)
             : a.dtype == FFN_BF16 ? reinterpret_cast<const void*>(k_quant_column_most<__nv_bfloat16>)
                                   : reinterpret_cast<const void*>(k_quant_column_most<__half>);
    s.grid = dim3((unsigned)up(a.cols, kTileCols), (unsigned)p.parts, 1);
    const cudaError_t err = launch_spec(s, args, st);
    if (err != cudaSuccess) return err;
  }
  s.func = a.dtype == FFN_F32    ? columns_kernel<float>(a.format)
           : a.dtype == FFN_BF16 ? columns_kernel<__nv_bfloat16>(a.format)
                                 : columns_kernel<__half>(a.format);
  // block scales: rows of the operand up to a whole block of 128 get zero bytes
  const int64_t strips = scales > 0 ? up(a.cols, 128) * (128 / kTileCols) : up(a.cols, kTileCols);
  p.row_tiles = (int32_t)up(p.width, kTileRows);
  s.grid = dim3((unsigned)(p.row_tiles * strips), 1, 1);
  s.smem = (size_t)kTileRows * (size_t)(e == 2 ? kPitch<__half> * 2 : kPitch<float> * 4);
  const cudaError_t err = allow_smem_once(s.func, s.smem);
  if (err != cudaSuccess) return err;
  return launch_spec(s, args, st);
}

}  // namespace dgb
