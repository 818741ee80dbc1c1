// kernel_quant_columns.cu -- quantisation by columns: the operand of x^T, whose rows are x's
// columns.
//
// A CTA takes 256 rows x 64 columns of x through shared memory; a warp then takes 32 of the
// rows, which are one block of 32 or two of 16 of every column, and a lane two columns, whose
// codes (16 bytes of 4-bit ones or 32 of 8-bit ones) meet those of the other warps in shared memory.
// Where a column has a scale of its own, a first kernel finds the largest magnitudes of
// parts of the columns; x is then read twice, the second time from its end, which L2 still holds,
// and before that kernel has ended.
// Up to kTasks arrays go in one launch.
//
// Bound by memory: 2 bytes read per element, 0.53 to 1.03 written.  14336 x 4096 bf16: to MXFP8
// 32.8 us (5.4 TB/s), MXFP4 28.9; with a scale per column (read twice) 53, and 515 x 1097 9 where
// one kernel takes 6.  8192 x 4096 fp32 33 to 35, with a scale per column 57 to 61.  (Persistent CTAs
// that copy the next tile while they work on one gain nothing.)  Held whole in the shared memory of a
// cluster, so that they are read once, columns take longer: loads, the exchange of the magnitudes and
// the codes then follow one another (14336 x 4096 66 to 77 us).
#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "quant_format.cuh"
#include "quant_launch.h"

namespace dgb {

namespace {

constexpr int kTileRows = 256, kTileCols = 64;
constexpr int kThreads = 256;
constexpr int kMostParts = 32;     // parts of a column whose largest magnitudes are found apart
constexpr int kTasks = kQuantColumnTasks;

struct QuantColumnsTask {
  int64_t rows, cols;       // of x
  int64_t width;            // elements of the operand's rows (rows of x, padded)
  int32_t blocks;           // 512-byte scale blocks across one of them
  int32_t vec;              // x's rows start on 16-byte boundaries
  int32_t parts;
  int32_t row_tiles;
  int32_t strips;           // of 64 columns that x has
  int32_t all_strips;       // and that the scale array's rows have
  int64_t part_rows;
  const void* x;
  const void* x_end;        // the first byte past x's last element
  uint8_t* data;
  uint8_t* scales;
  float* row_scale;
  float* most;              // parts x cols
  int64_t ld_x, ld_data;
};

struct QuantColumnsParams {
  QuantColumnsTask task[kTasks];
  uint32_t first_most[kTasks + 1], first_tile[kTasks + 1];  // CTAs before each task's
};

// the task of this CTA, and its CTA there
__device__ __forceinline__ const QuantColumnsTask& task_of(const QuantColumnsParams& q, const uint32_t* first,
                                                           uint32_t& cta) {
  int t = 0;
#pragma unroll
  for (int i = 1; i < kTasks; ++i) t += blockIdx.x >= first[i] ? 1 : 0;
  cta = blockIdx.x - first[t];
  return q.task[t];
}

// 16 bytes of row r from column `col` on, zeros outside the array.  Off a boundary they come as the
// two aligned pieces that hold them, where those lie in the array.
template <typename T>
__device__ __forceinline__ uint4 load_piece(const QuantColumnsTask& p, int64_t r, int64_t col) {
  constexpr int n = 16 / (int)sizeof(T);
  const T* row = reinterpret_cast<const T*>(p.x) + r * p.ld_x;
  union {
    T e[n];
    uint4 u;
  } piece;
  piece.u = make_uint4(0u, 0u, 0u, 0u);
  if (r < p.rows && col + n <= p.cols) {
    if (p.vec) return __ldg(reinterpret_cast<const uint4*>(row + col));
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + col), first = at & ~(uintptr_t)15;
    if (first >= reinterpret_cast<uintptr_t>(p.x) && first + 32 <= reinterpret_cast<uintptr_t>(p.x_end)) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(first)), b = __ldg(reinterpret_cast<const uint4*>(first) + 1);
      uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      const uint32_t off = (uint32_t)(at & 15u);
#pragma unroll
      for (int j = 0; j < 6; ++j) w[j] = (off & 8u) != 0u ? w[j + 2] : w[j];
#pragma unroll
      for (int j = 0; j < 5; ++j) w[j] = (off & 4u) != 0u ? w[j + 1] : w[j];
      if (sizeof(T) == 2 && (off & 2u) != 0u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], 16);
      }
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
#pragma unroll
  for (int j = 0; j < n; ++j)
    if (r < p.rows && col + j < p.cols) piece.e[j] = row[col + j];
  return piece.u;
}

// Whether rows r0 .. r0 + n and columns c0 .. c0 + 63 are whole and aligned
__device__ __forceinline__ bool inside(const QuantColumnsTask& p, int64_t r0, int64_t n, int64_t c0) {
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

// the largest magnitudes of a part of 64 columns
template <typename T>
__global__ void __launch_bounds__(kThreads) k_quant_column_most(const __grid_constant__ QuantColumnsParams q) {
  constexpr int n = 16 / (int)sizeof(T), across = kTileCols / n, down = kThreads / across, U = 8;
  __shared__ float found[down][kTileCols + 1];
  wait_for_prior_kernel();
  let_next_kernel_start();
  uint32_t cta;
  const QuantColumnsTask& p = task_of(q, q.first_most, cta);
  const int64_t part = cta / (uint32_t)p.strips, strip = cta - part * p.strips;
  const int tx = (int)threadIdx.x % across, ty = (int)threadIdx.x / across;
  const int64_t c0 = strip * kTileCols;
  const int64_t r0 = part * p.part_rows, r1 = min(p.rows, r0 + p.part_rows);
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
    p.most[part * p.cols + c] = m;
  }
}

template <typename T>
constexpr int kPitch = kTileCols + (sizeof(T) == 2 ? 8 : 4);  // elements: 16-byte pieces, lanes on different banks

// two columns of 16 rows as a lane reads them, and the larger magnitudes of both
template <typename T>
struct Columns16 {
  using Two = typename std::conditional<sizeof(T) == 2, uint32_t, float2>::type;
  Two w[16];
  __device__ __forceinline__ void load(const T* tile) {
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = *reinterpret_cast<const Two*>(tile + j * kPitch<T>);
  }
  __device__ __forceinline__ void most(float (&m)[2]) const {
    if constexpr (sizeof(T) == 2) {
      using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
      T2 a = __habs2(reinterpret_cast<const T2&>(w[0]));
#pragma unroll
      for (int j = 1; j < 16; ++j) a = __hmax2_nan(a, __habs2(reinterpret_cast<const T2&>(w[j])));
      m[0] = to_f32(a.x);
      m[1] = to_f32(a.y);
    } else {
      m[0] = m[1] = 0.f;
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        m[0] = larger(m[0], w[j].x, w[j + 1].x);
        m[1] = larger(m[1], w[j].y, w[j + 1].y);
      }
    }
  }
  __device__ __forceinline__ void column(float (&v)[16], int half) const {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if constexpr (sizeof(T) == 4) {
        v[j] = half ? w[j].y : w[j].x;
      } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        v[j] = __uint_as_float(half ? w[j] & 0xffff0000u : w[j] << 16);
      } else {
        v[j] = __half2float(__ushort_as_half((unsigned short)(half ? w[j] >> 16 : w[j])));
      }
    }
  }
};

template <typename T, int F>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 2 : 4)
    k_quant_columns(const __grid_constant__ QuantColumnsParams q) {
  constexpr int n = 16 / (int)sizeof(T), across = kTileCols / n, down = kThreads / across;
  constexpr int kRuns = kTileRows / 16;          // of 16 rows, a byte of a scale each (or of two)
  constexpr int kWords = kFourBit<F> ? 2 : 4;    // of a run's codes
  extern __shared__ __align__(16) uint8_t smem[];
  T* tile = reinterpret_cast<T*>(smem);
  __shared__ uint8_t bytes[kRuns][kTileCols];
  __shared__ RowUnit units[kTileCols];
  // Where the kernel before found the largest magnitudes, its CTAs had all waited for what came
  // before them when this one was placed: x may be read at once, those values when it has ended.
  if constexpr (!kRowScaled<F>) wait_for_prior_kernel();
  uint32_t cta;
  const QuantColumnsTask& p = task_of(q, q.first_tile, cta);
  const int64_t row_tile = p.row_tiles - 1 - (int64_t)(cta / (uint32_t)p.all_strips);
  const int64_t strip = cta % (uint32_t)p.all_strips;
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
#pragma unroll 4
      for (int r = ty; r < kTileRows; r += down)
        *reinterpret_cast<uint4*>(tile + r * kPitch<T> + tx * n) = load_piece<T>(p, r0 + r, c0 + tx * n);
    }
  }
  if constexpr (kRowScaled<F>) wait_for_prior_kernel();
  let_next_kernel_start();
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
  const T* mine = tile + warp * 32 * kPitch<T> + 2 * lane;
  Columns16<T> run[2];
  float most[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    run[i].load(mine + 16 * i * kPitch<T>);
    run[i].most(most[i]);
  }
  // The codes of a column meet in shared memory, where the tile was, and go out as whole lines: a
  // lane's 16 or 32 bytes of a column stored by itself are four times as many requests (14336 x 4096
  // MXFP4 30.8 -> 28.9 us, NVFP4 54.0 -> 52.9).
  constexpr int kCodes = kFourBit<F> ? kTileRows / 2 : kTileRows;  // bytes of a column
  constexpr int kCodesPitch = kCodes + 16;
  static_assert(kTileCols * kCodesPitch <= kTileRows * kPitch<T> * (int)sizeof(T), "the codes fit the tile");
  __syncthreads();
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const RowUnit row = units[2 * lane + half];
    if constexpr (kBlock<F> == 32) most[0][half] = most[1][half] = larger(most[0][half], most[1][half]);
    uint32_t codes[2 * kWords];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      BlockUnit b{0u, row.inv, 1.f};
      if constexpr (kBlock<F> != 0) {
        b = block_unit<F, sizeof(T) == 4>(most[i][half], row);
        bytes[warp * 2 + i][2 * lane + half] = (uint8_t)b.byte;
      }
      float v[16];
      run[i].column(v, half);
      codes16<F, sizeof(T) == 4>(codes + i * kWords, v, row, b);
    }
#pragma unroll
    for (int j = 0; j < 2 * kWords; j += 4)
      *reinterpret_cast<uint4*>(smem + (2 * lane + half) * kCodesPitch + warp * (kCodes / 8) + 4 * j) =
          make_uint4(codes[j], codes[j + 1], codes[j + 2], codes[j + 3]);
  }
  __syncthreads();
  {
    constexpr int kPieces = kCodes / 16;
    const int64_t first = kFourBit<F> ? r0 / 2 : r0, all = kFourBit<F> ? p.width / 2 : p.width;
#pragma unroll
    for (int i = 0; i < kTileCols * kPieces; i += kThreads) {
      const int col = (i + (int)threadIdx.x) / kPieces, piece = (int)threadIdx.x % kPieces;
      if (c0 + col < p.cols && first + 16 * piece < all)
        *reinterpret_cast<uint4*>(p.data + (c0 + col) * p.ld_data + first + 16 * piece) =
            *reinterpret_cast<const uint4*>(smem + col * kCodesPitch + 16 * piece);
    }
  }
  if constexpr (kBlock<F> != 0) {
    constexpr int kPer = kBlock<F> / 16;           // runs of a scale
    constexpr int words = kRuns / kPer / 4;        // scale words of a column
    const int64_t scale0 = r0 / kBlock<F>;
    for (int i = (int)threadIdx.x; i < kTileCols * words; i += kThreads) {
      const int col = i % kTileCols, word = i / kTileCols;
      if (scale0 / 4 + word >= p.blocks) continue;
      uint32_t w = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int s = 4 * word + j;
        // (no scale in rows behind the last column, or in columns behind the last block)
        if (c0 + col < p.cols && (scale0 + s) * kBlock<F> < p.width) w |= (uint32_t)bytes[s * kPer][col] << (8 * j);
      }
      *reinterpret_cast<uint32_t*>(p.scales + scale_offset(c0 + col, scale0 + 4 * word, p.blocks)) = w;
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

bool row_scaled(int32_t format) { return format == QUANT_E4M3 || format == QUANT_NVFP4; }

// Parts of the columns: enough CTAs for the device, of 64 rows at least.
int parts_of(int64_t rows, int64_t cols) {
  const int64_t strips = std::max<int64_t>(1, up(cols, kTileCols));
  return (int)std::max<int64_t>(1, std::min({up(4 * 152, strips), up(rows, 64), (int64_t)kMostParts}));
}

}  // namespace

size_t quant_columns_workspace(const quant_rows_t& a) {
  return row_scaled(a.format) ? (size_t)parts_of(a.rows, a.cols) * (size_t)a.cols * sizeof(float) : 0;
}

cudaError_t launch_quant_columns(const quant_rows_t* args, int count, cudaStream_t st) {
  const int32_t dtype = args[0].dtype, format = args[0].format;
  const int e = dtype == FFN_F32 ? 4 : 2;
  QuantColumnsParams q{};
  uint64_t most = 0, tiles = 0;
  for (int i = 0; i < kTasks; ++i) {
    q.first_most[i] = (uint32_t)most;
    q.first_tile[i] = (uint32_t)tiles;
    if (i >= count) {
      // (no CTA belongs to it)
      q.first_most[i] = q.first_tile[i] = 0xffffffffu;
      continue;
    }
    const quant_rows_t& a = args[i];
    QuantColumnsTask& p = q.task[i];
    p.rows = a.rows;
    p.cols = a.cols;
    p.width = width_of(a.rows);
    const int64_t scales = scales_of(p.width, a.format);
    p.blocks = (int32_t)up(scales, 4);
    p.vec = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.ld_x * e % 16 == 0;
    p.parts = parts_of(a.rows, a.cols);
    p.part_rows = up(a.rows, p.parts);
    p.strips = (int32_t)up(a.cols, kTileCols);
    p.row_tiles = (int32_t)up(p.width, kTileRows);
    p.x = a.x;
    p.x_end = end_of_rows(a.x, a.rows, a.ld_x, a.cols, e);
    p.data = static_cast<uint8_t*>(a.data);
    p.scales = static_cast<uint8_t*>(a.scales);
    p.row_scale = a.row_scale;
    p.most = static_cast<float*>(a.workspace);
    p.ld_x = a.ld_x;
    p.ld_data = a.ld_data;
    most += (uint64_t)p.strips * (uint64_t)p.parts;
    // (block scales: rows of the operand up to a whole block of 128 get zero bytes)
    p.all_strips = scales > 0 ? (int32_t)(up(a.cols, 128) * (128 / kTileCols)) : p.strips;
    tiles += (uint64_t)p.row_tiles * (uint64_t)p.all_strips;
  }
  if (tiles >= 0x7fffffffu) return cudaErrorInvalidValue;  // (each task fits: see quant.cu)
  LaunchSpec s;
  s.pdl = true;
  s.block = dim3(kThreads, 1, 1);
  void* params[] = {&q};
  if (row_scaled(format)) {
    s.func = dtype == FFN_F32    ? reinterpret_cast<const void*>(k_quant_column_most<float>)
             : dtype == FFN_BF16 ? reinterpret_cast<const void*>(k_quant_column_most<__nv_bfloat16>)
                                 : reinterpret_cast<const void*>(k_quant_column_most<__half>);
    s.grid = dim3((unsigned)most, 1, 1);
    const cudaError_t err = launch_spec(s, params, st);
    if (err != cudaSuccess) return err;
  }
  s.func = dtype == FFN_F32    ? columns_kernel<float>(format)
           : dtype == FFN_BF16 ? columns_kernel<__nv_bfloat16>(format)
                               : columns_kernel<__half>(format);
  s.grid = dim3((unsigned)tiles, 1, 1);
  s.smem = (size_t)kTileRows * (size_t)(e == 2 ? kPitch<__half> * 2 : kPitch<float> * 4);
  const cudaError_t err = allow_smem_once(s.func, s.smem);
  if (err != cudaSuccess) return err;
  return launch_spec(s, params, st);
}

}  // namespace dgb
