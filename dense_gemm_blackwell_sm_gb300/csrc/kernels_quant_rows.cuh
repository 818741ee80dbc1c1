// kernels_quant_rows.cuh -- quantisation by rows, with or without the residual's addition
// and the RMS norm in front of it.
//
// A group of threads (a warp to 512 threads) takes a row; a thread holds NV runs of 16
// neighbouring columns in registers, so that a row is read once whatever its scales need:
//   norm:  s = rs * residual + bs * y,  r = 1 / sqrt(sum s^2 / D + eps),  v = s r weight
//   E4M3, NVFP4: the row's largest magnitude, from all its threads
//   block scales: the block's largest magnitude, from one thread (16) or two (32)
// and then the codes.  The grid is what the device holds at once: a group walks its rows and
// loads the next one before it works on the one it has.  Rows longer than a group holds (no
// norm) are read twice.
//
// Bound by memory: 2 bytes read and 0.53 to 1.03 written per element (norm: 4 and 2 more).  8192 x
// 4096 bf16: to E4M3 19.9 us, MXFP8 18.2 (5.6 TB/s), MXFP4 16.8, NVFP4 19.2; 8192 x 8192 33.7, 33.7 (6.0
// TB/s), 30.4 and 33.3; 4096 x 14336 29.1, 30.3, 26.5 and 29.6; the norm of 8192 x 4096 41.9, 39.3 (6.0 TB/s),
// 39.0 and 44.0.  fp32: 26 to 27.5 us (6.0 to 6.2 TB/s); the norm 64 to 70.  Rows of 4095 columns, off 16-byte
// boundaries, 24 to 30.  One row of 4096: 1.5 and 2.3 to 2.6 us, a launch and a row's latency.  (Launches
// of one graph over inputs in turn.)
#pragma once

#include <type_traits>

#include "quant_format.cuh"

namespace dgb {

struct QuantRowsParams {
  uint32_t rows;       // of the input
  uint32_t all_rows;   // and of the scale array: rows past the last one get zero bytes
  int32_t cols;
  int32_t chunks;      // runs of 16 elements of a padded row
  int32_t all_chunks;  // and of the scale array's columns
  int32_t blocks;      // 512-byte scale blocks across a row
  int32_t vec;         // rows start on boundaries of: 2 = 32 bytes, 1 = 16, 0 = neither
  const void* x;       // norm: y
  const void* residual;
  const void* weight;
  void* s;
  uint8_t* data;
  uint8_t* scales;
  float* row_scale;
  uint32_t ld_x, ld_residual, ld_s, ld_data;  // (below 2^31: an address is one wide multiplication)
  int32_t weight_f32;  // weight is fp32 (else the inputs' type)
  int32_t weight_vec;
  const void* x_end;   // the first byte past the last element of x, of the residual, of the weight
  const void* residual_end;
  const void* weight_end;
  float eps, residual_scale, branch_scale;
};

namespace {

// 16 columns as they are in memory
template <typename T>
struct Run {
  uint32_t w[4 * sizeof(T)];
  __device__ __forceinline__ float operator[](int j) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[j]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      return __uint_as_float((j & 1) ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    } else {
      return __half2float(__ushort_as_half((unsigned short)((j & 1) ? w[j / 2] >> 16 : w[j / 2])));
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < (int)(4 * sizeof(T)); ++j) w[j] = 0u;
  }
};

// The columns from `col` on, zeros from column `cols` on (plain loads: s may be y or the
// residual).  Rows off a 16-byte boundary (vec 0) come as the 16-byte pieces that hold the run,
// where those lie in the array [begin, end), and are shifted: 8192 x 4095 bf16 to MXFP8 takes
// 37 us by single elements.
template <typename T>
__device__ __forceinline__ void load16(Run<T>& v, const T* row, int32_t col, int32_t cols, int32_t vec,
                                       const void* begin, const void* end) {
  constexpr int words = 4 * (int)sizeof(T);
  if (vec != 0 && col + 16 <= cols) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(row + col);
    if (vec == 2) {
#pragma unroll
      for (int j = 0; j < words; j += 8)
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v.w[j]), "=r"(v.w[j + 1]), "=r"(v.w[j + 2]), "=r"(v.w[j + 3]), "=r"(v.w[j + 4]),
                       "=r"(v.w[j + 5]), "=r"(v.w[j + 6]), "=r"(v.w[j + 7])
                     : "l"(p + j)
                     : "memory");
    } else {
#pragma unroll
      for (int j = 0; j < words; j += 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(p + j);
        v.w[j] = u.x;
        v.w[j + 1] = u.y;
        v.w[j + 2] = u.z;
        v.w[j + 3] = u.w;
      }
    }
    return;
  }
  if (col >= cols) {  // (padding: nothing is there to load, and a row may have no values at all)
    v.clear();
    return;
  }
  const uintptr_t at = reinterpret_cast<uintptr_t>(row + col), first = at & ~(uintptr_t)15;
  if (first >= reinterpret_cast<uintptr_t>(begin) && first + 16 * sizeof(T) + 16 <= reinterpret_cast<uintptr_t>(end)) {
    uint32_t w[words + 4];
#pragma unroll
    for (int j = 0; j < words + 4; j += 4) {
      const uint4 u = *reinterpret_cast<const uint4*>(first + 4 * j);
      w[j] = u.x;
      w[j + 1] = u.y;
      w[j + 2] = u.z;
      w[j + 3] = u.w;
    }
    const uint32_t off = (uint32_t)(at & 15u);
#pragma unroll
    for (int j = 0; j < words + 2; ++j) w[j] = (off & 8u) != 0u ? w[j + 2] : w[j];
#pragma unroll
    for (int j = 0; j < words + 1; ++j) w[j] = (off & 4u) != 0u ? w[j + 1] : w[j];
#pragma unroll
    for (int j = 0; j < words; ++j) v.w[j] = sizeof(T) == 2 && (off & 2u) != 0u ? __funnelshift_r(w[j], w[j + 1], 16) : w[j];
    if (col + 16 > cols) {
      constexpr int per = 4 / (int)sizeof(T);  // columns of a word
#pragma unroll
      for (int j = 0; j < words; ++j) {
        if (col + per * j >= cols) v.w[j] = 0u;
        else if (per == 2 && col + per * j + 1 >= cols) v.w[j] &= 0xffffu;
      }
    }
    return;
  }
  T e[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) e[j] = col + j < cols ? row[col + j] : from_f32<T>(0.f);
#pragma unroll
  for (int j = 0; j < words; ++j) {
    if constexpr (sizeof(T) == 4) {
      v.w[j] = __float_as_uint(e[j]);
    } else {
      v.w[j] = (uint32_t)reinterpret_cast<const uint16_t&>(e[2 * j]) |
               (uint32_t)reinterpret_cast<const uint16_t&>(e[2 * j + 1]) << 16;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store16(T* row, const float (&v)[16], int32_t col, int32_t cols, int32_t vec) {
  if (vec != 0 && col + 16 <= cols) {
    constexpr int words = 4 * (int)sizeof(T);
    uint32_t w[words];
#pragma unroll
    for (int j = 0; j < words; ++j) {
      if constexpr (sizeof(T) == 4) {
        w[j] = __float_as_uint(v[j]);
      } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        w[j] = pack_bf16x2(__float_as_uint(v[2 * j]), __float_as_uint(v[2 * j + 1]));
      } else {
        const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    uint32_t* p = reinterpret_cast<uint32_t*>(row + col);
    if (vec == 2) {
#pragma unroll
      for (int j = 0; j < words; j += 8) st_global_v8(p + j, w + j);
    } else {
#pragma unroll
      for (int j = 0; j < words; j += 4) *reinterpret_cast<uint4*>(p + j) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (col + j < cols) row[col + j] = from_f32<T>(v[j]);
}

// A row's sum or largest magnitude from all its threads, in a fixed order.  Every thread of the
// row calls it; `shared` (a float per warp of the CTA) is another one than in the call before.
template <bool LARGEST>
__device__ __forceinline__ float over_warp(float v, int lanes) {
  if constexpr (LARGEST) {
    // (magnitudes order as their bits do, a NaN above an infinity)
    uint32_t r;
    asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(r) : "r"(__float_as_uint(v)));
    return __uint_as_float(r);
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
}
template <bool LARGEST>
__device__ __forceinline__ float over_row(float v, float* shared) {
  v = over_warp<LARGEST>(v, 32);
  if (blockDim.x == 32) return v;
  const uint32_t warps = blockDim.x / 32u, lane = threadIdx.x & 31u;
  float* mine = shared + threadIdx.y * warps;
  if (lane == 0) mine[threadIdx.x / 32u] = v;
  asm volatile("barrier.sync %0, %1;" ::"r"(threadIdx.y + 1u), "r"(blockDim.x) : "memory");  // (the row's threads)
  // (at most 16 warps)
  return over_warp<LARGEST>((lane & 15u) < warps ? mine[lane & 15u] : 0.f, 16);
}

// Registers a thread, for as many warps an SM as hide a row's steps behind one another: 16-bit rows of
// one run a thread take 40 (8192 x 4096 to MXFP8 17.2 us, with 48 17.5, with 56 18.6, with 36 and spills
// 20.6), of two 72, so that two CTAs of 448 threads fit (4096 x 14336 to MXFP8 28.5, with 77 34.3).  NVFP4's
// two runs need 99: WIDE are those that take what they need, for the rows that quant_rows.cu leaves
// them.  A norm of 16-bit rows needs 64.
template <typename T, bool NORM, int NV, bool WIDE>
constexpr int kRowRegisters = NV == 1 && sizeof(T) == 2            ? (NORM ? 64 : 40)
                              : NV == 1 && !NORM                   ? 64
                              : NV == 2 && sizeof(T) == 2 && !WIDE ? 72
                                                                   : 128;

template <typename T, int F, bool NORM, int NV, bool WIDE = NV == 2 && F == QUANT_NVFP4>
__global__ void __maxnreg__((kRowRegisters<T, NORM, NV, WIDE>)) k_quant_rows(const QuantRowsParams p) {
  constexpr bool AHEAD = NORM ? NV == 1 : NV <= 2;  // the next row's loads are under way while this one is worked on
  __shared__ float shared[2][2][16];
  wait_for_prior_kernel();
  let_next_kernel_start();
  const int32_t threads = (int32_t)blockDim.x, tx = (int32_t)threadIdx.x;
  const int32_t per = threads * NV;
  const uint32_t step = gridDim.x * blockDim.y;

  Run<T> raw[NV], raw_res[NORM ? NV : 1];
  auto load = [&](uint32_t r, int32_t base) {
    const T* x = reinterpret_cast<const T*>(p.x) + (uint64_t)r * p.ld_x;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t c = base + i * threads + tx;
      const bool in = r < p.rows && c < p.chunks;
      if (in) load16<T>(raw[i], x, 16 * c, p.cols, p.vec, p.x, p.x_end);
      else raw[i].clear();
      if constexpr (NORM) {
        if (in && p.residual != nullptr) {
          load16<T>(raw_res[i], reinterpret_cast<const T*>(p.residual) + (uint64_t)r * p.ld_residual, 16 * c, p.cols, p.vec,
                    p.residual, p.residual_end);
        } else {
          raw_res[i].clear();
        }
      }
    }
  };

  uint32_t turn = 0;
  const uint32_t row0 = blockIdx.x * blockDim.y;
  if (AHEAD) load(row0 + threadIdx.y, 0);
  for (uint32_t r0 = row0; r0 < p.all_rows; r0 += step, turn ^= 1u) {
    const uint32_t r = r0 + threadIdx.y;
    const bool live = r < p.rows;
    if (!AHEAD) load(r, 0);
    float v[NV][16], most[NV];  // (and each run's largest magnitude)
    auto take = [&]() {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) v[i][j] = raw[i][j];
    };
    auto find = [&](float of_row) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        most[i] = largest16(v[i]);
        of_row = larger(of_row, most[i]);
      }
      return of_row;
    };
    take();
    if constexpr (NORM) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          mul2(v[i][j], v[i][j + 1], p.branch_scale, p.branch_scale);
          fma2(v[i][j], v[i][j + 1], raw_res[i][j], raw_res[i][j + 1], p.residual_scale, p.residual_scale);
        }
    }
    if (AHEAD && (NORM || p.chunks <= per)) load(r + step, 0);
    if constexpr (NORM) {
      float sum = 0.f, sum1 = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int32_t c = i * threads + tx;
        if (live && c < p.chunks && p.s != nullptr)
          store16<T>(reinterpret_cast<T*>(p.s) + (uint64_t)r * p.ld_s, v[i], 16 * c, p.cols, p.vec);
#pragma unroll
        for (int j = 0; j < 16; j += 2) fma2(sum, sum1, v[i][j], v[i][j + 1], v[i][j], v[i][j + 1]);
      }
      sum = over_row<false>(sum + sum1, shared[0][turn]);
      const float unit = __frsqrt_rn(sum / (float)p.cols + p.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 16; j += 2) mul2(v[i][j], v[i][j + 1], unit, unit);
      // (the weight behind the factor: n may be a number where s weight is none.  Multiplied in first, while
      // the row's sum is found, 16-bit rows take 41.5 us for 8192 x 4096 to MXFP8 where this takes 39.0, and
      // 4.9 for 512 x 4096 where this takes 5.1.)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int32_t c = i * threads + tx;
        auto scale = [&](const auto& e) {
#pragma unroll
          for (int j = 0; j < 16; j += 2) mul2(v[i][j], v[i][j + 1], e[j], e[j + 1]);
        };
        if (c >= p.chunks || p.weight == nullptr) continue;
        if (p.weight_f32) {
          Run<float> e;
          load16<float>(e, reinterpret_cast<const float*>(p.weight), 16 * c, p.cols, p.weight_vec, p.weight, p.weight_end);
          scale(e);
        } else {
          Run<T> e;
          load16<T>(e, reinterpret_cast<const T*>(p.weight), 16 * c, p.cols, p.weight_vec, p.weight, p.weight_end);
          scale(e);
        }
      }
    }

    RowUnit row = row_unit<F>(0.f);
    if constexpr (kRowScaled<F>) {
      float of_row = find(0.f);
      if constexpr (!NORM) {
        for (int32_t base = per; base < p.chunks; base += per) {
          load(r, base);
          take();
          of_row = find(of_row);
        }
      }
      row = row_unit<F>(over_row<true>(of_row, shared[1][turn]));
      if (live && tx == 0) p.row_scale[r] = row.scale;
    }

    for (int32_t base = 0; base < p.all_chunks; base += per) {
      if (!NORM && (base > 0 || (kRowScaled<F> && per < p.chunks))) {
        load(r, base);
        take();
        if constexpr (kBlock<F> != 0) find(0.f);
      } else if constexpr (kBlock<F> != 0 && !kRowScaled<F>) {
        find(0.f);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int32_t c = base + i * threads + tx;
        BlockUnit b{0u, row.inv, 1.f};
        if constexpr (kBlock<F> != 0) {
          if constexpr (kBlock<F> == 32) most[i] = larger(most[i], __shfl_xor_sync(0xffffffffu, most[i], 1));
          b = block_unit<F, sizeof(T) == 4 && !NORM>(most[i], row);
          // four scales, of four or eight threads, are stored together
          constexpr int lanes = 4 * kBlock<F> / 16;
          uint32_t word = live && c < p.chunks ? b.byte << (8 * ((c * 16 / kBlock<F>) & 3)) : 0u;
#pragma unroll
          for (int o = kBlock<F> / 16; o < lanes; o *= 2) word |= __shfl_xor_sync(0xffffffffu, word, o);
          if (c % lanes == 0 && c < p.all_chunks && r < p.all_rows)
            *reinterpret_cast<uint32_t*>(p.scales + scale_offset(r, c * 16 / kBlock<F>, p.blocks)) = word;
        }
        if (live && c < p.chunks)
          store_codes<F, sizeof(T) == 4 && !NORM>(
              p.data + (uint64_t)r * p.ld_data + (uint32_t)c * (kFourBit<F> ? 8u : 16u), v[i], row, b);
      }
    }
    if (AHEAD && !NORM && p.chunks > per) load(r + step, 0);
  }
}

template <typename T, int F, bool NORM>
const void* rows_kernel(int nv, bool bounded) {
  if (nv == 1) return reinterpret_cast<const void*>(k_quant_rows<T, F, NORM, 1>);
  if constexpr (!NORM) {
    if constexpr (sizeof(T) == 2 && F == QUANT_NVFP4)
      if (nv == 2 && bounded) return reinterpret_cast<const void*>(k_quant_rows<T, F, NORM, 2, false>);
    if (nv == 2) return reinterpret_cast<const void*>(k_quant_rows<T, F, NORM, 2>);
  }
  return reinterpret_cast<const void*>(k_quant_rows<T, F, NORM, 4>);
}

template <typename T, bool NORM>
const void* rows_kernel_of(int format, int nv, bool bounded) {
  switch (format) {
    case QUANT_E4M3: return rows_kernel<T, QUANT_E4M3, NORM>(nv, bounded);
    case QUANT_MXE4M3: return rows_kernel<T, QUANT_MXE4M3, NORM>(nv, bounded);
    case QUANT_MXFP4: return rows_kernel<T, QUANT_MXFP4, NORM>(nv, bounded);
    default: return rows_kernel<T, QUANT_NVFP4, NORM>(nv, bounded);
  }
}

}  // namespace

// by the inputs' type (kernels_quant_rows_f16.cu and so on)
const void* quant_rows_f16(int format, bool norm, int nv, bool bounded);
const void* quant_rows_bf16(int format, bool norm, int nv, bool bounded);
const void* quant_rows_f32(int format, bool norm, int nv, bool bounded);

}  // namespace dgb
