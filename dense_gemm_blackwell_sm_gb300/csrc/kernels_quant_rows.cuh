// kernels_quant_rows.cuh -- quantisation by rows, with or without the residual's addition
// and the RMS norm in front of it.
//
// A group of threads (a warp to 512 threads) takes a row; a thread holds NV runs of 16
// neighbouring columns in registers, so that a row is read once whatever its scales need:
//   norm:  s = rs * residual + bs * y,  r = 1 / sqrt(sum s^2 / D + eps),  v = s r weight
//   E4M3, NVFP4: the row's largest magnitude, from all its threads
//   block scales: the block's largest magnitude, from one thread (16) or two (32)
// and then the codes.  Rows longer than a group holds (no norm) are read twice.
//
// Bound by memory: 2 bytes read and 0.56 to 1.03 written per element (norm: 4 and 3.03).
#pragma once

#include "quant_format.cuh"

namespace dgb {

struct QuantRowsParams {
  int64_t rows;        // of the input
  int64_t all_rows;    // and of the scale array: rows past the last one get zero bytes
  int32_t cols;
  int32_t chunks;      // runs of 16 elements of a padded row
  int32_t all_chunks;  // and of the scale array's columns
  int32_t blocks;      // 512-byte scale blocks across a row
  int32_t vec;         // rows start on 16-byte boundaries
  const void* x;       // norm: y
  const void* residual;
  const void* weight;
  void* s;
  uint8_t* data;
  uint8_t* scales;
  float* row_scale;
  int64_t ld_x, ld_residual, ld_s, ld_data;
  int32_t weight_f32;  // weight is fp32 (else the inputs' type)
  int32_t weight_vec;
  float eps, residual_scale, branch_scale;
};

namespace {

// 16 columns from `col` on, zeros from column `cols` on (plain loads: s may be y or the residual)
template <typename T>
__device__ __forceinline__ void load16(float (&v)[16], const T* row, int32_t col, int32_t cols, bool vec) {
  if (vec && col + 16 <= cols) {
    if constexpr (sizeof(T) == 2) {
      const uint4* p = reinterpret_cast<const uint4*>(row + col);
      const uint4 a = p[0], b = p[1];
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[2 * j] = to_f32(reinterpret_cast<const T*>(&w[j])[0]);
        v[2 * j + 1] = to_f32(reinterpret_cast<const T*>(&w[j])[1]);
      }
    } else {
      const float4* p = reinterpret_cast<const float4*>(row + col);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 f = p[j];
        v[4 * j] = f.x;
        v[4 * j + 1] = f.y;
        v[4 * j + 2] = f.z;
        v[4 * j + 3] = f.w;
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = col + j < cols ? to_f32(row[col + j]) : 0.f;
}

template <typename T>
__device__ __forceinline__ void store16(T* row, const float (&v)[16], int32_t col, int32_t cols, bool vec) {
  if (vec && col + 16 <= cols) {
    if constexpr (sizeof(T) == 2) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        reinterpret_cast<T*>(&w[j])[0] = from_f32<T>(v[2 * j]);
        reinterpret_cast<T*>(&w[j])[1] = from_f32<T>(v[2 * j + 1]);
      }
      uint4* p = reinterpret_cast<uint4*>(row + col);
      p[0] = make_uint4(w[0], w[1], w[2], w[3]);
      p[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
      float4* p = reinterpret_cast<float4*>(row + col);
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (col + j < cols) row[col + j] = from_f32<T>(v[j]);
}

struct Sum {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Largest {
  __device__ __forceinline__ float operator()(float a, float b) const { return larger(a, b); }
};

// Over the threads of a row, in a fixed order.  Every thread of the CTA calls it.
template <typename Op>
__device__ __forceinline__ float over_row(float v, Op op, float* shared) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (blockDim.x == 32) return v;
  const int warps = (int)blockDim.x / 32;
  float* mine = shared + threadIdx.y * warps;
  if ((threadIdx.x & 31u) == 0) mine[threadIdx.x / 32] = v;
  __syncthreads();
  v = mine[0];
  for (int i = 1; i < warps; ++i) v = op(v, mine[i]);
  return v;
}

template <typename T, int F, bool NORM, int NV>
__global__ void __launch_bounds__(512) k_quant_rows(const QuantRowsParams p) {
  __shared__ float shared[2][16];
  wait_for_prior_kernel();
  let_next_kernel_start();
  const int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = r < p.rows;
  const int32_t threads = (int32_t)blockDim.x, tx = (int32_t)threadIdx.x;
  const T* x = reinterpret_cast<const T*>(p.x) + r * p.ld_x;
  const int32_t per = threads * NV;

  float v[NV][16];
  auto load = [&](int32_t base) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t c = base + i * threads + tx;
      if (live && c < p.chunks) {
        load16<T>(v[i], x, 16 * c, p.cols, p.vec != 0);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[i][j] = 0.f;
      }
    }
  };
  auto largest = [&](float most) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) most = larger(most, v[i][j]);
    return most;
  };

  load(0);
  if constexpr (NORM) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t c = i * threads + tx;
      if (!live || c >= p.chunks) continue;
#pragma unroll
      for (int j = 0; j < 16; ++j) v[i][j] *= p.branch_scale;
      if (p.residual != nullptr) {
        float e[16];
        load16<T>(e, reinterpret_cast<const T*>(p.residual) + r * p.ld_residual, 16 * c, p.cols, p.vec != 0);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[i][j] = fmaf(p.residual_scale, e[j], v[i][j]);
      }
      if (p.s != nullptr) store16<T>(reinterpret_cast<T*>(p.s) + r * p.ld_s, v[i], 16 * c, p.cols, p.vec != 0);
#pragma unroll
      for (int j = 0; j < 16; ++j) sum = fmaf(v[i][j], v[i][j], sum);
    }
    sum = over_row(sum, Sum{}, shared[0]);
    const float unit = __frsqrt_rn(sum / (float)p.cols + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t c = i * threads + tx;
      if (!live || c >= p.chunks) continue;
#pragma unroll
      for (int j = 0; j < 16; ++j) v[i][j] *= unit;
      if (p.weight != nullptr) {
        float e[16];
        if (p.weight_f32) {
          load16<float>(e, reinterpret_cast<const float*>(p.weight), 16 * c, p.cols, p.weight_vec != 0);
        } else {
          load16<T>(e, reinterpret_cast<const T*>(p.weight), 16 * c, p.cols, p.weight_vec != 0);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) v[i][j] *= e[j];
      }
    }
  }

  RowUnit row = row_unit<F>(0.f);
  if constexpr (kRowScaled<F>) {
    float most = largest(0.f);
    if constexpr (!NORM) {
      for (int32_t base = per; base < p.chunks; base += per) {
        load(base);
        most = largest(most);
      }
    }
    row = row_unit<F>(over_row(most, Largest{}, shared[1]));
    if (live && tx == 0) p.row_scale[r] = row.scale;
  }

  for (int32_t base = 0; base < p.all_chunks; base += per) {
    if (!NORM && (base > 0 || (kRowScaled<F> && per < p.chunks))) load(base);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t c = base + i * threads + tx;
      BlockUnit b{0u, row.inv, 1.f};
      if constexpr (kBlock<F> != 0) {
        float most = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) most = larger(most, v[i][j]);
        if constexpr (kBlock<F> == 32) most = larger(most, __shfl_xor_sync(0xffffffffu, most, 1));
        b = block_unit<F>(most, row);
        // four scales, of four or eight threads, are stored together
        constexpr int lanes = 4 * kBlock<F> / 16;
        uint32_t word = live && c < p.chunks ? b.byte << (8 * ((c * 16 / kBlock<F>) & 3)) : 0u;
#pragma unroll
        for (int o = kBlock<F> / 16; o < lanes; o *= 2) word |= __shfl_xor_sync(0xffffffffu, word, o);
        if (c % lanes == 0 && c < p.all_chunks && r < p.all_rows)
          *reinterpret_cast<uint32_t*>(p.scales + scale_offset(r, c * 16 / kBlock<F>, p.blocks)) = word;
      }
      if (live && c < p.chunks)
        store_codes<F, sizeof(T) == 4 && !NORM>(p.data + r * p.ld_data + (int64_t)c * (kFourBit<F> ? 8 : 16), v[i], row, b);
    }
  }
}

template <typename T, int F, bool NORM>
const void* rows_kernel(int nv) {
  switch (nv) {
    case 1: return reinterpret_cast<const void*>(k_quant_rows<T, F, NORM, 1>);
    case 2: return reinterpret_cast<const void*>(k_quant_rows<T, F, NORM, 2>);
    default: return reinterpret_cast<const void*>(k_quant_rows<T, F, NORM, 4>);
  }
}

template <typename T, bool NORM>
const void* rows_kernel_of(int format, int nv) {
  switch (format) {
    case QUANT_E4M3: return rows_kernel<T, QUANT_E4M3, NORM>(nv);
    case QUANT_MXE4M3: return rows_kernel<T, QUANT_MXE4M3, NORM>(nv);
    case QUANT_MXFP4: return rows_kernel<T, QUANT_MXFP4, NORM>(nv);
    default: return rows_kernel<T, QUANT_NVFP4, NORM>(nv);
  }
}

}  // namespace

// by the inputs' type (quant_rows_f16.cu and so on)
const void* quant_rows_f16(int format, bool norm, int nv);
const void* quant_rows_bf16(int format, bool norm, int nv);
const void* quant_rows_f32(int format, bool norm, int nv);

}  // namespace dgb
