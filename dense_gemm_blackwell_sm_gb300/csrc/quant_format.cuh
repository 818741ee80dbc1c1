// quant_format.cuh -- how values become codes and scales, for every kernel that writes a
// quantised operand.  The formats are described in include/quant.h.
#pragma once

#include "ffn_common.cuh"
#include "quant.h"

namespace dgb {

template <int F>
inline constexpr bool kFourBit = F == QUANT_MXFP4 || F == QUANT_NVFP4;
template <int F>
inline constexpr bool kRowScaled = F == QUANT_E4M3 || F == QUANT_NVFP4;
// elements per block scale (0: none)
template <int F>
inline constexpr int kBlock = F == QUANT_E4M3 ? 0 : F == QUANT_NVFP4 ? 16 : 32;

constexpr uint32_t kInfBits = 0x7f800000u;

// Two fp32 operations at once
__device__ __forceinline__ void mul2(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "mul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}
__device__ __forceinline__ void mul2_rz(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "mul.rz.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}
// (a, b) = (x, y) * (u, v) + (a, b)
__device__ __forceinline__ void fma2(float& a, float& b, float x, float y, float u, float v) {
  asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmov.b64 r, {%4, %5};\n\t"
      "fma.rn.f32x2 p, q, r, p;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y), "f"(u), "f"(v));
}

// The larger magnitude; a NaN wins.  (Magnitudes are kept as floats: a NaN or an infinity
// among the values shows in the largest.)
__device__ __forceinline__ float larger(float most, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(most), "f"(fabsf(v)));
  return r;
}
__device__ __forceinline__ float larger(float most, float v, float w) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(most), "f"(v), "f"(w));
  return r;
}
__device__ __forceinline__ float largest16(const float (&v)[16]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 16; j += 2) m = larger(m, v[j], v[j + 1]);
  return m;
}
__device__ __forceinline__ bool finite(float magnitude) { return __float_as_uint(magnitude) < kInfBits; }

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127

// The smallest e with m <= top * 2^e, for top = (1 + over / 2^23) * 2^shift.  (A subnormal m
// gives a larger e; every user clamps e above it.)
__device__ __forceinline__ int covering(float m, int shift, uint32_t over) {
  const uint32_t bits = __float_as_uint(m);
  return (int)(bits >> 23) - 127 - shift + ((bits & 0x7fffffu) > over ? 1 : 0);
}

// ---------------------------------------------------------------- 16 elements

// codes of values already in units of their scale, the first one lowest
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ uint32_t e2m1x8(const float* t) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
  return r;
}

// What a row's scale is and what multiplies its values.
struct RowUnit {
  float scale;  // as written to row_scale
  float inv;    // E4M3: 1 / scale; NVFP4: 1 / row_scale, a power of two (0 where the row has no finite scale)
};
template <int F>
__device__ __forceinline__ RowUnit row_unit(float most) {
  RowUnit u{1.f, 1.f};
  if constexpr (F == QUANT_E4M3) {
    u.scale = fmaxf(__fdiv_rn(most, 448.f), 1.17549435e-38f);
    u.inv = __frcp_rn(u.scale);
  } else if constexpr (F == QUANT_NVFP4) {
    // 2688 = 1.3125 * 2^11
    const int k = most == 0.f ? 0 : max(covering(most, 11, 0x280000u), -100);
    u.scale = pow2(k);
    u.inv = pow2(-k);
  }
  if (kRowScaled<F> && !finite(most)) {
    u.scale = __uint_as_float(0x7fffffffu);
    u.inv = 0.f;
  }
  return u;
}

// A block's scale: the byte kept, and what multiplies the block's values.
struct BlockUnit {
  uint32_t byte;
  float inv;    // 0 where the values are to be 0 (NVFP4 in 32 bits: the scale's reciprocal alone)
  float scale;  // NVFP4 in 32 bits: the scale, to divide by
};
// The nearest float to 1 / s, for s an E4M3 value above 0: one Newton step from the approximate
// reciprocal.
__device__ __forceinline__ float reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return fmaf(r, fmaf(-r, s, 1.f), r);
}
// The smallest float not below it
__device__ __forceinline__ float reciprocal_up(float s) {
  const float r = reciprocal(s);
  return fmaf(r, s, -1.f) < 0.f ? __uint_as_float(__float_as_uint(r) + 1u) : r;
}

// v / s with r the nearest float to 1 / s: the product with r, corrected by its remainder, which is
// exact (Markstein's step).  Rounded to a few bits it goes where the exact quotient does: for a
// midpoint b of the codes b s is a float, so v = b s gives b, and any other v is a unit in its last
// place from b s at least, which is more than half a unit of b.  (A division takes a slow way for
// zeros, of which there are many: 300 x 520 fp32 to NVFP4 4.5 us with divisions, like
// this 2.0; 8192 x 4096 34 and 25.)
__device__ __forceinline__ float quotient(float v, float s, float r) {
  const float q = v * r;
  return fmaf(fmaf(-q, s, v), r, q);
}
__device__ __forceinline__ void quotient2(float& v, float& w, float s, float r) {
  const float v0 = v, w0 = w;
  float q0 = v, q1 = w;
  mul2(q0, q1, r, r);
  fma2(v, w, q0, q1, -s, -s);
  const uint32_t sv = __float_as_uint(v0) & 0x80000000u, sw = __float_as_uint(w0) & 0x80000000u;
  fma2(q0, q1, v, w, r, r);
  v = __uint_as_float(__float_as_uint(q0) | sv);  // (a zero keeps its sign)
  w = __uint_as_float(__float_as_uint(q1) | sw);
}

// EXACT: for 32-bit inputs, whose quotients may lie nearer to a tie than a reciprocal is exact.  (Not for
// what follows a norm, which is 32 bits wide too: its own rounding errors are as large as the
// reciprocals', 2^-22.)
template <int F, bool EXACT>
__device__ __forceinline__ BlockUnit block_unit(float most, const RowUnit& row) {
  BlockUnit b{0u, row.inv, 1.f};
  if constexpr (F == QUANT_MXE4M3 || F == QUANT_MXFP4) {
    // 448 = 1.75 * 2^8, 6 = 1.5 * 2^2
    const int e = most == 0.f ? -127
                              : max(F == QUANT_MXE4M3 ? covering(most, 8, 0x600000u) : covering(most, 2, 0x400000u), -127);
    b.byte = (uint32_t)(e + 127);
    b.inv = pow2(-e);
    if (!finite(most)) b = {255u, 0.f, 1.f};
  } else if constexpr (F == QUANT_NVFP4) {
    // (for 16-bit magnitudes a product with 1/6 rounded up, rounded towards zero, stays on a tie
    // that the quotient is on: see below)
    constexpr float kSixth = 0.166666671633720397949f;  // (the nearest float, above 1/6)
    const float q = EXACT ? quotient(most * row.inv, 6.f, kSixth) : __fmul_rz(most * row.inv, kSixth);
    uint32_t byte, half;
    asm("{\n\t.reg .b16 r;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 r, %2, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, r;\n\t"
        "cvt.u32.u16 %0, r;\n\t}"
        : "=r"(byte), "=r"(half)
        : "f"(q));
    b.byte = byte & 0xffu;
    b.scale = __half2float(__ushort_as_half((unsigned short)half));
    // The reciprocal rounded up and the products rounded towards zero: a value that lies on
    // the middle between two codes stays there (b * s * r is at least b and below b's
    // neighbour for every scale s and midpoint b), so that ties go to even as for the exact
    // quotient.  16-bit values that are no ties are 2^-11 from them at least.
    b.inv = b.byte == 0u ? 0.f : EXACT ? reciprocal(b.scale) : reciprocal_up(b.scale) * row.inv;
    if (row.inv == 0.f) b = {0x7fu, 0.f, 1.f};
  }
  return b;
}

// 16 values to codes: 4 words (E4M3) or 2 (E2M1).  EXACT: values that may lie nearer to a tie than
// the reciprocal is exact (32-bit inputs) get their quotients.
template <int F, bool EXACT>
__device__ __forceinline__ void codes16(uint32_t* w, const float (&v)[16], const RowUnit& row, const BlockUnit& b) {
  float t[16];
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    t[j] = v[j];
    t[j + 1] = v[j + 1];
    if constexpr (F == QUANT_NVFP4 && EXACT) {
      mul2(t[j], t[j + 1], row.inv, row.inv);
      quotient2(t[j], t[j + 1], b.scale, b.inv);
    } else if constexpr (F == QUANT_NVFP4) {
      mul2_rz(t[j], t[j + 1], b.inv, b.inv);
    } else {
      mul2(t[j], t[j + 1], b.inv, b.inv);
    }
  }
  const bool zero = b.inv == 0.f;  // (an infinity times 0 is no 0)
  if constexpr (kFourBit<F>) {
    w[0] = e2m1x8(t);
    w[1] = e2m1x8(t + 8);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = e4m3x4(t[4 * j], t[4 * j + 1], t[4 * j + 2], t[4 * j + 3]);
  }
  if (zero) {
#pragma unroll
    for (int j = 0; j < (kFourBit<F> ? 2 : 4); ++j) w[j] = 0u;
  }
}
// ... stored at `dst`
template <int F, bool EXACT>
__device__ __forceinline__ void store_codes(uint8_t* dst, const float (&v)[16], const RowUnit& row, const BlockUnit& b) {
  uint32_t w[kFourBit<F> ? 2 : 4];
  codes16<F, EXACT>(w, v, row, b);
  if constexpr (kFourBit<F>) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// byte offset of the tiled scale of row r, scale column c, of an array with `cb` blocks a row
__device__ __forceinline__ uint64_t scale_offset(uint32_t r, uint32_t c, uint32_t cb) {
  return ((uint64_t)(r >> 7) * cb + (c >> 2)) * 512u + (r & 31u) * 16u + ((r >> 5) & 3u) * 4u + (c & 3u);
}

}  // namespace dgb
