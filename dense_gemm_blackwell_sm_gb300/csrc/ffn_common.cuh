// ffn_common.cuh -- element types and activations (with derivatives) shared by
// the feed-forward block's kernels.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kernel_common.cuh"

namespace dgb {

// These kernels launch as programmatic dependents.  Each waits for the kernel before it
// ahead of its first access to global memory, and lets the next one be placed only after
// that wait, those that fill the SMs for long (tiles, the slopes' pass) when their own
// work is done: so at most two of them are on the device at once, and none stands beside
// a long one for its whole run.  (While every kernel let the next one start at its own
// start, a row of gradient calls queued behind other work could stop: erf GeLU, kept
// pre-activations, 4096 x 14336 x 4096.  No kernel here waits for a later one, and what
// stopped was not found by reading; with this order the same calls run.)
__device__ __forceinline__ void wait_for_prior_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The normal distribution p and e = e^(-g^2/2).  Its lower tail is
//   e t R(t),  t = 1 / (1 + 0.3 |g|),
// where R is smooth on (0, 1]: a polynomial of degree 7, fitted by reweighted least squares
// to the smallest relative error, 1.3e-7 for |g| <= 13.6 (beyond, e is below 2^-126).  So
// the tail is right to fp32 rounding of its own size; (1 + erf(g / sqrt 2)) / 2 cancels
// there (4 % off at g = -5, zero from -5.6 on), and erfcf costs an epilogue 12 to 18 %
// (8192 x 2048 x 1024: 54.0 us with erff, 63.6 with erfcf, 50.4 with this).
__device__ __forceinline__ void normal(float g, float& p, float& e) {
  float t;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.3f, fabsf(g), 1.f)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * g * -0.7213475204444817f));
  float r = 0.03587991f;
  r = fmaf(r, t, -0.158059299f);
  r = fmaf(r, t, 0.207831666f);
  r = fmaf(r, t, -0.0550470725f);
  r = fmaf(r, t, 0.129284695f);
  r = fmaf(r, t, 0.0996937826f);
  r = fmaf(r, t, 0.120789267f);
  r = fmaf(r, t, 0.119626991f);
  const float tail = r * t * e;
  p = g < 0.f ? tail : 1.f - tail;
}

// The activation a = act(g) and its derivative d.  SiLU and the tanh form of
// GeLU go through the logistic function s as in the fused GEMM epilogue:
//   silu: a = g s(g),   d = s + a (1 - s)
//   gelu (tanh): a = g s(v), v = 2 sqrt(2/pi) (g + c g^3),  d = s + a (1 - s) v'
// v' is taken at g clamped to [-16, 16], where s (1 - s) is already exactly 0,
// so that its square does not overflow; a NaN still arrives through s.
template <int ACT>
__device__ __forceinline__ void act_and_slope(float g, float& a, float& d) {
  if constexpr (ACT == EPI_ACT_RELU) {
    a = g < 0.f ? 0.f : g;  // (a NaN stays one)
    d = g > 0.f ? 1.f : 0.f;
  } else if constexpr (ACT == EPI_ACT_SILU) {
    const float s = logistic(g);
    a = g * s;
    d = fmaf(a, 1.f - s, s);
  } else if constexpr (ACT == EPI_ACT_GELU_TANH) {
    const float k2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float s = logistic(k2 * (g + 0.044715f * g * g * g));
    const float gc = fminf(fmaxf(g, -16.f), 16.f);
    a = g * s;
    d = fmaf(gc * s * (1.f - s), k2 * fmaf(3.f * 0.044715f * gc, gc, 1.f), s);
  } else if constexpr (ACT == EPI_ACT_GELU_ERF) {
    float p, e;
    normal(g, p, e);
    a = g * p;
    d = fmaf(g * 0.3989422804014327f, e, p);  // density e^(-g^2/2) / sqrt(2 pi)
  } else {
    a = g;
    d = 1.f;
  }
}

template <int ACT>
__device__ __forceinline__ float act_only(float g) {
  float a, d;
  act_and_slope<ACT>(g, a, d);
  return a;
}

}  // namespace dgb
