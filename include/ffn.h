/*
 * ffn.h -- C ABI of the feed-forward block's operators (same library as gemm.h,
 * libdgbgemm.so, GB300 / sm_103a):
 *
 *   - the gated projections, h = act(x Wg^T) * (x Wu^T), both products, the
 *     activation and the elementwise product in one kernel, and their backward
 *     pass (from kept pre-activations, or computing them again);
 *   - the norms around a block: the block's output is normalised, gated, scaled
 *     and added to the residual stream, and the new stream is normalised for the
 *     next block, in one kernel, and its backward pass.
 *
 * The calls follow gemm.h: plain integers and pointers, device memory owned by
 * the caller, gemm_status_t answers, argument problems returned at once with
 * nothing launched, no exception across the boundary, work enqueued on `stream`
 * and nothing synchronised.  No call allocates: everything a call needs besides
 * its inputs and outputs is a workspace argument.  Calls keep no state between
 * one another except one status word per device, so calls on different streams
 * may overlap as long as their buffers do not.
 *
 * Every array is row-major with its own row pitch `ld_*` in elements (0 means
 * dense: the row's length); elements of a row are adjacent.  Arrays named
 * "output" must not overlap any input unless a comment allows it.
 */
#ifndef DGB_FFN_H
#define DGB_FFN_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FFN_F16 = 0, FFN_BF16 = 1, FFN_F32 = 2 } ffn_dtype_t;

/* Test hook of the tensor-core kernels and of the norms' kernels that bring rows
 * through shared memory (every gradient, and many rows forward): one copy is left
 * out, or waited for in vain, so that a bounded wait runs out and ffn_check reports
 * it.  The call's outputs are then void. */
#define FFN_DEBUG_SKIP_ONE_LOAD 1

/* h = act(x Wg^T) * (x Wu^T): M tokens, K input features, F hidden features.
 * w holds 2F rows of K: the gate's projection Wg, then Wu.  Products are
 * accumulated in fp32, activation and product are fp32, and each output is
 * rounded once.  Needs K % 8 == 0, x and w 16-byte aligned with ld % 8 == 0 (a
 * TMA row pitch); h and gu only their elements' alignment.  M may be 0. */
typedef struct {
  int64_t M, F, K;
  int32_t dtype;        /* FFN_F16 or FFN_BF16: x, w, h and gu */
  int32_t activation;   /* gemm_activation_t */
  const void* x;        /* M x K */
  const void* w;        /* 2F x K */
  void* h;              /* M x F, output */
  void* gu;             /* M x 2F, output: the pre-activations x w^T (gate, then up) for the
                           backward pass, or NULL */
  int64_t ld_x, ld_w, ld_h, ld_gu;
  int64_t timeout_ns;   /* bound on every device-side wait, 0 = 2 s */
  int32_t debug_flags;  /* FFN_DEBUG_* */
  int32_t reserved[3];
} ffn_gated_t;

GEMM_API gemm_status_t ffn_gated(const ffn_gated_t* args, gemm_stream_t stream);

/* Gradients of ffn_gated given dh = dL/dh, with g = x Wg^T and u = x Wu^T:
 *   dgu = [dh * u * act'(g), dh * act(g)],  dx = dgu w,  dw = dgu^T x.
 * g and u are read from `gu` (as ffn_gated wrote it), or computed again from x
 * and w when gu is NULL.  dgu is rounded once to `dtype` (it is the operand of
 * both products); dx and dw are accumulated in fp32 and rounded once.  Every
 * element of dx and dw is summed in a fixed order: the same inputs give the same
 * bits.  act'(0) of ReLU is 0.  M may be 0 (dw is then zero). */
typedef struct {
  int64_t M, F, K;
  int32_t dtype;        /* FFN_F16 or FFN_BF16, of every array here */
  int32_t activation;
  const void* x;        /* M x K, 16-byte aligned, ld % 8 == 0 (may be NULL without dw if gu is given) */
  const void* w;        /* 2F x K, 16-byte aligned, ld % 8 == 0 (may be NULL without dx if gu is given) */
  const void* gu;       /* M x 2F, or NULL */
  const void* dh;       /* M x F */
  void* dgu;            /* M x 2F, output: gradient of the pre-activations; 16-byte aligned,
                           ld_dgu a multiple of 8 and at least 2F (always given; ld 0 means
                           2F rounded up to a multiple of 8) */
  void* dx;             /* M x K, output, or NULL */
  void* dw;             /* 2F x K, output, or NULL */
  void* workspace;      /* 32-byte aligned, ffn_gated_backward_workspace bytes; may be NULL if those are 0 */
  int64_t ld_x, ld_w, ld_gu, ld_dh, ld_dgu, ld_dx, ld_dw;
  int64_t timeout_ns;
  int32_t debug_flags;
  int32_t reserved[3];
} ffn_gated_grad_t;

/* Bytes of workspace that ffn_gated_backward needs for these sizes and this dx (0 for
 * dx NULL and where dx is summed in one piece), or -1 for arguments it refuses.  It
 * depends on M, F, K and on whether dx is NULL alone. */
GEMM_API int64_t ffn_gated_backward_workspace(const ffn_gated_grad_t* args);

GEMM_API gemm_status_t ffn_gated_backward(const ffn_gated_grad_t* args, gemm_stream_t stream);

/* Norm kinds: v / sqrt(mean(v^2) + eps), or (v - mean) / sqrt(var + eps) with the
 * biased variance. */
typedef enum { FFN_NORM_RMS = 0, FFN_NORM_LAYER = 1 } ffn_norm_kind_t;

#define FFN_NORM_POST 1 /* normalise the block's output y */
#define FFN_NORM_PRE 2  /* normalise the new stream s into n */

/* With unit(v) a row's normalised values:
 *   z = y, or with FFN_NORM_POST  unit(y) * post_weight + post_bias
 *   s = residual_scale * residual + branch_scale * gate[i / (M / groups)] * z
 *   n = unit(s) * pre_weight + pre_bias                        (FFN_NORM_PRE)
 * Absent (NULL) weights and gates count as one, biases and the residual as zero.
 * Everything between the inputs and the two roundings is fp32; n is computed
 * from s before s is rounded.  s may be `residual` itself and n may be y itself
 * (same pointer and pitch). */
typedef struct {
  int64_t M, D;           /* rows and their length, 1 <= D <= 32768; M may be 0 */
  int64_t groups;         /* rows of `gate`; M must be a multiple of it.  1: one gate for all rows
                             (a layer scale); M: a gate for every row */
  int32_t dtype;          /* FFN_*: y, residual, s and n */
  int32_t param_dtype;    /* dtype or FFN_F32: gate, weights and biases */
  int32_t kind;           /* ffn_norm_kind_t, of both norms */
  int32_t flags;          /* FFN_NORM_* */
  float eps, residual_scale, branch_scale;
  int32_t debug_flags;    /* FFN_DEBUG_* (their waits are bound by 2 s) */
  const void* y;          /* M x D */
  const void* residual;   /* M x D, or NULL */
  const void* gate;       /* groups x D, or NULL */
  const void* post_weight; /* D values, or NULL */
  const void* post_bias;
  const void* pre_weight;
  const void* pre_bias;
  void* s;                /* M x D, output, or NULL */
  void* n;                /* M x D, output; given exactly when FFN_NORM_PRE is set */
  int64_t ld_y, ld_residual, ld_gate, ld_s, ld_n;
} ffn_norm_t;

GEMM_API gemm_status_t ffn_norm(const ffn_norm_t* args, gemm_stream_t stream);

/* Gradients of ffn_norm given ds = dL/ds (what reaches the stream from later
 * blocks) and dn = dL/dn, from y and the stream s as ffn_norm wrote it:
 *   t     = ds + unit-norm gradient of dn * pre_weight at s
 *   dresidual = residual_scale * t
 *   dz    = branch_scale * gate * t
 *   dgate = branch_scale * sum of t * z over the group's rows
 *   dy    = dz, or with FFN_NORM_POST the unit-norm gradient of dz * post_weight at y
 *   d*_weight, d*_bias = sums over all rows of dn * unit(s), dn, dz * unit(y), dz
 * Parameter gradients are fp32, whatever param_dtype, summed in a fixed order. */
typedef struct {
  int64_t M, D, groups;
  int32_t dtype, param_dtype, kind, flags;
  float eps, residual_scale, branch_scale;
  int32_t debug_flags;
  const void* ds;         /* M x D, or NULL (zero) */
  const void* dn;         /* M x D; given exactly when FFN_NORM_PRE is set */
  const void* y;          /* M x D (may be NULL without FFN_NORM_POST and dgate) */
  const void* s;          /* M x D (may be NULL without FFN_NORM_PRE) */
  const void* gate;
  const void* post_weight;
  const void* post_bias;  /* read for dgate only */
  const void* pre_weight;
  void* dresidual;        /* M x D, output, or NULL */
  void* dy;               /* M x D, output, or NULL */
  float* dgate;           /* groups x D fp32 (dense), output, or NULL */
  float* dpost_weight;    /* D fp32, output, or NULL (needs FFN_NORM_POST) */
  float* dpost_bias;
  float* dpre_weight;     /* (needs FFN_NORM_PRE) */
  float* dpre_bias;
  void* workspace;        /* ffn_norm_backward_workspace bytes, 16-byte aligned (NULL when 0) */
  int64_t ld_ds, ld_dn, ld_y, ld_s, ld_gate, ld_dresidual, ld_dy;
} ffn_norm_grad_t;

/* Bytes of the workspace this call needs (its sizes, flags and which outputs are
 * given are read, no array); -1 for sizes ffn_norm_backward would refuse. */
GEMM_API int64_t ffn_norm_backward_workspace(const ffn_norm_grad_t* args);

GEMM_API gemm_status_t ffn_norm_backward(const ffn_norm_grad_t* args, gemm_stream_t stream);

/* Synchronise `stream`, then report (and clear) a device-side error recorded by
 * this header's kernels on the current device. */
GEMM_API gemm_status_t ffn_check(gemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DGB_FFN_H */
