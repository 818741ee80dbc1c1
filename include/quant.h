/*
 * quant.h -- C ABI of the low-precision operands and their 4-bit product (same
 * library as gemm.h, libdgbgemm.so, GB300 / sm_103a):
 *
 *   - quantisation of rows, or of columns (the operands of a backward pass), to
 *     E4M3 with a scale per row, to E4M3 or E2M1 with a power of two per 32
 *     elements, and to E2M1 with an E4M3 scale per 16 and a scale per row;
 *   - the residual's addition, the RMS norm before the next layer and the
 *     quantisation of its output, in one kernel;
 *   - the product of two microscaled 4-bit operands with a fused epilogue.
 *
 * The 8-bit operands are those of gemm.h's products: E4M3 with scale_a / scale_b of
 * gemm_plan_run_epilogue, MXFP8 with gemm_plan_run_mx.  Their plan's K is quant_width of
 * the values' number (1024 for rows of 1001): the padding's zeros are part of the rows.
 *
 * The calls follow gemm.h and ffn.h: plain integers and pointers, device memory owned
 * by the caller, gemm_status_t answers, argument problems returned at once with
 * nothing launched, no exception across the boundary, work enqueued on `stream`
 * and nothing synchronised.  No call allocates, and calls keep no state between one
 * another except one status word per device: calls on different streams may
 * overlap as long as their buffers (workspaces among them) do not.
 *
 * Arrays of elements are row-major with their own row pitch `ld_*` in elements (0
 * means dense: the row's length); elements of a row are adjacent.  Rows may have no
 * elements, whatever their pitch: nothing of such an array is read, and it may be NULL.
 * A pitch and a number of rows whose array would pass 2^62 bytes are refused.  Arrays
 * named "output" must not overlap any input unless a comment allows it.
 */
#ifndef DGB_QUANT_H
#define DGB_QUANT_H

#include "ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How an operand's rows are held.  A row of K values is padded with zeros to
 * quant_width(K) elements, so that it can be copied in 16-byte pieces.
 *
 * QUANT_E4M3: bytes q with x ~ q * row_scale[row].  row_scale = max(m / 448, 2^-126)
 *   for the row's largest magnitude m, and q = x * (1 / row_scale), both in fp32, q
 *   rounded to nearest even.
 * QUANT_MXE4M3, QUANT_MXFP4: q in units of 2^e, one e per 32 elements: the smallest e
 *   with m <= 448 * 2^e (E4M3) or m <= 6 * 2^e (E2M1) for the 32's largest magnitude
 *   m (-127 at least; -127 for 32 zeros), kept as the UE8M0 byte e + 127.  Nothing
 *   saturates.
 * QUANT_NVFP4: E2M1 values in units of scale * row_scale[row].  row_scale is the
 *   smallest power of two, 2^-100 at least, with m <= 2688 * row_scale for the row's
 *   largest magnitude m (1 for a row of zeros); scale, one UE4M3 byte per 16 elements,
 *   is m / (6 row_scale) for the 16's largest magnitude, rounded to nearest even.
 *   The values are x / (scale * row_scale), rounded to nearest even and limited to 6;
 *   0 where the scale is 0.
 *
 * Two of these are choices among conventions.  The MX formats' power of two covers its block, so
 * that nothing saturates; where it is taken as floor(log2 m) less the format's largest
 * exponent instead, values up to 2^(e + 1) are limited.  NVFP4's second scale is a power of two
 * per row; one float for the whole array does as well where an operand comes with it (every
 * row_scale that float).
 *
 * E2M1 has the values 0, 0.5, 1, 1.5, 2, 3, 4, 6 (codes 0 to 7) and their negatives
 * (codes 8 to 15); element 2 i of a row is the low half of byte i.  All roundings but
 * those of QUANT_E4M3 are of the exact values (for inputs whose row_scale or 2^e is
 * clamped or whose quotients leave fp32's normal range, of those values in fp32), and so
 * are those behind a norm but for QUANT_NVFP4 (see quant_norm).
 *
 * A row with a NaN or an infinity gives NaN in every product it takes part in:
 * row_scale is a NaN (E4M3, NVFP4; with NVFP4 its scales too), or the scale of the
 * block is (MX formats); the values beside it are 0.
 *
 * Block scales are kept as gemm_plan_run_mx reads them: 512-byte blocks of 128 rows x
 * 4 scales, block (rb, cb) at byte (rb * ceil(scales / 4) + cb) * 512, and inside a block
 * the scale of row r, scale column c at byte (r % 32) * 16 + ((r / 32) % 4) * 4 + c % 4.
 * The calls below write every byte of such an array; those that belong to no element
 * are 0.  A product must not be given a NaN there in the columns past K. */
typedef enum { QUANT_E4M3 = 0, QUANT_MXE4M3 = 1, QUANT_MXFP4 = 2, QUANT_NVFP4 = 3 } quant_format_t;

/* Elements of a quantised row of `cols` values: a multiple of 32, at least 32 (a row of no
 * values is 32 zeros); -1 for cols < 0 or >= 2^31 - 32. */
GEMM_API int64_t quant_width(int64_t cols);
/* Bytes of a quantised row (its pitch when dense); -1 for arguments that are refused. */
GEMM_API int64_t quant_row_bytes(int64_t cols, int32_t format);
/* Bytes of the tiled block scales of `rows` rows of `cols` values (0 for QUANT_E4M3 and for
 * no rows); -1 for arguments that are refused. */
GEMM_API int64_t quant_scale_bytes(int64_t rows, int64_t cols, int32_t format);

/* Quantises x, rows x cols, by rows; with `transpose` its columns: the operand then has
 * cols rows of quant_width(rows) elements. */
typedef struct {
  int64_t rows, cols;   /* of x; either may be 0 */
  int32_t dtype;        /* ffn_dtype_t of x */
  int32_t format;       /* quant_format_t */
  int32_t transpose;    /* 0 or 1 */
  int32_t reserved;
  const void* x;        /* rows x cols */
  void* data;           /* output, 16-byte aligned: the operand's rows */
  void* scales;         /* output, 16-byte aligned, quant_scale_bytes; NULL for QUANT_E4M3 */
  float* row_scale;     /* output, one per row of the operand; NULL for the MX formats */
  void* workspace;      /* quant_rows_workspace bytes, 16-byte aligned; may be NULL if those are 0 */
  int64_t ld_x;
  int64_t ld_data;      /* bytes between rows of data, a multiple of 16 (0: dense) */
} quant_rows_t;

/* Bytes of workspace of this call (it reads sizes, format and transpose, no array); -1 for
 * sizes it would refuse. */
GEMM_API int64_t quant_rows_workspace(const quant_rows_t* args);

GEMM_API gemm_status_t quant_rows(const quant_rows_t* args, gemm_stream_t stream);

/* The same for `count` arrays (0 allowed), each with a workspace of its own; columns of arrays of
 * one dtype and format that follow one another go in few launches.  All are checked before
 * anything is launched. */
GEMM_API gemm_status_t quant_rows_many(const quant_rows_t* args, int32_t count, gemm_stream_t stream);

/* s = residual_scale * residual + branch_scale * y
 * n = s / sqrt(mean(s^2) + eps) * weight, from s before it is rounded, in fp32
 * and n quantised by rows (a row whose sum of squares passes fp32's range comes as zeros).
 * To QUANT_NVFP4 the quotients m / (6 row_scale) and x / (scale * row_scale) are taken with
 * reciprocals and are within 2^-22 of themselves, about as n is of its exact value, before
 * they are rounded.  Absent (NULL) weight counts as one, an absent residual as
 * zero; s is written if given and may be `residual` or y itself (same pointer and
 * pitch).  The gradient with respect to y, residual and weight is ffn_norm_backward's,
 * dn being what reaches the values that the operand stands for. */
typedef struct {
  int64_t M, D;         /* rows and their length, 1 <= D <= 32768; M may be 0 */
  int32_t dtype;        /* ffn_dtype_t: y, residual and s */
  int32_t param_dtype;  /* dtype or FFN_F32: weight */
  int32_t format;
  int32_t reserved;
  float eps, residual_scale, branch_scale, reserved_f;
  const void* y;        /* M x D */
  const void* residual; /* M x D, or NULL */
  const void* weight;   /* D values, or NULL */
  void* s;              /* M x D, output, or NULL */
  void* data;           /* as quant_rows_t */
  void* scales;
  float* row_scale;
  int64_t ld_y, ld_residual, ld_s;
  int64_t ld_data;
} quant_norm_t;

GEMM_API gemm_status_t quant_norm(const quant_norm_t* args, gemm_stream_t stream);

/* B is not written by the kernels just before this one on the stream (weights): it may be
 * read before they have completed. */
#define QUANT_STATIC_B 1

/* Test hook: one copy of the first stage is left out, so that a bounded wait runs out and
 * quant_check reports it.  The call's output is then void. */
#define QUANT_DEBUG_SKIP_ONE_LOAD 1

/* C = act(row_scale_a[i] * row_scale_b[j] * sum_k A[i][k] B[j][k] + bias[j]) + residual[i][j]
 * for A (M x K) and B (N x K) of one 4-bit format, QUANT_MXFP4 or QUANT_NVFP4, each value
 * in units of its block's scale.  Sums are accumulated in fp32 on the Tensor Core, the
 * epilogue is fp32 and each element is rounded once.  The order of a sum depends on the
 * sizes alone: the same inputs give the same bits.  The sum is multiplied by row_scale_a and
 * then by row_scale_b, in fp32.  K is the operands' width, a multiple of 32 below 2^31.  M
 * and N may be 0 and are at most 2^31 - 512. */
typedef struct {
  int64_t M, N, K;
  int32_t format;       /* QUANT_MXFP4 or QUANT_NVFP4, of both operands */
  int32_t out_dtype;    /* FFN_BF16 or FFN_F32: C and residual */
  int32_t activation;   /* gemm_activation_t */
  int32_t flags;        /* QUANT_STATIC_B */
  const void* a;        /* M rows of K / 2 bytes, 16-byte aligned */
  const void* b;        /* N rows */
  const void* scales_a; /* tiled block scales, 16-byte aligned */
  const void* scales_b;
  const float* row_scale_a; /* M values, or NULL (one) */
  const float* row_scale_b; /* N values, or NULL */
  const float* bias;    /* N values, or NULL */
  const void* residual; /* M x N, or NULL; may be C itself (same pointer and pitch) */
  void* c;              /* M x N, output */
  int64_t ld_a, ld_b;   /* bytes between rows, a multiple of 16 (0: dense) */
  int64_t ld_residual, ld_c;
  int64_t timeout_ns;   /* bound on every device-side wait, 0 = 2 s */
  int32_t debug_flags;
  int32_t reserved[3];
} quant_product_t;

GEMM_API gemm_status_t quant_product(const quant_product_t* args, gemm_stream_t stream);

/* A linear layer: x's rows quantised to B's format, then the product,
 *   C = act(Q(x) B^T + bias) + residual,
 * with the bits of quant_rows and quant_product.  Up to 16 tokens go in one kernel where that
 * is as fast or faster with the launch it saves counted in (replayed in a graph it can take up to
 * 5 % longer than two: 1 x 14336 x 4096 to NVFP4 10.0 us and 9.6).  C must not share a byte with x
 * (a call where it does is refused). */
typedef struct {
  int64_t M, N, K;      /* K: values of a row of x; B's rows are quant_width(K) elements */
  int32_t dtype;        /* ffn_dtype_t of x */
  int32_t format;       /* QUANT_MXFP4 or QUANT_NVFP4, of B */
  int32_t out_dtype;    /* as quant_product_t, from here on */
  int32_t activation;
  int32_t flags;
  int32_t debug_flags;
  const void* x;        /* M x K */
  const void* b;
  const void* scales_b;
  const float* row_scale_b;
  const float* bias;
  const void* residual;
  void* c;
  void* workspace;      /* quant_linear_workspace bytes, 256-byte aligned; may be NULL if those are 0 */
  int64_t ld_x;
  int64_t ld_b;         /* bytes */
  int64_t ld_residual, ld_c;
  int64_t timeout_ns;
} quant_linear_t;

/* Bytes of workspace of this call (it reads sizes, types and format, no array); -1 for sizes it
 * would refuse. */
GEMM_API int64_t quant_linear_workspace(const quant_linear_t* args);

GEMM_API gemm_status_t quant_linear(const quant_linear_t* args, gemm_stream_t stream);

/* Synchronise `stream`, then report (and clear) a device-side error recorded by this
 * header's kernels on the current device. */
GEMM_API gemm_status_t quant_check(gemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DGB_QUANT_H */
