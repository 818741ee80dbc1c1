// quant.cu -- the C ABI of the low-precision operands (include/quant.h): argument
// validation, launches and status checks.
#include "quant_launch.h"

#include "launch.h"

using namespace dgb;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxNormD = 32768;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

gemm_status_t launched(cudaError_t e) {
  if (e == cudaSuccess) return GEMM_OK;
  cudaGetLastError();
  return e == cudaErrorMemoryAllocation ? GEMM_ERR_OOM : GEMM_ERR_CUDA;
}

// A row pitch: 0 means dense.  False where it is shorter than a row.
bool pitch(int64_t* ld, int64_t row) {
  if (*ld == 0) *ld = row;
  return *ld >= row && *ld < kMaxDim;
}

bool is_format(int32_t f) { return f >= QUANT_E4M3 && f <= QUANT_NVFP4; }
bool is_dtype(int32_t t) { return t >= FFN_F16 && t <= FFN_F32; }
uintptr_t elem(int32_t dtype) { return dtype == FFN_F32 ? 4 : 2; }

// The arrays of a quantised operand: each given exactly where its format has it.
gemm_status_t operand(const void* data, const void* scales, const float* row_scale, int32_t format) {
  const bool block = format != QUANT_E4M3, row = format == QUANT_E4M3 || format == QUANT_NVFP4;
  if (!data || (scales != nullptr) != block || (row_scale != nullptr) != row) return GEMM_ERR_INVALID_ARG;
  if (!aligned(data, 16) || !aligned(scales, 16) || !aligned(row_scale, 4)) return GEMM_ERR_MISALIGNED;
  return GEMM_OK;
}

gemm_status_t rows_sizes(const quant_rows_t& a) {
  if (!is_dtype(a.dtype) || !is_format(a.format)) return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (a.transpose != 0 && a.transpose != 1) return GEMM_ERR_INVALID_ARG;
  if (a.rows < 0 || a.cols < 0 || a.rows >= kMaxDim - 32 || a.cols >= kMaxDim - 32) return GEMM_ERR_INVALID_ARG;
  // (one CTA per tile of 256 x 64, in one dimension of the grid)
  if (a.transpose && ((a.rows + 287) / 256) * ((a.cols + 127) / 64) >= kMaxDim / 8) return GEMM_ERR_UNSUPPORTED_SHAPE;
  return GEMM_OK;
}

// The sizes and choices of a product or a linear layer (columns past N are counted in 32 bits, and
// so are tiles).
template <typename Args>
gemm_status_t product_sizes(const Args& a) {
  if (a.format != QUANT_MXFP4 && a.format != QUANT_NVFP4) return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (a.out_dtype != FFN_BF16 && a.out_dtype != FFN_F32) return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (a.M < 0 || a.N < 0 || a.M > kMaxDim - 512 || a.N > kMaxDim - 512 || a.timeout_ns < 0) return GEMM_ERR_INVALID_ARG;
  if (a.activation < GEMM_ACT_NONE || a.activation > GEMM_ACT_GELU_ERF || (a.flags & ~QUANT_STATIC_B) != 0)
    return GEMM_ERR_INVALID_ARG;
  if (((a.M + 255) / 256) * ((a.N + 255) / 256) >= kMaxDim / 4) return GEMM_ERR_UNSUPPORTED_SHAPE;
  return GEMM_OK;
}

gemm_status_t linear_sizes(const quant_linear_t& a) {
  if (!is_dtype(a.dtype)) return GEMM_ERR_UNSUPPORTED_DTYPE;
  const gemm_status_t st = product_sizes(a);
  if (st != GEMM_OK) return st;
  return a.K < 0 || a.K >= kMaxDim - 32 ? GEMM_ERR_INVALID_ARG : GEMM_OK;
}

// Whether rows x (of `x_row` bytes each, `x_pitch` apart) and rows c share a byte: columns of one
// array's rows do not.
bool rows_overlap(const void* x, int64_t rows, int64_t x_row, int64_t x_pitch, const void* c, int64_t c_row,
                  int64_t c_pitch) {
  const intptr_t x0 = reinterpret_cast<intptr_t>(x), c0 = reinterpret_cast<intptr_t>(c);
  if (x_row == 0 || c0 >= x0 + (rows - 1) * x_pitch + x_row || x0 >= c0 + (rows - 1) * c_pitch + c_row) return false;
  if (x_pitch != c_pitch) return true;
  const int64_t apart = ((c0 - x0) % x_pitch + x_pitch) % x_pitch;
  return apart < x_row || apart + c_row > x_pitch;
}

// where the quantised rows of a linear layer lie in its workspace
struct LinearWorkspace {
  size_t scales, row_scale, bytes;
  explicit LinearWorkspace(const quant_linear_t& a) {
    auto round = [](size_t n) { return (n + 255) / 256 * 256; };
    const int64_t width = width_of(a.K);
    scales = round((size_t)a.M * (size_t)(width / 2));
    row_scale = scales + round((size_t)((a.M + 127) / 128) * (size_t)((scales_of(width, a.format) + 3) / 4) * 512);
    bytes = row_scale + (a.format == QUANT_NVFP4 ? round((size_t)a.M * 4) : 0);
  }
};

// Checks a call and resolves its pitches.
gemm_status_t rows_checked(quant_rows_t* p) {
  quant_rows_t& a = *p;
  gemm_status_t st = rows_sizes(a);
  if (st != GEMM_OK) return st;
  if (!pitch(&a.ld_x, a.cols) || !pitch(&a.ld_data, bytes_of(width_of(a.transpose ? a.rows : a.cols), a.format)) ||
      !rows_fit(a.rows, a.ld_x, a.cols, (int64_t)elem(a.dtype)))
    return GEMM_ERR_INVALID_ARG;
  if ((a.transpose ? a.cols : a.rows) == 0) return GEMM_OK;
  if (!a.x && a.rows > 0 && a.cols > 0) return GEMM_ERR_INVALID_ARG;
  st = operand(a.data, a.scales, a.row_scale, a.format);
  if (st != GEMM_OK) return st;
  if (!aligned(a.x, elem(a.dtype)) || a.ld_data % 16 != 0 || !aligned(a.workspace, 16)) return GEMM_ERR_MISALIGNED;
  if (a.transpose && quant_columns_workspace(a) > 0 && !a.workspace) return GEMM_ERR_INVALID_ARG;
  return GEMM_OK;
}

}  // namespace

extern "C" {

int64_t quant_width(int64_t cols) { return cols < 0 || cols >= kMaxDim - 32 ? -1 : width_of(cols); }

int64_t quant_row_bytes(int64_t cols, int32_t format) {
  if (quant_width(cols) < 0 || !is_format(format)) return -1;
  return bytes_of(width_of(cols), format);
}

int64_t quant_scale_bytes(int64_t rows, int64_t cols, int32_t format) {
  if (quant_width(cols) < 0 || !is_format(format) || rows < 0 || rows >= kMaxDim) return -1;
  return (rows + 127) / 128 * ((scales_of(width_of(cols), format) + 3) / 4) * 512;
}

int64_t quant_rows_workspace(const quant_rows_t* args) {
  if (!args || rows_sizes(*args) != GEMM_OK) return -1;
  return args->transpose && args->cols > 0 ? (int64_t)quant_columns_workspace(*args) : 0;
}

gemm_status_t quant_rows(const quant_rows_t* args, gemm_stream_t stream) { return quant_rows_many(args, 1, stream); }

gemm_status_t quant_rows_many(const quant_rows_t* args, int32_t count, gemm_stream_t stream) {
  if (!args || count < 0) return GEMM_ERR_INVALID_ARG;
  // everything is checked before anything is launched
  for (int32_t i = 0; i < count; ++i) {
    quant_rows_t a = args[i];
    const gemm_status_t st = rows_checked(&a);
    if (st != GEMM_OK) return st;
  }
  FfnDevice dev{};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  quant_rows_t columns[kQuantColumnTasks];
  int waiting = 0;
  cudaError_t e = cudaSuccess;
  for (int32_t i = 0; i < count && e == cudaSuccess; ++i) {
    quant_rows_t a = args[i];
    rows_checked(&a);  // (resolves the pitches)
    if ((a.transpose ? a.cols : a.rows) == 0) continue;
    if (dev.status == nullptr) {
      const gemm_status_t st = device_of_call(1, &dev);
      if (st != GEMM_OK) return st;
    }
    if (!a.transpose) {
      e = launch_quant_rows(a, dev, s);
      continue;
    }
    // columns of arrays alike go together
    if (waiting > 0 && (waiting == kQuantColumnTasks || columns[0].dtype != a.dtype || columns[0].format != a.format)) {
      e = launch_quant_columns(columns, waiting, s);
      waiting = 0;
    }
    columns[waiting++] = a;
  }
  if (e == cudaSuccess && waiting > 0) e = launch_quant_columns(columns, waiting, s);
  return launched(e);
}

gemm_status_t quant_norm(const quant_norm_t* args, gemm_stream_t stream) {
  if (!args) return GEMM_ERR_INVALID_ARG;
  quant_norm_t a = *args;
  if (!is_dtype(a.dtype) || !is_format(a.format) || (a.param_dtype != a.dtype && a.param_dtype != FFN_F32))
    return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (a.M < 0 || a.D < 1 || a.M >= kMaxDim || a.D >= kMaxDim) return GEMM_ERR_INVALID_ARG;
  if (a.D > kMaxNormD) return GEMM_ERR_UNSUPPORTED_SHAPE;
  if (!pitch(&a.ld_y, a.D) || !pitch(&a.ld_residual, a.D) || !pitch(&a.ld_s, a.D) ||
      !pitch(&a.ld_data, bytes_of(width_of(a.D), a.format)))
    return GEMM_ERR_INVALID_ARG;
  const uintptr_t e = elem(a.dtype);
  if (!rows_fit(a.M, a.ld_y, a.D, (int64_t)e) || !rows_fit(a.M, a.ld_residual, a.D, (int64_t)e) ||
      !rows_fit(a.M, a.ld_s, a.D, (int64_t)e))
    return GEMM_ERR_INVALID_ARG;
  if (a.M == 0) return GEMM_OK;
  if (!a.y) return GEMM_ERR_INVALID_ARG;
  gemm_status_t st = operand(a.data, a.scales, a.row_scale, a.format);
  if (st != GEMM_OK) return st;
  if (!aligned(a.y, e) || !aligned(a.residual, e) || !aligned(a.s, e) || !aligned(a.weight, elem(a.param_dtype)) ||
      a.ld_data % 16 != 0)
    return GEMM_ERR_MISALIGNED;
  FfnDevice dev;
  st = device_of_call(1, &dev);
  if (st != GEMM_OK) return st;
  return launched(launch_quant_norm(a, dev, reinterpret_cast<cudaStream_t>(stream)));
}

gemm_status_t quant_product(const quant_product_t* args, gemm_stream_t stream) {
  if (!args) return GEMM_ERR_INVALID_ARG;
  quant_product_t a = *args;
  const gemm_status_t sizes = product_sizes(a);
  if (sizes != GEMM_OK) return sizes;
  if (a.K < 32 || a.K >= kMaxDim) return GEMM_ERR_INVALID_ARG;
  if (a.K % 32 != 0) return GEMM_ERR_UNSUPPORTED_SHAPE;
  const uintptr_t e = elem(a.out_dtype);
  if (!pitch(&a.ld_a, a.K / 2) || !pitch(&a.ld_b, a.K / 2) || !pitch(&a.ld_residual, a.N) || !pitch(&a.ld_c, a.N) ||
      !rows_fit(a.M, a.ld_residual, a.N, (int64_t)e) || !rows_fit(a.M, a.ld_c, a.N, (int64_t)e))
    return GEMM_ERR_INVALID_ARG;
  if (a.M == 0 || a.N == 0) return GEMM_OK;
  if (!a.a || !a.b || !a.scales_a || !a.scales_b || !a.c) return GEMM_ERR_INVALID_ARG;
  if (!aligned(a.a, 16) || !aligned(a.b, 16) || !aligned(a.scales_a, 16) || !aligned(a.scales_b, 16) ||
      a.ld_a % 16 != 0 || a.ld_b % 16 != 0 || !aligned(a.row_scale_a, 4) || !aligned(a.row_scale_b, 4) ||
      !aligned(a.bias, 4) || !aligned(a.residual, e) || !aligned(a.c, e))
    return GEMM_ERR_MISALIGNED;
  FfnDevice dev;
  const gemm_status_t st = device_of_call(1, &dev);
  if (st != GEMM_OK) return st;
  return launched(launch_fp4_product(a, dev, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t quant_linear_workspace(const quant_linear_t* args) {
  if (!args || linear_sizes(*args) != GEMM_OK) return -1;
  if (args->M == 0 || args->N == 0 || fp4_linear_fused(*args)) return 0;
  return (int64_t)LinearWorkspace(*args).bytes;
}

gemm_status_t quant_linear(const quant_linear_t* args, gemm_stream_t stream) {
  if (!args) return GEMM_ERR_INVALID_ARG;
  quant_linear_t a = *args;
  gemm_status_t st = linear_sizes(a);
  if (st != GEMM_OK) return st;
  const int64_t width = width_of(a.K);
  const uintptr_t e = elem(a.out_dtype);
  if (!pitch(&a.ld_x, a.K) || !pitch(&a.ld_b, width / 2) || !pitch(&a.ld_residual, a.N) || !pitch(&a.ld_c, a.N) ||
      !rows_fit(a.M, a.ld_x, a.K, (int64_t)elem(a.dtype)) || !rows_fit(a.M, a.ld_residual, a.N, (int64_t)e) ||
      !rows_fit(a.M, a.ld_c, a.N, (int64_t)e))
    return GEMM_ERR_INVALID_ARG;
  if (a.M == 0 || a.N == 0) return GEMM_OK;
  if ((!a.x && a.K > 0) || !a.b || !a.scales_b || !a.c) return GEMM_ERR_INVALID_ARG;
  if (!aligned(a.x, elem(a.dtype)) || !aligned(a.b, 16) || !aligned(a.scales_b, 16) || a.ld_b % 16 != 0 ||
      !aligned(a.row_scale_b, 4) || !aligned(a.bias, 4) || !aligned(a.residual, e) || !aligned(a.c, e) ||
      !aligned(a.workspace, 256))
    return GEMM_ERR_MISALIGNED;
  if (rows_overlap(a.x, a.M, a.K * (int64_t)elem(a.dtype), a.ld_x * (int64_t)elem(a.dtype), a.c, a.N * (int64_t)e,
                   a.ld_c * (int64_t)e))
    return GEMM_ERR_INVALID_ARG;
  const bool fused = fp4_linear_fused(a);
  if (!fused && !a.workspace) return GEMM_ERR_INVALID_ARG;
  FfnDevice dev;
  st = device_of_call(1, &dev);
  if (st != GEMM_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (fused) return launched(launch_fp4_linear(a, dev, s));
  const LinearWorkspace ws(a);
  uint8_t* base = static_cast<uint8_t*>(a.workspace);
  quant_rows_t q{};
  q.rows = a.M;
  q.cols = a.K;
  q.dtype = a.dtype;
  q.format = a.format;
  q.x = a.x;
  q.data = base;
  q.scales = base + ws.scales;
  q.row_scale = a.format == QUANT_NVFP4 ? reinterpret_cast<float*>(base + ws.row_scale) : nullptr;
  q.ld_x = a.ld_x;
  q.ld_data = width / 2;
  const cudaError_t err = launch_quant_rows(q, dev, s);
  if (err != cudaSuccess) return launched(err);
  quant_product_t p{};
  p.M = a.M;
  p.N = a.N;
  p.K = width;
  p.format = a.format;
  p.out_dtype = a.out_dtype;
  p.activation = a.activation;
  p.flags = a.flags;
  p.a = q.data;
  p.b = a.b;
  p.scales_a = q.scales;
  p.scales_b = a.scales_b;
  p.row_scale_a = q.row_scale;
  p.row_scale_b = a.row_scale_b;
  p.bias = a.bias;
  p.residual = a.residual;
  p.c = a.c;
  p.ld_a = q.ld_data;
  p.ld_b = a.ld_b;
  p.ld_residual = a.ld_residual;
  p.ld_c = a.ld_c;
  p.timeout_ns = a.timeout_ns;
  p.debug_flags = a.debug_flags;
  return launched(launch_fp4_product(p, dev, s));
}

gemm_status_t quant_check(gemm_stream_t stream) { return check_word(1, reinterpret_cast<cudaStream_t>(stream)); }

}  // extern "C"
