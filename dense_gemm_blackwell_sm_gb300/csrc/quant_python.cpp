// quant_python.cpp -- what quant.py calls: checks of the tensors, allocation of the outputs and
// the calls of include/quant.h, as a Python extension (see ffn_python.cpp for the reason).
//
// A quantised operand travels as five values: data, scales or None, row_scale or None, format,
// columns.  Its arrays are one allocation: an allocation costs a third of a small call.
#include <ATen/cuda/EmptyTensor.h>

#include "python_calls.h"
#include "quant.h"

namespace {

PyObject* format_codes = nullptr;  // {name: code}
PyObject* format_names = nullptr;  // names by code

struct Operand {
  Tensor memory;  // of a new operand; a given one has its tensors'
  Tensor data_tensor, scales_tensor, row_scale_tensor;
  uint8_t* data = nullptr;
  uint8_t* scales = nullptr;
  float* row_scale = nullptr;
  int64_t rows = 0, cols = 0, ld = 0, scale_bytes = 0;
  int32_t format = 0;
  int index = 0;
};

// a format's name, or its code
int32_t format_of(PyObject* o) {
  if (!PyLong_Check(o)) {
    PyObject* code = PyDict_GetItemWithError(format_codes, o);
    if (code == nullptr) {
      if (PyErr_Occurred()) throw python_error();
      TORCH_CHECK_VALUE(false, "format must be one of e4m3, mxe4m3, mxfp4, nvfp4");
    }
    o = code;
  }
  const int64_t f = int_of(o);
  TORCH_CHECK_VALUE(f >= QUANT_E4M3 && f <= QUANT_NVFP4, "unknown format ", f);
  return (int32_t)f;
}

bool has_scales(int32_t format) { return format != QUANT_E4M3; }
bool has_row_scale(int32_t format) { return format == QUANT_E4M3 || format == QUANT_NVFP4; }

Tensor new_tensor(at::IntArrayRef sizes, at::ScalarType dtype, int index) {
  return Tensor(at::detail::empty_cuda(sizes, dtype, at::Device(at::kCUDA, (c10::DeviceIndex)index), std::nullopt));
}
Tensor new_rows(int64_t M, int64_t N, at::ScalarType dtype, int index) { return new_tensor({M, N}, dtype, index); }

// `sizes` values of `memory` from byte `offset` on, as a tensor
Tensor part_of(const Tensor& memory, int64_t offset, at::ScalarType dtype, at::IntArrayRef sizes) {
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(memory.storage()), memory.key_set(),
                                                      c10::scalarTypeToTypeMeta(dtype));
  c10::TensorImpl* impl = t.unsafeGetTensorImpl();
  impl->set_storage_offset(offset / (int64_t)c10::elementSize(dtype));
  impl->set_sizes_contiguous(sizes);
  return t;
}

int64_t round_up(int64_t n) { return (n + 255) / 256 * 256; }

// the operand of `rows` rows of `cols` values, allocated, with `more` bytes behind it
Operand empty_operand(int64_t rows, int64_t cols, int32_t format, int index, int64_t more = 0) {
  Operand o;
  o.rows = rows;
  o.cols = cols;
  o.format = format;
  o.index = index;
  const int64_t bytes = quant_row_bytes(cols, format);
  o.scale_bytes = quant_scale_bytes(rows, cols, format);
  TORCH_CHECK_VALUE(bytes >= 0 && o.scale_bytes >= 0, "rows of ", cols, " values are too long");
  o.ld = bytes;
  const int64_t scales_at = round_up(rows * bytes), row_scale_at = scales_at + round_up(o.scale_bytes);
  const int64_t more_at = row_scale_at + (has_row_scale(format) ? round_up(4 * rows) : 0);
  // (an array of no bytes has an address all the same)
  o.memory = new_tensor({more_at + more + 16}, at::kByte, index);
  uint8_t* base = static_cast<uint8_t*>(o.memory.data_ptr());
  o.data = base;
  if (has_scales(format)) o.scales = base + scales_at;
  if (has_row_scale(format)) o.row_scale = reinterpret_cast<float*>(base + row_scale_at);
  return o;
}
void* behind(const Operand& o) {
  const int64_t at = round_up(o.rows * o.ld) + round_up(o.scale_bytes) + (has_row_scale(o.format) ? round_up(4 * o.rows) : 0);
  return static_cast<uint8_t*>(o.memory.data_ptr()) + at;
}

// a given operand: p points at its five values
Operand operand_of(const char* name, PyObject* const* p) {
  Operand o;
  const Tensor& data = o.data_tensor = tensor_of(p[0], name);
  const Tensor *scales = optional_of(p[1], name), *row_scale = optional_of(p[2], name);
  o.format = format_of(p[3]);
  o.cols = int_of(p[4]);
  TORCH_CHECK_VALUE(o.format == QUANT_MXFP4 || o.format == QUANT_NVFP4, name, " must be a 4-bit operand (mxfp4 or nvfp4)");
  o.index = index_of(data);
  TORCH_CHECK_VALUE(data.dim() == 2, name, "'s data must be a 2-D tensor, not ", data.sizes());
  o.rows = data.size(0);
  const int64_t bytes = quant_row_bytes(o.cols, o.format);
  TORCH_CHECK_VALUE(bytes >= 0, name, " has ", o.cols, " columns");
  o.ld = rows_of(name, data, o.rows, bytes, at::kByte, o.index);
  const int64_t want = quant_scale_bytes(o.rows, o.cols, o.format);
  TORCH_CHECK_VALUE(scales != nullptr && scales->scalar_type() == at::kByte && scales->is_contiguous() &&
                        scales->numel() == want && scales->is_cuda() && scales->get_device() == o.index,
                    name, "'s scales must be ", want, " dense bytes on cuda:", o.index);
  o.scales_tensor = *scales;
  o.data = static_cast<uint8_t*>(data.data_ptr());
  o.scales = static_cast<uint8_t*>(scales->data_ptr());
  if (row_scale != nullptr) {
    TORCH_CHECK_VALUE(row_scale->scalar_type() == at::kFloat && row_scale->is_contiguous() && row_scale->dim() == 1 &&
                          row_scale->size(0) == o.rows && row_scale->is_cuda() && row_scale->get_device() == o.index,
                      name, "'s row scales must be ", o.rows, " dense values of float32 on cuda:", o.index);
    o.row_scale_tensor = *row_scale;
    o.row_scale = static_cast<float*>(row_scale->data_ptr());
  }
  return o;
}

// the five values of a new operand
PyObject* operand_tuple(const Operand& o) {
  const bool four = o.format == QUANT_MXFP4 || o.format == QUANT_NVFP4;
  const uint8_t* base = static_cast<const uint8_t*>(o.memory.data_ptr());
  const Tensor data = part_of(o.memory, 0, four ? at::kByte : at::kFloat8_e4m3fn, {o.rows, o.ld});
  Tensor scales, row_scale;
  if (o.scales) scales = part_of(o.memory, o.scales - base, at::kByte, {o.scale_bytes});
  if (o.row_scale) row_scale = part_of(o.memory, reinterpret_cast<const uint8_t*>(o.row_scale) - base, at::kFloat, {o.rows});
  THPObjectPtr out(PyTuple_New(5));
  if (!out) throw python_error();
  PyTuple_SET_ITEM(out.get(), 0, wrapped(data));
  PyTuple_SET_ITEM(out.get(), 1, wrapped(scales));
  PyTuple_SET_ITEM(out.get(), 2, wrapped(row_scale));
  PyTuple_SET_ITEM(out.get(), 3, Py_NewRef(PyTuple_GET_ITEM(format_names, o.format)));
  PyObject* cols = PyLong_FromLongLong(o.cols);
  if (cols == nullptr) throw python_error();
  PyTuple_SET_ITEM(out.get(), 4, cols);
  return out.release();
}

// x's rows or columns, to be quantised by the call whose arguments these are
Operand to_quantise(quant_rows_t* a, const char* name, const Tensor& x, int32_t format, bool transpose) {
  TORCH_CHECK_VALUE(x.dim() == 2, name, " must be a 2-D tensor, not ", x.sizes());
  const int index = index_of(x);
  const at::ScalarType dtype = x.scalar_type();
  a->rows = x.size(0);
  a->cols = x.size(1);
  a->dtype = code_of(dtype);
  TORCH_CHECK_VALUE(a->dtype >= 0, name, " must be float16, bfloat16 or float32, not ", dtype);
  a->format = format;
  a->transpose = transpose;
  a->ld_x = rows_of(name, x, a->rows, a->cols, dtype, index);
  // (a refused call asks for -1 bytes and is refused when it is made)
  const int64_t workspace = std::max<int64_t>(0, quant_rows_workspace(a));
  Operand o = empty_operand(transpose ? a->cols : a->rows, transpose ? a->rows : a->cols, format, index, workspace);
  a->x = x.data_ptr();
  a->data = o.data;
  a->scales = o.scales;
  a->row_scale = o.row_scale;
  a->workspace = behind(o);
  return o;
}

struct Several {
  quant_rows_t args[4];
  int32_t count;
};
gemm_status_t quant_several(const Several* s, gemm_stream_t stream) { return quant_rows_many(s->args, s->count, stream); }

struct Finish {
  const Tensor *bias, *residual, *out;
  int32_t activation, flags, debug_flags;
  at::ScalarType dtype;
  int64_t timeout_ns;
};

// what becomes of the sums, for a product or a linear layer of M x N; the output
template <typename Args>
Tensor finish_arguments(Args* a, const Finish& f, int index) {
  TORCH_CHECK_VALUE(f.dtype == at::kBFloat16 || f.dtype == at::kFloat, "the output must be bfloat16 or float32, not ",
                    f.dtype);
  a->out_dtype = code_of(f.dtype);
  a->activation = f.activation;
  a->flags = f.flags;
  a->timeout_ns = f.timeout_ns;
  a->debug_flags = f.debug_flags;
  if (f.bias != nullptr) {
    TORCH_CHECK_VALUE(f.bias->dim() == 1 && f.bias->size(0) == a->N && f.bias->scalar_type() == at::kFloat &&
                          f.bias->is_contiguous() && f.bias->is_cuda() && f.bias->get_device() == index,
                      "bias must be ", a->N, " dense values of float32 on cuda:", index);
    a->bias = static_cast<const float*>(f.bias->data_ptr());
  }
  if (f.residual != nullptr) {
    a->ld_residual = rows_of("residual", *f.residual, a->M, a->N, f.dtype, index);
    a->residual = f.residual->data_ptr();
  }
  Tensor c;
  if (f.out != nullptr) {
    a->ld_c = rows_of("out", *f.out, a->M, a->N, f.dtype, index);
    c = *f.out;
  } else {
    c = new_rows(a->M, a->N, f.dtype, index);
  }
  a->c = c.data_ptr();
  return c;
}

Tensor multiplied(const Operand& a, const Operand& b, const Finish& f, PyObject* stream) {
  TORCH_CHECK_VALUE(a.format == b.format && a.cols == b.cols, "operands must have one format and as many columns, not ",
                    a.cols, " and ", b.cols);
  TORCH_CHECK_VALUE(a.index == b.index, "operands must be on one device");
  quant_product_t p{};
  p.M = a.rows;
  p.N = b.rows;
  p.K = quant_width(a.cols);
  p.format = a.format;
  p.a = a.data;
  p.b = b.data;
  p.scales_a = a.scales;
  p.scales_b = b.scales;
  p.row_scale_a = a.row_scale;
  p.row_scale_b = b.row_scale;
  p.ld_a = a.ld;
  p.ld_b = b.ld;
  const Tensor c = finish_arguments(&p, f, a.index);
  call(quant_product, "quant_product", p, a.index, stream, {&c});
  return c;
}

// p: out dtype code, bias, act, residual, out, static_b, stream, timeout_ns, debug_flags
Finish finish_of(PyObject* const* p) {
  Finish f{};
  const int64_t code = int_of(p[0]);
  TORCH_CHECK_VALUE(code == FFN_BF16 || code == FFN_F32, "the output must be bfloat16 or float32");
  f.dtype = code == FFN_F32 ? at::kFloat : at::kBFloat16;
  f.bias = optional_of(p[1], "bias");
  f.activation = (int32_t)int_of(p[2]);
  f.residual = optional_of(p[3], "residual");
  f.out = optional_of(p[4], "out");
  f.flags = flag_of(p[5]) ? QUANT_STATIC_B : 0;
  f.timeout_ns = int_of(p[7]);
  f.debug_flags = (int32_t)int_of(p[8]);
  return f;
}

// (x, format, transpose, stream) -> an operand's five values
PyObject* quantise(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 4);
  quant_rows_t a{};
  const Operand o = to_quantise(&a, "x", tensor_of(p[0], "x"), format_of(p[1]), flag_of(p[2]));
  call(quant_rows, "quant_rows", a, o.index, p[3], {&o.memory});
  return operand_tuple(o);
  END_HANDLE_TH_ERRORS
}

// (y, residual, weight, format, eps, residual_scale, branch_scale, need_s, s, stream)
// -> (s or None, the operand's five values)
PyObject* norm_quantise(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 10);
  const Tensor &y = tensor_of(p[0], "y"), *residual = optional_of(p[1], "residual"), *weight = optional_of(p[2], "weight"),
               *s_given = optional_of(p[8], "s");
  TORCH_CHECK_VALUE(y.dim() == 2, "y must be a 2-D tensor, not ", y.sizes());
  quant_norm_t a{};
  const int index = index_of(y);
  const at::ScalarType dtype = y.scalar_type();
  a.M = y.size(0);
  a.D = y.size(1);
  a.dtype = a.param_dtype = code_of(dtype);
  TORCH_CHECK_VALUE(a.dtype >= 0, "y must be float16, bfloat16 or float32, not ", dtype);
  a.format = format_of(p[3]);
  a.eps = float_of(p[4]);
  a.residual_scale = float_of(p[5]);
  a.branch_scale = float_of(p[6]);
  a.ld_y = rows_of("y", y, a.M, a.D, dtype, index);
  if (residual != nullptr) a.ld_residual = rows_of("residual", *residual, a.M, a.D, dtype, index);
  if (weight != nullptr) {
    TORCH_CHECK_VALUE(weight->dim() == 1 && weight->size(0) == a.D && weight->is_contiguous() && weight->is_cuda() &&
                          weight->get_device() == index &&
                          (weight->scalar_type() == dtype || weight->scalar_type() == at::kFloat),
                      "weight must be ", a.D, " dense values of ", dtype, " or float32 on cuda:", index);
    a.param_dtype = code_of(weight->scalar_type());
  }
  Tensor s;
  a.ld_s = a.D;
  if (s_given != nullptr) {
    a.ld_s = rows_of("s", *s_given, a.M, a.D, dtype, index);
    s = *s_given;
  } else if (flag_of(p[7])) {
    s = new_rows(a.M, a.D, dtype, index);
  }
  Operand o = empty_operand(a.M, a.D, a.format, index);
  a.y = y.data_ptr();
  a.residual = data_of(residual);
  a.weight = data_of(weight);
  a.s = s.defined() ? s.data_ptr() : nullptr;
  a.data = o.data;
  a.scales = o.scales;
  a.row_scale = o.row_scale;
  call(quant_norm, "quant_norm", a, index, p[9], {&s, &o.memory});
  THPObjectPtr q(operand_tuple(o)), out(PyTuple_New(2));
  if (!out) throw python_error();
  PyTuple_SET_ITEM(out.get(), 0, wrapped(s));
  PyTuple_SET_ITEM(out.get(), 1, q.release());
  return out.release();
  END_HANDLE_TH_ERRORS
}

// (a's five values, b's five, out dtype, bias, act, residual, out, static_b, stream, timeout_ns,
//  debug_flags) -> c
PyObject* product(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 19);
  return wrapped(multiplied(operand_of("a", p), operand_of("b", p + 5), finish_of(p + 10), p[16]));
  END_HANDLE_TH_ERRORS
}

// (x, w's five values, and as product from out dtype on) -> y
PyObject* linear(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 15);
  const Tensor& x = tensor_of(p[0], "x");
  const Operand w = operand_of("w", p + 1);
  const Finish f = finish_of(p + 6);
  TORCH_CHECK_VALUE(x.dim() == 2 && x.size(1) == w.cols, "x must be (M, ", w.cols, "), not ", x.sizes());
  TORCH_CHECK_VALUE(index_of(x) == w.index, "x and w must be on one device");
  const at::ScalarType dtype = x.scalar_type();
  quant_linear_t a{};
  a.M = x.size(0);
  a.N = w.rows;
  a.K = w.cols;
  a.dtype = code_of(dtype);
  TORCH_CHECK_VALUE(a.dtype >= 0, "x must be float16, bfloat16 or float32, not ", dtype);
  a.format = w.format;
  a.ld_x = rows_of("x", x, a.M, a.K, dtype, w.index);
  a.x = x.data_ptr();
  a.b = w.data;
  a.scales_b = w.scales;
  a.row_scale_b = w.row_scale;
  a.ld_b = w.ld;
  const Tensor c = finish_arguments(&a, f, w.index);
  const Tensor workspace = workspace_of(quant_linear_workspace(&a), w.index);
  a.workspace = workspace.defined() ? workspace.data_ptr() : nullptr;
  call(quant_linear, "quant_linear", a, w.index, p[12], {&c, &workspace});
  return wrapped(c);
  END_HANDLE_TH_ERRORS
}

// (dy, x, w, format, need_dx, need_dw, out dtype, stream, timeout_ns) -> (dx or None, dw or None)
PyObject* linear_backward(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 9);
  const Tensor &dy = tensor_of(p[0], "dy"), *x = optional_of(p[1], "x"), *w = optional_of(p[2], "w");
  const int32_t format = format_of(p[3]);
  const bool need_dx = flag_of(p[4]), need_dw = flag_of(p[5]);
  TORCH_CHECK_VALUE(format == QUANT_MXFP4 || format == QUANT_NVFP4, "the format must be a 4-bit one (mxfp4 or nvfp4)");
  TORCH_CHECK_VALUE((!need_dx || w != nullptr) && (!need_dw || x != nullptr), "dx needs w, dw needs x");
  TORCH_CHECK_VALUE(dy.dim() == 2 && (!need_dw || (x->dim() == 2 && x->size(0) == dy.size(0))) &&
                        (!need_dx || (w->dim() == 2 && w->size(0) == dy.size(1))),
                    "dy must be (M, N), x (M, K) and w (N, K)");
  const int index = index_of(dy);
  TORCH_CHECK_VALUE((!need_dw || index_of(*x) == index) && (!need_dx || index_of(*w) == index),
                    "tensors must be on one device");
  Finish f{};
  const int64_t code = int_of(p[6]);
  TORCH_CHECK_VALUE(code == FFN_BF16 || code == FFN_F32, "the output must be bfloat16 or float32");
  f.dtype = code == FFN_F32 ? at::kFloat : at::kBFloat16;
  f.activation = GEMM_ACT_NONE;
  f.timeout_ns = int_of(p[8]);
  Tensor dx, dw;
  // (columns one after the other: they go in few launches)
  Several s{};
  Operand dy_rows, w_columns, dy_columns, x_columns;
  if (need_dx) dy_rows = to_quantise(&s.args[s.count++], "dy", dy, format, false);
  if (need_dw) {
    dy_columns = to_quantise(&s.args[s.count++], "dy", dy, format, true);
    x_columns = to_quantise(&s.args[s.count++], "x", *x, format, true);
  }
  if (need_dx) w_columns = to_quantise(&s.args[s.count++], "w", *w, format, true);
  call(quant_several, "quant_rows_many", s, index, p[7],
       {&dy_rows.memory, &w_columns.memory, &dy_columns.memory, &x_columns.memory});
  if (need_dx) dx = multiplied(dy_rows, w_columns, f, p[7]);
  if (need_dw) dw = multiplied(dy_columns, x_columns, f, p[7]);
  return tuple_of({&dx, &dw});
  END_HANDLE_TH_ERRORS
}

// (GemmError, share, {name: code}, names by code)
PyObject* bind_formats(PyObject* self, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 4);
  TORCH_CHECK_TYPE(PyDict_Check(p[2]) && PyTuple_Check(p[3]) && PyTuple_GET_SIZE(p[3]) == 4, "formats");
  Py_XSETREF(format_codes, Py_NewRef(p[2]));
  Py_XSETREF(format_names, Py_NewRef(p[3]));
  return bind(self, p, 2);
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {method<bind_formats>("bind"), method<quantise>("quantise"), method<norm_quantise>("norm_quantise"),
                         method<product>("product"), method<linear>("linear"),     method<linear_backward>("linear_backward"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_quant_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__quant_calls() { return PyModule_Create(&module); }
