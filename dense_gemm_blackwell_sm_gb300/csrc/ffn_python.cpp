// ffn_python.cpp -- what ffn.py calls: checks of the tensors, allocation of the outputs and
// the call of include/ffn.h, as a Python extension.  The operators' small calls take
// less time on the device than their marshalling does in Python (a norm of one token:
// 2.7 us on the device, 14.8 us a call through ctypes), hence this file.
//
// Every function takes its arguments by position (ffn.py has the names and defaults) and
// raises as torch does: ValueError for a refused argument, torch.OutOfMemoryError, and
// the binding's GemmError for a status of the library.
#include "python_calls.h"

namespace {

// ------------------------------------------------------------ gated projections

// x (M, K) and w (2F, K): sizes, type, device and pitches of both
template <typename Args>
int gated_inputs(Args* a, const Tensor& x, const Tensor& w, at::ScalarType* dtype) {
  TORCH_CHECK_VALUE(x.dim() == 2 && w.dim() == 2 && w.size(0) % 2 == 0 && x.size(1) == w.size(1),
                    "x must be (M, K) and w (2F, K), not ", x.sizes(), " and ", w.sizes());
  const int index = index_of(x);
  *dtype = x.scalar_type();
  TORCH_CHECK_VALUE(*dtype == at::kHalf || *dtype == at::kBFloat16, "x must be float16 or bfloat16, not ", *dtype);
  a->M = x.size(0);
  a->K = x.size(1);
  a->F = w.size(0) / 2;
  a->dtype = code_of(*dtype);
  a->ld_x = rows_of("x", x, a->M, a->K, *dtype, index);
  a->ld_w = rows_of("w", w, 2 * a->F, a->K, *dtype, index);
  a->x = x.data_ptr();
  a->w = w.data_ptr();
  return index;
}

// (x, w, act, save, out, gu, stream, timeout_ns, debug_flags) -> (h, gu or None)
PyObject* gated(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 9);
  ffn_gated_t a{};
  at::ScalarType dtype;
  const int index = gated_inputs(&a, tensor_of(p[0], "x"), tensor_of(p[1], "w"), &dtype);
  a.activation = (int32_t)int_of(p[2]);
  const Tensor *out = optional_of(p[4], "out"), *kept = optional_of(p[5], "gu");
  a.ld_h = a.F;
  a.ld_gu = 2 * a.F;
  Tensor h, gu;
  if (out != nullptr) a.ld_h = rows_of("out", *out, a.M, a.F, dtype, index);
  h = out != nullptr ? *out : empty_rows(a.M, a.F, dtype, index);
  if (kept != nullptr) {
    a.ld_gu = rows_of("gu", *kept, a.M, 2 * a.F, dtype, index);
    gu = *kept;
  } else if (flag_of(p[3])) {
    gu = empty_rows(a.M, 2 * a.F, dtype, index);
  }
  a.h = h.data_ptr();
  a.gu = gu.defined() ? gu.data_ptr() : nullptr;
  a.timeout_ns = int_of(p[7]);
  a.debug_flags = (int32_t)int_of(p[8]);
  call(ffn_gated, "ffn_gated", a, index, p[6], {&h, &gu});
  return tuple_of({&h, &gu});
  END_HANDLE_TH_ERRORS
}

// (dh, x, w, gu, act, need_dx, need_dw, stream, timeout_ns, debug_flags) -> (dx, dw)
PyObject* gated_backward(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 10);
  ffn_gated_grad_t a{};
  at::ScalarType dtype;
  const int index = gated_inputs(&a, tensor_of(p[1], "x"), tensor_of(p[2], "w"), &dtype);
  const Tensor &dh = tensor_of(p[0], "dh"), *gu = optional_of(p[3], "gu");
  a.ld_dh = rows_of("dh", dh, a.M, a.F, dtype, index);
  if (gu != nullptr) a.ld_gu = rows_of("gu", *gu, a.M, 2 * a.F, dtype, index);
  a.activation = (int32_t)int_of(p[4]);
  a.ld_dgu = (2 * a.F + 7) / 8 * 8;
  a.ld_dx = a.ld_dw = a.K;
  const Tensor dgu = empty_rows(a.M, a.ld_dgu, dtype, index);
  Tensor dx, dw;
  if (flag_of(p[5])) dx = empty_rows(a.M, a.K, dtype, index);
  if (flag_of(p[6])) dw = empty_rows(2 * a.F, a.K, dtype, index);
  a.dh = dh.data_ptr();
  a.gu = data_of(gu);
  a.dgu = dgu.data_ptr();
  a.dx = dx.defined() ? dx.data_ptr() : nullptr;
  a.dw = dw.defined() ? dw.data_ptr() : nullptr;
  a.timeout_ns = int_of(p[8]);
  a.debug_flags = (int32_t)int_of(p[9]);
  const Tensor workspace = workspace_of(ffn_gated_backward_workspace(&a), index);
  a.workspace = workspace.defined() ? workspace.data_ptr() : nullptr;
  call(ffn_gated_backward, "ffn_gated_backward", a, index, p[7], {&dgu, &dx, &dw, &workspace});
  return tuple_of({&dx, &dw});
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------------ norms

struct Parameters {
  const Tensor *gate, *post_weight, *post_bias, *pre_weight, *pre_bias;
};

// What both directions share: sizes, types, the gate and the vectors; p: post_norm,
// post_weight, post_bias, gate, pre_norm, pre_weight, pre_bias, kind, eps, residual_scale,
// branch_scale.
template <typename Args>
Parameters norm_parameters(Args* a, const Tensor& like, PyObject* const* p, int* index) {
  TORCH_CHECK_VALUE(like.dim() == 2, "rows must be a 2-D tensor, not ", like.sizes());
  const bool post = flag_of(p[0]), pre = flag_of(p[4]);
  const Parameters v{optional_of(p[3], "gate"), optional_of(p[1], "post_weight"), optional_of(p[2], "post_bias"),
                     optional_of(p[5], "pre_weight"), optional_of(p[6], "pre_bias")};
  const at::ScalarType dtype = like.scalar_type();
  *index = index_of(like);
  a->M = like.size(0);
  a->D = like.size(1);
  a->dtype = code_of(dtype);
  TORCH_CHECK_VALUE(a->dtype >= 0, "rows must be float16, bfloat16 or float32, not ", dtype);
  TORCH_CHECK_VALUE(post || (!v.post_weight && !v.post_bias), "post_weight and post_bias need post_norm");
  TORCH_CHECK_VALUE(pre || (!v.pre_weight && !v.pre_bias), "pre_weight and pre_bias need pre_norm");
  std::optional<at::ScalarType> param;
  a->groups = 1;
  a->ld_gate = a->D;
  if (v.gate != nullptr) {
    const Tensor& g = *v.gate;
    param = g.scalar_type();
    if (g.dim() == 2) a->groups = g.size(0);
    TORCH_CHECK_VALUE((g.dim() == 1 || g.dim() == 2) && a->groups >= 1 && a->M % a->groups == 0,
                      "gate must be (D) or (groups, D) with the rows a multiple of the groups");
    if (g.dim() == 2) a->ld_gate = rows_of("gate", g, a->groups, a->D, *param, *index);
    a->gate = g.data_ptr();
  }
  for (const Tensor* t : {v.gate, v.post_weight, v.post_bias, v.pre_weight, v.pre_bias}) {
    if (t == nullptr || (t == v.gate && t->dim() == 2)) continue;
    if (!param) param = t->scalar_type();
    TORCH_CHECK_VALUE(t->dim() == 1 && t->size(0) == a->D && t->scalar_type() == *param && t->is_cuda() &&
                          t->get_device() == *index && t->is_contiguous(),
                      "weights, biases and a single gate must be ", a->D, " dense values of ", *param, " on cuda:", *index);
  }
  TORCH_CHECK_VALUE(!param || *param == dtype || *param == at::kFloat, "weights, biases and gate must be ", dtype,
                    " or float32, not ", *param);
  a->param_dtype = code_of(param.value_or(dtype));
  a->post_weight = data_of(v.post_weight);
  a->post_bias = data_of(v.post_bias);
  a->pre_weight = data_of(v.pre_weight);
  a->flags = (post ? FFN_NORM_POST : 0) | (pre ? FFN_NORM_PRE : 0);
  a->kind = (int32_t)int_of(p[7]);
  a->eps = float_of(p[8]);
  a->residual_scale = float_of(p[9]);
  a->branch_scale = float_of(p[10]);
  return v;
}

// (y, residual, post_norm, post_weight, post_bias, gate, pre_norm, pre_weight, pre_bias,
//  kind, eps, residual_scale, branch_scale, need_s, s, n, stream) -> (s or None, n or None)
PyObject* block_norm(PyObject*, PyObject* const* p, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  expect(nargs, 17);
  ffn_norm_t a{};
  int index;
  const Tensor &y = tensor_of(p[0], "y"), *residual = optional_of(p[1], "residual");
  const Parameters v = norm_parameters(&a, y, p + 2, &index);
  const at::ScalarType dtype = y.scalar_type();
  a.pre_bias = data_of(v.pre_bias);
  a.ld_residual = a.ld_s = a.ld_n = a.D;
  a.ld_y = rows_of("y", y, a.M, a.D, dtype, index);
  if (residual != nullptr) a.ld_residual = rows_of("residual", *residual, a.M, a.D, dtype, index);
  const Tensor *s_given = optional_of(p[14], "s"), *n_given = optional_of(p[15], "n");
  const bool pre = (a.flags & FFN_NORM_PRE) != 0;
  TORCH_CHECK_VALUE(n_given == nullptr || pre, "n needs pre_norm");
  if (s_given != nullptr) a.ld_s = rows_of("s", *s_given, a.M, a.D, dtype, index);
  if (n_given != nullptr) a.ld_n = rows_of("n", *n_given, a.M, a.D, dtype, index);
  Tensor s, n;
  if (s_given != nullptr) {
    s = *s_given;
  } else if (flag_of(p[13])) {
    s = empty_rows(a.M, a.D, dtype, index);
  }
  if (n_given != nullptr) {
    n = *n_given;
  } else if (pre) {
    n = empty_rows(a.M, a.D, dtype, index);
  }
  a.y = y.data_ptr();
  a.residual = data_of(residual);
  a.s = s.defined() ? s.data_ptr() : nullptr;
  a.n = n.defined() ? n.data_ptr() : nullptr;
  call(ffn_norm, "ffn_norm", a, index, p[16], {&s, &n});
  return tuple_of({&s, &n});
  END_HANDLE_TH_ERRORS
}

// (ds, dn, y, s, post_norm, post_weight, post_bias, gate, pre_norm, pre_weight, pre_bias,
//  kind, eps, residual_scale, branch_scale, need_dresidual, need_dy, need_dparams, stream)
// -> the seven gradients, None where there is none
PyObject* block_norm_backward(PyObject*, PyObject* const* p, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  expect(nargs, 19);
  const Tensor *ds = optional_of(p[0], "ds"), *dn = optional_of(p[1], "dn"), *y = optional_of(p[2], "y"),
               *s = optional_of(p[3], "s");
  const bool post = flag_of(p[4]), pre = flag_of(p[8]), params = flag_of(p[17]);
  TORCH_CHECK_VALUE(ds != nullptr || dn != nullptr, "ds or dn must be given");
  TORCH_CHECK_VALUE(pre ? dn != nullptr && s != nullptr : dn == nullptr,
                    "dn and s are needed with pre_norm, and dn only then");
  TORCH_CHECK_VALUE(y != nullptr || (!post && !(p[7] != Py_None && params)),
                    "y is needed with post_norm or a gate");
  ffn_norm_grad_t a{};
  int index;
  const Tensor& like = dn != nullptr ? *dn : *ds;
  const Parameters v = norm_parameters(&a, like, p + 4, &index);
  const at::ScalarType dtype = like.scalar_type();
  a.ld_ds = a.ld_dn = a.ld_y = a.ld_s = a.ld_dresidual = a.ld_dy = a.D;
  if (ds != nullptr) a.ld_ds = rows_of("ds", *ds, a.M, a.D, dtype, index);
  if (dn != nullptr) a.ld_dn = rows_of("dn", *dn, a.M, a.D, dtype, index);
  if (y != nullptr) a.ld_y = rows_of("y", *y, a.M, a.D, dtype, index);
  if (s != nullptr) a.ld_s = rows_of("s", *s, a.M, a.D, dtype, index);
  a.ds = data_of(ds);
  a.dn = data_of(dn);
  a.y = data_of(y);
  a.s = data_of(s);
  Tensor dresidual, dy, dgate, dpost_weight, dpost_bias, dpre_weight, dpre_bias, workspace;
  if (flag_of(p[15])) a.dresidual = (dresidual = empty_rows(a.M, a.D, dtype, index)).data_ptr();
  if (flag_of(p[16])) a.dy = (dy = empty_rows(a.M, a.D, dtype, index)).data_ptr();
  const auto f32 = at::TensorOptions().dtype(at::kFloat).device(at::kCUDA, (c10::DeviceIndex)index);
  auto gradient = [&](const Tensor* of, Tensor& g) -> float* {
    if (of == nullptr || !params) return nullptr;
    g = at::empty(of->sizes(), f32);
    return g.data_ptr<float>();
  };
  a.dgate = gradient(v.gate, dgate);
  a.dpost_weight = gradient(v.post_weight, dpost_weight);
  a.dpost_bias = gradient(v.post_bias, dpost_bias);
  a.dpre_weight = gradient(v.pre_weight, dpre_weight);
  a.dpre_bias = gradient(v.pre_bias, dpre_bias);
  workspace = workspace_of(ffn_norm_backward_workspace(&a), index);
  a.workspace = workspace.defined() ? workspace.data_ptr() : nullptr;
  call(ffn_norm_backward, "ffn_norm_backward", a, index, p[18],
       {&dresidual, &dy, &dgate, &dpost_weight, &dpost_bias, &dpre_weight, &dpre_bias, &workspace});
  return tuple_of({&dresidual, &dy, &dgate, &dpost_weight, &dpost_bias, &dpre_weight, &dpre_bias});
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {method<bind>("bind"), method<gated>("gated"), method<gated_backward>("gated_backward"),
                         method<block_norm>("block_norm"), method<block_norm_backward>("block_norm_backward"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ffn_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__ffn_calls() { return PyModule_Create(&module); }
