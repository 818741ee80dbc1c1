// python_calls.h -- what the Python extensions (ffn_python.cpp, quant_python.cpp) share: checks
// of tensors, allocation, the call on a stream, errors.
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <initializer_list>
#include <optional>

#include "ffn.h"

namespace {

PyObject* gemm_error = nullptr;  // the exception of a status
PyObject* share = nullptr;       // share(stream, device index, tensors) -> the stream's handle

using at::Tensor;

const Tensor& tensor_of(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor, not ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
const Tensor* optional_of(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor_of(o, name); }
void* data_of(const Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }
bool flag_of(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
int64_t int_of(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
float float_of(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)v;
}

int index_of(const Tensor& t) {
  TORCH_CHECK_VALUE(t.is_cuda(), "tensors must be on a CUDA device");
  return (int)t.get_device();
}

int code_of(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return FFN_F16;
    case at::kBFloat16: return FFN_BF16;
    case at::kFloat: return FFN_F32;
    default: return -1;
  }
}

// A tensor of dense rows, M x N, of one type and device: its pitch.
int64_t rows_of(const char* name, const Tensor& t, int64_t M, int64_t N, at::ScalarType dtype, int index) {
  TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == M && t.size(1) == N && t.scalar_type() == dtype && t.is_cuda() &&
                        t.get_device() == index,
                    name, " must be (", M, ", ", N, ") of ", dtype, " on cuda:", index, ", not ", t.sizes(), " of ",
                    t.scalar_type(), " on ", t.device());
  if (t.is_contiguous()) return N;
  const int64_t pitch = t.stride(0);
  TORCH_CHECK_VALUE((N <= 1 || t.stride(1) == 1) && (M <= 1 || pitch >= N), name,
                    " must have dense, non-overlapping rows");
  return M > 1 ? pitch : N;
}

Tensor empty_rows(int64_t M, int64_t N, at::ScalarType dtype, int index) {
  return at::empty({M, N}, at::TensorOptions().dtype(dtype).device(at::kCUDA, (c10::DeviceIndex)index));
}

// (a refused call asks for -1 bytes and is refused when it is made)
Tensor workspace_of(int64_t bytes, int index) {
  if (bytes <= 0) return Tensor();
  return at::empty({bytes}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, (c10::DeviceIndex)index));
}

// The call on the given stream, or the current one.  `made`: memory of this call, which
// another stream has to know of.
template <typename Args>
void call(gemm_status_t (*f)(const Args*, gemm_stream_t), const char* name, const Args& args, int index,
          PyObject* stream, std::initializer_list<const Tensor*> made) {
  gemm_stream_t handle;
  if (stream == Py_None) {
    handle = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
  } else {
    THPObjectPtr list(PyList_New(0));
    if (!list) throw python_error();
    for (const Tensor* t : made) {
      if (t == nullptr || !t->defined()) continue;
      THPObjectPtr o(THPVariable_Wrap(*t));
      if (!o || PyList_Append(list.get(), o.get()) != 0) throw python_error();
    }
    THPObjectPtr h(PyObject_CallFunction(share, "OiO", stream, index, list.get()));
    if (!h) throw python_error();
    handle = reinterpret_cast<gemm_stream_t>(PyLong_AsVoidPtr(h.get()));
    if (PyErr_Occurred()) throw python_error();
  }
  gemm_status_t status;
  {
    pybind11::gil_scoped_release no_gil;
    const c10::cuda::OptionalCUDAGuard guard(
        c10::cuda::current_device() == index ? std::nullopt
                                             : std::optional<c10::Device>(c10::Device(at::kCUDA, (c10::DeviceIndex)index)));
    status = f(&args, handle);
  }
  if (status != GEMM_OK) {
    THPObjectPtr e(PyObject_CallFunction(gemm_error, "is", (int)status, name));
    if (e) PyErr_SetObject(gemm_error, e.get());
    throw python_error();
  }
}

void expect(Py_ssize_t got, Py_ssize_t want) {
  TORCH_CHECK_TYPE(got == want, "takes ", want, " arguments, not ", got);
}

PyObject* wrapped(const Tensor& t) {
  PyObject* o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
  if (o == nullptr) throw python_error();
  return o;
}
PyObject* tuple_of(std::initializer_list<const Tensor*> tensors) {
  THPObjectPtr out(PyTuple_New((Py_ssize_t)tensors.size()));
  if (!out) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor* t : tensors) PyTuple_SET_ITEM(out.get(), i++, wrapped(*t));
  return out.release();
}

// (GemmError, share): what `gemm_error` and `share` are
PyObject* bind(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 2);
  Py_XSETREF(gemm_error, Py_NewRef(p[0]));
  Py_XSETREF(share, Py_NewRef(p[1]));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, (PyCFunction)(void (*)())f, METH_FASTCALL, nullptr};
}

}  // namespace
