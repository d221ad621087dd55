// The binding's calls whose kernels take a few microseconds, marshalled in C++:
// a call of several tensors costs 4 us of the caller's time through ctypes
// (attribute by attribute, then a structure), 0.5 us here.
//
// Each function checks its tensors' types, sizes, strides and place and makes the
// C ABI's call on them. It returns the status, or None where a check fails: the
// Python side then says which one. A stream is a handle, or None for the current
// one of the first tensor's device.

#include <Python.h>

#include <vector>

#include <torch/csrc/autograd/python_variable.h>

#include "fsdp_shard.h"

namespace {

PyObject* g_current_stream = nullptr;   // device index -> handle

const at::Tensor* tensor(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// A contiguous device tensor of `type` with at least n elements; None is a null
// pointer where that is allowed.
template <typename P>
bool flat(PyObject* o, at::ScalarType type, int64_t n, bool may_be_none, P** p) {
  *p = nullptr;
  if (o == Py_None) return may_be_none;
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda() || t->scalar_type() != type || !t->is_contiguous() || t->numel() < n) return false;
  *p = static_cast<P*>(t->data_ptr());
  return true;
}

// A rows x dim device tensor of `type` whose rows are contiguous and do not overlap.
template <typename P>
bool matrix(PyObject* o, at::ScalarType type, int64_t rows, int64_t dim, bool may_be_none, P** p, int64_t* ld) {
  *p = nullptr;
  *ld = 0;
  if (o == Py_None) return may_be_none;
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda() || t->scalar_type() != type || t->dim() != 2 || t->size(0) != rows || t->size(1) != dim)
    return false;
  *ld = rows <= 1 ? dim : t->stride(0);
  if ((dim > 1 && t->stride(1) != 1) || *ld < dim) return false;
  *p = static_cast<P*>(t->data_ptr());
  return true;
}

bool stream_of(PyObject* o, const at::Tensor& first, hipStream_t* s) {
  PyObject* handle = nullptr;
  if (o == Py_None) {
    PyObject* index = PyLong_FromLong(first.get_device());
    if (!index) return false;
    handle = PyObject_CallFunctionObjArgs(g_current_stream, index, nullptr);
    Py_DECREF(index);
    if (!handle) return false;
  } else {
    Py_INCREF(handle = o);
  }
  *s = static_cast<hipStream_t>(PyLong_AsVoidPtr(handle));
  Py_DECREF(handle);
  return !PyErr_Occurred();
}

bool wants(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) PyErr_Format(PyExc_TypeError, "need %zd arguments, got %zd", want, n);
  return n == want;
}

template <typename F>
PyObject* status_of(F&& call) {
  fsdp_status st;
  Py_BEGIN_ALLOW_THREADS
  st = call();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

bool element_type(const at::Tensor& x, fsdp_dtype* code) {
  *code = x.scalar_type() == at::kFloat ? FSDP_F32 : FSDP_BF16;
  return x.dim() == 2 && (x.scalar_type() == at::kFloat || x.scalar_type() == at::kBFloat16);
}

// x, weight, out, residual, residual_out, rstd, scales, eps, stream
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!wants(n, 9)) return nullptr;
  fsdp_rms_norm_args c{};
  c.eps = PyFloat_AsDouble(a[7]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor* x = tensor(a[0]);
  if (!x || !element_type(*x, &c.dtype)) Py_RETURN_NONE;
  const at::ScalarType type = x->scalar_type();
  c.rows = x->size(0);
  c.dim = x->size(1);
  if ((a[3] == Py_None) != (a[4] == Py_None) ||
      !matrix(a[0], type, c.rows, c.dim, false, &c.x, &c.x_pitch) ||
      !matrix(a[2], a[6] == Py_None ? type : at::kFloat8_e4m3fn, c.rows, c.dim, false, &c.out, &c.out_pitch) ||
      !matrix(a[3], type, c.rows, c.dim, true, &c.residual, &c.residual_pitch) ||
      !matrix(a[4], type, c.rows, c.dim, true, &c.residual_out, &c.residual_out_pitch) ||
      !flat(a[1], type, c.dim, false, &c.weight) || !flat(a[5], at::kFloat, c.rows, true, &c.rstd) ||
      !flat(a[6], at::kFloat, c.rows, true, &c.scales))
    Py_RETURN_NONE;
  hipStream_t s;
  if (!stream_of(a[8], *x, &s)) return nullptr;
  return status_of([&] { return fsdp_rms_norm(&c, s); });
}

// dy, x, weight, rstd, dx, dweight, workspace, dresidual, stream
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!wants(n, 9)) return nullptr;
  fsdp_rms_norm_backward_args c{};
  const at::Tensor* x = tensor(a[1]);
  if (!x || !element_type(*x, &c.dtype)) Py_RETURN_NONE;
  const at::ScalarType type = x->scalar_type();
  c.rows = x->size(0);
  c.dim = x->size(1);
  if (!matrix(a[0], type, c.rows, c.dim, false, &c.dy, &c.dy_pitch) ||
      !matrix(a[1], type, c.rows, c.dim, false, &c.x, &c.x_pitch) ||
      !matrix(a[4], type, c.rows, c.dim, false, &c.dx, &c.dx_pitch) ||
      !matrix(a[7], type, c.rows, c.dim, true, &c.dresidual, &c.dresidual_pitch) ||
      !flat(a[2], type, c.dim, false, &c.weight) || !flat(a[3], at::kFloat, c.rows, false, &c.rstd) ||
      !flat(a[5], type, c.dim, true, &c.dweight))
    Py_RETURN_NONE;
  if (c.dweight && a[6] != Py_None) {
    if (!flat(a[6], at::kByte, 0, false, &c.workspace)) Py_RETURN_NONE;
    c.workspace_bytes = tensor(a[6])->numel();
  }
  hipStream_t s;
  if (!stream_of(a[8], *x, &s)) return nullptr;
  return status_of([&] { return fsdp_rms_norm_backward(&c, s); });
}

// lr, momentum, weight decay, nesterov
bool hparams(PyObject* const* a, double grad_scale, fsdp_muon_hparams* hp) {
  hp->lr = PyFloat_AsDouble(a[0]);
  hp->momentum = PyFloat_AsDouble(a[1]);
  hp->weight_decay = PyFloat_AsDouble(a[2]);
  hp->nesterov = PyObject_IsTrue(a[3]);
  hp->grad_scale = grad_scale;
  return !PyErr_Occurred();
}

struct Items {                       // a list's or tuple's elements
  explicit Items(PyObject* o) : seq(PySequence_Fast(o, "a list or tuple is needed")) {}
  ~Items() { Py_XDECREF(seq); }
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
  PyObject* seq;
};

// unit, its elements, its window's elements, grads, momentum, update, lr, momentum,
// weight decay, nesterov, gradient scale, stream
PyObject* reduce_momentum_shard(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!wants(n, 12)) return nullptr;
  const fsdp_unit* unit = static_cast<const fsdp_unit*>(PyLong_AsVoidPtr(a[0]));
  const int64_t total = PyLong_AsLongLong(a[1]), valid = PyLong_AsLongLong(a[2]);
  const double scale = PyFloat_AsDouble(a[10]);
  fsdp_muon_hparams hp{};
  if (PyErr_Occurred() || !hparams(a + 6, scale, &hp)) return nullptr;
  const Items grads(a[3]);
  if (!grads.seq) return nullptr;
  const Py_ssize_t rows = grads.size();
  if (rows < 1 || rows > FSDP_MAX_RANKS) Py_RETURN_NONE;
  const void* g[FSDP_MAX_RANKS];
  for (Py_ssize_t k = 0; k < rows; ++k)
    if (!flat(grads[k], at::kBFloat16, total, false, &g[k])) Py_RETURN_NONE;
  float* m;
  void* u;
  if (!flat(a[4], at::kFloat, valid, false, &m) || !flat(a[5], at::kBFloat16, valid, false, &u)) Py_RETURN_NONE;
  hipStream_t s;
  if (!stream_of(a[11], *tensor(a[4]), &s)) return nullptr;
  return status_of([&] { return fsdp_reduce_momentum_shard(unit, int32_t(rows), g, m, u, &hp, s); });
}

// unit, its tensors' elements, its window's begin and elements, tensors, scales, master,
// parameter, lr, momentum, weight decay, nesterov, stream. A tensor and a scale that do not
// reach into the window may be None.
PyObject* muon_apply_shard(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!wants(n, 13)) return nullptr;
  const fsdp_unit* unit = static_cast<const fsdp_unit*>(PyLong_AsVoidPtr(a[0]));
  const int64_t begin = PyLong_AsLongLong(a[2]), valid = PyLong_AsLongLong(a[3]);
  fsdp_muon_hparams hp{};
  if (PyErr_Occurred() || !hparams(a + 8, 0.0, &hp)) return nullptr;
  const Items sizes(a[1]), tensors(a[4]), scales(a[5]);
  if (!sizes.seq || !tensors.seq || !scales.seq) return nullptr;
  const Py_ssize_t count = sizes.size();
  if (tensors.size() != count || scales.size() != count) Py_RETURN_NONE;
  std::vector<const void*> t(static_cast<size_t>(count) + 1);
  std::vector<double> k(static_cast<size_t>(count) + 1);
  int64_t offset = 0;
  for (Py_ssize_t i = 0; i < count; ++i) {
    const int64_t need = PyLong_AsLongLong(sizes[i]);
    const bool outside = offset + need <= begin || offset >= begin + valid || need == 0;
    offset += need;
    if (!outside || scales[i] != Py_None) k[i] = PyFloat_AsDouble(scales[i]);
    if (PyErr_Occurred()) return nullptr;
    if (!flat(tensors[i], at::kBFloat16, need, outside, &t[i])) Py_RETURN_NONE;
  }
  float* p;
  void* w;
  if (!flat(a[6], at::kFloat, valid, false, &p) || !flat(a[7], at::kBFloat16, valid, true, &w)) Py_RETURN_NONE;
  hipStream_t s;
  if (!stream_of(a[12], *tensor(a[6]), &s)) return nullptr;
  return status_of([&] { return fsdp_muon_apply_shard(unit, t.data(), k.data(), p, w, &hp, s); });
}

// The function that gives a device's current stream.
PyObject* set_current_stream(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_current_stream, f);
  Py_RETURN_NONE;
}

// The C ABI throws nothing; what torch or the containers throw becomes a Python error.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<rms_norm>("rms_norm"),
    method<rms_norm_backward>("rms_norm_backward"),
    method<reduce_momentum_shard>("reduce_momentum_shard"),
    method<muon_apply_shard>("muon_apply_shard"),
    {"set_current_stream", set_current_stream, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__calls() { return PyModule_Create(&g_module); }
