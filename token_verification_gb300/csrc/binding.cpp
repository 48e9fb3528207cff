// binding.cpp - the Python binding's short way to the draft operators
// (spec_top_logits, spec_distill, spec_distill_grad, spec_beam_select,
// spec_beam_reorder): argument checks, output allocation and the C call in one
// step.  From Python the same steps take 10 to 15 us a call, longer than the
// kernels of a single request.
//
// It handles the plain case only - CUDA tensors on the current device, of the
// right types and shapes, outputs allocated here - and answers None to
// anything else; api.py then takes the long way, which checks each argument
// and says what is wrong.  Otherwise it returns the outputs, or the C call's
// status when that is not SV_OK.  The C functions come in as addresses
// (init), so that this module and ctypes use one loaded library.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/spec_verify.h"

namespace {

decltype(&spec_top_logits) g_top;
decltype(&spec_distill) g_distill;
decltype(&spec_distill_grad) g_distill_grad;
decltype(&spec_beam_select) g_select;
decltype(&spec_beam_workspace_size) g_select_ws;
decltype(&spec_beam_reorder) g_reorder;

using at::Tensor;

PyObject* long_way() { Py_RETURN_NONE; }

// A tensor argument, or null.
const Tensor* tensor(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// Contiguous on the device, of a type and of up to three extents.
bool fits(const Tensor* t, c10::Device d, at::ScalarType type, at::IntArrayRef shape) {
  return t && t->scalar_type() == type && t->device() == d && t->is_contiguous() &&
         t->sizes() == shape;
}

// An optional one: None or fitting.
bool fits_or_none(PyObject* o, c10::Device d, at::ScalarType type, at::IntArrayRef shape,
                  const Tensor** out) {
  *out = nullptr;
  if (o == Py_None) return true;
  *out = tensor(o);
  return fits(*out, d, type, shape);
}

// Logits [a, b, V]: their sv_dtype, or -1 when they are not the plain case.
int logits_type(const Tensor* t) {
  if (!t || t->dim() != 3 || !t->is_cuda() || !t->is_contiguous() ||
      t->device().index() != c10::cuda::current_device())
    return -1;
  if (t->scalar_type() == at::kBFloat16) return SV_BF16;
  return t->scalar_type() == at::kFloat ? SV_F32 : -1;
}

bool number(PyObject* o, double* v) {
  *v = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

bool size(PyObject* o, int64_t lo, int64_t hi, int64_t* v) {
  if (!PyLong_Check(o)) return false;
  *v = PyLong_AsLongLong(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return *v >= lo && *v <= hi;
}

bool small(const Tensor& t) {  // extents the C interface can take
  for (int64_t n : t.sizes())
    if (n > INT32_MAX) return false;
  return true;
}

template <class T>
T* data(const Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

Tensor make(c10::Device d, at::ScalarType type, at::IntArrayRef shape) {
  return Tensor(at::detail::empty_cuda(shape, type, d, std::nullopt));
}

sv_stream_t stream_of(c10::Device d) {
  return reinterpret_cast<sv_stream_t>(c10::cuda::getCurrentCUDAStream(d.index()).stream());
}

// The outputs as a tuple (None for undefined ones), or the status.
template <size_t N>
PyObject* answer(sv_status rc, const Tensor (&out)[N]) {
  if (rc != SV_OK) return PyLong_FromLong(rc);
  PyObject* t = PyTuple_New(N);
  if (!t) return nullptr;
  for (size_t i = 0; i < N; ++i) {
    PyObject* o = nullptr;
    if (out[i].defined()) {
      o = THPVariable_Wrap(out[i]);
      if (!o) {
        Py_DECREF(t);
        return nullptr;
      }
    } else {
      o = Py_None;
      Py_INCREF(o);
    }
    PyTuple_SET_ITEM(t, (Py_ssize_t)i, o);
  }
  return t;
}

// C++ exceptions end here: an allocation that fails is Python's MemoryError
// from the long way (which allocates again and says so).
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
    return long_way();
  }
}

// top_logits(logits, k, temperature, lens, status)
PyObject* top_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) return long_way();
  return guarded([&]() -> PyObject* {
    const Tensor* x = tensor(a[0]);
    const int type = logits_type(x);
    int64_t k;
    double T;
    if (type < 0 || !small(*x) || !size(a[1], 1, SV_MAX_TOP, &k) || !number(a[2], &T))
      return long_way();
    const c10::Device d = x->device();
    const int64_t B = x->size(0), P = x->size(1);
    const Tensor* lens;
    if (!fits_or_none(a[3], d, at::kInt, {B}, &lens)) return long_way();
    const Tensor out[4] = {make(d, at::kInt, {B, P, k}), make(d, at::kFloat, {B, P, k}),
                           make(d, at::kFloat, {B, P}),
                           a[4] == Py_True ? make(d, at::kInt, {B, P}) : Tensor()};
    return answer(g_top(x->data_ptr(), (int)k, (float)T, data<int32_t>(lens),
                        data<int32_t>(&out[0]), data<float>(&out[1]), data<float>(&out[2]),
                        out[3].defined() ? data<int32_t>(&out[3]) : nullptr, (sv_dtype)type,
                        (int)B, (int)P, (int)x->size(2), stream_of(d)),
                  out);
  });
}

struct Record {
  const Tensor *student, *ids, *logits, *lse, *lens, *grad_loss;
  int type;
  int64_t B, P, V, k;
};

bool record(Record& r, PyObject* student, PyObject* ids, PyObject* logits, PyObject* lse,
            PyObject* lens, PyObject* grad_loss) {
  r.student = tensor(student);
  r.type = logits_type(r.student);
  r.ids = tensor(ids);
  if (r.type < 0 || !small(*r.student) || !r.ids || r.ids->dim() != 3) return false;
  const c10::Device d = r.student->device();
  r.B = r.student->size(0);
  r.P = r.student->size(1);
  r.V = r.student->size(2);
  r.k = r.ids->size(2);
  if (r.k > SV_MAX_TOP) return false;
  r.logits = tensor(logits);
  return fits(r.ids, d, at::kInt, {r.B, r.P, r.k}) && fits(r.logits, d, at::kFloat, {r.B, r.P, r.k}) &&
         fits_or_none(lse, d, at::kFloat, {r.B, r.P}, &r.lse) &&
         fits_or_none(lens, d, at::kInt, {r.B}, &r.lens) &&
         fits_or_none(grad_loss, d, at::kFloat, {r.B, r.P}, &r.grad_loss);
}

// distill(student, ids, logits, temperature, lse, lens, grad_loss, stats, status)
PyObject* distill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 9) return long_way();
  return guarded([&]() -> PyObject* {
    Record r;
    double T;
    if (!record(r, a[0], a[1], a[2], a[4], a[5], a[6]) || !number(a[3], &T)) return long_way();
    const c10::Device d = r.student->device();
    const Tensor out[4] = {
        make(d, at::kFloat, {r.B, r.P}),
        a[7] == Py_True ? make(d, at::kFloat, {r.B, r.P, 4}) : Tensor(),
        r.grad_loss ? make(d, r.student->scalar_type(), r.student->sizes()) : Tensor(),
        a[8] == Py_True ? make(d, at::kInt, {r.B, r.P}) : Tensor()};
    return answer(
        g_distill(r.student->data_ptr(), data<int32_t>(r.ids), data<float>(r.logits),
                  data<float>(r.lse), data<int32_t>(r.lens), data<float>(r.grad_loss), (float)T,
                  data<float>(&out[0]), out[1].defined() ? data<float>(&out[1]) : nullptr,
                  out[2].defined() ? out[2].data_ptr() : nullptr,
                  out[3].defined() ? data<int32_t>(&out[3]) : nullptr, (sv_dtype)r.type, (int)r.B,
                  (int)r.P, (int)r.V, (int)r.k, stream_of(d)),
        out);
  });
}

// distill_grad(student, ids, logits, temperature, stats, grad_loss, lse, lens)
PyObject* distill_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8 || a[5] == Py_None) return long_way();
  return guarded([&]() -> PyObject* {
    Record r;
    double T;
    if (!record(r, a[0], a[1], a[2], a[6], a[7], a[5]) || !number(a[3], &T)) return long_way();
    const c10::Device d = r.student->device();
    const Tensor* stats = tensor(a[4]);
    if (!fits(stats, d, at::kFloat, {r.B, r.P, 4})) return long_way();
    const Tensor out[1] = {make(d, r.student->scalar_type(), r.student->sizes())};
    return answer(g_distill_grad(r.student->data_ptr(), data<int32_t>(r.ids),
                                 data<float>(r.logits), data<float>(r.lse), data<int32_t>(r.lens),
                                 data<float>(stats), data<float>(r.grad_loss), (float)T,
                                 out[0].data_ptr(), (sv_dtype)r.type, (int)r.B, (int)r.P,
                                 (int)r.V, (int)r.k, stream_of(d)),
                  out);
  });
}

// beam_select(logits, scores, n, status)
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (nargs != 4) return long_way();
  return guarded([&]() -> PyObject* {
    const Tensor* x = tensor(a[0]);
    const int type = logits_type(x);
    int64_t n;
    if (type < 0 || !small(*x) || !size(a[2], 1, SV_MAX_TOP, &n)) return long_way();
    const c10::Device d = x->device();
    const int64_t B = x->size(0), W = x->size(1);
    const Tensor* scores = tensor(a[1]);
    if (!fits(scores, d, at::kFloat, {B, W})) return long_way();
    const Tensor out[4] = {make(d, at::kInt, {B, n}), make(d, at::kInt, {B, n}),
                           make(d, at::kFloat, {B, n}),
                           a[3] == Py_True ? make(d, at::kInt, {B}) : Tensor()};
    const size_t need = g_select_ws((sv_dtype)type, (int)B, (int)W, (int)x->size(2), (int)n);
    // scratch of this call alone (stream-ordered, and a captured graph's own)
    const Tensor ws = need ? make(d, at::kByte, {(int64_t)need}) : Tensor();
    return answer(g_select(x->data_ptr(), data<float>(scores), data<int32_t>(&out[0]),
                           data<int32_t>(&out[1]), data<float>(&out[2]),
                           out[3].defined() ? data<int32_t>(&out[3]) : nullptr, (sv_dtype)type,
                           (int)B, (int)W, (int)x->size(2), (int)n,
                           need ? ws.data_ptr() : nullptr, need, stream_of(d)),
                  out);
  });
}

// beam_reorder(state, parents, out, lens): the status (0: done).
PyObject* beam_reorder(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) return long_way();
  return guarded([&]() -> PyObject* {
    const Tensor *s = tensor(a[0]), *parents = tensor(a[1]), *out = tensor(a[2]);
    if (!s || !out || !parents || s->dim() != 6 || out->dim() != 6 || parents->dim() != 2 ||
        !s->is_cuda() || s->device().index() != c10::cuda::current_device() || !small(*s) ||
        !small(*out) || out->device() != s->device() || out->scalar_type() != s->scalar_type() ||
        s->layout() != at::kStrided || out->layout() != at::kStrided)
      return long_way();
    const c10::Device d = s->device();
    const int64_t G = s->size(0), B = s->size(1), W = s->size(2), H = s->size(3), L = s->size(4),
                  D = s->size(5), Wo = parents->size(1), e = s->element_size();
    const Tensor* lens;
    if (!fits(parents, d, at::kInt, {B, Wo}) || !fits_or_none(a[3], d, at::kInt, {B}, &lens) ||
        out->sizes() != at::IntArrayRef({G, B, Wo, H, L, D}) || D == 0 || D * e > INT32_MAX ||
        (D > 1 && (s->stride(5) != 1 || out->stride(5) != 1)))
      return long_way();
    int64_t ss[5], os[5];
    for (int i = 0; i < 5; ++i) {
      ss[i] = s->stride(i) * e;
      os[i] = out->stride(i) * e;
    }
    const sv_status rc = g_reorder(s->data_ptr(), ss, data<int32_t>(parents), data<int32_t>(lens),
                                   out->data_ptr(), os, nullptr, (int)G, (int)B, (int)W, (int)Wo,
                                   (int)H, (int)L, (int)(D * e), stream_of(d));
    // autograd notices the write (inference tensors have no version)
    if (rc == SV_OK && !out->is_inference()) out->unsafeGetTensorImpl()->bump_version();
    return PyLong_FromLong(rc);
  });
}

// init(addresses of the six C functions)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[6];
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "init takes six addresses");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_top = reinterpret_cast<decltype(g_top)>(p[0]);
  g_distill = reinterpret_cast<decltype(g_distill)>(p[1]);
  g_distill_grad = reinterpret_cast<decltype(g_distill_grad)>(p[2]);
  g_select = reinterpret_cast<decltype(g_select)>(p[3]);
  g_select_ws = reinterpret_cast<decltype(g_select_ws)>(p[4]);
  g_reorder = reinterpret_cast<decltype(g_reorder)>(p[5]);
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(init),        FAST(top_logits),  FAST(distill),
                           FAST(distill_grad), FAST(beam_select), FAST(beam_reorder),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
