// The 8-bit operators' usual call, from Python objects to the C ABI without the interpreter in
// between (module audio_encoder_tower_b200._fastcall): contiguous torch tensors of the expected
// types and shapes on the current device, outputs given, the device's current stream. A call of
// binding.py costs 8 to 12 us of host time, most of it in reading tensor attributes one by one;
// these functions do the same checks on the tensors themselves in about half a microsecond. They
// return the enc_status of the C call, or -1 without calling it where anything is not as above:
// binding.py then takes its general path, which says what is wrong.
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/enc_fp8.h"

namespace {

constexpr int kUnusual = -1;

// The tensor of an argument, or nullptr for anything else (subclasses too: what they do to an
// operation is for the general path).
const at::Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

bool is_matrix(const at::Tensor& t, int64_t rows, int64_t cols, c10::DeviceIndex dev) {
  return t.dim() == 2 && t.size(0) == rows && t.size(1) == cols && t.is_cuda() && t.get_device() == dev &&
         t.is_contiguous();
}

// An e4m3 [rows, cols] matrix with its scales.
bool is_fp8(const at::Tensor* q, const at::Tensor* s, int64_t rows, int64_t cols, c10::DeviceIndex dev) {
  return q && s && q->scalar_type() == at::kFloat8_e4m3fn &&
         (s->scalar_type() == at::kFloat8_e8m0fnu || s->scalar_type() == at::kByte) && is_matrix(*q, rows, cols, dev) &&
         is_matrix(*s, rows, (cols + 511) / 512 * 4, dev);
}

// A bf16 or fp32 matrix: its enc_dtype, or -1.
int dtype_of(const at::Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? ENC_DTYPE_BF16 : t.scalar_type() == at::kFloat ? ENC_DTYPE_FP32 : -1;
}

// An fp32 [n] vector, or None (*p null).
bool vector_or_none(PyObject* o, int64_t n, c10::DeviceIndex dev, const float** p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  if (!t || t->scalar_type() != at::kFloat || t->dim() != 1 || t->size(0) != n || !t->is_cuda() ||
      t->get_device() != dev || !t->is_contiguous())
    return false;
  *p = static_cast<const float*>(t->data_ptr());
  return true;
}

bool sizes_fit(int64_t rows, int64_t cols) { return rows <= INT32_MAX && cols <= INT32_MAX; }

PyObject* answer(int code) { return PyLong_FromLong(code); }

// The status of a C call made without the interpreter's lock: a launch waits for as long as the
// device's queue is full, and other Python threads run meanwhile.
struct WithoutLock {
  PyThreadState* state = PyEval_SaveThread();
  ~WithoutLock() { PyEval_RestoreThread(state); }
};
template <typename F> PyObject* answer_of(F&& call) {
  int code;
  {
    WithoutLock unlocked;
    code = call();
  }
  return answer(code);
}

// No C++ exception leaves a function that Python calls: one means that a tensor is unusual.
template <PyObject* (*f)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* v, Py_ssize_t n) {
  try {
    return f(v, n);
  } catch (...) {
    return answer(kUnusual);
  }
}

// linear(a, a_scales, w, w_scales, bias, out, out_scales, gelu)
PyObject* linear(PyObject* const* v, Py_ssize_t n) {
  if (n != 8) return answer(kUnusual);
  const at::Tensor *a = tensor(v[0]), *w = tensor(v[2]), *out = tensor(v[5]);
  if (!a || !w || !out || a->dim() != 2 || w->dim() != 2 || !a->is_cuda()) return answer(kUnusual);
  const auto dev = a->get_device();
  const int64_t M = a->size(0), K = a->size(1), N = w->size(0);
  const float* bias;
  if (dev != c10::cuda::current_device() || !sizes_fit(M, K) || !sizes_fit(N, K) ||
      !is_fp8(a, tensor(v[1]), M, K, dev) || !is_fp8(w, tensor(v[3]), N, K, dev) ||
      !vector_or_none(v[4], N, dev, &bias) || (v[7] != Py_True && v[7] != Py_False))
    return answer(kUnusual);
  void* out_scales = nullptr;
  int kind;
  if (out->scalar_type() == at::kFloat8_e4m3fn) {
    if (!is_fp8(out, tensor(v[6]), M, N, dev)) return answer(kUnusual);
    kind = ENC_FP8_OUT_FP8;
    out_scales = tensor(v[6])->data_ptr();
  } else {
    const int t = dtype_of(*out);
    if (t < 0 || v[6] != Py_None || !is_matrix(*out, M, N, dev)) return answer(kUnusual);
    kind = t == ENC_DTYPE_BF16 ? ENC_FP8_OUT_BF16 : ENC_FP8_OUT_FP32;
  }
  const void *ap = a->data_ptr(), *as = tensor(v[1])->data_ptr(), *wp = w->data_ptr(), *ws = tensor(v[3])->data_ptr();
  void* op = out->data_ptr();
  const int gelu = v[7] == Py_True;
  const auto stream = c10::cuda::getCurrentCUDAStream(dev).stream();
  return answer_of([&] {
    return enc_linear_fp8(ap, as, wp, ws, bias, op, out_scales, kind, (int32_t)M, (int32_t)N, (int32_t)K, gelu, nullptr,
                          stream);
  });
}

// norm(kind, x, gamma, beta, delta, eps, x_out, q, scales): kind an enc_norm_kind; x_out None without a delta
PyObject* norm(PyObject* const* v, Py_ssize_t n) {
  if (n != 9 || !PyLong_Check(v[0]) || !PyFloat_Check(v[5])) return answer(kUnusual);
  const at::Tensor *x = tensor(v[1]), *q = tensor(v[7]), *s = tensor(v[8]);
  if (!x || x->dim() != 2 || !x->is_cuda()) return answer(kUnusual);
  const auto dev = x->get_device();
  const int64_t rows = x->size(0), d = x->size(1);
  const int xt = dtype_of(*x);
  const float *gamma, *beta;
  if (dev != c10::cuda::current_device() || xt < 0 || !sizes_fit(rows, d) || !is_matrix(*x, rows, d, dev) ||
      !vector_or_none(v[2], d, dev, &gamma) || !gamma || !vector_or_none(v[3], d, dev, &beta) ||
      !is_fp8(q, s, rows, d, dev))
    return answer(kUnusual);
  const void* delta = nullptr;
  void* x_out = nullptr;
  int dt = ENC_DTYPE_BF16;
  if (v[4] != Py_None) {
    const at::Tensor* t = tensor(v[4]);
    if (!t || (dt = dtype_of(*t)) < 0 || !is_matrix(*t, rows, d, dev)) return answer(kUnusual);
    delta = t->data_ptr();
  }
  if (v[6] != Py_None) {
    const at::Tensor* t = tensor(v[6]);
    if (!t || dtype_of(*t) != xt || !is_matrix(*t, rows, d, dev)) return answer(kUnusual);
    x_out = t->data_ptr();
  }
  const int32_t kind = (int32_t)PyLong_AsLong(v[0]);
  const float eps = (float)PyFloat_AS_DOUBLE(v[5]);
  const void* xp = x->data_ptr();
  void *qp = q->data_ptr(), *sp = s->data_ptr();
  const auto stream = c10::cuda::getCurrentCUDAStream(dev).stream();
  return answer_of([&] {
    return enc_norm_fp8(kind, xp, xt, d, delta, dt, d, gamma, beta, eps, (int32_t)rows, (int32_t)d, x_out, d, qp, sp,
                        stream);
  });
}

// quantize(x, q, scales)
PyObject* quantize(PyObject* const* v, Py_ssize_t n) {
  if (n != 3) return answer(kUnusual);
  const at::Tensor *x = tensor(v[0]), *q = tensor(v[1]), *s = tensor(v[2]);
  if (!x || x->dim() != 2 || !x->is_cuda()) return answer(kUnusual);
  const auto dev = x->get_device();
  const int64_t rows = x->size(0), cols = x->size(1);
  const int xt = dtype_of(*x);
  if (dev != c10::cuda::current_device() || xt < 0 || !sizes_fit(rows, cols) || !is_matrix(*x, rows, cols, dev) ||
      !is_fp8(q, s, rows, cols, dev))
    return answer(kUnusual);
  const void* xp = x->data_ptr();
  void *qp = q->data_ptr(), *sp = s->data_ptr();
  const auto stream = c10::cuda::getCurrentCUDAStream(dev).stream();
  return answer_of([&] { return enc_quantize_fp8(xp, xt, cols, (int32_t)rows, (int32_t)cols, qp, sp, stream); });
}

PyMethodDef methods[] = {
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<linear>)), METH_FASTCALL, nullptr},
    {"norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<norm>)), METH_FASTCALL, nullptr},
    {"quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<quantize>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", ENC_TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
