// bind.cpp -- the Python side of the operators around the experts as a CPython
// module: one call checks every tensor (on the current device, type, shape, contiguity), takes the current stream and
// calls the C ABI. A call of a few microseconds on the GPU is bound by what the host does for it: on a Grace
// core moe_norm_fwd with four tensors took 4.7 us with the checks in Python (0.38 a tensor) and the call
// through ctypes (0.6), 2.25 here, 1.7 of them the launch.
//
// Every function returns the C ABI's status, or None when an argument is not what the operator takes;
// the Python wrapper then names the argument and raises. No exception leaves a function: one from the
// tensor library also becomes None. init() receives the C ABI's functions, so that the library is the
// one that is loaded already.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstring>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe.h"

namespace {

decltype(&moe_norm_fwd) g_norm_fwd = nullptr;
decltype(&moe_norm_bwd) g_norm_bwd = nullptr;
decltype(&moe_gate_fwd) g_gate_fwd = nullptr;
decltype(&moe_gate_bwd) g_gate_bwd = nullptr;
decltype(&moe_linear_fwd) g_linear_fwd = nullptr;
decltype(&moe_linear_bwd) g_linear_bwd = nullptr;
decltype(&moe_balance_fwd) g_balance_fwd = nullptr;
decltype(&moe_balance_bwd) g_balance_bwd = nullptr;
decltype(&moe_xent_fwd) g_xent_fwd = nullptr;
decltype(&moe_xent_bwd) g_xent_bwd = nullptr;
decltype(&moe_grad_norm) g_grad_norm = nullptr;
decltype(&moe_adamw_step) g_adamw_step = nullptr;

constexpr bool kNeeded = true, kMay = false;  // a tensor that has to be there, one that may be None

// The arguments of one call: args[0] the dims structure (dims null: something else), args[1] the stream (None: the
// current one).
class Call {
 public:
  Call(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, void* dims, Py_ssize_t dims_bytes) : args_(args) {
    ok_ = n == want;
    if (!ok_) return;
    device_ = c10::cuda::current_device();
    if (!dims) return;
    Py_buffer b;
    if (PyObject_GetBuffer(args[0], &b, PyBUF_SIMPLE) != 0) {
      PyErr_Clear();
      ok_ = false;
      return;
    }
    ok_ = b.len == dims_bytes;
    if (ok_) memcpy(dims, b.buf, (size_t)dims_bytes);
    PyBuffer_Release(&b);
  }
  // argument i: a contiguous tensor of the current device, of type st and shape [d0] or [d0, d1]
  template <typename P = void>
  P* tensor(int i, bool needed, at::ScalarType st, int64_t d0, int64_t d1 = -1) {
    const at::Tensor* t = get(i, needed);
    if (!t) return nullptr;
    const auto s = t->sizes();
    ok_ = here(*t) && t->scalar_type() == st && t->is_contiguous() &&
          (d1 < 0 ? s.size() == 1 && s[0] == d0 : s.size() == 2 && s[0] == d0 && s[1] == d1);
    return ok_ ? static_cast<P*>(t->data_ptr()) : nullptr;
  }
  void* workspace(int i, size_t* bytes) {
    const at::Tensor* t = get(i, kNeeded);
    if (!t) return nullptr;
    ok_ = here(*t) && t->scalar_type() == at::kByte && t->is_contiguous();
    *bytes = (size_t)t->numel();
    return ok_ ? t->data_ptr() : nullptr;
  }
  // argument i: the optimiser's list, as its address, with its length and its device behind it
  const moe_adamw_tensor* list(int i, int64_t* count) {
    if (!ok_) return nullptr;
    void* p = PyLong_AsVoidPtr(args_[i]);
    *count = PyLong_AsLongLong(args_[i + 1]);
    const long long device = args_[i + 2] == Py_None ? device_ : PyLong_AsLongLong(args_[i + 2]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok_ = false;
      return nullptr;
    }
    ok_ = device == device_;
    return static_cast<const moe_adamw_tensor*>(p);
  }
  bool ok() const { return ok_; }
  // the call itself, without the interpreter's lock
  template <typename F>
  PyObject* run(F f) {
    void* st;
    if (args_[1] == Py_None) {
      st = c10::cuda::getCurrentCUDAStream(device_).stream();
    } else {
      st = PyLong_AsVoidPtr(args_[1]);
      if (PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_NONE;
      }
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = f(st);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
  }

 private:
  const at::Tensor* get(int i, bool needed) {
    if (!ok_) return nullptr;
    PyObject* o = args_[i];
    if (o == Py_None) {
      ok_ = !needed;
      return nullptr;
    }
    ok_ = THPVariable_Check(o);
    return ok_ ? &THPVariable_Unpack(o) : nullptr;
  }
  // the kernels run on the current device
  bool here(const at::Tensor& t) const { return t.is_cuda() && t.get_device() == device_; }
  PyObject* const* args_;
  bool ok_;
  c10::DeviceIndex device_ = -1;
};

at::ScalarType io_type(int32_t dtype) { return dtype == MOE_BF16 ? at::kBFloat16 : at::kFloat; }

// f builds its Call and runs it; whatever is thrown on the way is an argument the wrapper looks at again
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
    Py_RETURN_NONE;
  }
}

PyObject* norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    moe_norm_dims d;
    Call c(a, n, 10, &d, sizeof d);
    if (!c.ok()) Py_RETURN_NONE;
    const at::ScalarType io = io_type(d.dtype);
    const void* x = c.tensor(2, kNeeded, io, d.T, d.H);
    const void* residual = c.tensor(3, kMay, io, d.T, d.H);
    const void* weight = c.tensor(4, kNeeded, io, d.H);
    const void* bias = c.tensor(5, kMay, io, d.H);
    void* y = c.tensor(6, kNeeded, io, d.T, d.H);
    void* sum = c.tensor(7, kMay, io, d.T, d.H);
    float* mean = c.tensor<float>(8, kMay, at::kFloat, d.T);
    float* rstd = c.tensor<float>(9, kMay, at::kFloat, d.T);
    if (!c.ok()) Py_RETURN_NONE;
    return c.run([&](void* st) { return g_norm_fwd(&d, st, x, residual, weight, bias, y, sum, mean, rstd); });
  });
}

PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    moe_norm_dims d;
    Call c(a, n, 12, &d, sizeof d);
    if (!c.ok()) Py_RETURN_NONE;
    const at::ScalarType io = io_type(d.dtype);
    size_t bytes = 0;
    void* ws = c.workspace(2, &bytes);
    const void* dy = c.tensor(3, kNeeded, io, d.T, d.H);
    const void* dsum = c.tensor(4, kMay, io, d.T, d.H);
    const void* x = c.tensor(5, kNeeded, io, d.T, d.H);
    const void* weight = c.tensor(6, kNeeded, io, d.H);
    const float* mean = c.tensor<float>(7, kMay, at::kFloat, d.T);
    const float* rstd = c.tensor<float>(8, kNeeded, at::kFloat, d.T);
    void* dx = c.tensor(9, kNeeded, io, d.T, d.H);
    void* dweight = c.tensor(10, kNeeded, io, d.H);
    void* dbias = c.tensor(11, kMay, io, d.H);
    if (!c.ok()) Py_RETURN_NONE;
    return c.run([&](void* st) {
      return g_norm_bwd(&d, ws, bytes, st, dy, dsum, x, weight, mean, rstd, dx, dweight, dbias);
    });
  });
}

PyObject* gate_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    moe_gate_dims d;
    Call c(a, n, 7, &d, sizeof d);
    if (!c.ok()) Py_RETURN_NONE;
    const void* logits = c.tensor(2, kNeeded, io_type(d.dtype), d.T, d.E);
    const float* bias = c.tensor<float>(3, kMay, at::kFloat, d.E);
    int32_t* idx = c.tensor<int32_t>(4, kNeeded, at::kInt, d.T, d.k);
    float* w = c.tensor<float>(5, kNeeded, at::kFloat, d.T, d.k);
    int32_t* count = c.tensor<int32_t>(6, kMay, at::kInt, d.E);
    if (!c.ok()) Py_RETURN_NONE;
    return c.run([&](void* st) { return g_gate_fwd(&d, st, logits, bias, idx, w, count); });
  });
}

PyObject* gate_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    moe_gate_dims d;
    Call c(a, n, 6, &d, sizeof d);
    if (!c.ok()) Py_RETURN_NONE;
    const void* logits = c.tensor(2, kNeeded, io_type(d.dtype), d.T, d.E);
    const int32_t* idx = c.tensor<int32_t>(3, kNeeded, at::kInt, d.T, d.k);
    const float* dw = c.tensor<float>(4, kNeeded, at::kFloat, d.T, d.k);
    void* dlogits = c.tensor(5, kNeeded, io_type(d.grad_dtype), d.T, d.E);
    if (!c.ok()) Py_RETURN_NONE;
    return c.run([&](void* st) { return g_gate_bwd(&d, st, logits, idx, dw, dlogits); });
  });
}

PyObject* linear_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    moe_linear_dims d;
    Call c(a, n, 9, &d, sizeof d);
    if (!c.ok()) Py_RETURN_NONE;
    const at::ScalarType io = io_type(d.dtype);
    size_t bytes = 0;
    void* ws = c.workspace(2, &bytes);
    const void* x = c.tensor(3, kNeeded, io, d.M, d.K);
    const void* w = c.tensor(4, kNeeded, io, d.K, d.N);
    const void* bias = c.tensor(5, kMay, io, d.N);
    const void* residual = c.tensor(6, kMay, io, d.M, d.N);
    void* y = c.tensor(7, kNeeded, d.out_f32 ? at::kFloat : io, d.M, d.N);
    void* pre = c.tensor(8, kMay, io, d.M, d.N);
    if (!c.ok()) Py_RETURN_NONE;
    return c.run([&](void* st) { return g_linear_fwd(&d, ws, bytes, st, x, w, bias, residual, y, pre); });
  });
}

PyObject* linear_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    moe_linear_dims d;
    Call c(a, n, 11, &d, sizeof d);
    if (!c.ok()) Py_RETURN_NONE;
    const at::ScalarType io = io_type(d.dtype);
    size_t bytes = 0;
    void* ws = c.workspace(2, &bytes);
    const void* dy = c.tensor(3, kNeeded, io, d.M, d.N);
    const void* x = c.tensor(4, kNeeded, io, d.M, d.K);
    const void* w = c.tensor(5, kNeeded, io, d.K, d.N);
    const void* pre = c.tensor(6, kMay, io, d.M, d.N);
    const void* dx_add = c.tensor(7, kMay, io, d.M, d.K);
    void* dx = c.tensor(8, kMay, io, d.M, d.K);
    void* dw = c.tensor(9, kMay, io, d.K, d.N);
    void* dbias = c.tensor(10, kMay, io, d.N);
    if (!c.ok()) Py_RETURN_NONE;
    return c.run([&](void* st) {
      return g_linear_bwd(&d, ws, bytes, st, dy, x, w, pre, dx_add, dx, dw, dbias);
    });
  });
}

PyObject* balance_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    moe_balance_dims d;
    Call c(a, n, 9, &d, sizeof d);
    if (!c.ok()) Py_RETURN_NONE;
    const int64_t S = d.S > 1 ? d.S : 1;
    size_t bytes = 0;
    void* ws = c.workspace(2, &bytes);
    const void* logits = c.tensor(3, kNeeded, io_type(d.dtype), d.T, d.E);
    const int32_t* idx = c.tensor<int32_t>(4, kNeeded, at::kInt, d.T, d.k);
    const int32_t* start = c.tensor<int32_t>(5, kMay, at::kInt, d.S + 1);
    float* loss = c.tensor<float>(6, kNeeded, at::kFloat, 2);
    int32_t* count = c.tensor<int32_t>(7, kNeeded, at::kInt, S, d.E);
    float* prob = c.tensor<float>(8, kMay, at::kFloat, S, d.E);
    if (!c.ok() || (start != nullptr) != (d.S > 0)) Py_RETURN_NONE;
    return c.run([&](void* st) { return g_balance_fwd(&d, ws, bytes, st, logits, idx, start, loss, count, prob); });
  });
}

PyObject* balance_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    moe_balance_dims d;
    Call c(a, n, 8, &d, sizeof d);
    if (!c.ok()) Py_RETURN_NONE;
    const at::ScalarType grad = io_type(d.grad_dtype);
    const void* logits = c.tensor(2, kNeeded, io_type(d.dtype), d.T, d.E);
    const int32_t* count = c.tensor<int32_t>(3, kNeeded, at::kInt, d.S > 1 ? d.S : 1, d.E);
    const int32_t* start = c.tensor<int32_t>(4, kMay, at::kInt, d.S + 1);
    const float* dloss = c.tensor<float>(5, kMay, at::kFloat, 1);
    const void* add = c.tensor(6, kMay, grad, d.T, d.E);
    void* dlogits = c.tensor(7, kNeeded, grad, d.T, d.E);
    if (!c.ok() || (start != nullptr) != (d.S > 0)) Py_RETURN_NONE;
    return c.run([&](void* st) { return g_balance_bwd(&d, st, logits, count, start, dloss, add, dlogits); });
  });
}

PyObject* xent_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    moe_xent_dims d;
    Call c(a, n, 9, &d, sizeof d);
    if (!c.ok()) Py_RETURN_NONE;
    const at::ScalarType io = io_type(d.dtype);
    size_t bytes = 0;
    void* ws = c.workspace(2, &bytes);
    const void* x = c.tensor(3, kNeeded, io, d.M, d.H);
    const void* w = c.tensor(4, kNeeded, io, d.tied ? d.V : d.H, d.tied ? d.H : d.V);
    const int32_t* target = c.tensor<int32_t>(5, kNeeded, at::kInt, d.M);
    float* loss = c.tensor<float>(6, kNeeded, at::kFloat, d.M);
    float* lse = c.tensor<float>(7, kNeeded, at::kFloat, d.M);
    float* total = c.tensor<float>(8, kMay, at::kFloat, 2);
    if (!c.ok()) Py_RETURN_NONE;
    return c.run([&](void* st) { return g_xent_fwd(&d, ws, bytes, st, x, w, target, loss, lse, total); });
  });
}

PyObject* xent_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    moe_xent_dims d;
    Call c(a, n, 11, &d, sizeof d);
    if (!c.ok()) Py_RETURN_NONE;
    const at::ScalarType io = io_type(d.dtype);
    const int64_t r = d.tied ? d.V : d.H, q = d.tied ? d.H : d.V;
    size_t bytes = 0;
    void* ws = c.workspace(2, &bytes);
    const void* x = c.tensor(3, kNeeded, io, d.M, d.H);
    const void* w = c.tensor(4, kNeeded, io, r, q);
    const int32_t* target = c.tensor<int32_t>(5, kNeeded, at::kInt, d.M);
    const float* lse = c.tensor<float>(6, kNeeded, at::kFloat, d.M);
    const float* dloss = c.tensor<float>(7, kMay, at::kFloat, d.M);
    const float* total = c.tensor<float>(8, kMay, at::kFloat, 2);
    void* dx = c.tensor(9, kMay, io, d.M, d.H);
    void* dw = c.tensor(10, kMay, io, r, q);
    if (!c.ok()) Py_RETURN_NONE;
    return c.run([&](void* st) { return g_xent_bwd(&d, ws, bytes, st, x, w, target, lse, dloss, total, dx, dw); });
  });
}

// (scale, stream, ws, list, count, device, norm)
PyObject* grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(a, n, 7, nullptr, 0);
    if (!c.ok()) Py_RETURN_NONE;
    const double scale = PyFloat_AsDouble(a[0]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    size_t bytes = 0;
    void* ws = c.workspace(2, &bytes);
    int64_t count = 0;
    const moe_adamw_tensor* list = c.list(3, &count);
    float* norm = c.tensor<float>(6, kNeeded, at::kFloat, 1);
    if (!c.ok()) Py_RETURN_NONE;
    return c.run([&](void* st) { return g_grad_norm(list, count, ws, bytes, st, (float)scale, norm); });
  });
}

// (dims, stream, list, count, device, norm, lr, step)
PyObject* adamw_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    moe_adamw_dims d;
    Call c(a, n, 8, &d, sizeof d);
    if (!c.ok()) Py_RETURN_NONE;
    int64_t count = 0;
    const moe_adamw_tensor* list = c.list(2, &count);
    const float* norm = c.tensor<float>(5, kMay, at::kFloat, 1);
    const float* lr = c.tensor<float>(6, kMay, at::kFloat, 1);
    const int32_t* step = c.tensor<int32_t>(7, kMay, at::kInt, 1);
    if (!c.ok()) Py_RETURN_NONE;
    return c.run([&](void* st) { return g_adamw_step(&d, list, count, st, norm, lr, step); });
  });
}

template <typename F>
void take(F& f, void* p) {
  f = reinterpret_cast<F>(p);
}

// init(addresses of the C ABI's functions, in the order below)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kCount = 12;
  if (n != kCount) {
    PyErr_Format(PyExc_TypeError, "init takes %d addresses", kCount);
    return nullptr;
  }
  void* p[kCount];
  for (int i = 0; i < kCount; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  take(g_norm_fwd, p[0]);
  take(g_norm_bwd, p[1]);
  take(g_gate_fwd, p[2]);
  take(g_gate_bwd, p[3]);
  take(g_linear_fwd, p[4]);
  take(g_linear_bwd, p[5]);
  take(g_balance_fwd, p[6]);
  take(g_balance_bwd, p[7]);
  take(g_xent_fwd, p[8]);
  take(g_xent_bwd, p[9]);
  take(g_grad_norm, p[10]);
  take(g_adamw_step, p[11]);
  Py_RETURN_NONE;
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(init),        METHOD(norm_fwd),    METHOD(norm_bwd),   METHOD(gate_fwd),
                         METHOD(gate_bwd),    METHOD(linear_fwd),  METHOD(linear_bwd), METHOD(balance_fwd),
                         METHOD(balance_bwd), METHOD(xent_fwd),    METHOD(xent_bwd),   METHOD(grad_norm),
                         METHOD(adamw_step),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the PyTorch and Python this was compiled against, whose structures it reads
PyMODINIT_FUNC PyInit__bind() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", MOE_BUILT_FOR) != 0) Py_CLEAR(m);
  return m;
}
