// marshal.cpp -- the torch conveniences of binding.py in native code: argument
// checks, allocation of results and the C call. A grouped product of a decode
// step takes some 10 us on the GPU; the same marshalling in Python took 25 us
// of host time a call, 60 for the two calls of an 8-bit layer.
//
// The module links nothing of the CUDA library: bind() gives it the addresses
// of the C functions that binding.py has loaded, and the exception class.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>
#include <vector>

namespace {

enum { kF32 = 0, kBf16 = 1, kF16 = 2 };

struct Functions {
  int (*grouped)(int, int, int, int, int, int, int, float, const void*, int, const void*, int,
                 long long, const int*, float, void*, int, void*);
  int (*wgrad)(int, int, int, int, int, int, float, const void*, int, const void*, int, const int*,
               float, void*, int, long long, void*);
  int (*quantize)(int, int, int, const void*, int, signed char*, int, float*, void*);
  int (*i8)(int, int, int, const signed char*, int, const float*, const signed char*, int,
            const float*, int, void*, int, void*);
  int (*clip)(int, const void* const*, void* const*, const long long*, const int*, float, float*,
              void*);
} fn;
PyObject* g_error = nullptr;   // SgemmError(status, name)

// What a call refuses (ValueError), and what the library returned (SgemmError).
struct Refusal {
  std::string what;
};
struct Status {
  int code;
  const char* name;
};
struct PythonError {};   // the exception is already set

void check(bool ok, const char* what) {
  if (!ok) throw Refusal{what};
}

bool is_none(PyObject* o) { return o == nullptr || o == Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refusal{std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

int type_of(at::ScalarType t, const char* name) {
  switch (t) {
    case at::kFloat: return kF32;
    case at::kBFloat16: return kBf16;
    case at::kHalf: return kF16;
    default: throw Refusal{std::string(name) + " must be float32, bfloat16 or float16"};
  }
}
int type_of(const at::Tensor& t, const char* name) {
  // (the imaginary part of a conjugate: what is stored has the other sign)
  if (t.is_neg()) throw Refusal{std::string(name) + " is a negated view: call resolve_neg() first"};
  return type_of(t.scalar_type(), name);
}

int to_int(int64_t v) {
  check(v >= 0 && v <= 0x7fffffff, "sizes must be below 2^31");
  return (int)v;
}

// Row pitch of a row-major matrix (or of the matrices of a 3-D tensor). Rows
// that overlap (an expanded tensor's have stride 0) have no pitch that the
// kernels take: read at the row length they would lie past the storage.
int pitch(const at::Tensor& t, const char* name) {
  const int64_t d = t.dim(), cols = t.size(d - 1), least = cols > 1 ? cols : 1;
  if (cols > 1 && t.stride(d - 1) != 1)
    throw Refusal{std::string(name) + " must be row-major (unit stride along rows)"};
  if (t.size(d - 2) < 2 || t.numel() == 0) return to_int(least);
  if (t.stride(d - 2) < least)
    throw Refusal{std::string(name) + " has overlapping rows (a row stride below the row length)"};
  return to_int(t.stride(d - 2));
}

// The matrices of a 3-D result may lie one after another or row by row beside
// each other; groups that write the same elements would race.
void check_apart(const at::Tensor& t, int64_t ld) {
  if (t.size(0) < 2 || t.numel() == 0) return;
  const int64_t gap = t.stride(0), rows = t.size(1), cols = t.size(2);
  check(gap >= (rows - 1) * ld + cols ||
            (gap >= cols && (rows < 2 || ld >= (t.size(0) - 1) * gap + cols)),
        "the groups' matrices in C overlap");
}

// Tensors of one call: on one CUDA device, which is current for its duration,
// and so is the stream it was given: a result is allocated as that stream's
// own (one of the current stream's could still be in use by work queued there,
// or be handed out again there before the kernel has written it).
class Launch {
 public:
  Launch(PyObject* stream, std::initializer_list<const at::Tensor*> tensors)
      : Launch(stream, device_of(**tensors.begin())) {
    for (const at::Tensor* t : tensors) check_device(*t);
  }
  Launch(PyObject* stream, int device) : device_(device) {
    if (is_none(stream)) {
      on_device_.emplace((c10::DeviceIndex)device);
      handle_ = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    } else {
      PyObject* h = PyObject_GetAttrString(stream, "cuda_stream");
      if (h == nullptr) throw PythonError{};
      handle_ = PyLong_AsVoidPtr(h);
      Py_DECREF(h);
      if (PyErr_Occurred()) throw PythonError{};
      on_stream_.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle_),
                                                          (c10::DeviceIndex)device));
    }
  }
  void* handle() const { return handle_; }
  void check_device(const at::Tensor& t) const {
    check(t.is_cuda() && t.get_device() == device_, "tensors must be on one CUDA device");
  }

 private:
  static int device_of(const at::Tensor& t) {
    check(t.is_cuda(), "tensors must be on one CUDA device");
    return t.get_device();
  }
  int device_;
  void* handle_ = nullptr;
  std::optional<c10::cuda::CUDAGuard> on_device_;
  std::optional<c10::cuda::CUDAStreamGuard> on_stream_;
};

at::ScalarType dtype_or(PyObject* o, at::ScalarType other) {
  if (o == nullptr || o == Py_None) return other;
  check(THPDtype_Check(o), "out_dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

const int* offsets_of(const at::Tensor& t, int64_t groups) {
  check(t.scalar_type() == at::kInt && t.dim() == 1 && t.is_contiguous(),
        "offsets must be a contiguous 1-D int32 tensor");
  check(t.numel() == groups + 1, "offsets must hold one bound more than there are groups");
  return static_cast<const int*>(t.data_ptr());
}

void vector_of(const at::Tensor& t, int64_t n, const char* what) {
  check(t.scalar_type() == at::kFloat && t.dim() == 1 && t.size(0) == n && t.is_contiguous() &&
            !t.is_neg(), what);
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}

// Tells autograd that a given tensor's values have changed: a graph that had
// saved it for its backward pass refuses to use it. (Inference tensors have no
// version.)
void overwritten(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// The given result object, or a wrapper of the new tensor.
PyObject* result(PyObject* given, const at::Tensor& t) {
  if (!is_none(given)) {
    overwritten(t);
    Py_INCREF(given);
    return given;
  }
  return THPVariable_Wrap(t);
}

// (X, W, offsets, Y, transposed, alpha, beta, out_dtype, stream)
PyObject* grouped_gemm(PyObject* const* a) {
  const at::Tensor &X = tensor(a[0], "X"), &W = tensor(a[1], "W"), &off = tensor(a[2], "offsets");
  const bool transposed = a[4] == Py_True;
  const double alpha = number(a[5]), beta = number(a[6]);
  check(X.dim() == 2 && W.dim() == 3, "X must be 2-D and W 3-D");
  const int64_t T = X.size(0), K = X.size(1), E = W.size(0), N = W.size(transposed ? 1 : 2);
  check(W.size(transposed ? 2 : 1) == K, "shape mismatch");
  check(W.scalar_type() == X.scalar_type(), "X and W must have one type");
  const int* bounds = offsets_of(off, E);
  const int type = type_of(X, "X"), ldx = pitch(X, "X"), ldw = pitch(W, "W");
  type_of(W, "W");
  at::Tensor Y;
  at::ScalarType out = X.scalar_type();
  if (is_none(a[3])) {
    check(beta == 0.0, "beta needs Y");
    out = dtype_or(a[7], out);
  } else {
    Y = tensor(a[3], "Y");
    check(Y.dim() == 2 && Y.size(0) == T && Y.size(1) == N, "shape mismatch");
    pitch(Y, "Y");
    type_of(Y, "Y");
    out = Y.scalar_type();
  }
  const int out_type = type_of(out, "Y");
  const Launch on(a[8], {&X, &W, &off});
  if (!Y.defined()) Y = at::empty({T, N}, X.options().dtype(out).requires_grad(false));
  on.check_device(Y);
  const int st = fn.grouped(transposed ? 1 : 0, type, out_type, to_int(E), to_int(T), to_int(N),
                            to_int(K), (float)alpha, X.data_ptr(), ldx, W.data_ptr(), ldw,
                            E > 1 ? W.stride(0) : 0, bounds, (float)beta, Y.data_ptr(),
                            pitch(Y, "Y"), on.handle());
  if (st != 0) throw Status{st, "sgemm_grouped"};
  return result(a[3], Y);
}

// (A, B, offsets, C, alpha, beta, out_dtype, stream)
PyObject* grouped_wgrad(PyObject* const* a) {
  const at::Tensor &A = tensor(a[0], "A"), &B = tensor(a[1], "B"), &off = tensor(a[2], "offsets");
  const double alpha = number(a[4]), beta = number(a[5]);
  check(A.dim() == 2 && B.dim() == 2 && A.size(0) == B.size(0), "shape mismatch");
  check(A.scalar_type() == B.scalar_type(), "A and B must have one type");
  const int64_t E = off.numel() - 1, T = A.size(0), M = A.size(1), N = B.size(1);
  check(E >= 0, "offsets must hold one bound more than there are groups");
  const int* bounds = offsets_of(off, E);
  const int type = type_of(A, "A"), lda = pitch(A, "A"), ldb = pitch(B, "B");
  type_of(B, "B");
  at::Tensor C;
  at::ScalarType out = A.scalar_type();
  if (is_none(a[3])) {
    check(beta == 0.0, "beta needs C");
    out = dtype_or(a[6], out);
  } else {
    C = tensor(a[3], "C");
    check(C.dim() == 3 && C.size(0) == E && C.size(1) == M && C.size(2) == N, "shape mismatch");
    check_apart(C, pitch(C, "C"));
    type_of(C, "C");
    out = C.scalar_type();
  }
  const int out_type = type_of(out, "C");
  const Launch on(a[7], {&A, &B, &off});
  if (!C.defined()) C = at::empty({E, M, N}, A.options().dtype(out).requires_grad(false));
  on.check_device(C);
  const int st = fn.wgrad(type, out_type, to_int(E), to_int(T), to_int(M), to_int(N), (float)alpha,
                          A.data_ptr(), lda, B.data_ptr(), ldb, bounds, (float)beta, C.data_ptr(),
                          pitch(C, "C"), E > 1 ? C.stride(0) : 0, on.handle());
  if (st != 0) throw Status{st, "sgemm_grouped_wgrad"};
  return result(a[3], C);
}

// (X, Q, scale, stream)
PyObject* i8_quantize(PyObject* const* a) {
  const at::Tensor& X = tensor(a[0], "X");
  check(X.dim() == 2, "X must be 2-D");
  const int64_t M = X.size(0), K = X.size(1);
  const int type = type_of(X, "X"), ldx = pitch(X, "X");
  at::Tensor Q, scale;
  if (!is_none(a[1])) {
    Q = tensor(a[1], "Q");
    check(Q.scalar_type() == at::kChar && Q.dim() == 2 && Q.size(0) == M && Q.size(1) == K,
          "Q must be int8 of X's shape");
    pitch(Q, "Q");
  }
  if (!is_none(a[2])) {
    scale = tensor(a[2], "scale");
    vector_of(scale, M, "scale must be a contiguous float32 vector with one value a row");
  }
  {
    const Launch on(a[3], {&X});
    if (!Q.defined()) {
      // rows padded to 16 bytes, so that sgemm_i8 reads them in place
      const int64_t ld = (K + 15) / 16 * 16;
      const auto options = X.options().dtype(at::kChar).requires_grad(false);
      Q = ld == K ? at::empty({M, K}, options) : at::empty_strided({M, K}, {ld, 1}, options);
    }
    if (!scale.defined())
      scale = at::empty({M}, X.options().dtype(at::kFloat).requires_grad(false));
    on.check_device(Q);
    on.check_device(scale);
    const int st = fn.quantize(to_int(M), to_int(K), type, X.data_ptr(), ldx,
                               static_cast<signed char*>(Q.data_ptr()), pitch(Q, "Q"),
                               static_cast<float*>(scale.data_ptr()), on.handle());
    if (st != 0) throw Status{st, "sgemm_i8_quantize"};
  }
  PyObject* q = result(a[1], Q);
  PyObject* s = result(a[2], scale);
  PyObject* both = PyTuple_New(2);
  if (q == nullptr || s == nullptr || both == nullptr) throw PythonError{};
  PyTuple_SET_ITEM(both, 0, q);
  PyTuple_SET_ITEM(both, 1, s);
  return both;
}

// (A, scaleA, B, scaleB, C, out_dtype, stream)
PyObject* i8_gemm(PyObject* const* a) {
  const at::Tensor &A = tensor(a[0], "A"), &sa = tensor(a[1], "scaleA"), &B = tensor(a[2], "B"),
                   &sb = tensor(a[3], "scaleB");
  check(A.dim() == 2 && B.dim() == 2 && A.size(1) == B.size(1), "shape mismatch");
  check(A.scalar_type() == at::kChar && B.scalar_type() == at::kChar, "A and B must be int8");
  const int64_t M = A.size(0), K = A.size(1), N = B.size(0);
  vector_of(sa, M, "scaleA must be a contiguous float32 vector with a value for each row of A");
  vector_of(sb, N, "scaleB must be a contiguous float32 vector with a value for each row of B");
  const int lda = pitch(A, "A"), ldb = pitch(B, "B");
  at::Tensor C;
  at::ScalarType out = at::kBFloat16;
  if (is_none(a[4])) {
    out = dtype_or(a[5], out);
  } else {
    C = tensor(a[4], "C");
    check(C.dim() == 2 && C.size(0) == M && C.size(1) == N, "shape mismatch");
    pitch(C, "C");
    type_of(C, "C");
    out = C.scalar_type();
  }
  const int out_type = type_of(out, "C");
  const Launch on(a[6], {&A, &sa, &B, &sb});
  if (!C.defined()) C = at::empty({M, N}, A.options().dtype(out).requires_grad(false));
  on.check_device(C);
  const int st = fn.i8(to_int(M), to_int(N), to_int(K),
                       static_cast<const signed char*>(A.data_ptr()), lda,
                       static_cast<const float*>(sa.data_ptr()),
                       static_cast<const signed char*>(B.data_ptr()), ldb,
                       static_cast<const float*>(sb.data_ptr()), out_type, C.data_ptr(),
                       pitch(C, "C"), on.handle());
  if (st != 0) throw Status{st, "sgemm_i8"};
  return result(a[4], C);
}

// Holds a list or tuple of the items of any iterable.
struct Items {
  PyObject* fast;
  explicit Items(PyObject* o) : fast(PySequence_Fast(o, "gradients must be a sequence of tensors")) {
    if (fast == nullptr) throw PythonError{};
  }
  ~Items() { Py_DECREF(fast); }
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(fast); }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

// (grads, max_norm, out, stream)
PyObject* clip_grad_norm(PyObject* const* a) {
  const double max_norm = number(a[1]);
  const Items grads(a[0]);
  const Py_ssize_t n = grads.size();
  check(n > 0, "no gradients");
  check(n <= 0x7fffffff, "too many gradients");
  std::vector<const void*> in((size_t)n);
  std::vector<void*> to((size_t)n);
  std::vector<long long> sizes((size_t)n);
  std::vector<int> types((size_t)n);
  int device = -1;
  for (Py_ssize_t i = 0; i < n; ++i) {
    const at::Tensor& g = tensor(grads[i], "gradients");
    check(g.is_cuda() && (i == 0 || g.get_device() == device),
          "gradients must be on one CUDA device");
    device = g.get_device();
    check(g.is_contiguous(), "gradients must be contiguous");
    types[i] = type_of(g, "gradients");
    in[i] = to[i] = g.data_ptr();
    sizes[i] = g.numel();
  }
  const Items written(is_none(a[2]) ? grads.fast : a[2]);
  if (!is_none(a[2])) {
    const Items& out = written;
    check(out.size() == n, "out must hold a tensor for every gradient");
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor &o = tensor(out[i], "out"), &g = tensor(grads[i], "gradients");
      check(o.is_cuda() && o.get_device() == device, "gradients must be on one CUDA device");
      check(o.is_contiguous(), "gradients must be contiguous");
      type_of(o, "out");
      check(o.scalar_type() == g.scalar_type() && o.sizes() == g.sizes(),
            "out must have the gradients' types and shapes");
      to[i] = o.data_ptr();
    }
  }
  const Launch on(a[3], device);
  const at::Tensor norm =
      at::empty({}, tensor(grads[0], "gradients").options().dtype(at::kFloat).requires_grad(false));
  const int st = fn.clip((int)n, in.data(), to.data(), sizes.data(), types.data(), (float)max_norm,
                         static_cast<float*>(norm.data_ptr()), on.handle());
  if (st != 0) throw Status{st, "sgemm_grad_clip"};
  for (Py_ssize_t i = 0; i < n; ++i) overwritten(tensor(written[i], "out"));
  return THPVariable_Wrap(norm);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  try {
    if (fn.grouped == nullptr) throw Refusal{"the CUDA library is not bound"};
    if (nargs != N) throw Refusal{"wrong number of arguments"};
    return F(args);
  } catch (const Refusal& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
  } catch (const Status& s) {
    PyObject* value = PyObject_CallFunction(g_error, "is", s.code, s.name);
    if (value != nullptr) {
      PyErr_SetObject(g_error, value);
      Py_DECREF(value);
    }
  } catch (const PythonError&) {
  } catch (const std::exception& e) {   // an allocation that failed, for one
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (grouped, wgrad, quantize, i8, clip addresses, the exception class)
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long p[5];
  PyObject* error;
  if (!PyArg_ParseTuple(args, "KKKKKO", &p[0], &p[1], &p[2], &p[3], &p[4], &error)) return nullptr;
  fn.grouped = reinterpret_cast<decltype(fn.grouped)>(p[0]);
  fn.wgrad = reinterpret_cast<decltype(fn.wgrad)>(p[1]);
  fn.quantize = reinterpret_cast<decltype(fn.quantize)>(p[2]);
  fn.i8 = reinterpret_cast<decltype(fn.i8)>(p[3]);
  fn.clip = reinterpret_cast<decltype(fn.clip)>(p[4]);
  Py_INCREF(error);
  Py_XDECREF(g_error);
  g_error = error;
  Py_RETURN_NONE;
}

#define SGEMM_GB300_METHOD(NAME, N) \
  { #NAME, reinterpret_cast<PyCFunction>(&call<NAME, N>), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    SGEMM_GB300_METHOD(grouped_gemm, 9),
    SGEMM_GB300_METHOD(grouped_wgrad, 8),
    SGEMM_GB300_METHOD(i8_quantize, 4),
    SGEMM_GB300_METHOD(i8_gemm, 7),
    SGEMM_GB300_METHOD(clip_grad_norm, 4),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
