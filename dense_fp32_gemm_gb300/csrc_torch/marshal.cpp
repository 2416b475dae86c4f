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
  int (*norm)(int, int, int, const void*, int, const void*, int, const void*, int, float, void*, int,
              void*, int, float*, void*);
  int (*norm_i8)(int, int, int, const void*, int, const void*, int, const void*, int, float, void*,
                 int, signed char*, int, float*, void*);
  int (*norm_grad)(int, int, int, const void*, int, const void*, int, const void*, int, const float*,
                   const void*, int, void*, int, void*, void*);
  int (*ce)(int, int, int, int, const void*, int, const void*, int, const long long*, long long,
            float*, float*, void*);
  int (*ce_grad)(int, int, int, int, const void*, int, const void*, int, const long long*, long long,
                 const float*, const float*, void*, int, void*, int, void*);
  int (*mx4_quantize)(int, int, int, const void*, int, unsigned char*, int, unsigned char*, void*);
  int (*mx4_dequantize)(int, int, const unsigned char*, int, const unsigned char*, int, void*, int,
                        void*);
  int (*mx4)(int, int, int, const unsigned char*, int, const unsigned char*, const unsigned char*, int,
             const unsigned char*, int, void*, int, void*);
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

// 8-bit integers of X's shape, rows padded to 16 bytes, so that sgemm_i8 reads
// them in place.
at::Tensor padded_i8(const at::Tensor& X) {
  const int64_t M = X.size(0), K = X.size(1), ld = (K + 15) / 16 * 16;
  const auto options = X.options().dtype(at::kChar).requires_grad(false);
  return ld == K ? at::empty({M, K}, options) : at::empty_strided({M, K}, {ld, 1}, options);
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
    if (!Q.defined()) Q = padded_i8(X);
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

// A tuple of n objects; takes their references.
template <typename... O>
PyObject* tuple_of(O*... objects) {
  PyObject* all[] = {objects...};
  bool ok = true;
  for (PyObject* o : all) ok = ok && o != nullptr;
  PyObject* t = ok ? PyTuple_New(sizeof...(O)) : nullptr;
  if (t == nullptr) {
    for (PyObject* o : all) Py_XDECREF(o);
    throw PythonError{};
  }
  for (size_t i = 0; i < sizeof...(O); ++i) PyTuple_SET_ITEM(t, (Py_ssize_t)i, all[i]);
  return t;
}

// A matrix that was given as `name`: of X's shape and type.
void like(const at::Tensor& t, const at::Tensor& X, const char* name, const char* of = "X") {
  if (t.scalar_type() != X.scalar_type() || t.dim() != 2 || t.size(0) != X.size(0) ||
      t.size(1) != X.size(1))
    throw Refusal{std::string(name) + " must have the shape and type of " + of};
  type_of(t, name);
  pitch(t, name);
}

// The norm's weight: its type.
int weight_of(const at::Tensor& w, const at::Tensor& X) {
  check(w.dim() == 1 && w.size(0) == X.size(1) && w.is_contiguous(),
        "weight must be a contiguous vector with a value for each column");
  check(w.scalar_type() == X.scalar_type() || w.scalar_type() == at::kFloat,
        "weight must be of X's type or float32");
  return type_of(w, "weight");
}

// What rms_norm and rms_norm_i8 share: X, the residual and where their sum goes.
struct Rows {
  const at::Tensor &X, &weight;
  at::Tensor R, H;
  int type, weight_type, ldx, ldr = 1, M, N;
  Rows(PyObject* x, PyObject* w, PyObject* residual, PyObject* h)
      : X(tensor(x, "X")), weight(tensor(w, "weight")) {
    check(X.dim() == 2, "X must be 2-D");
    type = type_of(X, "X");
    ldx = pitch(X, "X");
    M = to_int(X.size(0));
    N = to_int(X.size(1));
    weight_type = weight_of(weight, X);
    ldr = N > 1 ? N : 1;
    if (!is_none(residual)) {
      R = tensor(residual, "residual");
      like(R, X, "residual");
      ldr = pitch(R, "residual");
    }
    if (!is_none(h)) {
      check(R.defined(), "H needs a residual");
      H = tensor(h, "H");
      like(H, X, "H");
    }
  }
  // (within the call's Launch) the sum's matrix, allocated if none was given
  void place(const Launch& on) {
    if (!R.defined()) return;
    on.check_device(R);
    if (!H.defined()) H = at::empty({X.size(0), X.size(1)}, X.options().requires_grad(false));
    on.check_device(H);
  }
  void* h() const { return H.defined() ? H.data_ptr() : nullptr; }
  int ldh() const { return H.defined() ? pitch(H, "H") : (N > 1 ? N : 1); }
  const void* r() const { return R.defined() ? R.data_ptr() : nullptr; }
  // the sum as an object: X itself without a residual
  PyObject* sum(PyObject* x, PyObject* given) const {
    if (R.defined()) return result(given, H);
    Py_INCREF(x);
    return x;
  }
};

// (X, weight, residual, eps, Y, H, rstd, stream)
PyObject* rms_norm(PyObject* const* a) {
  Rows in(a[0], a[1], a[2], a[5]);
  const double eps = number(a[3]);
  at::Tensor Y, rstd;
  if (!is_none(a[4])) {
    Y = tensor(a[4], "Y");
    like(Y, in.X, "Y");
  }
  if (!is_none(a[6])) {
    rstd = tensor(a[6], "rstd");
    vector_of(rstd, in.M, "rstd must be a contiguous float32 vector with one value a row");
  }
  {
    const Launch on(a[7], {&in.X, &in.weight});
    in.place(on);
    if (!Y.defined()) Y = at::empty({in.M, in.N}, in.X.options().requires_grad(false));
    if (!rstd.defined())
      rstd = at::empty({in.M}, in.X.options().dtype(at::kFloat).requires_grad(false));
    on.check_device(Y);
    on.check_device(rstd);
    const int st = fn.norm(in.M, in.N, in.type, in.X.data_ptr(), in.ldx, in.r(), in.ldr,
                           in.weight.data_ptr(), in.weight_type, (float)eps, in.h(), in.ldh(),
                           Y.data_ptr(), pitch(Y, "Y"), static_cast<float*>(rstd.data_ptr()),
                           on.handle());
    if (st != 0) throw Status{st, "sgemm_rms_norm"};
  }
  return tuple_of(result(a[4], Y), in.sum(a[0], a[5]), result(a[6], rstd));
}

// (X, weight, residual, eps, Q, scale, H, stream)
PyObject* rms_norm_i8(PyObject* const* a) {
  Rows in(a[0], a[1], a[2], a[6]);
  const double eps = number(a[3]);
  at::Tensor Q, scale;
  if (!is_none(a[4])) {
    Q = tensor(a[4], "Q");
    check(Q.scalar_type() == at::kChar && Q.dim() == 2 && Q.size(0) == in.M && Q.size(1) == in.N,
          "Q must be int8 of X's shape");
    pitch(Q, "Q");
  }
  if (!is_none(a[5])) {
    scale = tensor(a[5], "scale");
    vector_of(scale, in.M, "scale must be a contiguous float32 vector with one value a row");
  }
  {
    const Launch on(a[7], {&in.X, &in.weight});
    in.place(on);
    if (!Q.defined()) Q = padded_i8(in.X);
    if (!scale.defined())
      scale = at::empty({in.M}, in.X.options().dtype(at::kFloat).requires_grad(false));
    on.check_device(Q);
    on.check_device(scale);
    const int st = fn.norm_i8(in.M, in.N, in.type, in.X.data_ptr(), in.ldx, in.r(), in.ldr,
                              in.weight.data_ptr(), in.weight_type, (float)eps, in.h(), in.ldh(),
                              static_cast<signed char*>(Q.data_ptr()), pitch(Q, "Q"),
                              static_cast<float*>(scale.data_ptr()), on.handle());
    if (st != 0) throw Status{st, "sgemm_rms_norm_i8"};
  }
  return tuple_of(result(a[4], Q), result(a[5], scale), in.sum(a[0], a[6]));
}

// (dY, H, weight, rstd, dH, dX, dweight, want dX, want dweight, stream)
PyObject* rms_norm_grad(PyObject* const* a) {
  const at::Tensor &dY = tensor(a[0], "dY"), &H = tensor(a[1], "H"), &w = tensor(a[2], "weight"),
                   &rstd = tensor(a[3], "rstd");
  check(H.dim() == 2, "H must be 2-D");
  const int type = type_of(H, "H"), ldh = pitch(H, "H");
  like(dY, H, "dY", "H");
  const int weight_type = weight_of(w, H), M = to_int(H.size(0)), N = to_int(H.size(1));
  vector_of(rstd, M, "rstd must be a contiguous float32 vector with one value a row");
  const bool want_x = a[7] == Py_True, want_w = a[8] == Py_True;
  at::Tensor dH, dX, dw;
  if (!is_none(a[4])) {
    dH = tensor(a[4], "dH");
    like(dH, H, "dH", "H");
  }
  if (want_x && !is_none(a[5])) {
    dX = tensor(a[5], "dX");
    like(dX, H, "dX", "H");
  }
  if (want_w && !is_none(a[6])) {
    dw = tensor(a[6], "dweight");
    check(dw.dim() == 1 && dw.size(0) == N && dw.is_contiguous() && !dw.is_neg() &&
              dw.scalar_type() == w.scalar_type(), "dweight must have the shape and type of weight");
  }
  const int least = N > 1 ? N : 1;
  {
    const Launch on(a[9], {&dY, &H, &w, &rstd});
    if (dH.defined()) on.check_device(dH);
    if (want_x && !dX.defined()) dX = at::empty({M, N}, H.options().requires_grad(false));
    if (want_w && !dw.defined()) dw = at::empty({N}, w.options().requires_grad(false));
    if (want_x) on.check_device(dX);
    if (want_w) on.check_device(dw);
    const int st = fn.norm_grad(
        M, N, type, dY.data_ptr(), pitch(dY, "dY"), H.data_ptr(), ldh, w.data_ptr(), weight_type,
        static_cast<const float*>(rstd.data_ptr()), dH.defined() ? dH.data_ptr() : nullptr,
        dH.defined() ? pitch(dH, "dH") : least, want_x ? dX.data_ptr() : nullptr,
        want_x ? pitch(dX, "dX") : least, want_w ? dw.data_ptr() : nullptr, on.handle());
    if (st != 0) throw Status{st, "sgemm_rms_norm_grad"};
  }
  return tuple_of(want_x ? result(a[5], dX) : Py_NewRef(Py_None),
                  want_w ? result(a[6], dw) : Py_NewRef(Py_None));
}

// What both calls of the loss share.
struct Loss {
  const at::Tensor &X, &W, &target;
  long long ignore;
  int type, T, V, H, ldx, ldw;
  Loss(PyObject* x, PyObject* w, PyObject* words, PyObject* ignored)
      : X(tensor(x, "X")), W(tensor(w, "W")), target(tensor(words, "target")) {
    check(X.dim() == 2 && W.dim() == 2 && X.size(1) == W.size(1), "X and W must be 2-D with rows of one length");
    check(X.scalar_type() == W.scalar_type(), "X and W must have one type");
    type = type_of(X, "X");
    type_of(W, "W");
    ldx = pitch(X, "X");
    ldw = pitch(W, "W");
    T = to_int(X.size(0));
    V = to_int(W.size(0));
    H = to_int(X.size(1));
    check(target.scalar_type() == at::kLong && target.dim() == 1 && target.size(0) == T &&
              target.is_contiguous(), "target must be a contiguous int64 vector with a word for each row of X");
    ignore = PyLong_AsLongLong(ignored);
    if (ignore == -1 && PyErr_Occurred()) throw PythonError{};
  }
  const long long* words() const { return static_cast<const long long*>(target.data_ptr()); }
  at::Tensor row_values() const { return at::empty({T}, X.options().dtype(at::kFloat).requires_grad(false)); }
};

// (X, W, target, ignore_index, loss, lse, stream)
PyObject* linear_cross_entropy(PyObject* const* a) {
  const Loss in(a[0], a[1], a[2], a[3]);
  at::Tensor loss, lse;
  if (!is_none(a[4])) {
    loss = tensor(a[4], "loss");
    vector_of(loss, in.T, "loss must be a contiguous float32 vector with one value a row");
  }
  if (!is_none(a[5])) {
    lse = tensor(a[5], "lse");
    vector_of(lse, in.T, "lse must be a contiguous float32 vector with one value a row");
  }
  {
    const Launch on(a[6], {&in.X, &in.W, &in.target});
    if (!loss.defined()) loss = in.row_values();
    if (!lse.defined()) lse = in.row_values();
    on.check_device(loss);
    on.check_device(lse);
    const int st = fn.ce(in.type, in.T, in.V, in.H, in.X.data_ptr(), in.ldx, in.W.data_ptr(), in.ldw,
                         in.words(), in.ignore, static_cast<float*>(loss.data_ptr()),
                         static_cast<float*>(lse.data_ptr()), on.handle());
    if (st != 0) throw Status{st, "sgemm_linear_ce"};
  }
  return tuple_of(result(a[4], loss), result(a[5], lse));
}

// (X, W, target, lse, dloss, ignore_index, dX, dW, want dX, want dW, stream)
PyObject* linear_cross_entropy_grad(PyObject* const* a) {
  const Loss in(a[0], a[1], a[2], a[5]);
  const at::Tensor &lse = tensor(a[3], "lse"), &dloss = tensor(a[4], "dloss");
  vector_of(lse, in.T, "lse must be a contiguous float32 vector with one value a row");
  vector_of(dloss, in.T, "dloss must be a contiguous float32 vector with one value a row");
  const bool want_x = a[8] == Py_True, want_w = a[9] == Py_True;
  at::Tensor dX, dW;
  if (want_x && !is_none(a[6])) {
    dX = tensor(a[6], "dX");
    like(dX, in.X, "dX", "X");
  }
  if (want_w && !is_none(a[7])) {
    dW = tensor(a[7], "dW");
    like(dW, in.W, "dW", "W");
  }
  const int least = in.H > 1 ? in.H : 1;
  {
    const Launch on(a[10], {&in.X, &in.W, &in.target, &lse, &dloss});
    const auto options = in.X.options().requires_grad(false);
    if (want_x && !dX.defined()) dX = at::empty({in.T, in.H}, options);
    if (want_w && !dW.defined()) dW = at::empty({in.V, in.H}, options);
    if (want_x) on.check_device(dX);
    if (want_w) on.check_device(dW);
    const int st = fn.ce_grad(
        in.type, in.T, in.V, in.H, in.X.data_ptr(), in.ldx, in.W.data_ptr(), in.ldw, in.words(),
        in.ignore, static_cast<const float*>(lse.data_ptr()),
        static_cast<const float*>(dloss.data_ptr()), want_x ? dX.data_ptr() : nullptr,
        want_x ? pitch(dX, "dX") : least, want_w ? dW.data_ptr() : nullptr,
        want_w ? pitch(dW, "dW") : least, on.handle());
    if (st != 0) throw Status{st, "sgemm_linear_ce_grad"};
  }
  return tuple_of(want_x ? result(a[6], dX) : Py_NewRef(Py_None),
                  want_w ? result(a[7], dW) : Py_NewRef(Py_None));
}

// A matrix of 4-bit codes: rows of whole blocks of 16 bytes at 16-byte
// boundaries.
const at::Tensor& codes_of(const at::Tensor& t, const char* name) {
  if (t.scalar_type() != at::kByte || t.dim() != 2 || t.size(1) % 16 != 0)
    throw Refusal{std::string(name) + " must be a 2-D uint8 tensor with 16 bytes for every 32 values"};
  if (pitch(t, name) % 16 != 0 && t.size(0) > 1 && t.numel() > 0)
    throw Refusal{std::string(name) + " must have rows at multiples of 16 bytes"};
  return t;
}
int code_pitch(const at::Tensor& t, const char* name) {
  const int p = pitch(t, name);
  return t.size(1) == 0 ? 16 : p;       // (a pitch of 1 has no meaning here)
}
int64_t scale_bytes(int64_t rows, int64_t blocks) { return (rows + 127) / 128 * ((blocks + 3) / 4) * 512; }
const unsigned char* scales_of(const at::Tensor& t, int64_t rows, int64_t blocks, const char* name) {
  if (t.scalar_type() != at::kByte || t.dim() != 1 || !t.is_contiguous() ||
      t.numel() != scale_bytes(rows, blocks))
    throw Refusal{std::string(name) + " must be a contiguous uint8 vector with 512 bytes for every 128 rows x 4 blocks"};
  return static_cast<const unsigned char*>(t.data_ptr());
}

// (X, Q, scale, stream)
PyObject* mx4_quantize(PyObject* const* a) {
  const at::Tensor& X = tensor(a[0], "X");
  check(X.dim() == 2, "X must be 2-D");
  const int M = to_int(X.size(0)), K = to_int(X.size(1));
  const int64_t blocks = ((int64_t)K + 31) / 32;
  const int type = type_of(X, "X"), ldx = pitch(X, "X");
  at::Tensor Q, scale;
  if (!is_none(a[1])) {
    Q = codes_of(tensor(a[1], "Q"), "Q");
    check(Q.size(0) == M && Q.size(1) == blocks * 16, "Q must have a row of whole blocks for each of X");
  }
  if (!is_none(a[2])) {
    scale = tensor(a[2], "scale");
    scales_of(scale, M, blocks, "scale");
  }
  {
    const Launch on(a[3], {&X});
    const auto options = X.options().dtype(at::kByte).requires_grad(false);
    if (!Q.defined()) Q = at::empty({M, blocks * 16}, options);
    if (!scale.defined()) scale = at::empty({scale_bytes(M, blocks)}, options);
    on.check_device(Q);
    on.check_device(scale);
    const int st = fn.mx4_quantize(M, K, type, X.data_ptr(), ldx,
                                   static_cast<unsigned char*>(Q.data_ptr()), code_pitch(Q, "Q"),
                                   static_cast<unsigned char*>(scale.data_ptr()), on.handle());
    if (st != 0) throw Status{st, "sgemm_mx4_quantize"};
  }
  return tuple_of(result(a[1], Q), result(a[2], scale));
}

// (Q, scale, K, X, out_dtype, stream)
PyObject* mx4_dequantize(PyObject* const* a) {
  const at::Tensor &Q = codes_of(tensor(a[0], "Q"), "Q"), &scale = tensor(a[1], "scale");
  const long long k = PyLong_AsLongLong(a[2]);
  if (k == -1 && PyErr_Occurred()) throw PythonError{};
  const int M = to_int(Q.size(0)), K = to_int(k);
  check((k + 31) / 32 * 16 == Q.size(1), "K values are not the blocks of Q");
  scales_of(scale, M, Q.size(1) / 16, "scale");
  at::Tensor X;
  at::ScalarType out = at::kBFloat16;
  if (is_none(a[3])) {
    out = dtype_or(a[4], out);
  } else {
    X = tensor(a[3], "X");
    check(X.dim() == 2 && X.size(0) == M && X.size(1) == K, "shape mismatch");
    pitch(X, "X");
    type_of(X, "X");
    out = X.scalar_type();
  }
  const int type = type_of(out, "X");
  {
    const Launch on(a[5], {&Q, &scale});
    if (!X.defined()) X = at::empty({M, K}, Q.options().dtype(out).requires_grad(false));
    on.check_device(X);
    const int st = fn.mx4_dequantize(M, K, static_cast<const unsigned char*>(Q.data_ptr()),
                                     code_pitch(Q, "Q"),
                                     static_cast<const unsigned char*>(scale.data_ptr()), type,
                                     X.data_ptr(), pitch(X, "X"), on.handle());
    if (st != 0) throw Status{st, "sgemm_mx4_dequantize"};
  }
  return result(a[3], X);
}

// (A, scaleA, B, scaleB, C, out_dtype, stream)
PyObject* mx4_gemm(PyObject* const* a) {
  const at::Tensor &A = codes_of(tensor(a[0], "A"), "A"), &sa = tensor(a[1], "scaleA"),
                   &B = codes_of(tensor(a[2], "B"), "B"), &sb = tensor(a[3], "scaleB");
  check(A.size(1) == B.size(1), "shape mismatch");
  const int64_t blocks = A.size(1) / 16;
  const int M = to_int(A.size(0)), N = to_int(B.size(0)), K = to_int(blocks * 32);
  const unsigned char *scale_a = scales_of(sa, M, blocks, "scaleA"),
                      *scale_b = scales_of(sb, N, blocks, "scaleB");
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
  {
    const Launch on(a[6], {&A, &sa, &B, &sb});
    if (!C.defined()) C = at::empty({M, N}, A.options().dtype(out).requires_grad(false));
    on.check_device(C);
    const int st = fn.mx4(M, N, K, static_cast<const unsigned char*>(A.data_ptr()), code_pitch(A, "A"),
                          scale_a, static_cast<const unsigned char*>(B.data_ptr()),
                          code_pitch(B, "B"), scale_b, out_type, C.data_ptr(), pitch(C, "C"),
                          on.handle());
    if (st != 0) throw Status{st, "sgemm_mx4"};
  }
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

// (addresses of the C functions, in the order of Functions, the exception class)
PyObject* bind(PyObject*, PyObject* args) {
  constexpr int kFunctions = 13;
  PyObject *addresses, *error;
  if (!PyArg_ParseTuple(args, "O!O", &PyTuple_Type, &addresses, &error)) return nullptr;
  if (PyTuple_GET_SIZE(addresses) != kFunctions) {
    PyErr_SetString(PyExc_ValueError, "wrong number of functions");
    return nullptr;
  }
  unsigned long long p[kFunctions];
  for (int i = 0; i < kFunctions; ++i) {
    p[i] = PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(addresses, i));
    if (PyErr_Occurred()) return nullptr;
  }
  fn.grouped = reinterpret_cast<decltype(fn.grouped)>(p[0]);
  fn.wgrad = reinterpret_cast<decltype(fn.wgrad)>(p[1]);
  fn.quantize = reinterpret_cast<decltype(fn.quantize)>(p[2]);
  fn.i8 = reinterpret_cast<decltype(fn.i8)>(p[3]);
  fn.clip = reinterpret_cast<decltype(fn.clip)>(p[4]);
  fn.norm = reinterpret_cast<decltype(fn.norm)>(p[5]);
  fn.norm_i8 = reinterpret_cast<decltype(fn.norm_i8)>(p[6]);
  fn.norm_grad = reinterpret_cast<decltype(fn.norm_grad)>(p[7]);
  fn.ce = reinterpret_cast<decltype(fn.ce)>(p[8]);
  fn.ce_grad = reinterpret_cast<decltype(fn.ce_grad)>(p[9]);
  fn.mx4_quantize = reinterpret_cast<decltype(fn.mx4_quantize)>(p[10]);
  fn.mx4_dequantize = reinterpret_cast<decltype(fn.mx4_dequantize)>(p[11]);
  fn.mx4 = reinterpret_cast<decltype(fn.mx4)>(p[12]);
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
    SGEMM_GB300_METHOD(rms_norm, 8),
    SGEMM_GB300_METHOD(rms_norm_i8, 8),
    SGEMM_GB300_METHOD(rms_norm_grad, 10),
    SGEMM_GB300_METHOD(linear_cross_entropy, 7),
    SGEMM_GB300_METHOD(linear_cross_entropy_grad, 11),
    SGEMM_GB300_METHOD(mx4_quantize, 4),
    SGEMM_GB300_METHOD(mx4_dequantize, 6),
    SGEMM_GB300_METHOD(mx4_gemm, 7),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
