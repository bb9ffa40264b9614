// The layer operators' calls on torch tensors: argument checks, output and
// workspace memory, streams.  Only marshalling; every step of the computation
// is a call of the C ABI.  A decoded token's operators are a few microseconds
// of device work each, so this side of them is native: checking the tensors
// and taking the memory from Python cost 10 to 20 us a call.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <optional>
#include <stdexcept>
#include <string>

#include "ozemu.h"

namespace {

PyObject* g_status_error = nullptr;  // the package's OzemuError

// A refused argument (ValueError), and a Python error that is already set.
struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct Raised {};

const at::Tensor* tensor_or_none(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + ": expected a tensor");
  return &THPVariable_Unpack(o);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  const at::Tensor* t = tensor_or_none(o, name);
  if (!t) throw Refused(std::string(name) + ": expected a tensor");
  return *t;
}

int type_code(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return OZEMU_BF16;
    case at::kHalf: return OZEMU_F16;
    case at::kFloat: return OZEMU_F32;
    default: return -1;
  }
}

// Rows and columns of a 2-D argument, as the C ABI's int.
void sizes(const at::Tensor& t, const char* name, int* rows, int* cols) {
  if (t.dim() != 2) throw Refused(std::string(name) + ": expected a 2-D tensor");
  if (t.size(0) > INT_MAX || t.size(1) > INT_MAX) throw Refused(std::string(name) + ": too large");
  *rows = static_cast<int>(t.size(0));
  *cols = static_cast<int>(t.size(1));
}

struct Matrix {
  void* p = nullptr;
  int ld = 1;
};

// An optional row-major matrix of the given size, type and device.
Matrix matrix(const at::Tensor* t, int rows, int cols, const at::Tensor& like, const char* name) {
  Matrix m;
  m.ld = cols > 0 ? cols : 1;
  if (!t) return m;
  if (t->dim() != 2 || t->size(0) != rows || t->size(1) != cols || t->scalar_type() != like.scalar_type() ||
      t->device() != like.device() || t->layout() != at::kStrided)
    throw Refused(std::string(name) + ": expected a " + std::to_string(rows) + " x " + std::to_string(cols) +
                  " matrix of " + c10::toString(like.scalar_type()) + " on " + like.device().str());
  if (rows == 0 || cols == 0) return m;
  const int64_t outer = t->stride(0), inner = t->stride(1);
  if ((inner != 1 && cols > 1) || (rows > 1 && (outer < cols || outer > INT_MAX)))
    throw Refused(std::string(name) + ": expected a row-major matrix, got strides (" + std::to_string(outer) + ", " +
                  std::to_string(inner) + ")");
  m.p = t->data_ptr();
  if (rows > 1) m.ld = static_cast<int>(outer);
  return m;
}

// An optional dense vector.
void* vector(const at::Tensor* t, int n, at::ScalarType type, const at::Tensor& like, const char* name) {
  if (!t) return nullptr;
  if (t->dim() != 1 || t->size(0) != n || t->scalar_type() != type || t->device() != like.device() ||
      (n > 1 && t->stride(0) != 1))
    throw Refused(std::string(name) + ": expected a dense vector of " + std::to_string(n) + " " + c10::toString(type) +
                  " on " + like.device().str());
  return n > 0 ? t->data_ptr() : nullptr;
}

// Whether some row of `rows` rows of `width` bytes, `ld` bytes apart from `p`
// on, shares a byte with one of the other matrix's.
struct Area {
  intptr_t p;
  long long ld;
  int rows;
  long long width;
};
long long floor_div(long long a, long long b) { return a / b - (a % b < 0); }  // b > 0
bool share(const Area& a, const Area& b) {
  if (a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0) return false;
  if (a.p + (a.rows - 1) * a.ld + a.width <= b.p || b.p + (b.rows - 1) * b.ld + b.width <= a.p) return false;
  // A row at distance d from one of a's meets it where -b.width < d < a.width.
  // Of the distances d + t ld, t = first ... last, the first above -b.width:
  auto meets = [&](long long d, long long ld, long long first, long long last) {
    const long long t = std::max(first, floor_div(-b.width - d, ld) + 1);
    return t <= last && d + t * ld < a.width;
  };
  if (a.ld == b.ld) return meets(b.p - a.p, a.ld, 1 - a.rows, b.rows - 1);
  for (int i = 0; i < a.rows; ++i)  // matrices that lie within each other in rows of different lengths
    if (meets(b.p - (a.p + i * a.ld), b.ld, 0, b.rows - 1)) return true;
  return false;
}

// An output that the caller gives, against an input: they share nothing, or
// are the same matrix where the call takes it so.
class Output {
 public:
  Output(const at::Tensor* given, const Matrix& m, int rows, int cols, const at::Tensor& like)
      : given_(given), at_(area(m, rows, cols, static_cast<int>(like.element_size()))) {}
  void apart(const at::Tensor* input, const Matrix& m, int rows, int cols, const char* name, bool or_same = false) const {
    if (!given_ || !input) return;
    const Area in = area(m, rows, cols, static_cast<int>(input->element_size()));
    if (or_same && in.p == at_.p && (in.ld == at_.ld || rows <= 1)) return;
    if (share(at_, in)) throw Refused(std::string("out: overlaps ") + name);
  }
  void apart(const at::Tensor* input, void* p, int n, const char* name) const {
    Matrix m;
    m.p = p;
    m.ld = n > 0 ? n : 1;
    apart(input, m, 1, n, name);
  }

 private:
  static Area area(const Matrix& m, int rows, int cols, int size) {
    return {reinterpret_cast<intptr_t>(m.p), static_cast<long long>(m.ld) * size, m.p ? rows : 0,
            static_cast<long long>(cols) * size};
  }
  const at::Tensor* given_;
  Area at_;
};

// The stream of one call.  With a stream given, outputs and workspace are
// taken on it and the allocator learns of the inputs' use there; ordering
// their values is the caller's.
class OnStream {
 public:
  OnStream(const at::Tensor& like, PyObject* stream, std::initializer_list<const at::Tensor*> inputs) {
    if (!like.is_cuda()) throw Refused("expected CUDA tensors");
    if (like.device().index() != c10::cuda::current_device()) throw Refused("expected tensors on the current device");
    if (stream == Py_None) {
      handle = c10::cuda::getCurrentCUDAStream(like.device().index()).stream();
      return;
    }
    const c10::cuda::CUDAStream s(
        c10::Stream::unpack3(number(stream, "stream_id"), static_cast<c10::DeviceIndex>(number(stream, "device_index")),
                             static_cast<c10::DeviceType>(number(stream, "device_type"))));
    for (const at::Tensor* t : inputs)
      if (t) t->record_stream(s);
    guard_.emplace(s);
    handle = s.stream();
  }
  cudaStream_t handle;

 private:
  static int64_t number(PyObject* o, const char* name) {
    PyObject* v = PyObject_GetAttrString(o, name);
    if (!v) throw Raised();
    const long long n = PyLong_AsLongLong(v);
    Py_DECREF(v);
    if (n == -1 && PyErr_Occurred()) throw Raised();
    return n;
  }
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
};

// The calls record no graph: what requires a gradient would miss it without a
// word, so they say it (as a Python warning; an error where those are errors).
void no_graph(const char* call, const char* instead, std::initializer_list<const at::Tensor*> inputs) {
  if (!c10::GradMode::is_enabled()) return;
  for (const at::Tensor* t : inputs)
    if (t && t->requires_grad()) {
      const std::string text = std::string(call) +
                               ": an input requires a gradient, but this call records no graph for automatic "
                               "gradients; " + instead;
      if (PyErr_WarnEx(PyExc_UserWarning, text.c_str(), 2) < 0) throw Raised();
      return;
    }
}

// A workspace of `bytes` on the current stream, 256-byte aligned.
struct Scratch {
  Scratch(const at::Tensor& like, size_t n) : bytes(n) {
    if (n == 0) return;
    keep = at::empty({static_cast<int64_t>(n + 256)}, like.options().dtype(at::kByte));
    p = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(keep.data_ptr()) + 255) & ~uintptr_t(255));
  }
  at::Tensor keep;
  void* p = nullptr;
  size_t bytes;
};

void check(int status, const char* what) {
  if (status == OZEMU_OK) return;
  PyObject* e = PyObject_CallFunction(g_status_error, "is", status, what);
  if (e) {
    PyErr_SetObject(g_status_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

PyObject* wrapped(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

// (a, b, c): NULL with the error set if one of them could not be wrapped.
PyObject* triple(const at::Tensor& a, const at::Tensor& b, const at::Tensor& c) {
  PyObject *x = wrapped(a), *y = wrapped(b), *z = wrapped(c);
  PyObject* r = x && y && z ? PyTuple_Pack(3, x, y, z) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  Py_XDECREF(z);
  return r;
}

// Runs a call's body; no C++ exception leaves it.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F body) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

struct LinearSizes {
  int m, n, k, type, act;
};
LinearSizes linear_sizes(const at::Tensor& x, const at::Tensor& w, PyObject* act) {
  LinearSizes s;
  int k2;
  s.act = static_cast<int>(PyLong_AsLong(act));
  if (s.act == -1 && PyErr_Occurred()) throw Raised();
  s.type = type_code(x.scalar_type());
  if (s.type != OZEMU_BF16 && s.type != OZEMU_F16)
    throw Refused(std::string("expected bfloat16 or float16, got ") + c10::toString(x.scalar_type()));
  sizes(x, "x", &s.m, &s.k);
  sizes(w, "w", &s.n, &k2);
  return s;
}

// linear(x, w, bias, residual, activation, save_pre, out, stream)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 8, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w");
    const at::Tensor *bias = tensor_or_none(a[2], "bias"), *res = tensor_or_none(a[3], "residual");
    const at::Tensor* given = tensor_or_none(a[6], "out");
    const LinearSizes s = linear_sizes(x, w, a[4]);
    const bool save = truth(a[5]);
    const Matrix mx = matrix(&x, s.m, s.k, x, "x"), mw = matrix(&w, s.n, s.k, x, "w");
    const Matrix mr = matrix(res, s.m, s.n, x, "residual"), mo = matrix(given, s.m, s.n, x, "out");
    void* pb = vector(bias, s.n, x.scalar_type(), x, "bias");
    const Output o(given, mo, s.m, s.n, x);
    o.apart(&x, mx, s.m, s.k, "x");
    o.apart(&w, mw, s.n, s.k, "w");
    o.apart(bias, pb, s.n, "bias");
    o.apart(res, mr, s.m, s.n, "residual", true);
    OnStream on(x, a[7], {&x, &w, bias, res, given});
    no_graph("linear", "linear_backward computes them (torch.no_grad() says that none are wanted)", {&x, &w, bias, res});
    at::Tensor fresh, pre;
    Matrix my = mo, mp;
    if (!given) {
      fresh = at::empty({s.m, s.n}, x.options());
      my = matrix(&fresh, s.m, s.n, x, "out");
    }
    mp.ld = my.ld;
    if (save) {
      pre = at::empty({s.m, s.n}, x.options());
      mp = matrix(&pre, s.m, s.n, x, "pre");
    }
    const Scratch ws(x, ozemu_linear_bytes(s.m, s.n, s.k, mx.p, mx.ld, mw.p, mw.ld));
    check(ozemu_linear(s.m, s.n, s.k, s.type, mx.p, mx.ld, mw.p, mw.ld, pb, mr.p, mr.ld, s.act, mp.p, mp.ld, my.p,
                       my.ld, ws.p, ws.bytes, on.handle),
          "ozemu_linear");
    PyObject* y = a[6];
    if (given)
      Py_INCREF(y);
    else
      y = THPVariable_Wrap(fresh);
    if (!save || !y) return y;
    PyObject* z = THPVariable_Wrap(pre);
    PyObject* r = z ? PyTuple_Pack(2, y, z) : nullptr;
    Py_DECREF(y);
    Py_XDECREF(z);
    return r;
  });
}

// linear_backward(dy, x, w, pre, activation, x_grad, w_grad, bias_grad, stream)
PyObject* linear_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 9, [&]() -> PyObject* {
    const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x"), &w = tensor(a[2], "w");
    const LinearSizes s = linear_sizes(x, w, a[4]);
    const at::Tensor* pre = s.act == OZEMU_ACT_NONE ? nullptr : tensor_or_none(a[3], "pre");
    if (s.act != OZEMU_ACT_NONE && !pre) throw Refused("pre: this activation needs the pre-activation");
    const Matrix md = matrix(&dy, s.m, s.n, x, "dy"), mx = matrix(&x, s.m, s.k, x, "x");
    const Matrix mw = matrix(&w, s.n, s.k, x, "w"), mp = matrix(pre, s.m, s.n, x, "pre");
    OnStream on(x, a[8], {&dy, &x, &w, pre});
    no_graph("linear_backward", "torch.no_grad() says that none are wanted", {&dy, &x, &w, pre});
    at::Tensor dx, dw, db;
    if (truth(a[5])) dx = at::empty({s.m, s.k}, x.options());
    if (truth(a[6])) dw = at::empty({s.n, s.k}, x.options());
    if (truth(a[7])) db = at::empty({s.n}, x.options());
    const int ld = s.k > 0 ? s.k : 1;
    const Scratch ws(x, ozemu_linear_backward_bytes(s.m, s.n, s.k, md.p, md.ld, mx.p, mx.ld, mw.p, mw.ld, s.act));
    check(ozemu_linear_backward(s.m, s.n, s.k, s.type, md.p, md.ld, mx.p, mx.ld, mw.p, mw.ld, s.act, mp.p, mp.ld,
                                dx.defined() ? dx.data_ptr() : nullptr, ld, dw.defined() ? dw.data_ptr() : nullptr, ld,
                                db.defined() ? db.data_ptr() : nullptr, ws.p, ws.bytes, on.handle),
          "ozemu_linear_backward");
    return triple(dx, dw, db);
  });
}

// The type of a norm's parameters: their own, or x's where there are none.
at::ScalarType param_type(const at::Tensor& x, const at::Tensor* weight, const at::Tensor* bias) {
  const at::ScalarType t = weight ? weight->scalar_type() : bias ? bias->scalar_type() : x.scalar_type();
  if (type_code(x.scalar_type()) < 0)
    throw Refused(std::string("expected bfloat16, float16 or float32, got ") + c10::toString(x.scalar_type()));
  if (t != x.scalar_type() && t != at::kFloat)
    throw Refused(std::string("expected parameters of ") + c10::toString(x.scalar_type()) + " or Float, got " +
                  c10::toString(t));
  return t;
}

// layer_norm(x, weight, bias, eps, stats, out, stream)
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 7, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "x");
    const at::Tensor *weight = tensor_or_none(a[1], "weight"), *bias = tensor_or_none(a[2], "bias");
    const at::Tensor* given = tensor_or_none(a[5], "out");
    const at::ScalarType pt = param_type(x, weight, bias);
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised();
    const bool stats = truth(a[4]);
    int rows, cols;
    sizes(x, "x", &rows, &cols);
    const Matrix mx = matrix(&x, rows, cols, x, "x"), mo = matrix(given, rows, cols, x, "out");
    void *pw = vector(weight, cols, pt, x, "weight"), *pb = vector(bias, cols, pt, x, "bias");
    const Output o(given, mo, rows, cols, x);
    o.apart(&x, mx, rows, cols, "x", true);
    o.apart(weight, pw, cols, "weight");
    o.apart(bias, pb, cols, "bias");
    OnStream on(x, a[6], {&x, weight, bias, given});
    no_graph("layer_norm", "layer_norm_backward computes them (torch.no_grad() says that none are wanted)",
             {&x, weight, bias});
    at::Tensor fresh, mean, rstd;
    Matrix my = mo;
    if (!given) {
      fresh = at::empty({rows, cols}, x.options());
      my = matrix(&fresh, rows, cols, x, "out");
    }
    if (stats) {
      mean = at::empty({rows}, x.options().dtype(at::kFloat));
      rstd = at::empty({rows}, x.options().dtype(at::kFloat));
    }
    check(ozemu_layer_norm(rows, cols, type_code(x.scalar_type()), mx.p, mx.ld, type_code(pt), pw, pb,
                           static_cast<float>(eps), my.p, my.ld, stats ? mean.data_ptr<float>() : nullptr,
                           stats ? rstd.data_ptr<float>() : nullptr, on.handle),
          "ozemu_layer_norm");
    if (stats) return triple(given ? *given : fresh, mean, rstd);
    if (given) return Py_NewRef(a[5]);
    return THPVariable_Wrap(fresh);
  });
}

// layer_norm_backward(dy, x, mean, rstd, weight, dresidual, weight_grad, bias_grad, out, stream)
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 10, [&]() -> PyObject* {
    const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x");
    const at::Tensor &mean = tensor(a[2], "mean"), &rstd = tensor(a[3], "rstd");
    const at::Tensor *weight = tensor_or_none(a[4], "weight"), *dr = tensor_or_none(a[5], "dresidual");
    const at::Tensor* given = tensor_or_none(a[8], "out");
    const at::ScalarType pt = param_type(x, weight, nullptr);
    int rows, cols;
    sizes(x, "x", &rows, &cols);
    const Matrix md = matrix(&dy, rows, cols, x, "dy"), mx = matrix(&x, rows, cols, x, "x");
    const Matrix mr = matrix(dr, rows, cols, x, "dresidual"), mo = matrix(given, rows, cols, x, "out");
    void* pw = vector(weight, cols, pt, x, "weight");
    void *pm = vector(&mean, rows, at::kFloat, x, "mean"), *ps = vector(&rstd, rows, at::kFloat, x, "rstd");
    const Output o(given, mo, rows, cols, x);
    o.apart(&dy, md, rows, cols, "dy", true);
    o.apart(&x, mx, rows, cols, "x", true);
    o.apart(dr, mr, rows, cols, "dresidual", true);
    o.apart(weight, pw, cols, "weight");
    o.apart(&mean, pm, rows, "mean");
    o.apart(&rstd, ps, rows, "rstd");
    OnStream on(x, a[9], {&dy, &x, &mean, &rstd, weight, dr, given});
    no_graph("layer_norm_backward", "torch.no_grad() says that none are wanted", {&dy, &x, weight, dr});
    at::Tensor fresh, dw, db;
    Matrix mdx = mo;
    if (!given) {
      fresh = at::empty({rows, cols}, x.options());
      mdx = matrix(&fresh, rows, cols, x, "out");
    }
    if (truth(a[6])) dw = at::empty({cols}, x.options().dtype(pt));
    if (truth(a[7])) db = at::empty({cols}, x.options().dtype(pt));
    const Scratch ws(x, ozemu_layer_norm_backward_bytes(rows, cols));
    check(ozemu_layer_norm_backward(rows, cols, type_code(x.scalar_type()), md.p, md.ld, mx.p, mx.ld, type_code(pt), pw,
                                    static_cast<const float*>(pm), static_cast<const float*>(ps), mr.p, mr.ld, mdx.p,
                                    mdx.ld, dw.defined() ? dw.data_ptr() : nullptr,
                                    db.defined() ? db.data_ptr() : nullptr, ws.p, ws.bytes, on.handle),
          "ozemu_layer_norm_backward");
    return triple(given ? *given : fresh, dw, db);
  });
}

// setup(OzemuError)
PyObject* setup(PyObject*, PyObject* error) {
  Py_INCREF(error);
  Py_XDECREF(g_status_error);
  g_status_error = error;
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear)), METH_FASTCALL, nullptr},
    {"linear_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear_backward)), METH_FASTCALL,
     nullptr},
    {"layer_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(layer_norm)), METH_FASTCALL, nullptr},
    {"layer_norm_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(layer_norm_backward)),
     METH_FASTCALL, nullptr},
    {"setup", setup, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ozemu_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr,
                        nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ozemu_torch() { return PyModule_Create(&g_module); }
