// The layer operators' calls on torch tensors: argument checks, output and
// workspace memory, streams.  Only marshalling; every step of the computation
// is a call of the C ABI.  A decoded token's operators are a few microseconds
// of device work each, so this side of them is native: checking the tensors
// and taking the memory from Python cost 10 to 20 us a call.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
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
#include <vector>

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
  // Against an array of bytes.
  void apart(const at::Tensor& bytes, const char* name) const {
    const long long n = bytes.numel();
    if (given_ && share(at_, {reinterpret_cast<intptr_t>(bytes.data_ptr()), n, n > 0 ? 1 : 0, n}))
      throw Refused(std::string("out: overlaps ") + name);
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
  OnStream(const at::Tensor& like, PyObject* stream, const std::vector<const at::Tensor*>& inputs) {
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
void no_graph(const char* call, const char* instead, const std::vector<const at::Tensor*>& inputs) {
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

// The same for a gated layer, whose w has two rows for an output.
LinearSizes gated_sizes(const at::Tensor& x, const at::Tensor& w, PyObject* act) {
  LinearSizes s = linear_sizes(x, w, act);
  if (s.n % 2 != 0) throw Refused("w: expected an even number of rows, the gate's and as many of the up projection");
  s.n /= 2;
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

// gated_linear(x, w, bias, activation, save_pre, out, stream)
PyObject* gated_linear(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 7, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w");
    const at::Tensor *bias = tensor_or_none(a[2], "bias"), *given = tensor_or_none(a[5], "out");
    const LinearSizes s = gated_sizes(x, w, a[3]);
    const bool save = truth(a[4]);
    const Matrix mx = matrix(&x, s.m, s.k, x, "x"), mw = matrix(&w, 2 * s.n, s.k, x, "w");
    const Matrix mo = matrix(given, s.m, s.n, x, "out");
    void* pb = vector(bias, 2 * s.n, x.scalar_type(), x, "bias");
    const Output o(given, mo, s.m, s.n, x);
    o.apart(&x, mx, s.m, s.k, "x");
    o.apart(&w, mw, 2 * s.n, s.k, "w");
    o.apart(bias, pb, 2 * s.n, "bias");
    OnStream on(x, a[6], {&x, &w, bias, given});
    no_graph("gated_linear", "gated_linear_backward computes them (torch.no_grad() says that none are wanted)",
             {&x, &w, bias});
    at::Tensor fresh, pre;
    Matrix mh = mo, mp;
    if (!given) {
      fresh = at::empty({s.m, s.n}, x.options());
      mh = matrix(&fresh, s.m, s.n, x, "out");
    }
    mp.ld = s.n > 0 ? 2 * s.n : 1;
    if (save) {
      pre = at::empty({s.m, 2 * s.n}, x.options());
      mp = matrix(&pre, s.m, 2 * s.n, x, "pre");
    }
    const Scratch ws(x, ozemu_gated_linear_bytes(s.m, s.n, s.k, mx.p, mx.ld, mw.p, mw.ld));
    check(ozemu_gated_linear(s.m, s.n, s.k, s.type, mx.p, mx.ld, mw.p, mw.ld, pb, s.act, mp.p, mp.ld, mh.p, mh.ld, ws.p,
                             ws.bytes, on.handle),
          "ozemu_gated_linear");
    PyObject* h = given ? Py_NewRef(a[5]) : THPVariable_Wrap(fresh);
    if (!save || !h) return h;
    PyObject* z = THPVariable_Wrap(pre);
    PyObject* r = z ? PyTuple_Pack(2, h, z) : nullptr;
    Py_DECREF(h);
    Py_XDECREF(z);
    return r;
  });
}

// gated_linear_backward(dh, x, w, pre, activation, x_grad, w_grad, bias_grad, stream)
PyObject* gated_linear_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 9, [&]() -> PyObject* {
    const at::Tensor &dh = tensor(a[0], "dh"), &x = tensor(a[1], "x"), &w = tensor(a[2], "w"), &pre = tensor(a[3], "pre");
    const LinearSizes s = gated_sizes(x, w, a[4]);
    const Matrix md = matrix(&dh, s.m, s.n, x, "dh"), mx = matrix(&x, s.m, s.k, x, "x");
    const Matrix mw = matrix(&w, 2 * s.n, s.k, x, "w"), mp = matrix(&pre, s.m, 2 * s.n, x, "pre");
    OnStream on(x, a[8], {&dh, &x, &w, &pre});
    no_graph("gated_linear_backward", "torch.no_grad() says that none are wanted", {&dh, &x, &w, &pre});
    at::Tensor dx, dw, db;
    if (truth(a[5])) dx = at::empty({s.m, s.k}, x.options());
    if (truth(a[6])) dw = at::empty({2 * s.n, s.k}, x.options());
    if (truth(a[7])) db = at::empty({2 * s.n}, x.options());
    const int ld = s.k > 0 ? s.k : 1;
    const Scratch ws(x, ozemu_gated_linear_backward_bytes(s.m, s.n, s.k, mx.p, mx.ld, mw.p, mw.ld));
    check(ozemu_gated_linear_backward(s.m, s.n, s.k, s.type, md.p, md.ld, mx.p, mx.ld, mw.p, mw.ld, s.act, mp.p, mp.ld,
                                      dx.defined() ? dx.data_ptr() : nullptr, ld, dw.defined() ? dw.data_ptr() : nullptr,
                                      ld, db.defined() ? db.data_ptr() : nullptr, ws.p, ws.bytes, on.handle),
          "ozemu_gated_linear_backward");
    return triple(dx, dw, db);
  });
}

// A microscaled matrix in one array: the codes, then the scales from the next
// 256-byte boundary on.
struct MxData {
  MxData(int rows, int k) : rows(rows), k(k), codes(ozemu_mx_code_bytes(rows, k)) {
    at = (codes + 255) & ~static_cast<size_t>(255);
    bytes = static_cast<int64_t>(at + ozemu_mx_scale_bytes(rows, k));
  }
  void in(const at::Tensor& t, const at::Tensor& like, const char* name) {
    if (t.scalar_type() != at::kByte || t.device() != like.device() || t.dim() != 1 || t.size(0) != bytes ||
        (bytes > 1 && t.stride(0) != 1))
      throw Refused(std::string(name) + ": expected a dense vector of " + std::to_string(bytes) + " Byte on " +
                    like.device().str());
    p = static_cast<uint8_t*>(t.data_ptr());
    if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0) throw Refused(std::string(name) + ": not on a 16-byte boundary");
  }
  uint8_t* scales() const { return p + at; }
  int rows, k;
  size_t codes, at;
  int64_t bytes;
  uint8_t* p = nullptr;
};

int integer(PyObject* o) {
  const long long n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) throw Raised();
  if (n < 0 || n > INT_MAX) throw Refused("sizes: out of range");
  return static_cast<int>(n);
}

at::ScalarType scalar_type(int code) {
  return code == OZEMU_F32 ? at::kFloat : code == OZEMU_F16 ? at::kHalf : at::kBFloat16;
}

// mx_quantize(x, out, stream): the matrix's array, a fresh one for None
PyObject* mx_quantize(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 3, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "x");
    const at::Tensor* given = tensor_or_none(a[1], "out");
    int rows, k;
    sizes(x, "x", &rows, &k);
    if (type_code(x.scalar_type()) < 0)
      throw Refused(std::string("expected bfloat16, float16 or float32, got ") + c10::toString(x.scalar_type()));
    const Matrix mx = matrix(&x, rows, k, x, "x");
    MxData q(rows, k);
    if (given) {
      q.in(*given, x, "out");
      const long long size = x.element_size();
      if (share({reinterpret_cast<intptr_t>(q.p), q.bytes, q.bytes > 0 ? 1 : 0, q.bytes},
                {reinterpret_cast<intptr_t>(mx.p), mx.ld * size, mx.p ? rows : 0, k * size}))
        throw Refused("out: overlaps x");
    }
    OnStream on(x, a[2], {&x, given});
    no_graph("mx_quantize", "torch.no_grad() says that none are wanted", {&x});
    at::Tensor fresh;
    if (!given) {
      fresh = at::empty({q.bytes}, x.options().dtype(at::kByte));
      q.in(fresh, x, "out");
    }
    check(ozemu_mx_quantize(rows, k, type_code(x.scalar_type()), mx.p, mx.ld, q.p, q.scales(), on.handle),
          "ozemu_mx_quantize");
    return given ? Py_NewRef(a[1]) : THPVariable_Wrap(fresh);
  });
}

// mx_dequantize(data, rows, k, type, out, stream)
PyObject* mx_dequantize(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 6, [&]() -> PyObject* {
    const at::Tensor& data = tensor(a[0], "q");
    const int rows = integer(a[1]), k = integer(a[2]), type = integer(a[3]);
    const at::Tensor* given = tensor_or_none(a[4], "out");
    MxData q(rows, k);
    q.in(data, data, "q");
    const at::TensorOptions options = data.options().dtype(scalar_type(type));
    Matrix my;
    if (given) {
      if (given->scalar_type() != scalar_type(type) || given->device() != data.device())
        throw Refused(std::string("out: expected a matrix of ") + c10::toString(scalar_type(type)) + " on " +
                      data.device().str());
      my = matrix(given, rows, k, *given, "out");
      const Output o(given, my, rows, k, *given);
      o.apart(data, "q");
    }
    OnStream on(data, a[5], {&data, given});
    at::Tensor fresh;
    if (!given) {
      fresh = at::empty({rows, k}, options);
      my = matrix(&fresh, rows, k, fresh, "out");
    }
    check(ozemu_mx_dequantize(rows, k, type, q.p, q.scales(), my.p, my.ld, on.handle), "ozemu_mx_dequantize");
    return given ? Py_NewRef(a[4]) : THPVariable_Wrap(fresh);
  });
}

// mx_linear(x, m, w, n, k, bias, residual or factor, whether it is a factor, activation, type, out, stream)
PyObject* mx_linear(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 12, [&]() -> PyObject* {
    const at::Tensor &dx = tensor(a[0], "x"), &dw = tensor(a[2], "w");
    const int m = integer(a[1]), n = integer(a[3]), k = integer(a[4]), act = integer(a[8]), type = integer(a[9]);
    const bool times = truth(a[7]);
    const char* name = times ? "times" : "residual";
    const at::Tensor *bias = tensor_or_none(a[5], "bias"), *res = tensor_or_none(a[6], name);
    const at::Tensor* given = tensor_or_none(a[10], "out");
    MxData x(m, k), w(n, k);
    x.in(dx, dx, "x");
    w.in(dw, dx, "w");
    const at::ScalarType t = scalar_type(type);
    // The matrices of the call's type, against one of that type.
    const at::Tensor* like = given ? given : res ? res : bias;
    if (like && (like->scalar_type() != t || like->device() != dx.device()))
      throw Refused(std::string(given ? "out" : res ? name : "bias") + ": expected " + c10::toString(t) + " on " +
                    dx.device().str());
    Matrix mr, my;
    void* pb = nullptr;
    mr.ld = my.ld = n > 0 ? n : 1;
    if (like) {
      mr = matrix(res, m, n, *like, name);
      my = matrix(given, m, n, *like, "out");
      pb = vector(bias, n, t, *like, "bias");
      const Output o(given, my, m, n, *like);
      o.apart(bias, pb, n, "bias");
      o.apart(res, mr, m, n, name, true);
      o.apart(dx, "x");
      o.apart(dw, "w");
    }
    OnStream on(dx, a[11], {&dx, &dw, bias, res, given});
    no_graph("mx_linear", "torch.no_grad() says that none are wanted", {bias, res});
    at::Tensor fresh;
    if (!given) {
      fresh = at::empty({m, n}, dx.options().dtype(t));
      my = matrix(&fresh, m, n, fresh, "out");
    }
    check(ozemu_mx_linear(m, n, k, type, x.p, x.scales(), w.p, w.scales(), pb, mr.p, mr.ld, times, act, my.p, my.ld, on.handle),
          "ozemu_mx_linear");
    return given ? Py_NewRef(a[10]) : THPVariable_Wrap(fresh);
  });
}

// The tensors of a sequence, which `keep` holds a reference to.
struct Sequence {
  Sequence(PyObject* o, const char* name) : keep(PySequence_Fast(o, name)) {
    if (!keep) throw Raised();
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(keep); ++i) {
      PyObject* item = PySequence_Fast_GET_ITEM(keep, i);
      if (!THPVariable_Check(item)) {
        Py_DECREF(keep);
        throw Refused(std::string(name) + ": expected a sequence of tensors");
      }
      t.push_back(&THPVariable_Unpack(item));
    }
  }
  ~Sequence() { Py_DECREF(keep); }
  Sequence(const Sequence&) = delete;
  PyObject* keep;
  std::vector<const at::Tensor*> t;
};

struct Bytes {
  uintptr_t begin, end;
  size_t which;
};
bool before(const Bytes& a, const Bytes& b) { return a.begin < b.begin; }

// clip_grad_norm(grads, max_norm, eps, out, stream)
PyObject* clip_grad_norm(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 5, [&]() -> PyObject* {
    const Sequence grads(a[0], "grads: expected a sequence of tensors");
    const size_t n = grads.t.size();
    if (n == 0) throw Refused("grads: expected at least one tensor");
    if (n > static_cast<size_t>(INT_MAX)) throw Refused("grads: too many tensors");
    const double max_norm = PyFloat_AsDouble(a[1]);
    if (max_norm == -1.0 && PyErr_Occurred()) throw Raised();
    const double eps = PyFloat_AsDouble(a[2]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised();
    std::optional<Sequence> given;
    if (a[3] != Py_None) {
      given.emplace(a[3], "out: expected a sequence of tensors");
      if (given->t.size() != n) throw Refused("out: expected as many tensors as grads");
    }
    const at::Tensor& first = *grads.t[0];
    for (const at::Tensor* t : grads.t) {
      if (type_code(t->scalar_type()) < 0)
        throw Refused(std::string("grads: expected bfloat16, float16 or float32, got ") + c10::toString(t->scalar_type()));
      if (t->device() != first.device()) throw Refused("grads: expected tensors of one device");
      if (t->layout() != at::kStrided || !t->is_non_overlapping_and_dense())
        throw Refused("grads: expected dense tensors");
    }
    std::vector<const at::Tensor*> all = grads.t;
    if (given) all.insert(all.end(), given->t.begin(), given->t.end());
    std::vector<const void*> in(n);
    std::vector<void*> outs(n);
    std::vector<long long> sizes(n);
    std::vector<int> types(n);
    std::vector<Bytes> written;
    for (size_t i = 0; i < n; ++i) {
      const at::Tensor& g = *grads.t[i];
      in[i] = g.numel() > 0 ? g.data_ptr() : nullptr;
      sizes[i] = g.numel();
      types[i] = type_code(g.scalar_type());
      if (!given) continue;
      const at::Tensor& o = *given->t[i];
      if (o.scalar_type() != g.scalar_type() || o.device() != g.device() || o.layout() != at::kStrided ||
          o.sizes() != g.sizes())
        throw Refused("out: expected tensors of the gradients' sizes, types and device");
      if (g.numel() == 0) continue;
      for (int64_t d = 0; d < g.dim(); ++d)
        if (g.size(d) > 1 && o.stride(d) != g.stride(d)) throw Refused("out: expected tensors of the gradients' strides");
      outs[i] = o.data_ptr();
      const uintptr_t p = reinterpret_cast<uintptr_t>(outs[i]);
      written.push_back({p, p + g.nbytes(), i});
    }
    // Outputs share nothing with each other, nor with a gradient but their own.
    std::sort(written.begin(), written.end(), before);
    for (size_t i = 1; i < written.size(); ++i)
      if (written[i].begin < written[i - 1].end) throw Refused("out: overlaps another output");
    if (given)
      for (size_t i = 0; i < n; ++i) {
        if (sizes[i] == 0) continue;
        const uintptr_t p = reinterpret_cast<uintptr_t>(in[i]);
        const uintptr_t end = p + grads.t[i]->nbytes();
        // The last output that begins before this gradient's end, and those before it that reach into it.
        auto at = std::lower_bound(written.begin(), written.end(), Bytes{end, 0, 0}, before);
        while (at != written.begin()) {
          --at;
          if (at->end <= p) break;
          if (!(at->which == i && at->begin == p)) throw Refused("out: overlaps a gradient that is not its own");
        }
      }
    OnStream on(first, a[4], all);
    no_graph("clip_grad_norm", "torch.no_grad() says that none are wanted", grads.t);
    std::vector<at::Tensor> fresh;
    if (!given) {
      fresh.reserve(n);
      for (size_t i = 0; i < n; ++i) {
        fresh.push_back(at::empty_like(*grads.t[i]));
        outs[i] = sizes[i] > 0 ? fresh[i].data_ptr() : nullptr;
      }
    }
    const at::Tensor norm = at::empty({}, first.options().dtype(at::kFloat));
    const int total = static_cast<int>(n);
    const Scratch ws(first, ozemu_clip_grad_norm_bytes(total, in.data(), sizes.data(), types.data()));
    check(ozemu_clip_grad_norm(total, in.data(), sizes.data(), types.data(), outs.data(), static_cast<float>(max_norm),
                               static_cast<float>(eps), norm.data_ptr<float>(), ws.p, ws.bytes, on.handle),
          "ozemu_clip_grad_norm");
    PyObject* list = PyList_New(static_cast<Py_ssize_t>(n));
    if (!list) throw Raised();
    for (size_t i = 0; i < n; ++i) {
      PyObject* o = given ? Py_NewRef(PySequence_Fast_GET_ITEM(given->keep, static_cast<Py_ssize_t>(i)))
                          : THPVariable_Wrap(fresh[i]);
      if (!o) {
        Py_DECREF(list);
        throw Raised();
      }
      PyList_SET_ITEM(list, static_cast<Py_ssize_t>(i), o);
    }
    PyObject* length = THPVariable_Wrap(norm);
    PyObject* r = length ? PyTuple_Pack(2, length, list) : nullptr;
    Py_XDECREF(length);
    Py_DECREF(list);
    return r;
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
    {"gated_linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gated_linear)), METH_FASTCALL, nullptr},
    {"gated_linear_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gated_linear_backward)),
     METH_FASTCALL, nullptr},
    {"mx_quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(mx_quantize)), METH_FASTCALL, nullptr},
    {"mx_dequantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(mx_dequantize)), METH_FASTCALL,
     nullptr},
    {"mx_linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(mx_linear)), METH_FASTCALL, nullptr},
    {"clip_grad_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(clip_grad_norm)), METH_FASTCALL,
     nullptr},
    {"setup", setup, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ozemu_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr,
                        nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ozemu_torch() { return PyModule_Create(&g_module); }
