// The commonest calls of drop.py and quant.py without their Python: tensors that
// lie on the current device and its current stream, are contiguous and fit one
// another.  Each function checks that, allocates the outputs with PyTorch and
// calls the same entry point of the library; for anything else, and for what the
// library refuses, it returns None, and the caller's own path checks again and
// says what is wrong.  A call of norm_quant took 17 us through Python and ctypes,
// of which the launch is 2, so short calls waited for the host; here it takes 6 to 8.
// Outputs come from the CUDA allocator without the dispatcher, 0.3 us less each.
#include <Python.h>

#include <array>
#include <map>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/addln_dropout.h"
#include "../../include/addln_quant.h"

namespace {

// The library's entry points, by address (init).
struct Entries {
  decltype(&dropout_fwd) drop;
  decltype(&dropout_add_norm_fwd) fwd;
  decltype(&dropout_add_norm_bwd) bwd;
  decltype(&dropout_add_norm_bwd_workspace_size) bwd_size;
  decltype(&norm_quant_fwd) quant;
  decltype(&dequant_rows) dequant;
} lib{};

// Workspace sizes by what decides them.
std::map<std::array<int64_t, 4>, int64_t> sizes;

// The tensor of a Python object that is one (not of a subclass), or NULL.
const at::Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

int code_of(at::ScalarType t) {
  return t == at::kFloat ? ADDLN_FP32 : t == at::kHalf ? ADDLN_FP16 : t == at::kBFloat16 ? ADDLN_BF16 : -1;
}

// A call's first tensor: dense, contiguous, [..., H], on the current device.
struct Rows {
  const at::Tensor* t = nullptr;
  int64_t rows = 0, H = 0;
  int code = -1;
  void* stream = nullptr;

  bool take(PyObject* o) {
    t = tensor(o);
    if (t == nullptr || !t->defined() || !t->is_cuda() || t->layout() != at::kStrided || !t->is_contiguous() ||
        t->numel() == 0)
      return false;
    const auto index = t->get_device();
    if (index != c10::cuda::current_device()) return false;
    stream = c10::cuda::getCurrentCUDAStream(index).stream();
    return true;
  }
  bool take_rows(PyObject* o) {
    if (!take(o) || t->dim() < 1 || t->size(-1) < 1) return false;
    code = code_of(t->scalar_type());
    H = t->size(-1);
    rows = t->numel() / H;
    return code >= 0;
  }
  bool fits(const at::Tensor* o, at::ScalarType type) const {
    return o != nullptr && o->defined() && o->is_cuda() && o->layout() == at::kStrided && o->scalar_type() == type &&
           o->get_device() == t->get_device() && o->is_contiguous();
  }
  // The address of a tensor that stands beside this one, or of None (NULL).
  bool beside(PyObject* o, const void** at) const {
    *at = nullptr;
    if (o == Py_None) return true;
    const at::Tensor* b = tensor(o);
    if (!fits(b, t->scalar_type()) || !b->sizes().equals(t->sizes())) return false;
    *at = b->const_data_ptr();
    return true;
  }
  // The same of an fp32 vector of n elements.
  bool vector(PyObject* o, int64_t n, const float** at) const {
    *at = nullptr;
    if (o == Py_None) return true;
    const at::Tensor* b = tensor(o);
    if (!fits(b, at::kFloat) || b->numel() != n) return false;
    *at = b->const_data_ptr<float>();
    return true;
  }
  at::Tensor same(at::ScalarType type) const { return at::detail::empty_cuda(t->sizes(), type, t->device(), std::nullopt); }
  at::Tensor floats(at::IntArrayRef sizes) const { return at::detail::empty_cuda(sizes, at::kFloat, t->device(), std::nullopt); }
};

// A dropout's p and rng: two whole numbers of up to 64 bits, or an int64 tensor of
// two on the device of `like`.
struct Drop {
  double p;
  const int64_t* rng = nullptr;
  uint64_t seed = 0, offset = 0;

  bool take(PyObject* po, PyObject* ro, const Rows& like) {
    if (!PyFloat_CheckExact(po)) return false;
    p = PyFloat_AS_DOUBLE(po);
    if (PyTuple_CheckExact(ro) && PyTuple_GET_SIZE(ro) == 2 && PyLong_CheckExact(PyTuple_GET_ITEM(ro, 0)) &&
        PyLong_CheckExact(PyTuple_GET_ITEM(ro, 1))) {
      seed = PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(ro, 0));
      if (!PyErr_Occurred()) offset = PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(ro, 1));
      if (!PyErr_Occurred()) return true;
      PyErr_Clear();  // negative, or too large
      return false;
    }
    const at::Tensor* t = tensor(ro);
    if (!like.fits(t, at::kLong) || t->numel() != 2) return false;
    rng = t->const_data_ptr<int64_t>();
    return true;
  }
};

bool number(PyObject* o, double* v) {
  if (!PyFloat_CheckExact(o)) return false;
  *v = PyFloat_AS_DOUBLE(o);
  return true;
}
bool number(PyObject* o, int64_t* v) {
  if (!PyLong_CheckExact(o)) return false;
  *v = PyLong_AsLongLong(o);
  if (!PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}

// True or False itself: what Python merely takes for one is left to its path.
bool truth(PyObject* o, bool* v) {
  *v = o == Py_True;
  return *v || o == Py_False;
}

PyObject* none() { Py_RETURN_NONE; }
PyObject* wrap(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : none(); }
void* ptr(const at::Tensor& t) { return t.defined() ? t.mutable_data_ptr() : nullptr; }
float* fptr(const at::Tensor& t) { return static_cast<float*>(ptr(t)); }

template <typename... T>
PyObject* tuple(const T&... t) {
  PyObject* out = PyTuple_New(sizeof...(T));
  if (out == nullptr) return nullptr;
  int i = 0;
  bool ok = true;
  auto put = [&](PyObject* o) {
    ok = ok && o != nullptr;
    PyTuple_SET_ITEM(out, i++, o);
  };
  (put(wrap(t)), ...);
  if (ok) return out;
  Py_DECREF(out);
  return nullptr;
}

// Whether a vector's gradient, which is made with one dimension, has its shape.
bool one_dimension(PyObject* o) { return o == Py_None || THPVariable_Unpack(o).dim() == 1; }

// Runs a call's body; a C++ exception (no memory, say) becomes None.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
    PyErr_Clear();
    return none();
  }
}

// dropout(x, p, rng)
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Rows x;
    Drop d;
    if (n != 3 || lib.drop == nullptr || !x.take(a[0])) return none();
    const int code = code_of(x.t->scalar_type());
    if (code < 0 || !d.take(a[1], a[2], x)) return none();
    const at::Tensor y = x.same(x.t->scalar_type());
    if (lib.drop(x.t->const_data_ptr(), ptr(y), x.t->numel(), d.p, d.rng, d.seed, d.offset, code, x.stream)) return none();
    return wrap(y);
  });
}

// dropout_add_norm(f, x, p, rng, bias, norm, gamma, beta, eps, want_stats):
// h, y, mean, rstd
PyObject* dropout_add_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Rows f;
    Drop d;
    const void* x;
    const float *bias, *gamma, *beta;
    int64_t norm;
    double eps;
    bool stats;
    if (n != 10 || lib.fwd == nullptr || !f.take_rows(a[0]) || !f.beside(a[1], &x) || !d.take(a[2], a[3], f) ||
        !f.vector(a[4], f.H, &bias) || !number(a[5], &norm) || !f.vector(a[6], f.H, &gamma) || !f.vector(a[7], f.H, &beta) ||
        !number(a[8], &eps) || !truth(a[9], &stats))
      return none();
    stats = stats && norm != ADDLN_NORM_NONE;
    at::Tensor y, mean, rstd;
    const at::Tensor h = f.same(f.t->scalar_type());
    if (norm != ADDLN_NORM_NONE) y = f.same(f.t->scalar_type());
    if (stats) rstd = f.floats({f.rows});
    if (stats && norm == ADDLN_NORM_LAYER) mean = f.floats({f.rows});
    if (lib.fwd(f.t->const_data_ptr(), x, bias, d.p, d.rng, d.seed, d.offset, static_cast<int>(norm), gamma, beta, ptr(h),
                ptr(y), fptr(mean), fptr(rstd), f.rows, f.H, static_cast<float>(eps), f.code, f.stream))
      return none();
    return tuple(h, y, mean, rstd);
  });
}

// dropout_add_norm_backward(dy, dh, h, mean, rstd, p, rng, bias, norm, gamma,
// beta): df, dx, dbias, dgamma, dbeta (dx None without a norm)
PyObject* dropout_add_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Rows g;
    Drop d;
    const void *dy, *dh, *h;
    const float *mean, *rstd, *bias, *gamma, *beta;
    int64_t norm;
    if (n != 11 || lib.bwd == nullptr || !g.take_rows(a[0] == Py_None ? a[1] : a[0]) || !g.beside(a[0], &dy) ||
        !g.beside(a[1], &dh) || !g.beside(a[2], &h) || !g.vector(a[3], g.rows, &mean) || !g.vector(a[4], g.rows, &rstd) ||
        !d.take(a[5], a[6], g) || !g.vector(a[7], g.H, &bias) || !number(a[8], &norm) || !g.vector(a[9], g.H, &gamma) ||
        !g.vector(a[10], g.H, &beta) || !one_dimension(a[7]) || !one_dimension(a[9]) || !one_dimension(a[10]))
      return none();
    const at::Tensor df = g.same(g.t->scalar_type());
    at::Tensor dx, dbias, dgamma, dbeta, ws;
    if (norm != ADDLN_NORM_NONE) dx = g.same(g.t->scalar_type());
    if (bias) dbias = g.floats({g.H});
    if (gamma) dgamma = g.floats({g.H});
    if (beta) dbeta = g.floats({g.H});
    int64_t size = 0;
    if (bias || gamma || beta) {
      const std::array<int64_t, 4> key{g.rows, g.H, g.code, g.t->get_device()};
      const auto it = sizes.find(key);
      size = it != sizes.end() ? it->second : lib.bwd_size(g.rows, g.H, g.code);
      if (size < 0) return none();
      if (it == sizes.end()) {
        if (sizes.size() >= 256) sizes.clear();
        sizes[key] = size;
      }
      ws = at::detail::empty_cuda({size}, at::kByte, g.t->device(), std::nullopt);
    }
    if (lib.bwd(dy, dh, h, d.p, d.rng, d.seed, d.offset, static_cast<int>(norm), gamma, mean, rstd, ptr(df), ptr(dx),
                fptr(dbias), fptr(dgamma), fptr(dbeta), g.rows, g.H, g.code, ptr(ws), size, g.stream))
      return none();
    return tuple(df, dx, dbias, dgamma, dbeta);
  });
}

at::ScalarType q_type(int64_t format) {
  return format == ADDLN_Q_E4M3 ? at::kFloat8_e4m3fn : format == ADDLN_Q_E5M2 ? at::kFloat8_e5m2 : at::kChar;
}

// norm_quant(x, residual, gamma, beta, eps, norm, format, scaling, group,
// want_stats), the groups' scales row by row: q, scale, h, mean, rstd
PyObject* norm_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Rows x;
    const void* r;
    const float *gamma, *beta;
    double eps;
    int64_t norm, format, scaling, group;
    bool stats;
    if (n != 10 || lib.quant == nullptr || !x.take_rows(a[0]) || !x.beside(a[1], &r) || !x.vector(a[2], x.H, &gamma) ||
        !x.vector(a[3], x.H, &beta) || !number(a[4], &eps) || !number(a[5], &norm) || !number(a[6], &format) ||
        !number(a[7], &scaling) || !number(a[8], &group) || !truth(a[9], &stats) || scaling == ADDLN_SCALE_TENSOR)
      return none();
    stats = stats && norm != ADDLN_NORM_NONE;
    at::Tensor h, mean, rstd;
    const at::Tensor q = x.same(q_type(format));
    at::DimVector shape(x.t->sizes().begin(), x.t->sizes().end());
    shape.back() = group ? (x.H + group - 1) / group : 1;
    const at::Tensor scale = at::detail::empty_cuda(
        shape, scaling == ADDLN_SCALE_POW2 ? at::kFloat8_e8m0fnu : at::kFloat, x.t->device(), std::nullopt);
    if (r) h = x.same(x.t->scalar_type());
    if (stats) rstd = x.floats({x.rows});
    if (stats && norm == ADDLN_NORM_LAYER) mean = x.floats({x.rows});
    if (lib.quant(x.t->const_data_ptr(), r, static_cast<int>(norm), gamma, beta, ptr(q), static_cast<int>(format),
                  static_cast<int>(scaling), group, 0, ptr(scale), ptr(h), fptr(mean), fptr(rstd), x.rows, x.H,
                  static_cast<float>(eps), x.code, x.stream))
      return none();
    return tuple(q, scale, h, mean, rstd);
  });
}

// dequantise(q, scale, code): scales row by row, of q's rows or groups
PyObject* dequantise(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Rows q;
    int64_t code;
    if (n != 3 || lib.dequant == nullptr || !q.take(a[0]) || q.t->dim() < 1 || q.t->size(-1) < 1 || !number(a[2], &code) ||
        code < ADDLN_FP32 || code > ADDLN_BF16)
      return none();
    const auto type = q.t->scalar_type();
    const int format = type == at::kFloat8_e4m3fn ? ADDLN_Q_E4M3 : type == at::kFloat8_e5m2 ? ADDLN_Q_E5M2
                       : type == at::kChar ? ADDLN_Q_INT8 : -1;
    const at::Tensor* s = tensor(a[1]);
    if (format < 0 || s == nullptr || s->dim() != q.t->dim() || s->dim() < 2) return none();
    const bool pow2 = s->scalar_type() == at::kFloat8_e8m0fnu;
    if (!q.fits(s, pow2 ? at::kFloat8_e8m0fnu : at::kFloat)) return none();
    for (int64_t i = 0; i + 1 < s->dim(); ++i)
      if (s->size(i) != q.t->size(i)) return none();
    const int64_t H = q.t->size(-1), G = s->size(-1);
    int64_t group = 0;
    if (G != 1 || pow2) {
      // no two of these cut a row into the same number, but for one
      for (group = 128; group >= 32 && G != (H + group - 1) / group;) group /= 2;
      if (group < 32) return none();
    }
    const at::Tensor out = q.same(code == ADDLN_FP32 ? at::kFloat : code == ADDLN_FP16 ? at::kHalf : at::kBFloat16);
    if (lib.dequant(q.t->const_data_ptr(), format, pow2 ? ADDLN_SCALE_POW2 : group ? ADDLN_SCALE_GROUP : ADDLN_SCALE_ROW, group,
                    0, s->const_data_ptr(), ptr(out), q.t->numel() / H, H, static_cast<int>(code), q.stream))
      return none();
    return wrap(out);
  });
}

// init(addresses of the six entry points, in the order of Entries)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  uintptr_t at[6];
  if (n != 6) return PyErr_Format(PyExc_TypeError, "init takes six addresses");
  for (int i = 0; i < 6; ++i) {
    at[i] = static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(a[i]));
    if (PyErr_Occurred()) return nullptr;
  }
  lib.drop = reinterpret_cast<decltype(lib.drop)>(at[0]);
  lib.fwd = reinterpret_cast<decltype(lib.fwd)>(at[1]);
  lib.bwd = reinterpret_cast<decltype(lib.bwd)>(at[2]);
  lib.bwd_size = reinterpret_cast<decltype(lib.bwd_size)>(at[3]);
  lib.quant = reinterpret_cast<decltype(lib.quant)>(at[4]);
  lib.dequant = reinterpret_cast<decltype(lib.dequant)>(at[5]);
  sizes.clear();
  return none();
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(init), METHOD(dropout), METHOD(dropout_add_norm), METHOD(dropout_add_norm_backward),
                         METHOD(norm_quant), METHOD(dequantise), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "addln_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit_addln_fast() { return PyModule_Create(&module); }
