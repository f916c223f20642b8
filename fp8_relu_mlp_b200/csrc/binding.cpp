// Argument marshalling of the calls that a training or serving loop makes per
// layer and token: tensors are unpacked and checked here instead of by five
// Python calls each, which takes longer than the kernels of a single token.
// The functions themselves are the library's, handed over by address.  The
// module is optional: without it the Python binding makes the same checks.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/headeronly/version.h>

#include <climits>
#include <cstdint>

namespace {

enum Fn {
  kQuantize,
  kWeight,
  kLinearFwd,
  kLinear,
  kUp,
  kMlp,
  kNormFwd,
  kNormBwd,
  kNormBwdWorkspace,
  kGradNorm,
  kGradNormWorkspace,
  kAdamW,
  kCount
};
const char* const kNames[kCount] = {
    "fp8mlp_quantize_block",  "fp8mlp_weight_block_cache_refresh",      "fp8mlp_linear_fwd_block",
    "fp8mlp_linear_block",    "fp8mlp_up_proj_block",                   "fp8mlp_mlp_fwd_block",
    "fp8mlp_norm_gate_fwd",   "fp8mlp_norm_gate_bwd",                   "fp8mlp_norm_gate_bwd_workspace_size",
    "fp8mlp_grad_norm",       "fp8mlp_grad_norm_workspace_size",        "fp8mlp_adamw_step"};
void* g_fn[kCount];
unsigned g_bound = 0;  // one bit per function that is set

// Without the interpreter's lock: a launch waits where the stream's queue is full.
template <class... A>
int invoke(Fn f, A... a) {
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = reinterpret_cast<int (*)(A...)>(g_fn[f])(a...);
  Py_END_ALLOW_THREADS;
  return rc;
}

size_t blocks(long long n) { return n > 0 ? static_cast<size_t>((n + 127) / 128) : 0; }

// One call's arguments, taken in order.  After a failure (a Python exception
// is set) every further one is a no-op.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, i = 0;
  int dev = -2;  // no tensor is on it
  bool ok = true;

  Args(PyObject* const* args, Py_ssize_t nargs, Py_ssize_t want) : a(args), n(nargs) {
    if (nargs != want) {
      PyErr_Format(PyExc_TypeError, "%zd arguments are needed, %zd were given", want, nargs);
      ok = false;
    } else if (g_bound != (1u << kCount) - 1) {
      PyErr_SetString(PyExc_RuntimeError, "the library's functions are not bound");
      ok = false;
    } else if (has_gpu()) {
      dev = static_cast<int>(c10::cuda::current_device());
    }
  }
  static bool has_gpu() {
    static const bool seen = c10::cuda::device_count() > 0;
    return seen;
  }
  int integer() {
    if (!ok) return 0;
    const long v = PyLong_AsLong(a[i++]);
    if (v == -1 && PyErr_Occurred()) {
      ok = false;
    } else if (v < INT_MIN || v > INT_MAX) {
      PyErr_Format(PyExc_OverflowError, "argument %zd does not fit an int", i);
      ok = false;
    }
    return static_cast<int>(v);
  }
  // an integer further on: a gate's size needs the argument behind it
  int peek_integer(Py_ssize_t at) {
    const Py_ssize_t here = i;
    i = at;
    const int v = integer();
    i = here;
    return v;
  }
  float real() {
    if (!ok) return 0.f;
    const double v = PyFloat_AsDouble(a[i++]);
    if (v == -1.0 && PyErr_Occurred()) ok = false;
    return static_cast<float>(v);
  }
  void* address(PyObject* o, const char* name) {
    void* p = PyLong_AsVoidPtr(o);
    if (p == nullptr && PyErr_Occurred()) {
      ok = false;
      if (PyErr_ExceptionMatches(PyExc_OverflowError)) PyErr_Format(PyExc_OverflowError, "%s: an address has 64 bits", name);
    }
    return p;
  }
  // device address of a tensor with at least `need` bytes (None: NULL; an int
  // is an address the caller vouches for)
  template <class T = void>
  T* buf(size_t need, const char* name) {
    if (!ok) return nullptr;
    PyObject* o = a[i++];
    if (o == Py_None) return nullptr;
    void* p = nullptr;
    if (THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (!t.is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s: tensor arguments must be contiguous", name);
      } else if (!t.is_cuda()) {
        PyErr_Format(PyExc_ValueError, "%s: a CUDA tensor is needed", name);
      } else if (t.nbytes() < need) {
        PyErr_Format(PyExc_ValueError, "%s: %zu bytes are needed, the tensor has %zu", name, need, t.nbytes());
      } else if (t.get_device() != dev) {
        PyErr_Format(PyExc_ValueError, "%s is on device %d, the current device is %d", name,
                     static_cast<int>(t.get_device()), dev);
      } else {
        return static_cast<T*>(t.data_ptr());
      }
      ok = false;
    } else if (PyLong_CheckExact(o)) {
      p = address(o, name);
    } else {
      PyErr_Format(PyExc_TypeError, "%s: cannot pass %R as a pointer", name, reinterpret_cast<PyObject*>(Py_TYPE(o)));
      ok = false;
    }
    return static_cast<T*>(p);
  }
  // None: torch's current stream; an int is a handle; else an object with one
  void* stream() {
    if (!ok) return nullptr;
    PyObject* o = a[i++];
    if (o == Py_None) return dev >= 0 ? c10::cuda::getCurrentCUDAStream().stream() : nullptr;
    if (PyLong_CheckExact(o)) return address(o, "stream");
    PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
    if (h == nullptr) {
      ok = false;
      return nullptr;
    }
    void* s = address(h, "stream");
    Py_DECREF(h);
    return s;
  }
};

// 0 where the library refuses the sizes (negative ones, and widths whose
// products could wrap)
size_t bytes(long long a, long long b, long long each) {
  return a > 0 && b > 0 ? static_cast<size_t>(a) * static_cast<size_t>(b) * static_cast<size_t>(each) : 0;
}
long long gate_rows(int M, int rows) { return rows > 0 && M > 0 ? (static_cast<long long>(M) + rows - 1) / rows : 0; }

PyObject* finish(const Args& x, int rc) { return x.ok ? PyLong_FromLong(rc) : nullptr; }

// C++ exceptions of torch's accessors end here
template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

#define BINDING(name) PyObject* name(PyObject*, PyObject* const* args, Py_ssize_t nargs)

BINDING(quantize_block) {
  return guarded([&]() -> PyObject* {
    Args x(args, nargs, 6);
    const int M = x.integer(), K = x.integer();
    void *in = x.buf(bytes(M, K, 2), "x"), *xq = x.buf(bytes(M, K, 1), "xq"), *xs = x.buf(bytes(M, blocks(K), 4), "xs");
    void* s = x.stream();
    return finish(x, x.ok ? invoke(kQuantize, M, K, in, xq, xs, s) : 0);
  });
}

BINDING(weight_block_cache_refresh) {
  return guarded([&]() -> PyObject* {
    Args x(args, nargs, 8);
    const int N = x.integer(), K = x.integer();
    const size_t sc = bytes(blocks(K), blocks(N), 4);
    void *W = x.buf(bytes(N, K, 2), "W"), *Wq = x.buf(bytes(N, K, 1), "Wq"), *ws = x.buf(sc, "ws");
    void *Wqt = x.buf(bytes(N, K, 1), "Wq_t"), *wst = x.buf(sc, "ws_t");
    void* s = x.stream();
    return finish(x, x.ok ? invoke(kWeight, N, K, W, Wq, ws, Wqt, wst, s) : 0);
  });
}

BINDING(linear_fwd_block) {
  return guarded([&]() -> PyObject* {
    Args x(args, nargs, 9);
    const int M = x.integer(), K = x.integer(), N = x.integer();
    void *xq = x.buf(bytes(M, K, 1), "xq"), *xs = x.buf(bytes(M, blocks(K), 4), "xs"), *Wq = x.buf(bytes(N, K, 1), "Wq");
    void *ws = x.buf(bytes(blocks(K), blocks(N), 4), "ws"), *y = x.buf(bytes(M, N, 2), "y");
    void* s = x.stream();
    return finish(x, x.ok ? invoke(kLinearFwd, M, K, N, xq, xs, Wq, ws, y, s) : 0);
  });
}

BINDING(linear_block) {
  return guarded([&]() -> PyObject* {
    Args x(args, nargs, 10);
    const int M = x.integer(), K = x.integer(), N = x.integer();
    void *in = x.buf(bytes(M, K, 2), "x"), *Wq = x.buf(bytes(N, K, 1), "Wq");
    void *ws = x.buf(bytes(blocks(K), blocks(N), 4), "ws"), *xq = x.buf(bytes(M, K, 1), "xq");
    void *xs = x.buf(bytes(M, blocks(K), 4), "xs"), *y = x.buf(bytes(M, N, 2), "y");
    void* s = x.stream();
    return finish(x, x.ok ? invoke(kLinear, M, K, N, in, Wq, ws, xq, xs, y, s) : 0);
  });
}

BINDING(up_proj_block) {
  return guarded([&]() -> PyObject* {
    Args x(args, nargs, 11);
    const int M = x.integer(), d = x.integer(), h = x.integer();
    void *xq = x.buf(bytes(M, d, 1), "xq"), *xs = x.buf(bytes(M, blocks(d), 4), "xs"), *W = x.buf(bytes(h, d, 1), "W1q");
    void *ws = x.buf(bytes(blocks(d), blocks(h), 4), "w1s"), *post = x.buf(bytes(M, h, 2), "post");
    void *pq = x.buf(bytes(M, h, 1), "post_q"), *ps = x.buf(bytes(M, blocks(h), 4), "post_s");
    void* s = x.stream();
    return finish(x, x.ok ? invoke(kUp, M, d, h, xq, xs, W, ws, post, pq, ps, s) : 0);
  });
}

BINDING(mlp_fwd_block) {
  return guarded([&]() -> PyObject* {
    Args x(args, nargs, 15);
    const int M = x.integer(), d = x.integer(), h = x.integer();
    const size_t w = bytes(h, d, 1), sc = bytes(blocks(d), blocks(h), 4);
    void *in = x.buf(bytes(M, d, 2), "x"), *W1 = x.buf(w, "W1q"), *s1 = x.buf(sc, "w1s"), *W2 = x.buf(w, "W2q_t");
    void *s2 = x.buf(sc, "w2s_t"), *xq = x.buf(bytes(M, d, 1), "xq"), *xs = x.buf(bytes(M, blocks(d), 4), "xs");
    void *post = x.buf(bytes(M, h, 2), "post"), *pq = x.buf(bytes(M, h, 1), "post_q");
    void *ps = x.buf(bytes(M, blocks(h), 4), "post_s"), *out = x.buf(bytes(M, d, 2), "out");
    void* s = x.stream();
    return finish(x, x.ok ? invoke(kMlp, M, d, h, in, W1, s1, W2, s2, xq, xs, post, pq, ps, out, s) : 0);
  });
}

BINDING(norm_gate_fwd) {
  return guarded([&]() -> PyObject* {
    Args x(args, nargs, 17);
    const int M = x.integer(), d = x.integer();
    const size_t n = bytes(M, d, 2), g = bytes(1, d, 2), m = bytes(M, 1, 4);
    const int rows = x.peek_integer(6);
    void *r = x.buf(n, "r"), *y = x.buf(n, "y"), *wpost = x.buf(g, "w_post"), *gate = x.buf(bytes(gate_rows(M, rows), d, 2), "gate");
    const int rpg = x.integer();
    void *alpha = x.buf(4, "alpha"), *wpre = x.buf(g, "w_pre");
    const float eps = x.real();
    void *rn = x.buf(n, "r_next"), *sp = x.buf(m, "rstd_post"), *xx = x.buf(n, "x"), *sr = x.buf(m, "rstd_pre");
    void *xq = x.buf(bytes(M, d, 1), "xq"), *xs = x.buf(bytes(M, blocks(d), 4), "xs");
    void* s = x.stream();
    return finish(x, x.ok ? invoke(kNormFwd, M, d, r, y, wpost, gate, rpg, alpha, wpre, eps, rn, sp, xx, sr, xq, xs, s) : 0);
  });
}

BINDING(norm_gate_bwd) {
  return guarded([&]() -> PyObject* {
    Args x(args, nargs, 22);
    const int M = x.integer(), d = x.integer();
    const size_t n = bytes(M, d, 2), g = bytes(1, d, 2), f = bytes(1, d, 4), m = bytes(M, 1, 4);
    const int rows = x.peek_integer(6);
    void *r = x.buf(n, "r"), *y = x.buf(n, "y"), *wpost = x.buf(g, "w_post"), *gate = x.buf(bytes(gate_rows(M, rows), d, 2), "gate");
    const int rpg = x.integer();
    void *alpha = x.buf(4, "alpha"), *sp = x.buf(m, "rstd_post"), *rn = x.buf(n, "r_next"), *wpre = x.buf(g, "w_pre");
    void *sr = x.buf(m, "rstd_pre"), *dx = x.buf(n, "dx"), *drn = x.buf(n, "dr_next"), *dr = x.buf(n, "dr"), *dy = x.buf(n, "dy");
    void *dwpost = x.buf(f, "dw_post"), *dgate = x.buf(bytes(gate_rows(M, rows), d, 4), "dgate"), *da = x.buf(4, "dalpha");
    void* dwpre = x.buf(f, "dw_pre");
    const size_t need = x.ok ? reinterpret_cast<size_t (*)(int, int, int)>(g_fn[kNormBwdWorkspace])(M, d, rpg) : 0;
    void* ws = x.buf(need, "workspace");
    void* s = x.stream();
    return finish(x, x.ok ? invoke(kNormBwd, M, d, r, y, wpost, gate, rpg, alpha, sp, rn, wpre, sr, dx, drn, dr, dy, dwpost,
                                   dgate, da, dwpre, ws, s)
                          : 0);
  });
}

BINDING(grad_norm) {
  return guarded([&]() -> PyObject* {
    Args x(args, nargs, 6);
    const int n = x.integer();
    void* t = x.buf(0, "tensors");
    const float max_norm = x.real();
    const size_t need = x.ok ? reinterpret_cast<size_t (*)(int, void*)>(g_fn[kGradNormWorkspace])(n, t) : 0;
    void *out = x.buf(8, "norm_coef"), *ws = x.buf(need, "workspace"), *s = x.stream();
    return finish(x, x.ok ? invoke(kGradNorm, n, t, max_norm, out, ws, s) : 0);
  });
}

BINDING(adamw_step) {
  return guarded([&]() -> PyObject* {
    Args x(args, nargs, 9);
    const int n = x.integer();
    void *t = x.buf(0, "tensors"), *st = x.buf(32, "st");
    const int bits = x.integer();
    const float b1 = x.real(), b2 = x.real(), eps = x.real();
    void *coef = x.buf(4, "grad_coef"), *s = x.stream();
    return finish(x, x.ok ? invoke(kAdamW, n, t, st, bits, b1, b2, eps, coef, s) : 0);
  });
}

// bind(name, address): one of the library's functions; all of names() have to
// be bound before the first call
BINDING(bind) {
  if (nargs != 2) {
    PyErr_SetString(PyExc_TypeError, "bind(name, address)");
    return nullptr;
  }
  const char* name = PyUnicode_AsUTF8(args[0]);
  if (name == nullptr) return nullptr;
  for (int k = 0; k < kCount; ++k) {
    if (PyUnicode_CompareWithASCIIString(args[0], kNames[k]) == 0) {
      void* f = PyLong_AsVoidPtr(args[1]);
      if (PyErr_Occurred()) return nullptr;
      if (f == nullptr) break;
      g_fn[k] = f;
      g_bound |= 1u << k;
      Py_RETURN_NONE;
    }
  }
  PyErr_Format(PyExc_KeyError, "%s", name);
  return nullptr;
}

PyObject* names(PyObject*, PyObject*) {
  PyObject* l = PyList_New(kCount);
  for (int k = 0; l != nullptr && k < kCount; ++k) PyList_SET_ITEM(l, k, PyUnicode_FromString(kNames[k]));
  return l;
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {METHOD(quantize_block), METHOD(weight_block_cache_refresh),
                          METHOD(linear_fwd_block), METHOD(linear_block),
                          METHOD(up_proj_block), METHOD(mlp_fwd_block),
                          METHOD(norm_gate_fwd), METHOD(norm_gate_bwd),
                          METHOD(grad_norm), METHOD(adamw_step),
                          METHOD(bind), {"names", names, METH_NOARGS, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", "Argument marshalling of the per-layer calls.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&kModule);
  if (m != nullptr && PyModule_AddStringConstant(m, "TORCH_VERSION", TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
