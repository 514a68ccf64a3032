// layers_binding.cpp -- the compiled half of the Python binding of the layers'
// entry points (include/ag.h): checks tensors, allocates outputs and
// workspaces, and calls libag.
//
// At a few rows such a call is mostly the caller's time: checking a handful of
// tensors, allocating and filling a foreign-function call from Python took 7 to
// 70 us where the library's own call takes 4 to 14 (one row through a 1024 x 1536
// layer: 11.3 us from Python, 126 gradients to clip: 84 us).
//
// The module links nothing of libag: __init__.py hands it the addresses of the
// library's functions, so that both halves use the one loaded library.  Every
// function here takes its arguments by position, in the order of its caller in
// __init__.py, which has the defaults and the documentation.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <string>
#include <vector>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/ag.h"

namespace {

// libag's functions and the binding's exception, from bind().
struct Library {
  decltype(&ag_linear_fwd) linear_fwd;
  decltype(&ag_linear_fwd_workspace) linear_fwd_workspace;
  decltype(&ag_linear_bwd) linear_bwd;
  decltype(&ag_linear_bwd_workspace) linear_bwd_workspace;
  decltype(&ag_qk_norm_rope_fwd) qk_fwd;
  decltype(&ag_qk_norm_rope_bwd) qk_bwd;
  decltype(&ag_qk_norm_rope_bwd_workspace) qk_bwd_workspace;
  decltype(&ag_grad_clip) clip;
  decltype(&ag_grad_clip_workspace) clip_workspace;
  PyObject *error;
} lib;

// An argument that the binding refuses.
struct Refusal {
  PyObject *type;
  std::string text;
};
[[noreturn]] void refuse(PyObject *type, const std::string &text) { throw Refusal{type, text}; }

// A status of libag other than AG_OK: raises AgError(function, status).
[[noreturn]] void raise_status(const char *fn, int status) {
  PyObject *e = PyObject_CallFunction(lib.error, "si", fn, status);
  if (e) {
    PyErr_SetObject(lib.error, e);
    Py_DECREF(e);
  }
  throw python_error();
}
void check_status(const char *fn, int status) {
  if (status != AG_OK) raise_status(fn, status);
}

// Every entry point: C++ exceptions become Python's.
template <typename F>
PyObject *guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refusal &r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// The library's calls enqueue work: other threads may run meanwhile.
template <typename F>
int unlocked(F f) {
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st;
}

// --------------------------------------------------------------------------
// Arguments
using at::ScalarType;
using at::Tensor;

std::string sizes_text(at::IntArrayRef s) {
  std::string t = "[";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? "," : "") + std::to_string(s[i]);
  return t + "]";
}

int code_of(ScalarType t) {
  return t == at::kFloat ? AG_F32 : t == at::kBFloat16 ? AG_BF16 : t == at::kHalf ? AG_F16 : -1;
}
bool is_half(ScalarType t) { return t == at::kBFloat16 || t == at::kHalf; }

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
  const Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be on a CUDA device");
  if (t.layout() != at::kStrided) refuse(PyExc_TypeError, std::string(name) + " must be a strided tensor");
  // (A view that only notes a change of sign: its memory holds the other values.)
  if (t.is_neg() || t.is_conj())
    refuse(PyExc_ValueError, std::string(name) + " is a lazily negated view: resolve it first");
  return t;
}
const Tensor &tensor_of(PyObject *o, const char *name, ScalarType type, at::Device dev) {
  const Tensor &t = tensor(o, name);
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", got " +
                                c10::toString(t.scalar_type()));
  if (t.device() != dev)
    refuse(PyExc_ValueError, std::string("all tensors of a call must be on ") + dev.str() + "; " +
                                 name + " is on " + t.device().str());
  return t;
}

ScalarType dtype_of(PyObject *o, const char *name) {
  if (!THPDtype_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a torch.dtype");
  return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

// A row-major matrix (its rows may be apart): pointer and row stride.
struct Matrix {
  void *p = nullptr;
  int64_t ld = 0;
};
Matrix matrix(const Tensor &t, const char *name, int64_t rows, int64_t cols) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    refuse(PyExc_ValueError, std::string(name) + " must be [" + std::to_string(rows) + "," +
                                 std::to_string(cols) + "], got " + sizes_text(t.sizes()));
  if (t.stride(1) != 1 && cols > 1)
    refuse(PyExc_ValueError, std::string("the rows of ") + name + " must be dense");
  const int64_t ld = t.stride(0);
  return {t.data_ptr(), rows > 1 || ld > cols ? ld : cols};
}
Matrix matrix(PyObject *o, const char *name, ScalarType type, int64_t rows, int64_t cols,
              at::Device dev) {
  return matrix(tensor_of(o, name, type, dev), name, rows, cols);
}

// An optional dense float32 vector.
float *vector(PyObject *o, const char *name, int64_t n, at::Device dev) {
  if (o == Py_None) return nullptr;
  const Tensor &t = tensor_of(o, name, at::kFloat, dev);
  if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    refuse(PyExc_ValueError, std::string(name) + " must be a contiguous [" + std::to_string(n) + "]");
  return t.data_ptr<float>();
}

void *dense(PyObject *o, const char *name, ScalarType type, at::IntArrayRef shape, at::Device dev) {
  const Tensor &t = tensor_of(o, name, type, dev);
  if (t.sizes() != shape || !t.is_contiguous())
    refuse(PyExc_ValueError, std::string(name) + " must be a contiguous " + sizes_text(shape) +
                                 ", got " + sizes_text(t.sizes()));
  return t.data_ptr();
}

int integer(PyObject *o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return static_cast<int>(v);
}
float number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(v);
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

Tensor make(at::IntArrayRef shape, ScalarType type, at::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}
void *stream_of(at::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(PyExc_TypeError, "wrong number of arguments");
}

// --------------------------------------------------------------------------
// linear_fwd(x, W, bias, act, residual, preact, out, out_dtype)
PyObject *linear_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 8);
    const Tensor &x = tensor(a[0], "x");
    const ScalarType T = x.scalar_type();
    if (!is_half(T))
      refuse(PyExc_TypeError, std::string("x must be bfloat16 or float16, got ") + c10::toString(T));
    const at::Device dev = x.device();
    const Tensor &W = tensor_of(a[1], "W", T, dev);
    if (x.dim() != 2 || W.dim() != 2) refuse(PyExc_ValueError, "x must be [M,K] and W [N,K]");
    const c10::cuda::CUDAGuard guard(dev);
    const int64_t M = x.size(0), K = x.size(1), N = W.size(0);
    const Matrix mx = matrix(x, "x", M, K), mw = matrix(W, "W", N, K);
    const int act = integer(a[3]);
    const ScalarType O = a[7] != Py_None ? dtype_of(a[7], "out_dtype")
                         : a[6] != Py_None ? tensor(a[6], "out").scalar_type()
                                           : T;
    if (O != T && O != at::kFloat)
      refuse(PyExc_TypeError, std::string("out_dtype must be the type of x or float32, got ") +
                                  c10::toString(O));
    const float *bias = vector(a[2], "bias", N, dev);
    Matrix mr, mz;
    if (a[4] != Py_None) mr = matrix(a[4], "residual", O, M, N, dev);
    Tensor y = a[6] == Py_None ? make({M, N}, O, dev) : tensor_of(a[6], "out", O, dev);
    const Matrix my = matrix(y, "out", M, N);
    Tensor z;
    if (a[5] != Py_None && a[5] != Py_False) {
      z = a[5] == Py_True ? make({M, N}, T, dev) : tensor_of(a[5], "preact", T, dev);
      mz = matrix(z, "preact", M, N);
    }
    void *const stream = stream_of(dev);
    const auto call = [&](void *ws, int64_t bytes) {
      return unlocked([&] {
        return lib.linear_fwd(mx.p, mx.ld, mw.p, mw.ld, bias, mr.p, mr.ld, M, N, K, code_of(T), act,
                              mz.p, mz.ld, my.p, my.ld, code_of(O), ws, bytes, stream);
      });
    };
    // Most calls need no workspace; the others say so before they do anything.
    int st = call(nullptr, 0);
    if (st == AG_ERR_SCRATCH) {
      int64_t bytes = 0;
      check_status("ag_linear_fwd_workspace",
                   lib.linear_fwd_workspace(mx.p, mx.ld, mw.p, mw.ld, M, N, K, &bytes));
      const Tensor ws = make({bytes}, at::kByte, dev);
      st = call(ws.data_ptr(), bytes);
    }
    check_status("ag_linear_fwd", st);
    if (!z.defined()) return THPVariable_Wrap(y);
    return Py_BuildValue("(NN)", THPVariable_Wrap(y), THPVariable_Wrap(z));
  });
}

// linear_bwd(dy, x, W, act, preact, need_dx, need_dW, need_db, dx_dtype, dW_dtype, dx, dW)
PyObject *linear_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 12);
    const Tensor &dy = tensor(a[0], "dy");
    const ScalarType T = dy.scalar_type();
    if (!is_half(T))
      refuse(PyExc_TypeError, std::string("dy must be bfloat16 or float16, got ") + c10::toString(T));
    const at::Device dev = dy.device();
    const Tensor &x = tensor_of(a[1], "x", T, dev);
    if (dy.dim() != 2 || x.dim() != 2) refuse(PyExc_ValueError, "dy must be [M,N] and x [M,K]");
    const c10::cuda::CUDAGuard guard(dev);
    const int64_t M = dy.size(0), N = dy.size(1), K = x.size(1);
    const Matrix mdy = matrix(dy, "dy", M, N), mx = matrix(x, "x", M, K),
                 mw = matrix(a[2], "W", T, N, K, dev);
    const int act = integer(a[3]);
    Matrix mz;
    if (a[4] != Py_None) mz = matrix(a[4], "preact", T, M, K, dev);
    else if (act != AG_ACT_NONE) refuse(PyExc_ValueError, "an act needs the preact of x");
    const auto type = [&](PyObject *wanted, PyObject *given, ScalarType usual, const char *name) {
      const ScalarType t = given != Py_None    ? tensor(given, name).scalar_type()
                           : wanted != Py_None ? dtype_of(wanted, name)
                                               : usual;
      if ((t != T && t != at::kFloat) || (given != Py_None && wanted != Py_None &&
                                          dtype_of(wanted, name) != t))
        refuse(PyExc_TypeError, std::string(name) + " must be of the type of x or float32, got " +
                                    c10::toString(t));
      return t;
    };
    Tensor dx, dW, db;
    Matrix mdx, mdw;
    ScalarType xt = T, wt = T;
    if (truth(a[5])) {
      xt = type(a[8], a[10], T, "dx");
      dx = a[10] == Py_None ? make({M, K}, xt, dev) : tensor_of(a[10], "dx", xt, dev);
      mdx = matrix(dx, "dx", M, K);
    }
    if (truth(a[6])) {
      wt = type(a[11] == Py_None ? a[9] : Py_None, a[11], at::kFloat, "dW");
      dW = a[11] == Py_None ? make({N, K}, wt, dev) : tensor_of(a[11], "dW", wt, dev);
      mdw = matrix(dW, "dW", N, K);
    }
    float *dbp = nullptr;
    if (truth(a[7])) {
      db = make({N}, at::kFloat, dev);
      dbp = db.data_ptr<float>();
    }
    int64_t bytes = 0;
    check_status("ag_linear_bwd_workspace",
                 lib.linear_bwd_workspace(mdy.p, mdy.ld, mx.p, mx.ld, mw.p, mw.ld, M, N, K, mdx.p,
                                          mdw.p, dbp, &bytes));
    const Tensor ws = bytes ? make({bytes}, at::kByte, dev) : Tensor();
    void *const stream = stream_of(dev);
    check_status("ag_linear_bwd", unlocked([&] {
      return lib.linear_bwd(mdy.p, mdy.ld, mx.p, mx.ld, mw.p, mw.ld, mz.p, mz.ld, act, M, N, K,
                            code_of(T), mdx.p, mdx.ld, code_of(xt), mdw.p, mdw.ld, code_of(wt), dbp,
                            bytes ? ws.data_ptr() : nullptr, bytes, stream);
    }));
    // (An undefined tensor becomes None.)
    return Py_BuildValue("(NNN)", THPVariable_Wrap(dx), THPVariable_Wrap(dW), THPVariable_Wrap(db));
  });
}

// --------------------------------------------------------------------------
// Queries and keys
struct Heads {
  void *p = nullptr;
  int64_t H = 0, sb = 0, sl = 0, sh = 0;
  bool flat = false;  // [B, L, D]
};
// A [B,L,H,D] (or [B,L,D]: one head) tensor with dense heads.
Heads heads(const Tensor &t, const char *name, int64_t B, int64_t L, int64_t D) {
  const int64_t d = t.dim();
  if ((d != 3 && d != 4) || t.size(0) != B || t.size(1) != L || t.size(d - 1) != D)
    refuse(PyExc_ValueError, std::string(name) + " must be [B,L,H,D] or [B,L,D] with the sizes of " +
                                 "the others, got " + sizes_text(t.sizes()));
  if (t.stride(d - 1) != 1 && D > 1)
    refuse(PyExc_ValueError, std::string("the heads of ") + name + " must be dense");
  return {t.data_ptr(), d == 4 ? t.size(2) : 1, t.stride(0), t.stride(1), d == 4 ? t.stride(2) : 0,
          d == 3};
}

// The arguments that both directions take: q, k, q_weight, k_weight, q_bias,
// k_bias, norm, eps, inv_freq, rope, positions.
struct QkCall {
  ScalarType T;
  at::Device dev = at::Device(at::kCPU);
  int64_t B, L, D, R = 0, pos_sb = 0;
  Heads side[2];
  float *w[2], *b[2];
  int norm, rope;
  float eps;
  double *freq = nullptr;
  int64_t *positions = nullptr;

  explicit QkCall(PyObject *const *a) {
    static const char *const names[2] = {"q", "k"};
    const int of = a[0] != Py_None ? 0 : 1;
    if (a[of] == Py_None) refuse(PyExc_ValueError, "q and k are both None");
    const Tensor &first = tensor(a[of], names[of]);
    T = first.scalar_type();
    if (code_of(T) < 0)
      refuse(PyExc_TypeError, std::string(names[of]) + " must be float32, bfloat16 or float16, got " +
                                  c10::toString(T));
    if (first.dim() != 3 && first.dim() != 4)
      refuse(PyExc_ValueError, std::string(names[of]) + " must be [B,L,H,D] or [B,L,D]");
    dev = first.device();
    B = first.size(0), L = first.size(1), D = first.size(first.dim() - 1);
    for (int i = 0; i < 2; ++i)
      if (a[i] != Py_None) side[i] = heads(tensor_of(a[i], names[i], T, dev), names[i], B, L, D);
    w[0] = vector(a[2], "q_weight", D, dev), w[1] = vector(a[3], "k_weight", D, dev);
    b[0] = vector(a[4], "q_bias", D, dev), b[1] = vector(a[5], "k_bias", D, dev);
    norm = integer(a[6]), eps = number(a[7]), rope = integer(a[9]);
    if (a[8] != Py_None) {
      const Tensor &f = tensor_of(a[8], "inv_freq", at::kDouble, dev);
      if (f.dim() != 1 || !f.is_contiguous())
        refuse(PyExc_ValueError, "inv_freq must be a contiguous [R/2]");
      R = 2 * f.size(0), freq = f.data_ptr<double>();
    }
    if (a[10] != Py_None) {
      const Tensor &p = tensor_of(a[10], "positions", at::kLong, dev);
      const bool two = p.dim() == 2;
      if (!(p.dim() == 1 && p.size(0) == L) && !(two && p.size(0) == B && p.size(1) == L))
        refuse(PyExc_ValueError, "positions must be [L] or [B,L], got " + sizes_text(p.sizes()));
      if (L > 1 && p.stride(p.dim() - 1) != 1)
        refuse(PyExc_ValueError, "the rows of positions must be dense");
      positions = p.data_ptr<int64_t>();
      pos_sb = two && B > 1 ? p.stride(0) : 0;
    }
  }
  // The attention's layout of a side.
  std::vector<int64_t> layout(int i) const {
    if (side[i].flat) return {B, L, D};
    return {B, side[i].H, L, D};
  }
};

// qk_fwd(<the eleven of QkCall>, out_dtype, q_out, k_out)
PyObject *qk_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 14);
    const QkCall c(a);
    const c10::cuda::CUDAGuard guard(c.dev);
    const ScalarType O = dtype_of(a[11], "out_dtype");
    if (code_of(O) < 0)
      refuse(PyExc_TypeError, std::string("out_dtype must be float32, bfloat16 or float16, got ") +
                                  c10::toString(O));
    Tensor out[2];
    void *p[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; ++i) {
      if (a[i] == Py_None) continue;
      const auto shape = c.layout(i);
      if (a[12 + i] == Py_None) {
        out[i] = make(shape, O, c.dev);
        p[i] = out[i].data_ptr();
      } else {
        p[i] = dense(a[12 + i], i ? "k_out" : "q_out", O, shape, c.dev);
        out[i] = THPVariable_Unpack(a[12 + i]);
      }
    }
    void *const stream = stream_of(c.dev);
    const Heads &q = c.side[0], &k = c.side[1];
    check_status("ag_qk_norm_rope_fwd", unlocked([&] {
      return lib.qk_fwd(q.p, q.sb, q.sl, q.sh, k.p, k.sb, k.sl, k.sh, code_of(c.T), c.w[0], c.b[0],
                        c.w[1], c.b[1], c.norm, c.eps, c.freq, c.R, c.rope, c.positions, c.pos_sb,
                        c.B, q.H, k.H, c.L, c.D, p[0], p[1], code_of(O), stream);
    }));
    return Py_BuildValue("(NN)", THPVariable_Wrap(out[0]), THPVariable_Wrap(out[1]));
  });
}

// qk_bwd(<the eleven of QkCall>, dq_out, dk_out, dq, dk)
PyObject *qk_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 15);
    const QkCall c(a);
    const c10::cuda::CUDAGuard guard(c.dev);
    const Tensor &g0 = tensor(a[a[0] != Py_None ? 11 : 12], a[0] != Py_None ? "dq_out" : "dk_out");
    const ScalarType G = g0.scalar_type();
    if (code_of(G) < 0)
      refuse(PyExc_TypeError, std::string("dq_out and dk_out must be float32, bfloat16 or float16, ") +
                                  "got " + c10::toString(G));
    void *g[2] = {nullptr, nullptr};
    Tensor dx[2], params[4];  // of the queries and keys; q_weight, k_weight, q_bias, k_bias
    Heads out[2];
    for (int i = 0; i < 2; ++i) {
      if (a[i] == Py_None) continue;
      g[i] = dense(a[11 + i], i ? "dk_out" : "dq_out", G, c.layout(i), c.dev);
      const Tensor &x = THPVariable_Unpack(a[i]);
      const char *name = i ? "dk" : "dq";
      dx[i] = a[13 + i] == Py_None ? make(x.sizes(), c.T, c.dev)
                                   : tensor_of(a[13 + i], name, c.T, c.dev);
      if (dx[i].sizes() != x.sizes())
        refuse(PyExc_ValueError, std::string(name) + " must be " + sizes_text(x.sizes()) + ", got " +
                                     sizes_text(dx[i].sizes()));
      out[i] = heads(dx[i], name, c.B, c.L, c.D);
    }
    float *p[4] = {nullptr, nullptr, nullptr, nullptr};
    int64_t bytes = 0;
    for (int i = 0; i < 4; ++i) {
      if (a[2 + i] == Py_None) continue;
      params[i] = make({c.D}, at::kFloat, c.dev);
      p[i] = params[i].data_ptr<float>();
    }
    const Heads &q = c.side[0], &k = c.side[1];
    Tensor ws;
    if (p[0] || p[1] || p[2] || p[3])
      check_status("ag_qk_norm_rope_bwd_workspace",
                   lib.qk_bwd_workspace(c.B, q.H, k.H, c.L, c.D, 1, &bytes));
    if (bytes) ws = make({bytes}, at::kByte, c.dev);
    void *const stream = stream_of(c.dev);
    check_status("ag_qk_norm_rope_bwd", unlocked([&] {
      return lib.qk_bwd(g[0], g[1], code_of(G), q.p, q.sb, q.sl, q.sh, k.p, k.sb, k.sl, k.sh,
                        code_of(c.T), c.w[0], c.w[1], c.norm, c.eps, c.freq, c.R, c.rope,
                        c.positions, c.pos_sb, c.B, q.H, k.H, c.L, c.D, out[0].p, out[0].sb,
                        out[0].sl, out[0].sh, out[1].p, out[1].sb, out[1].sl, out[1].sh, p[0], p[2],
                        p[1], p[3], bytes ? ws.data_ptr() : nullptr, bytes, stream);
    }));
    return Py_BuildValue("(NNNNNN)", THPVariable_Wrap(dx[0]), THPVariable_Wrap(dx[1]),
                         THPVariable_Wrap(params[0]), THPVariable_Wrap(params[1]),
                         THPVariable_Wrap(params[2]), THPVariable_Wrap(params[3]));
  });
}

// --------------------------------------------------------------------------
// grad_clip(grads, max_norm, eps, norm): grads a list or tuple.
PyObject *grad_clip(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 4);
    const Py_ssize_t all = PySequence_Fast_GET_SIZE(a[0]);
    PyObject **items = PySequence_Fast_ITEMS(a[0]);
    std::vector<void *> ptrs;
    std::vector<int64_t> counts;
    std::vector<int> codes;
    ptrs.reserve(all), counts.reserve(all), codes.reserve(all);
    at::Device dev = at::Device(at::kCPU);
    for (Py_ssize_t i = 0; i < all; ++i) {
      if (items[i] == Py_None) continue;
      const Tensor &t = tensor(items[i], "every gradient");
      if (ptrs.empty()) dev = t.device();
      if (t.device() != dev)
        refuse(PyExc_ValueError, std::string("all tensors of a call must be on ") + dev.str() +
                                     "; one is on " + t.device().str());
      const int code = code_of(t.scalar_type());
      if (code < 0)
        refuse(PyExc_TypeError,
               std::string("every gradient must be float32, bfloat16 or float16, got ") +
                   c10::toString(t.scalar_type()));
      if (!t.is_contiguous() && !t.is_non_overlapping_and_dense())
        refuse(PyExc_ValueError, "every gradient must be dense");
      ptrs.push_back(t.data_ptr()), counts.push_back(t.numel()), codes.push_back(code);
    }
    if (ptrs.empty()) refuse(PyExc_ValueError, "grads has no tensor");
    const float max_norm = number(a[1]), eps = number(a[2]);
    const c10::cuda::CUDAGuard guard(dev);
    const Tensor norm = a[3] == Py_None ? make({}, at::kFloat, dev)
                                        : tensor_of(a[3], "norm", at::kFloat, dev);
    if (norm.numel() != 1) refuse(PyExc_ValueError, "norm must have one element");
    const int64_t m = static_cast<int64_t>(ptrs.size());
    int64_t bytes = 0;
    check_status("ag_grad_clip_workspace", lib.clip_workspace(m, &bytes));
    const Tensor ws = make({bytes}, at::kByte, dev);
    void *const stream = stream_of(dev);
    check_status("ag_grad_clip", unlocked([&] {
      return lib.clip(ptrs.data(), counts.data(), codes.data(), m, max_norm, eps,
                      norm.data_ptr<float>(), ws.data_ptr(), bytes, stream);
    }));
    return a[3] == Py_None ? THPVariable_Wrap(norm) : Py_NewRef(a[3]);
  });
}

// is_dense(t): whether the elements fill one block of memory, in any order of
// the dimensions.
PyObject *is_dense(PyObject *, PyObject *o) {
  return guarded([&]() -> PyObject * {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "t must be a torch.Tensor");
    const Tensor &t = THPVariable_Unpack(o);
    return PyBool_FromLong(t.is_contiguous() || t.is_non_overlapping_and_dense());
  });
}

// bind(addresses, AgError): addresses of libag's functions in the order of
// Library.
PyObject *bind(PyObject *, PyObject *args) {
  unsigned long long f[9];
  PyObject *error = nullptr;
  if (!PyArg_ParseTuple(args, "(KKKKKKKKK)O", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &f[7],
                        &f[8], &error))
    return nullptr;
  lib.linear_fwd = reinterpret_cast<decltype(lib.linear_fwd)>(f[0]);
  lib.linear_fwd_workspace = reinterpret_cast<decltype(lib.linear_fwd_workspace)>(f[1]);
  lib.linear_bwd = reinterpret_cast<decltype(lib.linear_bwd)>(f[2]);
  lib.linear_bwd_workspace = reinterpret_cast<decltype(lib.linear_bwd_workspace)>(f[3]);
  lib.qk_fwd = reinterpret_cast<decltype(lib.qk_fwd)>(f[4]);
  lib.qk_bwd = reinterpret_cast<decltype(lib.qk_bwd)>(f[5]);
  lib.qk_bwd_workspace = reinterpret_cast<decltype(lib.qk_bwd_workspace)>(f[6]);
  lib.clip = reinterpret_cast<decltype(lib.clip)>(f[7]);
  lib.clip_workspace = reinterpret_cast<decltype(lib.clip_workspace)>(f[8]);
  Py_XSETREF(lib.error, Py_NewRef(error));
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"linear_fwd", fast(linear_fwd), METH_FASTCALL, nullptr},
    {"linear_bwd", fast(linear_bwd), METH_FASTCALL, nullptr},
    {"qk_fwd", fast(qk_fwd), METH_FASTCALL, nullptr},
    {"qk_bwd", fast(qk_bwd), METH_FASTCALL, nullptr},
    {"grad_clip", fast(grad_clip), METH_FASTCALL, nullptr},
    {"is_dense", is_dense, METH_O, nullptr},
    {"bind", bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layers",
                      "Compiled half of the binding of libag's layers.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// `built_for` says which torch and Python this was compiled for (build.py).
PyMODINIT_FUNC PyInit__layers() {
  PyObject *m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", AG_BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
