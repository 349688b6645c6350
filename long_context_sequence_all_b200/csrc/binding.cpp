// Python binding of the token-wise operators: argument checks, allocation of
// outputs and workspaces on the current stream, and the call of the C ABI
// (include/ulysses.h) in libulysses.so.  Marshalling only; all arithmetic is in
// the library's kernels.
//
// A one-token call takes the GPU 3 to 9 microseconds; checked, allocated for and
// passed on from Python it took the host 12 (residual norm) to 28 (its backward),
// from here 5 and 11; the loss with its gradient (six launches) 46, from here 24.
#include <Python.h>
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "ulysses.h"

namespace {

struct Api {
  decltype(&ulysses_linear_workspace_size) linear_size;
  decltype(&ulysses_linear) linear;
  decltype(&ulysses_linear_bwd_workspace_size) linear_bwd_size;
  decltype(&ulysses_linear_bwd) linear_bwd;
  decltype(&ulysses_residual_norm) norm;
  decltype(&ulysses_residual_norm_bwd_workspace_size) norm_bwd_size;
  decltype(&ulysses_residual_norm_bwd) norm_bwd;
  decltype(&ulysses_linear_loss_workspace_size) loss_size;
  decltype(&ulysses_linear_loss) loss;
  decltype(&ulysses_linear_loss_bwd_workspace_size) loss_bwd_size;
  decltype(&ulysses_linear_loss_bwd) loss_bwd;
} api;
PyObject *error_class = nullptr;   // UlyssesError(status, where)

struct Refused {
  int status;
  std::string what;
};
[[noreturn]] void refuse(int status, const char *where, const std::string &what) {
  throw Refused{status, std::string(where) + ": " + what};
}
void check(uly_status st, const char *where) {
  if (st != ULY_OK) throw Refused{(int)st, where};
}

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

using Tensor = const at::Tensor *;   // null: None

Tensor tensor(PyObject *o, const char *where, const char *name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(ULY_ERR_DTYPE, where, std::string(name) + " is no tensor");
  return &THPVariable_Unpack(o);
}

// One tensor of a call: there, of this type and shape, contiguous, on device `dev`.
struct Call {
  const char *where;
  int dev;
  void want(const char *name, Tensor t, at::IntArrayRef shape, at::ScalarType type) const {
    if (!t) refuse(ULY_ERR_NULL, where, std::string(name) + " is missing");
    if (t->scalar_type() != type)
      refuse(ULY_ERR_DTYPE, where, std::string(name) + " has dtype " + c10::toString(t->scalar_type()) + ", expected " +
                                       c10::toString(type));
    if (t->sizes() != shape)
      refuse(ULY_ERR_SHAPE, where, std::string(name) + " has shape " + text(t->sizes()) + ", expected " + text(shape));
    if (!t->is_contiguous())
      refuse(ULY_ERR_UNSUPPORTED, where, std::string(name) + " is not contiguous (strides " + text(t->strides()) + ")");
    if (t->get_device() != dev)
      refuse(ULY_ERR_CUDA, where, std::string(name) + " is on another device than the call's first tensor");
  }
  void maybe(const char *name, Tensor t, at::IntArrayRef shape, at::ScalarType type) const {
    if (t) want(name, t, shape, type);
  }
  // The tensors are on the current CUDA device, where the call launches.
  void here() const {
    if (dev < 0 || dev != (int)c10::cuda::current_device())
      refuse(ULY_ERR_CUDA, where, "tensors on device " + std::to_string(dev) + ", not on the current CUDA device");
  }
};

// Past the dispatcher (nothing here is differentiated or batched by torch).
at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like) {
  return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}

// An output: the caller's, or a new one if wanted.
struct Out {
  at::Tensor own;
  Tensor t = nullptr;
  PyObject *given = nullptr;
  void take(PyObject *o, const Call &c, const char *name, bool wanted, at::IntArrayRef shape, at::ScalarType type,
            const at::Tensor &like) {
    t = tensor(o, c.where, name);
    if (t) {
      c.want(name, t, shape, type);
      given = o;
    } else if (wanted) {
      own = empty(shape, type, like);
      t = &own;
    }
  }
  void *ptr() const { return t ? t->data_ptr() : nullptr; }
  PyObject *result() const {   // a new reference
    if (given) return Py_NewRef(given);
    if (t) return THPVariable_Wrap(own);
    return Py_NewRef(Py_None);
  }
};

struct Workspace {
  at::Tensor own;
  void *p = nullptr;
  size_t bytes = 0;
  void take(PyObject *o, const Call &c, size_t need, const at::Tensor &like) {
    if (Tensor t = tensor(o, c.where, "workspace")) {
      if (t->scalar_type() != at::kByte || !t->is_contiguous() || t->get_device() != c.dev)
        refuse(ULY_ERR_DTYPE, c.where, "the workspace is not contiguous bytes on the call's device");
      p = t->data_ptr();
      bytes = t->numel();
    } else if (need) {
      own = empty({(int64_t)need}, at::kByte, like);
      p = own.data_ptr();
      bytes = need;
    }
  }
};

const void *ptr(Tensor t) { return t ? t->data_ptr() : nullptr; }
void *stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
int type_code(at::ScalarType t, const char *where) {
  if (t == at::kBFloat16) return ULY_BF16;
  if (t == at::kFloat) return ULY_F32;
  refuse(ULY_ERR_DTYPE, where, std::string("dtype ") + c10::toString(t));
}
at::ScalarType code_type(long code, const char *where) {
  if (code == ULY_BF16) return at::kBFloat16;
  if (code == ULY_F32) return at::kFloat;
  refuse(ULY_ERR_DTYPE, where, "gradient type");
}
int32_t to_i32(int64_t v) { return v > INT32_MAX ? INT32_MAX : (int32_t)v; }   // refused by the library as a shape

long integer(PyObject *o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int32_t integer32(PyObject *o) {
  const long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "an argument is out of 32 bits");
    throw python_error();
  }
  return (int32_t)v;
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}
float real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)v;
}

// Without the interpreter's lock: a launch may wait for room in its queue.
template <class F>
void call(const char *where, F f) {
  uly_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  check(st, where);
}

struct Features {
  at::SmallVector<int64_t, 6> x, y, z;   // shapes [..., K], [..., N], [..., rows of w]
  int64_t k, n, nz, tokens;
  Features(const char *where, Tensor a, Tensor w, int32_t act) {
    if (!a || !w) refuse(ULY_ERR_NULL, where, "x or w is missing");
    if (a->dim() < 1 || w->dim() != 2 || (act == ULY_ACT_SWIGLU && w->size(0) % 2))
      refuse(ULY_ERR_SHAPE, where, "x " + text(a->sizes()) + ", w " + text(w->sizes()));
    nz = w->size(0);
    k = w->size(1);
    n = act == ULY_ACT_SWIGLU ? nz / 2 : nz;
    x.append(a->sizes().begin(), a->sizes().end());
    x.back() = k;
    y = z = x;
    y.back() = n;
    z.back() = nz;
    tokens = k ? a->numel() / k : 0;
  }
};

// linear(x, w, bias, residual, activation, save_pre, y, pre, workspace) -> y, pre
PyObject *linear(PyObject *const *a) {
  static const char *where = "ulysses_linear";
  Tensor x = tensor(a[0], where, "x"), w = tensor(a[1], where, "w"), bias = tensor(a[2], where, "bias"),
         res = tensor(a[3], where, "residual");
  const int32_t act = integer32(a[4]);
  const Features f(where, x, w, act);
  const Call c{where, (int)x->get_device()};
  c.want("x", x, f.x, at::kBFloat16);
  c.want("w", w, {f.nz, f.k}, at::kBFloat16);
  c.maybe("bias", bias, {f.nz}, at::kBFloat16);
  c.maybe("residual", res, f.y, at::kBFloat16);
  Out y, pre;
  y.take(a[6], c, "y", x->is_cuda(), f.y, at::kBFloat16, *x);
  pre.take(a[7], c, "pre", x->is_cuda() && truth(a[5]), f.z, at::kBFloat16, *x);
  c.here();
  size_t need = 0;
  const int32_t k = to_i32(f.k), n = to_i32(f.n);
  check(api.linear_size(f.tokens, k, n, act, &need), "ulysses_linear_workspace_size");
  Workspace ws;
  ws.take(a[8], c, need, *x);
  void *s = stream_of(c.dev);
  call(where, [&] {
    return api.linear(f.tokens, k, n, act, ptr(x), ptr(w), ptr(bias), ptr(res), y.ptr(), pre.ptr(), ws.p,
                      ws.bytes, s);
  });
  if (!pre.t) return y.result();
  return Py_BuildValue("(NN)", y.result(), pre.result());
}

// linear_bwd(x, w, dy, pre, activation, bias_grad, grad type, dx, dw, dbias, workspace) -> dx, dw, dbias
PyObject *linear_bwd(PyObject *const *a) {
  static const char *where = "ulysses_linear_bwd";
  Tensor x = tensor(a[0], where, "x"), w = tensor(a[1], where, "w"), dy = tensor(a[2], where, "dy"),
         pre = tensor(a[3], where, "pre");
  const int32_t act = integer32(a[4]);
  const Features f(where, x, w, act);
  const Call c{where, (int)x->get_device()};
  c.want("x", x, f.x, at::kBFloat16);
  c.want("w", w, {f.nz, f.k}, at::kBFloat16);
  c.want("dy", dy, f.y, at::kBFloat16);
  if (act == ULY_ACT_NONE) pre = nullptr;
  else c.want("pre", pre, f.z, at::kBFloat16);
  const bool cuda = x->is_cuda();
  Out dx, dw, db;
  dx.take(a[7], c, "dx", cuda, f.x, at::kBFloat16, *x);
  Tensor given = tensor(a[8], where, "dw");
  const at::ScalarType wt = given ? given->scalar_type() : code_type(integer(a[6]), where);
  const int code = type_code(wt, where);
  dw.take(a[8], c, "dw", cuda, {f.nz, f.k}, wt, *x);
  db.take(a[9], c, "dbias", cuda && truth(a[5]), {f.nz}, at::kFloat, *x);
  c.here();
  size_t need = 0;
  const int32_t k = to_i32(f.k), n = to_i32(f.n);
  check(api.linear_bwd_size(f.tokens, k, n, act, &need), "ulysses_linear_bwd_workspace_size");
  Workspace ws;
  ws.take(a[10], c, need, *x);
  void *s = stream_of(c.dev);
  call(where, [&] {
    return api.linear_bwd(f.tokens, k, n, act, ptr(x), ptr(w), ptr(pre), ptr(dy), dx.ptr(), dw.ptr(), code,
                          static_cast<float *>(db.ptr()), ws.p, ws.bytes, s);
  });
  return Py_BuildValue("(NNN)", dx.result(), dw.result(), db.result());
}

// What both directions of the norm check of the gate and the weights.
void want_norm(const Call &c, at::IntArrayRef shape, at::ScalarType type, Tensor w_pre, Tensor w_post, Tensor gate,
               int32_t mode) {
  if (shape.size() != 4) refuse(ULY_ERR_SHAPE, c.where, "shape " + text(shape) + ", expected [P][B][n/P][hidden]");
  type_code(type, c.where);
  const int64_t d = shape[3];
  c.maybe("w_pre", w_pre, {d}, type);
  c.maybe("w_post", w_post, {d}, type);
  switch (mode) {
    case ULY_GATE_NONE:
      if (gate) refuse(ULY_ERR_SHAPE, c.where, "a gate with GATE_NONE");
      break;
    case ULY_GATE_CHANNEL: c.want("gate", gate, {d}, type); break;
    case ULY_GATE_SEQUENCE: c.want("gate", gate, {shape[1], d}, type); break;
    case ULY_GATE_TOKEN: c.want("gate", gate, shape, type); break;
    default: refuse(ULY_ERR_UNSUPPORTED, c.where, "gate mode " + std::to_string(mode));
  }
}
struct NormShape {
  int32_t P, B, n, d;
  NormShape(const char *where, at::IntArrayRef s) : P(to_i32(s[0])), B(to_i32(s[1])), d(to_i32(s[3])) {
    // P s within an int32, else refused as a shape
    n = s[2] > 0 && s[0] > INT32_MAX / s[2] ? -1 : (int32_t)(s[0] * s[2]);
    if (n < 0) refuse(ULY_ERR_SHAPE, where, "shape " + text(s));
  }
};

// residual_norm(x, h, w_pre, w_post, gate, gate_mode, res_scale, eps, r, u) -> r, u
PyObject *residual_norm(PyObject *const *a) {
  static const char *where = "ulysses_residual_norm";
  Tensor x = tensor(a[0], where, "x"), h = tensor(a[1], where, "h"), w_pre = tensor(a[2], where, "w_pre"),
         w_post = tensor(a[3], where, "w_post"), gate = tensor(a[4], where, "gate");
  const int32_t mode = integer32(a[5]);
  if (!x) refuse(ULY_ERR_NULL, where, "x is missing");
  const Call c{where, (int)x->get_device()};
  const auto shape = x->sizes();
  const auto type = x->scalar_type();
  want_norm(c, shape, type, w_pre, w_post, gate, mode);
  c.want("x", x, shape, type);
  c.maybe("h", h, shape, type);
  Out r, u;
  r.take(a[8], c, "r", x->is_cuda() && (h || !w_pre), shape, type, *x);
  u.take(a[9], c, "u", x->is_cuda() && w_pre, shape, type, *x);
  c.here();
  const NormShape s(where, shape);
  const float scale = real(a[6]), eps = real(a[7]);
  const int code = type_code(type, where);
  void *st = stream_of(c.dev);
  call(where, [&] {
    return api.norm(s.B, s.n, s.P, s.d, code, ptr(x), ptr(h), ptr(gate), mode, ptr(w_post), ptr(w_pre), scale,
                    eps, r.ptr(), u.ptr(), st);
  });
  return Py_BuildValue("(NN)", r.result(), u.result());
}

// residual_norm_bwd(r, h, dr, du, w_pre, w_post, gate, gate_mode, res_scale, eps, dx, dh, dw_pre, dw_post, dgate,
//                   workspace) -> dx, dh, dw_pre, dw_post, dgate
PyObject *residual_norm_bwd(PyObject *const *a) {
  static const char *where = "ulysses_residual_norm_bwd";
  Tensor r = tensor(a[0], where, "r"), h = tensor(a[1], where, "h"), dr = tensor(a[2], where, "dr"),
         du = tensor(a[3], where, "du"), w_pre = tensor(a[4], where, "w_pre"), w_post = tensor(a[5], where, "w_post"),
         gate = tensor(a[6], where, "gate");
  const int32_t mode = integer32(a[7]);
  if (!r) refuse(ULY_ERR_NULL, where, "r is missing");
  const Call c{where, (int)r->get_device()};
  const auto shape = r->sizes();
  const auto type = r->scalar_type();
  want_norm(c, shape, type, w_pre, w_post, gate, mode);
  c.want("r", r, shape, type);
  c.maybe("h", h, shape, type);
  c.maybe("dr", dr, shape, type);
  c.maybe("du", du, shape, type);
  const int64_t d = shape[3];
  const bool cuda = r->is_cuda();
  Out dx, dh, dw_pre, dw_post, dgate;
  dx.take(a[10], c, "dx", cuda, shape, type, *r);
  dh.take(a[11], c, "dh", cuda && h, shape, type, *r);
  dw_pre.take(a[12], c, "dw_pre", cuda && du, {d}, at::kFloat, *r);
  dw_post.take(a[13], c, "dw_post", cuda && w_post, {d}, at::kFloat, *r);
  if (!gate && a[14] != Py_None) refuse(ULY_ERR_SHAPE, where, "dgate without a gate");
  if (gate)
    dgate.take(a[14], c, "dgate", cuda, gate->sizes(), mode == ULY_GATE_TOKEN ? type : at::kFloat, *r);
  c.here();
  const NormShape s(where, shape);
  const float scale = real(a[8]), eps = real(a[9]);
  const int code = type_code(type, where);
  size_t need = 0;
  check(api.norm_bwd_size(s.B, s.n, s.d, code, mode, &need), "ulysses_residual_norm_bwd_workspace_size");
  Workspace ws;
  ws.take(a[15], c, need, *r);
  void *st = stream_of(c.dev);
  call(where, [&] {
    return api.norm_bwd(s.B, s.n, s.P, s.d, code, ptr(r), ptr(h), ptr(dr), ptr(du), ptr(gate), mode, ptr(w_post),
                        ptr(w_pre), scale, eps, dx.ptr(), dh.ptr(), static_cast<float *>(dw_post.ptr()),
                        static_cast<float *>(dw_pre.ptr()), dgate.ptr(), ws.p, ws.bytes, st);
  });
  return Py_BuildValue("(NNNNN)", dx.result(), dh.result(), dw_pre.result(), dw_post.result(), dgate.result());
}

// What both loss calls take: x, w, labels, P, ignore_index and the three results.
struct LossCall {
  Tensor x, w, labels;
  Call c;
  int32_t P, d, V, ignore;
  int64_t T;
  Out sum, count, loss;
  LossCall(const char *where, PyObject *const *a, PyObject *const *outs) {
    x = tensor(a[0], where, "x");
    w = tensor(a[1], where, "w");
    labels = tensor(a[2], where, "labels");
    if (!x || !w) refuse(ULY_ERR_NULL, where, "x or w is missing");
    if (x->dim() != 2 || w->dim() != 2) refuse(ULY_ERR_SHAPE, where, "x " + text(x->sizes()) + ", w " + text(w->sizes()));
    c = Call{where, (int)x->get_device()};
    c.want("x", x, x->sizes(), at::kBFloat16);
    c.want("w", w, {w->size(0), x->size(1)}, at::kBFloat16);
    if (labels && labels->numel() == x->size(0)) c.want("labels", labels, labels->sizes(), at::kInt);   // or the seq layout
    else c.want("labels", labels, {x->size(0)}, at::kInt);
    T = x->size(0);
    d = to_i32(x->size(1));
    V = to_i32(w->size(0));
    const long p = integer(a[3]);
    if (p < 1 || p > 65535) refuse(ULY_ERR_SHAPE, where, "P = " + std::to_string(p));
    P = (int32_t)p;
    ignore = integer32(a[4]);
    const bool cuda = x->is_cuda();
    sum.take(outs[0], c, "shard_sum", cuda, {P}, at::kFloat, *x);
    count.take(outs[1], c, "shard_count", cuda, {P}, at::kLong, *x);
    loss.take(outs[2], c, "loss", cuda, {1}, at::kFloat, *x);
  }
  float *sums() const { return static_cast<float *>(sum.ptr()); }
  int64_t *counts() const { return static_cast<int64_t *>(count.ptr()); }
  float *value() const { return static_cast<float *>(loss.ptr()); }
};

// linear_loss(x, w, labels, P, ignore_index, shard_sum, shard_count, loss, workspace)
PyObject *linear_loss(PyObject *const *a) {
  static const char *where = "ulysses_linear_loss";
  LossCall l(where, a, a + 5);
  l.c.here();
  size_t need = 0;
  check(api.loss_size(l.P, l.T, l.d, l.V, &need), "ulysses_linear_loss_workspace_size");
  Workspace ws;
  ws.take(a[8], l.c, need, *l.x);
  void *s = stream_of(l.c.dev);
  call(where, [&] {
    return api.loss(l.P, l.T, l.d, l.V, ptr(l.x), ptr(l.w), static_cast<const int32_t *>(ptr(l.labels)), l.ignore,
                    l.sums(), l.counts(), l.value(), ws.p, ws.bytes, s);
  });
  return Py_BuildValue("(NNN)", l.sum.result(), l.count.result(), l.loss.result());
}

// linear_loss_bwd(x, w, labels, P, ignore_index, grad type, piece_tokens, dx, dw, shard_sum, shard_count, loss, workspace)
PyObject *linear_loss_bwd(PyObject *const *a) {
  static const char *where = "ulysses_linear_loss_bwd";
  LossCall l(where, a, a + 9);
  const bool cuda = l.x->is_cuda();
  Out dx, dw;
  dx.take(a[7], l.c, "dx", cuda, l.x->sizes(), at::kBFloat16, *l.x);
  Tensor given = tensor(a[8], where, "dw");
  const at::ScalarType wt = given ? given->scalar_type() : code_type(integer(a[5]), where);
  const int code = type_code(wt, where);
  dw.take(a[8], l.c, "dw", cuda, l.w->sizes(), wt, *l.x);
  l.c.here();
  const int64_t piece = integer(a[6]);
  size_t need = 0;
  check(api.loss_bwd_size(l.P, l.T, l.d, l.V, code, piece, &need), "ulysses_linear_loss_bwd_workspace_size");
  Workspace ws;
  ws.take(a[12], l.c, need, *l.x);
  void *s = stream_of(l.c.dev);
  call(where, [&] {
    return api.loss_bwd(l.P, l.T, l.d, l.V, ptr(l.x), ptr(l.w), static_cast<const int32_t *>(ptr(l.labels)), l.ignore,
                        dx.ptr(), dw.ptr(), code, piece, l.sums(), l.counts(), l.value(), ws.p, ws.bytes, s);
  });
  return Py_BuildValue("(NNNNN)", l.sum.result(), l.count.result(), l.loss.result(), dx.result(), dw.result());
}

// Positional arguments only, in number `n`; refusals become UlyssesError.
template <PyObject *(*F)(PyObject *const *), int n>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != n) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", n, nargs);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused &r) {
    PyObject *e = PyObject_CallFunction(error_class ? error_class : PyExc_RuntimeError, "is", r.status, r.what.c_str());
    if (e) {
      PyErr_SetObject((PyObject *)Py_TYPE(e), e);
      Py_DECREF(e);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// init(path of libulysses.so, the exception class of refusals)
PyObject *init(PyObject *, PyObject *args) {
  const char *path = nullptr;
  PyObject *cls = nullptr;
  if (!PyArg_ParseTuple(args, "sO", &path, &cls)) return nullptr;
  void *lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  if (!lib) {
    PyErr_Format(PyExc_RuntimeError, "%s", dlerror());
    return nullptr;
  }
  const struct {
    const char *name;
    void *to;
  } names[] = {{"ulysses_linear_workspace_size", &api.linear_size},
               {"ulysses_linear", &api.linear},
               {"ulysses_linear_bwd_workspace_size", &api.linear_bwd_size},
               {"ulysses_linear_bwd", &api.linear_bwd},
               {"ulysses_residual_norm", &api.norm},
               {"ulysses_residual_norm_bwd_workspace_size", &api.norm_bwd_size},
               {"ulysses_residual_norm_bwd", &api.norm_bwd},
               {"ulysses_linear_loss_workspace_size", &api.loss_size},
               {"ulysses_linear_loss", &api.loss},
               {"ulysses_linear_loss_bwd_workspace_size", &api.loss_bwd_size},
               {"ulysses_linear_loss_bwd", &api.loss_bwd}};
  for (const auto &n : names) {
    void *f = dlsym(lib, n.name);
    if (!f) {
      PyErr_Format(PyExc_RuntimeError, "%s has no %s", path, n.name);
      return nullptr;
    }
    *static_cast<void **>(n.to) = f;
  }
  Py_XSETREF(error_class, Py_NewRef(cls));
  Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), int n>
constexpr PyMethodDef method(const char *name) {
  return {name, (PyCFunction)(void (*)(void))(PyObject * (*)(PyObject *, PyObject *const *, Py_ssize_t)) entry<F, n>,
          METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {{"init", init, METH_VARARGS, nullptr},
                         method<linear, 9>("linear"),
                         method<linear_bwd, 11>("linear_bwd"),
                         method<residual_norm, 10>("residual_norm"),
                         method<residual_norm_bwd, 16>("residual_norm_bwd"),
                         method<linear_loss, 9>("linear_loss"),
                         method<linear_loss_bwd, 13>("linear_loss_bwd"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", "Binding of the token-wise operators", -1, methods};

}  // namespace

#ifndef ULY_BINDING_TAG
#error "the build says what the binding is for (build.py)"
#endif
PyMODINIT_FUNC PyInit__native(void) {
  PyObject *m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "tag", ULY_BINDING_TAG) < 0) Py_CLEAR(m);
  return m;
}
