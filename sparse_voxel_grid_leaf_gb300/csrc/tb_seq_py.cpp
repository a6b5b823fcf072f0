// The sequence operators' Python entry points: checks of the tensors, outputs
// and workspaces from torch's allocator, and the C calls of include/tb.h on
// torch's current stream.  The module is C++ because the calls are short: in
// Python the marshalling alone took 8 to 12 us of a call of 14 to 18 us.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <string>

#include "../../include/tb.h"

namespace {

PyObject* g_error = nullptr;  // TBError(status, message)

struct Refused {
  int status;
  std::string message;
};

[[noreturn]] void refuse(const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  throw Refused{TB_ERR_INVALID_ARG, buf};
}

void check(tb_status st) {
  if (st != TB_OK) throw Refused{(int)st, tb_last_error()};
}

PyObject* raise(const Refused& r) {
  PyObject* e = PyObject_CallFunction(g_error, "is", r.status, r.message.c_str());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

// An error that Python has set already.
struct PythonError {};

#define TB_ENTRY(name, count)                                            \
  PyObject* name##_body(PyObject* const* a);                             \
  PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n) {          \
    HANDLE_TH_ERRORS                                                     \
    if (n != count) {                                                    \
      PyErr_SetString(PyExc_TypeError, #name ": wrong argument count");  \
      return nullptr;                                                    \
    }                                                                    \
    try {                                                                \
      return name##_body(a);                                             \
    } catch (const Refused& r) {                                         \
      return raise(r);                                                   \
    } catch (const PythonError&) {                                       \
      return nullptr;                                                    \
    }                                                                    \
    END_HANDLE_TH_ERRORS                                                 \
  }                                                                      \
  PyObject* name##_body(PyObject* const* a)

// ------------------------------------------------------------------ arguments

const at::Tensor& tensor(const char* what, const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) refuse("%s: %s must be a tensor", what, name);
  return THPVariable_Unpack(o);
}
const at::Tensor* maybe(const char* what, const char* name, PyObject* o) {
  return o == Py_None ? nullptr : &tensor(what, name, o);
}
double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw PythonError{};
  return x;
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw PythonError{};
  return x != 0;
}

// Whether a gradient is asked for, or one of the tensors carries a forward-mode
// tangent, which the operators do not make either: the autograd functions, and
// the calls that refuse, say so.
template <class... T>
bool tracked(const T*... t) {
  return (c10::GradMode::is_enabled() && ((t && t->requires_grad()) || ...)) ||
         ((t && t->_fw_grad(/*level=*/0).defined()) || ...);
}

// The backward calls record nothing.
[[noreturn]] void refuse_second(const char* what) { refuse("%s: gradients of gradients are not made", what); }

// Tells autograd of a write to t's memory: a backward pass that saved it, or a
// view of the same memory, then raises instead of reading what is new.
void written(const at::Tensor& t) { t.unsafeGetTensorImpl()->bump_version(); }

int device_of(const char* what, const at::Tensor& t) {
  if (!t.is_cuda()) refuse("%s: tensors must be on the GPU", what);
  const int d = t.get_device(), now = c10::cuda::current_device();
  if (d != now) refuse("%s: tensors live on device %d, current device is %d", what, d, now);
  return d;
}

tb_stream stream_of(int device) {
  return (tb_stream)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
}

int32_t type_of(const char* what, const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return TB_TYPE_F32;
    case at::kHalf: return TB_TYPE_F16;
    case at::kBFloat16: return TB_TYPE_BF16;
    default: refuse("%s: expected dtype float32/float16/bfloat16, got %s", what, c10::toString(t.scalar_type()));
  }
}

std::string shape_text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

void same(const char* what, const char* name, const at::Tensor& t, at::IntArrayRef shape, at::ScalarType dtype,
          int device) {
  if (t.sizes() != shape || t.scalar_type() != dtype || !t.is_cuda() || t.get_device() != device)
    refuse("%s: %s must be %s %s on device %d, got %s %s on %s", what, name, c10::toString(dtype),
           shape_text(shape).c_str(), device, c10::toString(t.scalar_type()), shape_text(t.sizes()).c_str(),
           t.device().str().c_str());
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, int device) {
  return at::Tensor(at::detail::empty_cuda(shape, dtype, c10::Device(c10::kCUDA, (c10::DeviceIndex)device), c10::nullopt));
}

// Rows [rows, heads, elements] with unit stride inside a head: the tensor, or
// a copy that this holds.
struct Rows {
  at::Tensor copy;
  void* p = nullptr;
  int64_t rows = 0, heads = 0, dim = 0, row = 0, head = 0;
  Rows() = default;
  Rows(const char* what, const char* name, const at::Tensor& t) {
    if (t.dim() != 3) refuse("%s: %s must have 3 dimensions (rows, heads, elements), got %d", what, name, (int)t.dim());
    const at::Tensor* x = &t;
    if (t.stride(2) != 1 && t.size(2) > 1) {
      copy = t.contiguous();
      x = &copy;
    }
    p = x->data_ptr();
    rows = x->size(0), heads = x->size(1), dim = x->size(2);
    row = x->stride(0), head = x->stride(1);
  }
};

// Contiguous, as it is or as a copy that `hold` keeps.
void* contiguous(const at::Tensor& t, at::Tensor& hold) {
  if (t.is_contiguous()) return t.data_ptr();
  hold = t.contiguous();
  return hold.data_ptr();
}

// [rows, width] of a tensor whose last dimension is the width.
struct Flat {
  at::Tensor copy;
  void* p = nullptr;
  int64_t rows = 0, width = 0, row = 0;
  Flat() = default;
  Flat(const char* what, const char* name, const at::Tensor& t) {
    if (t.dim() < 1) refuse("%s: %s has no rows", what, name);
    const at::Tensor* x = &t;
    width = t.size(t.dim() - 1);
    if (t.dim() != 2) {
      rows = 1;
      for (int64_t i = 0; i + 1 < t.dim(); ++i) rows *= t.size(i);
      copy = t.reshape({rows, width});
      x = &copy;
    }
    if (x->stride(1) != 1 && width > 1) {
      copy = x->contiguous();
      x = &copy;
    }
    rows = x->size(0);
    row = x->stride(0);
    p = x->data_ptr();
  }
};

PyObject* wrap(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
PyObject* tuple(std::initializer_list<PyObject*> items) {
  PyObject* r = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* x : items) {
    if (!r || !x) {
      Py_XDECREF(x);
      Py_CLEAR(r);
      continue;
    }
    PyTuple_SET_ITEM(r, i++, x);
  }
  return r;
}
PyObject* keep(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// --------------------------------------------------------------------- rotary

// (q, k or None, positions, frequencies, layout, sections or None, amplitude,
// inplace, inverse) -> (q, k), or None where gradients are asked for
TB_ENTRY(rotary, 9) {
  const bool inplace = truth(a[7]), inverse = truth(a[8]);
  const char* what = inverse ? "rotary_backward" : "rotary";
  const at::Tensor& q = tensor(what, "q", a[0]);
  const at::Tensor* k = maybe(what, "k", a[1]);
  const at::Tensor& positions = tensor(what, "positions", a[2]);
  const at::Tensor& turns = tensor(what, "frequencies", a[3]);
  if (tracked(&q, k)) {
    if (inplace) refuse("%s: in place is for tensors without gradients", what);
    Py_RETURN_NONE;
  }
  const int device = device_of(what, q);
  tb_rotary_args r{};
  r.type = type_of(what, q);
  auto fits = [&](const char* name, const at::Tensor& t) {
    if (!inplace) return;
    bool ok = t.dim() == 3 && (t.stride(2) == 1 || t.size(2) == 1);
    for (int64_t i = 0; ok && i < 3; ++i) ok = t.stride(i) != 0 || t.size(i) <= 1;
    if (!ok) refuse("%s: %s cannot be turned in place (unit stride inside a head, no repeated rows)", what, name);
  };
  fits("q", q);
  const Rows rq(what, "q", q);
  Rows rk;
  if (k) {
    if (k->dim() != 3) refuse("%s: k must have 3 dimensions (rows, heads, elements), got %d", what, (int)k->dim());
    const int64_t shape[3] = {rq.rows, k->size(1), rq.dim};
    same(what, "k", *k, shape, q.scalar_type(), device);
    fits("k", *k);
    rk = Rows(what, "k", *k);
  }
  if (turns.dim() != 1 || turns.scalar_type() != at::kLong || !turns.is_cuda() || turns.get_device() != device)
    refuse("%s: frequencies must be int64 [pairs] on device %d", what, device);
  at::Tensor turns_copy, positions_copy;
  const int64_t pairs = turns.size(0);
  r.turns = (const int64_t*)contiguous(turns, turns_copy);
  const bool wide = positions.scalar_type() == at::kLong;
  if (!wide && positions.scalar_type() != at::kInt)
    refuse("%s: positions must be int32 or int64, got %s", what, c10::toString(positions.scalar_type()));
  const int64_t axes = positions.dim() == 1 ? 1 : positions.dim() == 2 ? positions.size(1) : 0;
  if (axes < 1 || axes > 3 || positions.size(0) != rq.rows || !positions.is_cuda() || positions.get_device() != device)
    refuse("%s: positions must be [%lld] or [%lld, 1 to 3] on device %d, got %s", what, (long long)rq.rows,
           (long long)rq.rows, device, shape_text(positions.sizes()).c_str());
  const at::Tensor* pos = &positions;
  if (axes > 1 && positions.stride(1) != 1) {
    positions_copy = positions.contiguous();
    pos = &positions_copy;
  }
  int64_t section[3] = {};
  if (a[5] == Py_None) {
    for (int64_t i = 0; i < axes; ++i) section[i] = pairs / axes + (i < pairs % axes);
  } else {
    PyObject* s = PySequence_Fast(a[5], "sections must be a sequence of numbers");
    if (!s) throw PythonError{};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(s);
    int64_t sum = 0;
    for (Py_ssize_t i = 0; i < n && i < 3; ++i) sum += section[i] = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(s, i));
    Py_DECREF(s);
    if (PyErr_Occurred()) throw PythonError{};
    if (n != axes || sum != pairs)
      refuse("%s: %d sections of %lld pairs, for %lld pairs on %lld axes", what, (int)n, (long long)sum, (long long)pairs,
             (long long)axes);
  }
  const char* layout = PyUnicode_Check(a[4]) ? PyUnicode_AsUTF8(a[4]) : nullptr;
  if (!layout) {
    PyErr_Clear();
    refuse("%s: the layout must be \"half\" or \"interleaved\"", what);
  }
  const std::string lay = layout;
  if (lay != "half" && lay != "interleaved") refuse("%s: unknown layout '%s'", what, layout);
  if (pairs > INT32_MAX || rq.heads > INT32_MAX || rk.heads > INT32_MAX || rq.dim > INT32_MAX)
    refuse("%s: sizes beyond 2^31", what);
  r.q = rq.p, r.q_row = rq.row, r.q_head = rq.head, r.q_heads = (int32_t)rq.heads;
  r.k = rk.p, r.k_row = rk.row, r.k_head = rk.head, r.k_heads = (int32_t)rk.heads;
  r.positions = pos->data_ptr();
  r.positions64 = wide;
  r.position_row = pos->stride(0);
  r.tokens = rq.rows;
  r.dim = (int32_t)rq.dim, r.pairs = (int32_t)pairs, r.axes = (int32_t)axes;
  r.section[0] = (int32_t)section[0], r.section[1] = (int32_t)section[1];
  r.layout = lay != "half";
  r.inverse = inverse;
  r.amplitude = (float)number(a[6]);
  at::Tensor qo, ko;
  if (inplace) {
    r.q_out = rq.p, r.q_out_row = rq.row, r.q_out_head = rq.head;
    r.k_out = rk.p, r.k_out_row = rk.row, r.k_out_head = rk.head;
    written(q);
    if (k) written(*k);
  } else {
    qo = empty({rq.rows, rq.heads, rq.dim}, q.scalar_type(), device);
    r.q_out = qo.data_ptr(), r.q_out_row = rq.heads * rq.dim, r.q_out_head = rq.dim;
    if (k) {
      ko = empty({rk.rows, rk.heads, rk.dim}, q.scalar_type(), device);
      r.k_out = ko.data_ptr(), r.k_out_row = rk.heads * rk.dim, r.k_out_head = rk.dim;
    }
  }
  check(tb_rotary(&r, stream_of(device)));
  if (inplace) return tuple({keep(a[0]), keep(a[1])});
  return tuple({wrap(qo), wrap(ko)});
}

// ----------------------------------------------------------------------- norm

void weight_of(const char* what, const at::Tensor& w, int64_t width, const at::Tensor& x, int device, at::Tensor& hold,
               const void** p) {
  const int64_t shape[1] = {width};
  same(what, "weight", w, shape, x.scalar_type(), device);
  *p = contiguous(w, hold);
}

// (x, weight, residual or None, eps, fp8) -> (y, h, scale), h the input x and
// scale None where they are not made; or None where gradients are asked for
TB_ENTRY(norm, 5) {
  const bool fp8 = truth(a[4]);
  const char* what = fp8 ? "rms_norm_fp8" : "rms_norm";
  const at::Tensor& x = tensor(what, "x", a[0]);
  const at::Tensor& weight = tensor(what, "weight", a[1]);
  const at::Tensor* residual = maybe(what, "residual", a[2]);
  if (tracked(&x, &weight, residual)) {
    if (fp8) refuse("%s: the 8-bit output has no gradient", what);
    Py_RETURN_NONE;
  }
  const int device = device_of(what, x);
  tb_norm_args r{};
  r.type = type_of(what, x);
  const Flat fx(what, "x", x);
  Flat fr;
  at::Tensor weight_copy, h, y, scale;
  weight_of(what, weight, fx.width, x, device, weight_copy, &r.weight);
  if (fx.width > INT32_MAX) refuse("%s: sizes beyond 2^31", what);
  r.x = fx.p, r.x_row = fx.row, r.rows = fx.rows, r.width = (int32_t)fx.width;
  if (residual) {
    same(what, "residual", *residual, x.sizes(), x.scalar_type(), device);
    fr = Flat(what, "residual", *residual);
    h = empty(x.sizes(), x.scalar_type(), device);
    r.residual = fr.p, r.residual_row = fr.row;
    r.h_out = h.data_ptr(), r.h_row = fx.width;
  }
  y = empty(x.sizes(), fp8 ? at::kFloat8_e4m3fn : x.scalar_type(), device);
  r.y = y.data_ptr(), r.y_row = fx.width;
  if (fp8) {
    scale = empty(x.sizes().slice(0, x.dim() - 1), at::kFloat, device);
    r.scale = (float*)scale.data_ptr();
    r.fp8 = 1;
  }
  r.eps = (float)number(a[3]);
  if (r.rows) check(tb_rms_norm(&r, stream_of(device)));
  return tuple({wrap(y), residual ? wrap(h) : keep(a[0]), wrap(scale)});
}

// (dy, h, weight, dh or None, eps) -> (dx, dweight)
TB_ENTRY(norm_backward, 5) {
  const char* what = "rms_norm_backward";
  const at::Tensor& dy = tensor(what, "dy", a[0]);
  const at::Tensor& h = tensor(what, "h", a[1]);
  const at::Tensor& weight = tensor(what, "weight", a[2]);
  const at::Tensor* dh = maybe(what, "dh", a[3]);
  if (tracked(&dy, &h, &weight, dh)) refuse_second(what);
  const int device = device_of(what, h);
  tb_norm_backward_args r{};
  r.type = type_of(what, h);
  const Flat fh(what, "h", h);
  same(what, "dy", dy, h.sizes(), h.scalar_type(), device);
  const Flat fd(what, "dy", dy);
  Flat fg;
  at::Tensor weight_copy;
  weight_of(what, weight, fh.width, h, device, weight_copy, &r.weight);
  if (dh) {
    same(what, "dh", *dh, h.sizes(), h.scalar_type(), device);
    fg = Flat(what, "dh", *dh);
  }
  if (fh.width > INT32_MAX) refuse("%s: sizes beyond 2^31", what);
  at::Tensor dx = empty(h.sizes(), h.scalar_type(), device), dw = empty({fh.width}, h.scalar_type(), device);
  r.workspace_bytes = tb_rms_norm_backward_workspace(fh.rows, (int32_t)fh.width);
  at::Tensor work = empty({r.workspace_bytes}, at::kByte, device);
  r.dy = fd.p, r.dy_row = fd.row;
  r.h = fh.p, r.h_row = fh.row, r.rows = fh.rows, r.width = (int32_t)fh.width;
  r.dh = fg.p, r.dh_row = fg.row;
  r.dx = dx.data_ptr(), r.dx_row = fh.width;
  r.dweight = dw.data_ptr();
  r.workspace = (float*)work.data_ptr();
  r.eps = (float)number(a[4]);
  check(tb_rms_norm_backward(&r, stream_of(device)));
  return tuple({wrap(dx), wrap(dw)});
}

// ----------------------------------------------------------- linear attention

struct Linear {
  int device;
  Rows q, k, v;
  at::Tensor decay_copy, offsets_copy, state_copy, work;
  tb_linear_args r{};
  at::ScalarType dtype;

  // a: q, k, v, decay, offsets or None, state or None, scale or None
  Linear(const char* what, PyObject* const* a) {
    const at::Tensor& tq = tensor(what, "q", a[0]);
    const at::Tensor& tk = tensor(what, "k", a[1]);
    const at::Tensor& tv = tensor(what, "v", a[2]);
    const at::Tensor& decay = tensor(what, "decay", a[3]);
    const at::Tensor* offsets = maybe(what, "offsets", a[4]);
    const at::Tensor* state = maybe(what, "state", a[5]);
    device = device_of(what, tq);
    r.type = type_of(what, tq);
    dtype = tq.scalar_type();
    q = Rows(what, "q", tq);
    if (tv.dim() != 3) refuse("%s: v must have 3 dimensions (rows, heads, elements), got %d", what, (int)tv.dim());
    same(what, "k", tk, tq.sizes(), dtype, device);
    const int64_t shape_v[3] = {q.rows, q.heads, tv.size(2)}, shape_d[1] = {q.heads};
    same(what, "v", tv, shape_v, dtype, device);
    same(what, "decay", decay, shape_d, at::kFloat, device);
    k = Rows(what, "k", tk);
    v = Rows(what, "v", tv);
    int64_t grids = 1;
    if (offsets) {
      grids = offsets->dim() == 1 ? offsets->size(0) - 1 : -1;
      if (grids < 0 || offsets->scalar_type() != at::kLong || !offsets->is_cuda() || offsets->get_device() != device)
        refuse("%s: offsets must be int64 [grids + 1] on device %d", what, device);
      r.offsets = (const int64_t*)contiguous(*offsets, offsets_copy);
    }
    const int64_t shape_s[4] = {grids, q.heads, q.dim, v.dim};
    if (state) {
      same(what, "state", *state, shape_s, at::kFloat, device);
      r.state = (const float*)contiguous(*state, state_copy);
    }
    if (grids > INT32_MAX || q.heads > INT32_MAX || q.dim > INT32_MAX || v.dim > INT32_MAX)
      refuse("%s: sizes beyond 2^31", what);
    r.q = q.p, r.q_row = q.row, r.q_head = q.head;
    r.k = k.p, r.k_row = k.row, r.k_head = k.head;
    r.v = v.p, r.v_row = v.row, r.v_head = v.head;
    r.decay = (const float*)contiguous(decay, decay_copy);
    r.tokens = q.rows;
    r.grids = (int32_t)grids, r.heads = (int32_t)q.heads, r.key = (int32_t)q.dim, r.value = (int32_t)v.dim;
    r.scale = a[6] == Py_None ? 1.f / std::sqrt((float)q.dim) : (float)number(a[6]);
  }
  at::Tensor states() const { return empty({r.grids, r.heads, r.key, r.value}, at::kFloat, device); }
  at::Tensor rows(int64_t dim) const { return empty({q.rows, q.heads, dim}, dtype, device); }
  void workspace(bool backward) {
    r.workspace_bytes = tb_linear_attention_workspace(r.tokens, r.grids, r.heads, r.key, r.value, r.type, backward);
    if (!r.workspace_bytes) return;
    work = empty({r.workspace_bytes}, at::kByte, device);
    r.workspace = work.data_ptr();
  }
};

// (q, k, v, decay, offsets or None, state or None, scale or None,
// return_state) -> (o, last states or None), or None where gradients are asked for
TB_ENTRY(linear, 8) {
  const char* what = "linear_attention";
  const at::Tensor* decay = &tensor(what, "decay", a[3]);
  if (tracked(decay)) refuse("%s: the decay is a constant and has no gradient", what);
  if (tracked(&tensor(what, "q", a[0]), &tensor(what, "k", a[1]), &tensor(what, "v", a[2]), maybe(what, "state", a[5])))
    Py_RETURN_NONE;
  Linear l(what, a);
  at::Tensor out = l.rows(l.v.dim), last;
  if (truth(a[7])) last = l.states();
  l.r.out = out.data_ptr(), l.r.out_row = l.q.heads * l.v.dim, l.r.out_head = l.v.dim;
  l.r.state_out = last.defined() ? (float*)last.data_ptr() : nullptr;
  l.workspace(false);
  check(tb_linear_attention(&l.r, stream_of(l.device)));
  return tuple({wrap(out), wrap(last)});
}

// (q, k, v, decay, offsets or None, state or None, scale or None, do, dstate
// or None, want) -> (dq, dk, dv, gradient of the first states or None)
TB_ENTRY(linear_backward, 10) {
  const char* what = "linear_attention_backward";
  const at::Tensor& grad = tensor(what, "do", a[7]);
  const at::Tensor* dstate = maybe(what, "dstate", a[8]);
  if (tracked(&tensor(what, "q", a[0]), &tensor(what, "k", a[1]), &tensor(what, "v", a[2]), &tensor(what, "decay", a[3]),
              maybe(what, "state", a[5]), &grad, dstate))
    refuse_second(what);
  Linear l(what, a);
  const int64_t shape_o[3] = {l.q.rows, l.q.heads, l.v.dim}, shape_s[4] = {l.r.grids, l.r.heads, l.r.key, l.r.value};
  same(what, "do", grad, shape_o, l.dtype, l.device);
  const Rows g(what, "do", grad);
  tb_linear_backward_args b{};
  at::Tensor dstate_copy, dq = l.rows(l.q.dim), dk = l.rows(l.q.dim), dv = l.rows(l.v.dim), first;
  if (dstate) {
    same(what, "dstate", *dstate, shape_s, at::kFloat, l.device);
    b.dstate_out = (const float*)contiguous(*dstate, dstate_copy);
  }
  if (truth(a[9])) {
    first = l.states();
    b.dstate = (float*)first.data_ptr();
  }
  l.workspace(true);
  b.f = l.r;
  b.grad = g.p, b.grad_row = g.row, b.grad_head = g.head;
  b.dq = dq.data_ptr(), b.dq_row = l.q.heads * l.q.dim, b.dq_head = l.q.dim;
  b.dk = dk.data_ptr(), b.dk_row = l.q.heads * l.q.dim, b.dk_head = l.q.dim;
  b.dv = dv.data_ptr(), b.dv_row = l.q.heads * l.v.dim, b.dv_head = l.v.dim;
  check(tb_linear_attention_backward(&b, stream_of(l.device)));
  return tuple({wrap(dq), wrap(dk), wrap(dv), wrap(first)});
}

// (q, k, v, decay, state, slots or None, scale or None) -> o
TB_ENTRY(step, 7) {
  const char* what = "linear_attention_step";
  const at::Tensor& tq = tensor(what, "q", a[0]);
  const at::Tensor& tk = tensor(what, "k", a[1]);
  const at::Tensor& tv = tensor(what, "v", a[2]);
  const at::Tensor& decay = tensor(what, "decay", a[3]);
  const at::Tensor& state = tensor(what, "state", a[4]);
  const at::Tensor* slots = maybe(what, "slots", a[5]);
  const int device = device_of(what, tq);
  tb_linear_step_args r{};
  r.type = type_of(what, tq);
  const Rows q(what, "q", tq);
  if (tv.dim() != 3) refuse("%s: v must have 3 dimensions (rows, heads, elements), got %d", what, (int)tv.dim());
  same(what, "k", tk, tq.sizes(), tq.scalar_type(), device);
  const int64_t shape_v[3] = {q.rows, q.heads, tv.size(2)}, shape_d[1] = {q.heads};
  same(what, "v", tv, shape_v, tq.scalar_type(), device);
  same(what, "decay", decay, shape_d, at::kFloat, device);
  const Rows k(what, "k", tk), v(what, "v", tv);
  const int64_t shape_s[4] = {state.dim() == 4 ? state.size(0) : 0, q.heads, q.dim, v.dim};
  same(what, "state", state, shape_s, at::kFloat, device);
  if (!state.is_contiguous()) refuse("%s: the states must be contiguous", what);
  at::Tensor decay_copy, slots_copy;
  if (slots) {
    const int64_t shape_n[1] = {q.rows};
    same(what, "slots", *slots, shape_n, at::kInt, device);
    r.slots = (const int32_t*)contiguous(*slots, slots_copy);
  }
  if (tracked(&tq, &tk, &tv, &decay, &state))
    refuse("%s: a step in place has no gradient (linear_attention has)", what);
  if (q.heads > INT32_MAX || q.dim > INT32_MAX || v.dim > INT32_MAX) refuse("%s: sizes beyond 2^31", what);
  at::Tensor out = empty(shape_v, tq.scalar_type(), device);
  r.q = q.p, r.q_row = q.row, r.q_head = q.head;
  r.k = k.p, r.k_row = k.row, r.k_head = k.head;
  r.v = v.p, r.v_row = v.row, r.v_head = v.head;
  r.out = out.data_ptr(), r.out_row = q.heads * v.dim, r.out_head = v.dim;
  r.decay = (const float*)contiguous(decay, decay_copy);
  r.state = (float*)state.data_ptr();
  r.streams = q.rows, r.num_slots = shape_s[0];
  r.heads = (int32_t)q.heads, r.key = (int32_t)q.dim, r.value = (int32_t)v.dim;
  r.scale = a[6] == Py_None ? 1.f / std::sqrt((float)q.dim) : (float)number(a[6]);
  written(state);
  check(tb_linear_attention_step(&r, stream_of(device)));
  return wrap(out);
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

#define TB_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {TB_METHOD(rotary),          TB_METHOD(norm), TB_METHOD(norm_backward), TB_METHOD(linear),
                           TB_METHOD(linear_backward), TB_METHOD(step), {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_seq", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__seq(void) { return PyModule_Create(&g_module); }
