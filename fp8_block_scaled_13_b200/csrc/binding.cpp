// The argument handling of the Python wrappers in block.py and muon.py: the
// checks, the allocation of outputs and the call into libpuro_fp8.so.  These
// operators run for a few microseconds on small inputs and take up to 20
// tensors; checking those in Python took two to three times as long as the GPU
// needed (the norm of 16 rows: 13 us of 20; its backward pass: 30 of 43).
// Everything is refused here as the Python wrappers of the linear layers refuse
// it: ValueError before any launch; a status of the library is returned as the
// first value and raised there.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cstdarg>
#include <initializer_list>
#include <set>
#include <string>

#include "../../include/puro_fp8.h"

namespace {

struct PythonError {};  // a Python exception is set

[[noreturn]] void value_error(const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(PyExc_ValueError, format, args);
  va_end(args);
  throw PythonError();
}

// A tensor argument, or none.
struct Arg {
  const char* name;
  const at::Tensor* t = nullptr;

  Arg(PyObject* o, const char* n, bool optional = true) : name(n) {
    if (optional && o == Py_None) return;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "%s must be a tensor, got %s", n, Py_TYPE(o)->tp_name);
      throw PythonError();
    }
    t = &THPVariable_Unpack(o);
  }
  explicit operator bool() const { return t != nullptr; }
  void* ptr() const { return t ? t->data_ptr() : nullptr; }
  int64_t ld() const { return t ? t->stride(0) : 0; }
};

std::string type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kByte: return "torch.uint8";
    default: return std::string("torch.") + c10::toString(t);
  }
}

std::string shape_name(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

void need_cuda(const Arg& a) {
  if (!a.t->is_cuda()) value_error("%s must be a CUDA tensor", a.name);
}

void need_type(const Arg& a, at::ScalarType t) {
  if (a.t->scalar_type() != t)
    value_error("%s must be %s, got %s", a.name, type_name(t).c_str(), type_name(a.t->scalar_type()).c_str());
}

// A row-major matrix of the given type and shape (wider: at least that many columns).
void need_matrix(const Arg& a, at::ScalarType type, int64_t rows, int64_t cols, bool wider = false) {
  need_cuda(a);
  need_type(a, type);
  const at::Tensor& t = *a.t;
  const bool shape = t.dim() == 2 && t.size(0) == rows && (wider ? t.size(1) >= cols : t.size(1) == cols);
  if (!shape || (t.numel() && t.stride(1) != 1))
    value_error("%s must be a row-major (%lld, %lld) tensor, got %s", a.name, (long long)rows, (long long)cols,
                shape_name(t).c_str());
}

// The matrix that a call's sizes come from.
void need_any_matrix(const Arg& a) {
  need_cuda(a);
  need_type(a, at::kBFloat16);
  if (a.t->dim() != 2 || a.t->stride(1) != 1) value_error("%s must be a row-major 2-D tensor", a.name);
}

// A contiguous FP32 vector.
void need_vector(const Arg& a, int64_t n) {
  const at::Tensor& t = *a.t;
  if (!t.is_cuda() || t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    value_error("%s must be a contiguous CUDA float32 [%lld] tensor", a.name, (long long)n);
}

void need_weight(const Arg& a, int64_t cols) {
  need_cuda(a);
  const at::Tensor& t = *a.t;
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)
    value_error("%s must be torch.bfloat16 or torch.float32, got %s", a.name, type_name(t.scalar_type()).c_str());
  if (t.dim() != 1 || t.size(0) != cols || !t.is_contiguous())
    value_error("%s must be a contiguous [%lld] tensor, got %s", a.name, (long long)cols, shape_name(t).c_str());
}

void need_bytes(const Arg& a, int64_t n) {
  const at::Tensor& t = *a.t;
  if (!t.is_cuda() || t.scalar_type() != at::kByte || !t.is_contiguous() || t.numel() < n)
    value_error("%s must be a contiguous CUDA uint8 tensor of at least %lld bytes", a.name, (long long)n);
}

// 1 for FP32 weights, 0 for BF16 ones.
int weight_type(const Arg& w_pre, const Arg& w_post) {
  if (w_post && w_post.t->scalar_type() != w_pre.t->scalar_type())
    value_error("w_pre and w_post must have one type, got %s and %s", type_name(w_pre.t->scalar_type()).c_str(),
                type_name(w_post.t->scalar_type()).c_str());
  return w_pre.t->scalar_type() == at::kFloat;
}

void need_branch(const Arg& h, const Arg& w_post, const Arg& gate) {
  if (!h && (w_post || gate)) value_error("w_post and gate act on the block output h, which is missing");
}

struct Gate {
  int kind = PURO_GATE_NONE, f32 = 0;
  int64_t ld = 0;
};

// The kind of a gate [rows, 1], [1, cols] or [rows, cols].
Gate gate_of(const Arg& a, int64_t rows, int64_t cols) {
  Gate g;
  if (!a) return g;
  need_cuda(a);
  const at::Tensor& t = *a.t;
  const int64_t r = t.dim() == 2 ? t.size(0) : -1, c = t.dim() == 2 ? t.size(1) : -1;
  if (!((r == rows && c == 1) || (r == 1 && c == cols) || (r == rows && c == cols)))
    value_error("gate must be [%lld, 1], [1, %lld] or [%lld, %lld], got %s", (long long)rows, (long long)cols,
                (long long)rows, (long long)cols, shape_name(t).c_str());
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)
    value_error("gate must be torch.bfloat16 or torch.float32, got %s", type_name(t.scalar_type()).c_str());
  g.f32 = t.scalar_type() == at::kFloat;
  if (c == 1) {
    if (!t.is_contiguous()) value_error("a gate per token must be contiguous");
    g.kind = PURO_GATE_TOKEN;
  } else if (r == 1) {  // also one row of elements: the same products
    if (!t.is_contiguous()) value_error("a gate per channel must be contiguous");
    g.kind = PURO_GATE_CHANNEL;
  } else {
    if (g.f32) value_error("a gate per element must be torch.bfloat16");
    if (t.numel() && t.stride(1) != 1) value_error("gate must be a row-major 2-D tensor");
    g.kind = PURO_GATE_FULL;
    g.ld = t.stride(0);
  }
  return g;
}

int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

// Runs with the operands' device current, as the library launches on the
// current one; operands on several devices are refused.
class OnDevice {
 public:
  OnDevice(const char* call, std::initializer_list<const Arg*> args) {
    const at::Tensor* first = nullptr;
    for (const Arg* a : args)
      if (*a) {
        if (!first) first = a->t;
        if (a->t->device() != first->device()) refuse(call, args);
      }
    device_ = first->device();
    if (!device_.is_cuda()) return;  // the checks say which operand
    before_ = c10::cuda::current_device();
    if (device_.index() != before_) c10::cuda::set_device(device_.index());
  }
  ~OnDevice() {
    if (before_ >= 0 && device_.index() != before_) {
      try {
        c10::cuda::set_device(before_);
      } catch (...) {
      }
    }
  }
  OnDevice(const OnDevice&) = delete;
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device_.index()).stream(); }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(device_));
  }

 private:
  [[noreturn]] static void refuse(const char* call, std::initializer_list<const Arg*> args) {
    std::set<std::string> names;
    for (const Arg* a : args)
      if (*a) names.insert(a->t->device().str());
    std::string all;
    for (const std::string& n : names) all += (all.empty() ? "" : ", ") + n;
    value_error("%s: operands are on different devices (%s)", call, all.c_str());
  }
  c10::Device device_{c10::kCPU};
  int before_ = -1;
};

// Where a [rows, cols] result goes: the caller's QuantAct or BF16 tensor, or new
// memory.  `out` is None, a tensor, or an object with the fields of a QuantAct.
struct Field {
  PyObject* o = nullptr;
  Field(PyObject* out, const char* name) {
    if (out == Py_None) return;
    o = PyObject_GetAttrString(out, name);
    if (!o) {
      if (!PyErr_ExceptionMatches(PyExc_AttributeError)) throw PythonError();
      PyErr_Clear();
    }
  }
  ~Field() { Py_XDECREF(o); }
  Field(const Field&) = delete;
  PyObject* get() const { return o ? o : Py_None; }
};

struct Result {
  int layout;
  PyObject* out;
  bool tensor;                // `out` is a tensor
  Field fq, fs, fqt, fst;
  Arg q, s, qt, st, bf;       // the caller's
  at::Tensor nq, ns, nqt, nst, nbf;  // new ones

  Result(PyObject* o, int flag)
      : layout(flag), out(o), tensor(o != Py_None && THPVariable_Check(o)),
        fq(tensor ? Py_None : o, "q"), fs(tensor ? Py_None : o, "s"), fqt(tensor ? Py_None : o, "qt"),
        fst(tensor ? Py_None : o, "st"), q(fq.get(), "out.q"), s(fs.get(), "out.s"), qt(fqt.get(), "out.qt"),
        st(fst.get(), "out.st"), bf(tensor ? o : Py_None, "out") {}

  static const Arg& given(const Arg& a, const char* what) {
    if (!a) value_error("out has no %s", what);
    return a;
  }
  static bool is(PyObject* o, const char* name, int64_t n) {
    Field f(o, name);
    if (!f.o || !PyLong_Check(f.o)) return false;
    const long long v = PyLong_AsLongLong(f.o);
    if (v == -1 && PyErr_Occurred()) PyErr_Clear();
    return v == n;
  }

  void resolve(int64_t rows, int64_t cols, const OnDevice& dev) {
    const int64_t tiles = (rows + 127) / 128;
    if (layout == PURO_BF16) {
      if (out == Py_None) {
        nbf = dev.empty({rows, cols}, at::kBFloat16);
        return;
      }
      if (!tensor) value_error("out must be a BF16 tensor for layout 'bf16'");
      need_matrix(bf, at::kBFloat16, rows, cols);
      return;
    }
    if (out == Py_None) {
      auto scales = [&](int64_t r, int64_t groups) {
        const int64_t n = puro_fp8_blocked_scale_bytes(r, groups);
        return dev.empty({n > 16 ? n : 16}, at::kByte);
      };
      if (layout & PURO_ROWWISE) {
        nq = dev.empty({rows, cols}, at::kByte);
        ns = scales(rows, cols / 128);
      }
      if (layout & PURO_COLWISE) {
        nqt = dev.empty({cols, round16(rows)}, at::kByte);
        nst = scales(cols, tiles);
      }
      return;
    }
    if (tensor || !is(out, "rows", rows) || !is(out, "cols", cols))
      value_error("out must be a QuantAct made for a [%lld, %lld] input", (long long)rows, (long long)cols);
    if (layout & PURO_ROWWISE) {
      need_matrix(given(q, "row-wise codes"), at::kByte, rows, cols);
      need_bytes(given(s, "row-wise scales"), puro_fp8_blocked_scale_bytes(rows, cols / 128));
    }
    if (layout & PURO_COLWISE) {
      need_matrix(given(qt, "transposed codes"), at::kByte, cols, round16(rows), true);
      need_bytes(given(st, "transposed scales"), puro_fp8_blocked_scale_bytes(cols, tiles));
    }
  }

  // the C call's arguments
  static void* at_(const Arg& a, const at::Tensor& n) { return a ? a.ptr() : n.defined() ? n.data_ptr() : nullptr; }
  static int64_t ld_(const Arg& a, const at::Tensor& n) { return a ? a.ld() : n.defined() ? n.stride(0) : 0; }
  bool row() const { return layout != PURO_BF16 && (layout & PURO_ROWWISE); }
  bool col() const { return layout != PURO_BF16 && (layout & PURO_COLWISE); }
  void* q_() const { return row() ? at_(q, nq) : nullptr; }
  int64_t ld_q() const { return row() ? ld_(q, nq) : 0; }
  void* s_() const { return row() ? at_(s, ns) : nullptr; }
  void* qt_() const { return col() ? at_(qt, nqt) : nullptr; }
  int64_t ld_qt() const { return col() ? ld_(qt, nqt) : 0; }
  void* st_() const { return col() ? at_(st, nst) : nullptr; }
  void* bf_() const { return layout == PURO_BF16 ? at_(bf, nbf) : nullptr; }
  int64_t ld_bf() const { return layout == PURO_BF16 ? ld_(bf, nbf) : 0; }
};

PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

// (status, new tensors...): None for each that was given or is not wanted.
PyObject* results(int status, std::initializer_list<const at::Tensor*> tensors) {
  PyObject* r = PyTuple_New((Py_ssize_t)tensors.size() + 1);
  if (!r) throw PythonError();
  PyTuple_SET_ITEM(r, 0, PyLong_FromLong(status));
  Py_ssize_t i = 1;
  for (const at::Tensor* t : tensors) {
    PyObject* o = wrap(*t);
    if (!o) {
      Py_DECREF(r);
      throw PythonError();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError();
  return v;
}

int integer(PyObject* o, const char* name) {
  int overflow = 0;
  const long v = PyLong_AsLongAndOverflow(o, &overflow);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  if (overflow || v < INT_MIN || v > INT_MAX) value_error("%s is out of range", name);
  return (int)v;
}

void need_count(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
  throw PythonError();
}

// The library's calls only queue work, but may wait for room in the queue.
template <class F>
int unlocked(F f) {
  int st;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  Py_END_ALLOW_THREADS;
  return st;
}

// Turns C++ exceptions into Python ones, torch's (out of memory among them) into
// what torch makes of them.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const PythonError&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// x, w_pre, h, w_post, gate, scale, eps, layout, y, out
//   -> status, y, rstd, rstd_post, q, s, qt, st, bf16
PyObject* residual_norm(PyObject* const* a, Py_ssize_t n) {
  need_count(n, 10);
  const Arg x(a[0], "x", false), w_pre(a[1], "w_pre", false), h(a[2], "h"), w_post(a[3], "w_post"), gate(a[4], "gate"),
      y(a[8], "y");
  const float scale = (float)number(a[5]), eps = (float)number(a[6]);
  Result res(a[9], integer(a[7], "layout"));
  const OnDevice dev("residual_norm", {&x, &w_pre, &h, &w_post, &gate, &y, &res.q, &res.s, &res.qt, &res.st, &res.bf});
  need_any_matrix(x);
  const int64_t rows = x.t->size(0), cols = x.t->size(1);
  need_branch(h, w_post, gate);
  if (!(eps > 0)) value_error("eps must be positive");
  need_weight(w_pre, cols);
  const int w_f32 = weight_type(w_pre, w_post);
  at::Tensor ny;
  if (h) {
    need_matrix(h, at::kBFloat16, rows, cols);
    if (y)
      need_matrix(y, at::kBFloat16, rows, cols);
    else
      ny = dev.empty({rows, cols}, at::kBFloat16);
    if (w_post) need_weight(w_post, cols);
  } else if (y) {
    value_error("y is only written with a block output h");
  }
  const Gate g = gate_of(gate, rows, cols);
  res.resolve(rows, cols, dev);
  at::Tensor rstd = dev.empty({rows}, at::kFloat), rstd_post, ws;
  if (w_post) rstd_post = dev.empty({rows}, at::kFloat);
  const int64_t need = puro_fp8_residual_norm_workspace_bytes(rows, cols, res.layout, 0);
  if (need) ws = dev.empty({need}, at::kByte);
  void* stream = dev.stream();
  const int st = unlocked([&] {
    return puro_fp8_residual_norm(
        x.ptr(), x.ld(), h.ptr(), h.ld(), w_pre.ptr(), w_post.ptr(), w_f32, gate.ptr(), g.ld, g.kind, g.f32, scale, eps,
        rows, cols, Result::at_(y, ny), Result::ld_(y, ny), rstd.data_ptr<float>(),
        w_post ? rstd_post.data_ptr<float>() : nullptr, res.layout, res.q_(), res.ld_q(), res.s_(), res.qt_(),
        res.ld_qt(), res.st_(), res.bf_(), res.ld_bf(), need ? ws.data_ptr() : nullptr, stream);
  });
  return results(st, {&ny, &rstd, &rstd_post, &res.nq, &res.ns, &res.nqt, &res.nst, &res.nbf});
}

// dn, y, rstd, w_pre, h, dy, w_post, rstd_post, gate, scale, layout, dx, out, dw_pre, dw_post, dgate, accumulate
//   -> status, dx, dw_pre, dw_post, dgate, q, s, qt, st, bf16
PyObject* residual_norm_backward(PyObject* const* a, Py_ssize_t n) {
  need_count(n, 17);
  const Arg dn(a[0], "dn", false), y(a[1], "y", false), rstd(a[2], "rstd", false), w_pre(a[3], "w_pre", false),
      h(a[4], "h"), dy(a[5], "dy"), w_post(a[6], "w_post"), rstd_post(a[7], "rstd_post"), gate(a[8], "gate"),
      dx(a[11], "dx"), dw_pre(a[13], "dw_pre"), dw_post(a[14], "dw_post"), dgate(a[15], "dgate");
  const float scale = (float)number(a[9]);
  const int accumulate = PyObject_IsTrue(a[16]);
  if (accumulate < 0) throw PythonError();
  Result res(a[12], integer(a[10], "layout"));
  const OnDevice dev("residual_norm_backward",
                     {&dn, &y, &rstd, &w_pre, &h, &dy, &w_post, &rstd_post, &gate, &dx, &dw_pre, &dw_post, &dgate,
                      &res.q, &res.s, &res.qt, &res.st, &res.bf});
  need_any_matrix(dn);
  const int64_t rows = dn.t->size(0), cols = dn.t->size(1);
  need_branch(h, w_post, gate);
  need_matrix(y, at::kBFloat16, rows, cols);
  need_vector(rstd, rows);
  need_weight(w_pre, cols);
  const int w_f32 = weight_type(w_pre, w_post);
  if (dy) need_matrix(dy, at::kBFloat16, rows, cols);
  if (h) need_matrix(h, at::kBFloat16, rows, cols);
  if (w_post) {
    need_weight(w_post, cols);
    if (!rstd_post) value_error("w_post needs the rstd_post of the forward pass");
    need_vector(rstd_post, rows);
  }
  const Gate g = gate_of(gate, rows, cols);
  if (dx) need_matrix(dx, at::kBFloat16, rows, cols);
  if (!h && res.out != Py_None) value_error("out holds the gradient of h, which is missing");
  if ((!w_post && dw_post) || (!gate && dgate)) value_error("dw_post and dgate need w_post and gate");
  if (accumulate && (!dw_pre || (w_post && !dw_post) || (g.kind == PURO_GATE_CHANNEL && !dgate)))
    value_error("accumulate=True needs the FP32 buffers to add into");
  if (dw_pre) need_vector(dw_pre, cols);
  if (dw_post) need_vector(dw_post, cols);
  const at::ScalarType gate_type = g.kind == PURO_GATE_FULL ? at::kBFloat16 : at::kFloat;
  if (dgate) {
    need_matrix(dgate, gate_type, gate.t->size(0), gate.t->size(1));
    if (g.kind == PURO_GATE_TOKEN && !dgate.t->is_contiguous()) value_error("dgate must be contiguous");
  }
  at::Tensor ndx, ndw_pre, ndw_post, ndgate;
  if (!dx) ndx = dev.empty({rows, cols}, at::kBFloat16);
  if (!dw_pre) ndw_pre = dev.empty({cols}, at::kFloat);
  if (w_post && !dw_post) ndw_post = dev.empty({cols}, at::kFloat);
  if (gate && !dgate) ndgate = dev.empty({gate.t->size(0), gate.t->size(1)}, gate_type);
  if (h) res.resolve(rows, cols, dev);
  const int64_t need = puro_fp8_residual_norm_workspace_bytes(rows, cols, h ? res.layout : 0, 1);
  at::Tensor ws = dev.empty({need > 16 ? need : 16}, at::kByte);
  void* stream = dev.stream();
  const int st = unlocked([&] {
    return puro_fp8_residual_norm_backward(
        dn.ptr(), dn.ld(), dy.ptr(), dy.ld(), y.ptr(), y.ld(), static_cast<const float*>(rstd.ptr()), h.ptr(), h.ld(),
        static_cast<const float*>(rstd_post.ptr()), w_pre.ptr(), w_post.ptr(), w_f32, gate.ptr(), g.ld, g.kind, g.f32,
        scale, rows, cols, Result::at_(dx, ndx), Result::ld_(dx, ndx),
        static_cast<float*>(Result::at_(dw_pre, ndw_pre)), static_cast<float*>(Result::at_(dw_post, ndw_post)),
        Result::at_(dgate, ndgate), Result::ld_(dgate, ndgate), accumulate, res.layout, h ? res.q_() : nullptr,
        h ? res.ld_q() : 0, h ? res.s_() : nullptr, h ? res.qt_() : nullptr, h ? res.ld_qt() : 0,
        h ? res.st_() : nullptr, h ? res.bf_() : nullptr, h ? res.ld_bf() : 0, ws.data_ptr(), stream);
  });
  return results(st, {&ndx, &ndw_pre, &ndw_post, &ndgate, &res.nq, &res.ns, &res.nqt, &res.nst, &res.nbf});
}

// gu, layout, out -> status, q, s, qt, st, bf16
PyObject* swiglu(PyObject* const* a, Py_ssize_t n) {
  need_count(n, 3);
  const Arg gu(a[0], "gu", false);
  Result res(a[2], integer(a[1], "layout"));
  const OnDevice dev("swiglu", {&gu, &res.q, &res.s, &res.qt, &res.st, &res.bf});
  need_any_matrix(gu);
  const int64_t rows = gu.t->size(0), f2 = gu.t->size(1);
  if (f2 % 2) value_error("gu must hold two halves of equal width, got %lld columns", (long long)f2);
  res.resolve(rows, f2 / 2, dev);
  void* stream = dev.stream();
  const int st = unlocked([&] {
    return puro_fp8_swiglu(gu.ptr(), gu.ld(), rows, f2 / 2, res.layout, res.q_(), res.ld_q(), res.s_(), res.qt_(),
                           res.ld_qt(), res.st_(), res.bf_(), res.ld_bf(), stream);
  });
  return results(st, {&res.nq, &res.ns, &res.nqt, &res.nst, &res.nbf});
}

// da, gu, layout, out -> status, q, s, qt, st, bf16
PyObject* swiglu_backward(PyObject* const* a, Py_ssize_t n) {
  need_count(n, 4);
  const Arg da(a[0], "da", false), gu(a[1], "gu", false);
  Result res(a[3], integer(a[2], "layout"));
  const OnDevice dev("swiglu_backward", {&da, &gu, &res.q, &res.s, &res.qt, &res.st, &res.bf});
  need_any_matrix(da);
  const int64_t rows = da.t->size(0), f = da.t->size(1);
  need_matrix(gu, at::kBFloat16, rows, 2 * f);
  res.resolve(rows, 2 * f, dev);
  void* stream = dev.stream();
  const int st = unlocked([&] {
    return puro_fp8_swiglu_backward(da.ptr(), da.ld(), gu.ptr(), gu.ld(), rows, f, res.layout, res.q_(), res.ld_q(),
                                    res.s_(), res.qt_(), res.ld_qt(), res.st_(), res.bf_(), res.ld_bf(), stream);
  });
  return results(st, {&res.nq, &res.ns, &res.nqt, &res.nst, &res.nbf});
}

// A row-major matrix of any row stride, also a view into a wider one: its row stride.
int64_t need_rows(const Arg& a) {
  const at::Tensor& t = *a.t;
  if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1) || (t.size(0) > 1 && t.stride(0) < t.size(1)))
    value_error("%s must be a row-major 2-D tensor", a.name);
  return t.size(0) > 1 ? t.stride(0) : std::max(t.stride(0), t.size(1));
}

// g, steps, a, b, c, eps, out, workspace -> status, out
PyObject* orthogonalize(PyObject* const* a, Py_ssize_t n_args) {
  need_count(n_args, 8);
  const Arg g(a[0], "g", false), out(a[6], "out"), workspace(a[7], "workspace");
  const int steps = integer(a[1], "steps");
  const float ca = (float)number(a[2]), cb = (float)number(a[3]), cc = (float)number(a[4]), eps = (float)number(a[5]);
  const OnDevice dev("orthogonalize", {&g, &out, &workspace});
  need_cuda(g);
  const at::ScalarType type = g.t->scalar_type();
  if (type != at::kFloat && type != at::kBFloat16)
    value_error("g must be torch.float32 or torch.bfloat16, got %s", type_name(type).c_str());
  const int64_t ld_g = need_rows(g), n = g.t->size(0), k = g.t->size(1);
  if (n > 65536 || k > 65536)
    value_error("g must be at most [65536, 65536], got [%lld, %lld]", (long long)n, (long long)k);
  if (steps < 1 || steps > 64) value_error("steps must be 1 to 64, got %d", steps);
  if (!(eps >= 0)) value_error("eps must not be negative");
  at::Tensor result;
  int64_t ld_out = k;
  if (out) {
    need_type(out, at::kBFloat16);
    ld_out = need_rows(out);
    if (out.t->size(0) != n || out.t->size(1) != k)
      value_error("out must be [%lld, %lld], got %s", (long long)n, (long long)k, shape_name(*out.t).c_str());
    const char *g0 = static_cast<const char*>(g.ptr()), *o0 = static_cast<const char*>(out.ptr());
    if (n && k && g0 < o0 + ((n - 1) * ld_out + k) * 2 && o0 < g0 + ((n - 1) * ld_g + k) * (type == at::kFloat ? 4 : 2))
      value_error("out must not overlap g");
  } else {
    result = dev.empty({n, k}, at::kBFloat16);
  }
  const int64_t need = puro_fp8_orthogonalize_workspace_bytes(n, k);
  at::Tensor ws;
  if (workspace) {
    need_bytes(workspace, need);
    if (reinterpret_cast<uintptr_t>(workspace.ptr()) % 256) value_error("workspace must start on a multiple of 256 bytes");
    const char *w0 = static_cast<const char*>(workspace.ptr()), *w1 = w0 + need;
    auto meets = [&](const Arg& a, int64_t ld, int64_t element) {
      const char* p0 = static_cast<const char*>(a.ptr());
      return n && k && w0 < p0 + ((n - 1) * ld + k) * element && p0 < w1;
    };
    if (meets(g, ld_g, type == at::kFloat ? 4 : 2)) value_error("workspace must not overlap g");
    if (out && meets(out, ld_out, 2)) value_error("workspace must not overlap out");
  } else {
    ws = dev.empty({need > 256 ? need : 256}, at::kByte);
  }
  void* stream = dev.stream();
  const int st = unlocked([&] {
    return puro_fp8_orthogonalize(g.ptr(), ld_g, type == at::kFloat, n, k, steps, ca, cb, cc, eps,
                                  Result::at_(out, result), ld_out, Result::at_(workspace, ws), stream);
  });
  return results(st, {&result});
}

#define ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<f>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(residual_norm), ENTRY(residual_norm_backward), ENTRY(swiglu), ENTRY(swiglu_backward),
                         ENTRY(orthogonalize),
                         {nullptr, nullptr, 0, nullptr}};
#undef ENTRY

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
