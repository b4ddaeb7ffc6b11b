// The row operators' calls (bs_grec and bs_gnorm calls of bsolve.h) from Python: reads devices, types,
// shapes, row distances and pointers from torch tensors, checks them against each other and calls the
// C ABI. A call costs about 3 us with its launch; reading as much tensor by tensor in Python
// takes 5 us warm and twice that between a program's other work, more than a small call's kernel.
#include <Python.h>

#include <cstdint>
#include <stdexcept>
#include <string>

#include <ATen/core/Tensor.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include "bsolve.h"

namespace {

struct Refused {};  // a Python error is set

[[noreturn]] void type_error(const std::string& what) {
  PyErr_SetString(PyExc_TypeError, what.c_str());
  throw Refused();
}
[[noreturn]] void value_error(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Refused();
}

std::string text(c10::IntArrayRef s) {
  std::string t = "(";
  for (size_t k = 0; k < s.size(); ++k) t += (k ? ", " : "") + std::to_string(s[k]);
  return t + ")";
}

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) type_error(std::string(name) + ": a torch tensor expected");
  return &THPVariable_Unpack(o);
}

// The operand that the others are compared with.
struct Like {
  at::ScalarType type;
  c10::IntArrayRef shape;
  int64_t device;
  int64_t width;
  bs_dtype code;

  Like(PyObject* o, const char* name) {
    const at::Tensor* t = tensor(o, name);
    if (!t) type_error(std::string(name) + ": a torch tensor expected");
    type = t->scalar_type();
    switch (type) {
      case at::kFloat: code = BS_FP32; break;
      case at::kBFloat16: code = BS_BF16; break;
      case at::kHalf: code = BS_FP16; break;
      default:
        type_error(std::string("unsupported dtype ") + c10::toString(type) +
                   ": float32, bfloat16 or float16");
    }
    shape = t->sizes();
    if (shape.size() != 2 && shape.size() != 3)
      value_error(std::string(name) + ": shape " + text(shape) +
                  ", expected (rows, width) or (batch, length, width)");
    if (!t->is_cuda())
      value_error(std::string(name) + ": bsolve operands are device tensors of one device");
    device = t->get_device();
    width = shape.back();
    if (width > INT32_MAX) value_error(std::string(name) + ": rows too long");
  }
  int64_t rows() const { return shape.size() == 3 ? shape[0] * shape[1] : shape[0]; }
};

// The address of a tensor's first element, as stored: a view that torch reads with the other sign
// (the imaginary part of a conjugate) would be taken for its negative.
void* address(const at::Tensor& t, const char* name) {
  if (t.is_neg())
    value_error(std::string(name) + ": a view with a pending sign; resolve_neg() it first");
  return t.data_ptr();
}

struct Row {
  void* p = nullptr;
  int64_t ld = 0;
};

// A row operand: of the type and shape, on the device, the last stride 1 and the rows at one
// distance. None: null.
Row row(PyObject* o, const char* name, const Like& like) {
  const at::Tensor* t = tensor(o, name);
  Row r;
  if (!t) return r;
  if (t->scalar_type() != like.type)
    type_error(std::string(name) + ": dtype " + c10::toString(t->scalar_type()) + ", expected " +
               c10::toString(like.type));
  const auto s = t->sizes();
  if (s != like.shape)
    value_error(std::string(name) + ": shape " + text(s) + ", expected " + text(like.shape));
  if (!t->is_cuda() || t->get_device() != like.device)
    value_error(std::string(name) + ": bsolve operands are device tensors of one device");
  const auto st = t->strides();
  if (like.width > 1 && st.back() != 1)
    value_error(std::string(name) + ": the elements of a row must be contiguous");
  if (s.size() == 3) {
    r.ld = s[1] > 1 ? st[1] : (s[0] > 1 ? st[0] : like.width);
    if (s[0] > 1 && s[1] > 1 && st[0] != s[1] * r.ld)
      value_error(std::string(name) + ": the rows of all sequences must lie at one distance");
  } else {
    r.ld = s[0] > 1 ? st[0] : like.width;
  }
  if (r.ld < like.width) {
    if (t->numel()) value_error(std::string(name) + ": rows overlap");
    r.ld = like.width;
  }
  r.p = address(*t, name);
  return r;
}

// A contiguous operand of numel elements. None: null.
template <typename V>
V* vec(PyObject* o, const char* name, const Like& like, int64_t numel, at::ScalarType type) {
  const at::Tensor* t = tensor(o, name);
  if (!t) return nullptr;
  if (t->scalar_type() != type)
    type_error(std::string(name) + ": dtype " + c10::toString(t->scalar_type()) + ", expected " +
               c10::toString(type));
  if (numel >= 0 && t->numel() != numel)
    value_error(std::string(name) + ": " + std::to_string(t->numel()) + " elements, expected " +
                std::to_string(numel));
  if (!t->is_cuda() || t->get_device() != like.device)
    value_error(std::string(name) + ": bsolve operands are device tensors of one device");
  if (!t->is_contiguous()) value_error(std::string(name) + ": must be contiguous");
  return static_cast<V*>(address(*t, name));
}
float* f32(PyObject* o, const char* name, const Like& like, int64_t numel) {
  return vec<float>(o, name, like, numel, at::kFloat);
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}
long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
// An int argument: what does not fit is -1, which the calls refuse.
int small(PyObject* o) {
  const long long v = integer(o);
  return v < INT32_MIN || v > INT32_MAX ? -1 : static_cast<int>(v);
}
void* handle(PyObject* o) {
  void* v = PyLong_AsVoidPtr(o);
  if (!v && PyErr_Occurred()) throw Refused();
  return v;
}

// Sequences of a recurrence call.
struct Sequences {
  int64_t batch, rows;
  const int64_t* offsets = nullptr;

  Sequences(const Like& x, PyObject* o) {
    const at::Tensor* t = tensor(o, "offsets");
    if (!t) {
      if (x.shape.size() != 3)
        value_error("x: shape " + text(x.shape) +
                    ", expected (batch, length, channels), or (rows, channels) with offsets");
      batch = x.shape[0];
      rows = batch * x.shape[1];
      return;
    }
    if (x.shape.size() != 2)
      value_error("x: shape " + text(x.shape) + ", expected (rows, channels) with offsets");
    if (t->numel() < 1) value_error("offsets: batch + 1 row numbers expected");
    offsets = vec<int64_t>(o, "offsets", x, t->numel(), at::kLong);
    batch = t->numel() - 1;
    rows = x.shape[0];
  }
};

// Makes a device current while it lives.
class OnDevice {
 public:
  explicit OnDevice(int64_t device) {
    check(cudaGetDevice(&before_));
    if (device == before_) return;
    check(cudaSetDevice(static_cast<int>(device)));
    changed_ = true;
  }
  ~OnDevice() {
    if (changed_) cudaSetDevice(before_);
  }
  OnDevice(const OnDevice&) = delete;
  OnDevice& operator=(const OnDevice&) = delete;

 private:
  static void check(cudaError_t e) {
    if (e != cudaSuccess) throw std::runtime_error(cudaGetErrorString(e));
  }
  int before_ = 0;
  bool changed_ = false;
};

// Lets the program's other threads run: a launch behind a full queue waits for the GPU.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

// An entry of the C ABI, its arguments all worked out, on the operands' device: the entries launch
// on the current one, and the null stream that they are often given is every device's.
template <typename... P, typename... A>
bs_status enter(const Like& like, bs_status (*entry)(P...), A... args) {
  const Unlocked unlocked;
  const OnDevice device(like.device);
  return entry(args...);
}

template <typename F>
PyObject* guarded(const char* name, Py_ssize_t given, Py_ssize_t wanted, F&& f) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%s: %zd arguments, %zd expected", name, given, wanted);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* grec(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("grec", n, 11, [&] {
    const Like l(a[0], "x");
    const Sequences s(l, a[7]);
    const Row x = row(a[0], "x", l), r = row(a[1], "r", l), i = row(a[2], "i", l),
              h = row(a[4], "h", l);
    const int c = static_cast<int>(l.width);
    return enter(
        l, bs_grec_batched, l.code, c, s.batch, s.rows, s.offsets, x.p, x.ld, r.p, r.ld, i.p, i.ld,
        f32(a[3], "lam", l, c), number(a[9]), f32(a[5], "h0", l, s.batch * c), h.p, h.ld,
        f32(a[6], "hT", l, s.batch * c),
        f32(a[8], "tape", l, bs_grec_tape_rows(s.batch, s.rows) * c), handle(a[10]));
  });
}

PyObject* grec_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("grec_backward", n, 16, [&] {
    const Like l(a[0], "x");
    const Sequences s(l, a[13]);
    const Row x = row(a[0], "x", l), r = row(a[1], "r", l), i = row(a[2], "i", l),
              dh = row(a[5], "dh", l), dx = row(a[6], "dx", l), dr = row(a[7], "dr", l),
              di = row(a[8], "di", l);
    const int c = static_cast<int>(l.width);
    void* work = vec<void>(a[10], "work", l, -1, at::kByte);
    const size_t bytes = work ? static_cast<size_t>(tensor(a[10], "work")->numel()) : 0;
    return enter(
        l, bs_grec_backward_batched, l.code, c, s.batch, s.rows, s.offsets, x.p, x.ld, r.p, r.ld,
        i.p, i.ld, f32(a[3], "lam", l, c), number(a[14]),
        f32(a[4], "tape", l, bs_grec_tape_rows(s.batch, s.rows) * c), dh.p, dh.ld,
        f32(a[11], "dhT", l, s.batch * c), dx.p, dx.ld, dr.p, dr.ld, di.p, di.ld,
        f32(a[9], "dlam", l, c), f32(a[12], "dh0", l, s.batch * c), work, bytes, handle(a[15]));
  });
}

PyObject* grec_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("grec_step", n, 9, [&] {
    const Like l(a[0], "x");
    if (l.shape.size() != 2)
      value_error("x: shape " + text(l.shape) + ", expected (batch, channels)");
    const Row x = row(a[0], "x", l), r = row(a[1], "r", l), i = row(a[2], "i", l),
              y = row(a[5], "y", l);
    const int64_t batch = l.shape[0], c = l.width;
    const at::Tensor* state = tensor(a[4], "state");
    if (!state || state->dim() != 2 || state->size(1) != c)
      value_error("state: shape " + (state ? text(state->sizes()) : std::string("None")) +
                  ", expected (num_slots, " + std::to_string(c) + ")");
    return enter(
        l, bs_grec_step_batched, l.code, static_cast<int>(c), batch, x.p, x.ld, r.p, r.ld, i.p,
        i.ld, f32(a[3], "lam", l, c), number(a[7]), f32(a[4], "state", l, state->size(0) * c),
        state->size(0), vec<int32_t>(a[6], "slots", l, batch, at::kInt), y.p, y.ld, handle(a[8]));
  });
}

PyObject* gnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("gnorm", n, 11, [&] {
    const Like l(a[0], "f");
    const Row f = row(a[0], "f", l), y = row(a[1], "y", l), z = row(a[2], "z", l),
              x = row(a[3], "x", l), u = row(a[7], "u", l);
    const int w = static_cast<int>(l.width);
    return enter(
        l, bs_gnorm_batched, l.code, l.rows(), w, f.p, f.ld, z.p, z.ld, x.p, x.ld,
        f32(a[4], "w_post", l, w), f32(a[5], "scale", l, w), f32(a[6], "w_pre", l, w),
        number(a[8]), static_cast<bs_gate>(small(a[9])), y.p, y.ld, u.p, u.ld, handle(a[10]));
  });
}

PyObject* gnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("gnorm_backward", n, 18, [&] {
    const Like l(a[0], "f");
    const Row f = row(a[0], "f", l), dy = row(a[1], "dy", l), df = row(a[2], "df", l),
              z = row(a[4], "z", l), x = row(a[5], "x", l), du = row(a[9], "du", l),
              dz = row(a[10], "dz", l), dx = row(a[11], "dx", l);
    const int w = static_cast<int>(l.width);
    void* work = vec<void>(a[3], "work", l, -1, at::kByte);
    const size_t bytes = work ? static_cast<size_t>(tensor(a[3], "work")->numel()) : 0;
    return enter(
        l, bs_gnorm_backward_batched, l.code, l.rows(), w, f.p, f.ld, z.p, z.ld, x.p, x.ld,
        f32(a[6], "w_post", l, w), f32(a[7], "scale", l, w), f32(a[8], "w_pre", l, w), number(a[15]),
        static_cast<bs_gate>(small(a[16])), dy.p, dy.ld, du.p, du.ld, df.p, df.ld, dz.p, dz.ld,
        dx.p, dx.ld, f32(a[12], "dw_post", l, w), f32(a[13], "dscale", l, w),
        f32(a[14], "dw_pre", l, w), work, bytes, handle(a[17]));
  });
}

// The size queries: n integers in, one out.
template <typename F>
PyObject* query(Py_ssize_t given, Py_ssize_t wanted, F&& f) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", given, wanted);
    return nullptr;
  }
  try {
    return PyLong_FromLongLong(static_cast<long long>(f()));
  } catch (const Refused&) {
    return nullptr;
  }
}

PyObject* grec_tape_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return query(n, 2, [&] { return bs_grec_tape_rows(integer(a[0]), integer(a[1])); });
}
PyObject* grec_backward_workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return query(n, 3, [&] {
    return bs_grec_backward_workspace(small(a[0]), integer(a[1]), integer(a[2]));
  });
}
PyObject* gnorm_backward_workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return query(n, 2, [&] { return bs_gnorm_backward_workspace(small(a[0]), integer(a[1])); });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL,
          nullptr};
}

PyMethodDef methods[] = {method<grec>("grec"), method<grec_backward>("grec_backward"),
                         method<grec_step>("grec_step"), method<gnorm>("gnorm"),
                         method<gnorm_backward>("gnorm_backward"),
                         method<grec_tape_rows>("grec_tape_rows"),
                         method<grec_backward_workspace>("grec_backward_workspace"),
                         method<gnorm_backward_workspace>("gnorm_backward_workspace"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rowcall", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rowcall() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "target", BSOLVE_ROWCALL_TARGET) != 0) Py_CLEAR(m);
  return m;
}
