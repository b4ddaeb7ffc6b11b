// The row operators' calls (bs_grec, bs_gnorm, bs_gemm_q8 and bs_gdelta calls of bsolve.h) from Python: reads
// devices, types, shapes, row distances and pointers from torch tensors, checks them against each other and calls the
// C ABI. A call costs about 3 us with its launch; reading as much tensor by tensor in Python
// takes 5 us warm and twice that between a program's other work, more than a small call's kernel.
#include <Python.h>

#include <cmath>
#include <cstdint>
#include <stdexcept>
#include <string>
#include <tuple>
#include <vector>

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

  // dims 0: rows of elements, (rows, width) or (batch, length, width).
  Like(PyObject* o, const char* name, size_t dims = 0) {
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
    if (dims && shape.size() != dims)
      value_error(std::string(name) + ": shape " + text(shape) + ", expected " +
                  (dims == 4 ? "(batch, length, heads, size), or (rows, heads, size) with offsets"
                             : "(rows, heads, size)"));
    if (!dims && shape.size() != 2 && shape.size() != 3)
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

// A row operand of a type and shape, on the device, the last stride 1 and the rows at one distance.
// None: null.
Row row_of(PyObject* o, const char* name, const Like& like, at::ScalarType type,
           c10::IntArrayRef shape) {
  const at::Tensor* t = tensor(o, name);
  Row r;
  if (!t) return r;
  if (t->scalar_type() != type)
    type_error(std::string(name) + ": dtype " + c10::toString(t->scalar_type()) + ", expected " +
               c10::toString(type));
  const auto s = t->sizes();
  const int64_t width = shape.back();
  if (s != shape)
    value_error(std::string(name) + ": shape " + text(s) + ", expected " + text(shape));
  if (!t->is_cuda() || t->get_device() != like.device)
    value_error(std::string(name) + ": bsolve operands are device tensors of one device");
  const auto st = t->strides();
  if (width > 1 && st.back() != 1)
    value_error(std::string(name) + ": the elements of a row must be contiguous");
  if (s.size() == 3) {
    r.ld = s[1] > 1 ? st[1] : (s[0] > 1 ? st[0] : width);
    if (s[0] > 1 && s[1] > 1 && st[0] != s[1] * r.ld)
      value_error(std::string(name) + ": the rows of all sequences must lie at one distance");
  } else {
    r.ld = s[0] > 1 ? st[0] : width;
  }
  if (r.ld < width) {
    if (t->numel()) value_error(std::string(name) + ": rows overlap");
    r.ld = width;
  }
  r.p = address(*t, name);
  return r;
}
Row row(PyObject* o, const char* name, const Like& like) {
  return row_of(o, name, like, like.type, like.shape);
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

// The shape of rows that lie beside others', `width` elements each.
std::vector<int64_t> beside(c10::IntArrayRef shape, int64_t width) {
  std::vector<int64_t> v(shape.begin(), shape.end());
  v.back() = width;
  return v;
}

PyObject* gnorm_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("gnorm_q8", n, 12, [&] {
    const Like l(a[0], "f");
    const Row f = row(a[0], "f", l), q = row_of(a[1], "q", l, at::kFloat8_e4m3fn, l.shape),
              s = row_of(a[2], "scales", l, at::kFloat, beside(l.shape, (l.width + 127) / 128)),
              y = row(a[3], "y", l), z = row(a[4], "z", l), x = row(a[5], "x", l);
    const int w = static_cast<int>(l.width);
    return enter(l, bs_gnorm_q8_batched, l.code, l.rows(), w, f.p, f.ld, z.p, z.ld, x.p, x.ld,
                 f32(a[6], "w_post", l, w), f32(a[7], "scale", l, w), f32(a[8], "w_pre", l, w),
                 number(a[9]), static_cast<bs_gate>(small(a[10])), y.p, y.ld,
                 static_cast<uint8_t*>(q.p), q.ld, static_cast<float*>(s.p), s.ld, handle(a[11]));
  });
}

PyObject* gemm_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("gemm_q8", n, 6, [&] {
    const Like l(a[4], "y");
    const at::Tensor* w = tensor(a[2], "w");
    if (!w || w->dim() != 2)
      value_error("w: shape " + (w ? text(w->sizes()) : std::string("None")) + ", expected (n, k)");
    const int64_t k = w->size(1), blocks = (k + 127) / 128;
    const int64_t own[] = {l.width, k}, groups[] = {(l.width + 127) / 128, blocks};
    const Row y = row(a[4], "y", l),
              ra = row_of(a[0], "a", l, at::kFloat8_e4m3fn, beside(l.shape, k)),
              sa = row_of(a[1], "sa", l, at::kFloat, beside(l.shape, blocks)),
              rw = row_of(a[2], "w", l, at::kFloat8_e4m3fn, own),
              sw = row_of(a[3], "sw", l, at::kFloat, groups);
    // the rows of a contiguous tensor of another width than a multiple of 16 do not lie so
    for (auto [r, rows, name] : {std::tuple(&ra, l.rows(), "a"), std::tuple(&rw, own[0], "w")})
      if (k > 0 && rows > 1 && r->ld % 16)
        value_error(std::string(name) + ": rows " + std::to_string(r->ld) + " bytes apart, a multiple of 16 expected");
    return enter(l, bs_gemm_q8, l.code, l.rows(), l.width, k, static_cast<const uint8_t*>(ra.p), ra.ld,
                 static_cast<const float*>(sa.p), sa.ld, static_cast<const uint8_t*>(rw.p), rw.ld,
                 static_cast<const float*>(sw.p), sw.ld, y.p, y.ld, handle(a[5]));
  });
}

// Row operands of the gated delta rule: heads of contiguous elements, one after another in a row.
struct Heads {
  Like q;               // its shape: the rows' and (heads, elements)
  c10::IntArrayRef lead;  // the rows' part
  int64_t heads_k, dk, heads_v, dv, batch, rows;
  const int64_t* offsets = nullptr;

  // Of q and v; `packed`: with offsets, else (batch, length) or, for a step, (batch).
  Heads(PyObject* q_, PyObject* v_, PyObject* offsets_, bool step)
      : q(q_, "q", step || offsets_ != Py_None ? 3 : 4) {
    lead = q.shape.slice(0, q.shape.size() - 2);
    heads_k = q.shape[lead.size()], dk = q.width;
    const at::Tensor* v = tensor(v_, "v");
    if (!v) type_error("v: a torch tensor expected");
    if (v->dim() != static_cast<int64_t>(lead.size()) + 2)
      value_error("v: shape " + text(v->sizes()) + ", expected " + std::to_string(lead.size() + 2) +
                  " dimensions");
    heads_v = v->size(lead.size()), dv = v->size(lead.size() + 1);
    for (int64_t n : {heads_k, heads_v, dv})
      if (n > INT32_MAX) value_error("heads too many or too long");
    rows = lead[0] * (lead.size() == 2 ? lead[1] : 1);
    batch = lead[0];
    if (const at::Tensor* t = tensor(offsets_, "offsets")) {
      if (t->numel() < 1) value_error("offsets: batch + 1 row numbers expected");
      offsets = vec<int64_t>(offsets_, "offsets", q, t->numel(), at::kLong);
      batch = t->numel() - 1;
    }
  }

  // A row operand of `heads` x `size` elements a row (size 0: of `heads` numbers).
  Row row(PyObject* o, const char* name, int64_t heads, int64_t size, at::ScalarType type) const {
    const at::Tensor* t = tensor(o, name);
    if (!t) type_error(std::string(name) + ": a torch tensor expected");
    if (t->scalar_type() != type)
      type_error(std::string(name) + ": dtype " + c10::toString(t->scalar_type()) + ", expected " +
                 c10::toString(type));
    std::vector<int64_t> want(lead.begin(), lead.end());
    want.push_back(heads);
    if (size) want.push_back(size);
    const auto s = t->sizes(), st = t->strides();
    if (s != c10::IntArrayRef(want))
      value_error(std::string(name) + ": shape " + text(s) + ", expected " + text(want));
    if (!t->is_cuda() || t->get_device() != q.device)
      value_error(std::string(name) + ": bsolve operands are device tensors of one device");
    const size_t n = lead.size();
    const int64_t inner = size ? size : 1, width = heads * inner;
    if ((size > 1 && st[n + 1] != 1) || (heads > 1 && st[n] != inner))
      value_error(std::string(name) + ": the heads of a row must be contiguous");
    Row r;
    if (n == 2) {
      r.ld = s[1] > 1 ? st[1] : (s[0] > 1 ? st[0] : width);
      if (s[0] > 1 && s[1] > 1 && st[0] != s[1] * r.ld)
        value_error(std::string(name) + ": the rows of all sequences must lie at one distance");
    } else {
      r.ld = s[0] > 1 ? st[0] : width;
    }
    if (r.ld < width) {
      if (t->numel()) value_error(std::string(name) + ": rows overlap");
      r.ld = width;
    }
    r.p = address(*t, name);
    return r;
  }
  Row keys(PyObject* o, const char* name) const { return row(o, name, heads_k, dk, q.type); }
  Row values(PyObject* o, const char* name) const { return row(o, name, heads_v, dv, q.type); }
  Row gates(PyObject* o, const char* name) const { return row(o, name, heads_v, 0, at::kFloat); }
  int64_t states() const { return batch * heads_v * dk * dv; }
  double scale(PyObject* o) const {
    return o == Py_None ? 1.0 / std::sqrt(static_cast<double>(dk)) : number(o);
  }
};

// A buffer of at least `need` bytes. None: null.
void* bytes_of(PyObject* o, const char* name, const Like& like, size_t need, size_t* have = nullptr) {
  void* p = vec<void>(o, name, like, -1, at::kByte);
  const size_t n = p ? static_cast<size_t>(tensor(o, name)->numel()) : 0;
  if (p && n < need)
    value_error(std::string(name) + ": " + std::to_string(n) + " bytes, " + std::to_string(need) +
                " needed");
  if (have) *have = n;
  return p;
}

PyObject* gdelta(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("gdelta", n, 13, [&] {
    const Heads s(a[0], a[2], a[9], false);
    const Row q = s.keys(a[0], "q"), k = s.keys(a[1], "k"), v = s.values(a[2], "v"),
              g = s.gates(a[3], "g"), beta = s.gates(a[4], "beta"), o = s.values(a[5], "o");
    size_t bytes = 0;
    void* work = bytes_of(a[6], "work", s.q, bs_gdelta_workspace(s.heads_v, s.batch, s.rows), &bytes);
    return enter(
        s.q, bs_gdelta_batched, s.q.code, static_cast<int>(s.heads_k), static_cast<int>(s.heads_v),
        static_cast<int>(s.dk), static_cast<int>(s.dv), s.batch, s.rows, s.offsets, q.p, q.ld, k.p,
        k.ld, v.p, v.ld, static_cast<float*>(g.p), g.ld, static_cast<float*>(beta.p), beta.ld,
        s.scale(a[11]), f32(a[7], "h0", s.q, s.states()), o.p, o.ld,
        f32(a[8], "hT", s.q, s.states()),
        bytes_of(a[10], "tape", s.q, bs_gdelta_tape(s.heads_v, s.dk, s.dv, s.batch, s.rows)), work,
        bytes, handle(a[12]));
  });
}

PyObject* gdelta_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("gdelta_backward", n, 18, [&] {
    const Heads s(a[0], a[2], a[15], false);
    const Row q = s.keys(a[0], "q"), k = s.keys(a[1], "k"), v = s.values(a[2], "v"),
              g = s.gates(a[3], "g"), beta = s.gates(a[4], "beta"), o = s.values(a[6], "do"),
              dq = s.keys(a[7], "dq"), dk = s.keys(a[8], "dk"), dv = s.values(a[9], "dv"),
              dg = s.gates(a[10], "dg"), dbeta = s.gates(a[11], "dbeta");
    size_t bytes = 0;
    void* work = bytes_of(
        a[12], "work", s.q, bs_gdelta_backward_workspace(s.heads_v, s.dk, s.dv, s.batch, s.rows), &bytes);
    return enter(
        s.q, bs_gdelta_backward_batched, s.q.code, static_cast<int>(s.heads_k),
        static_cast<int>(s.heads_v), static_cast<int>(s.dk), static_cast<int>(s.dv), s.batch, s.rows,
        s.offsets, q.p, q.ld, k.p, k.ld, v.p, v.ld, static_cast<float*>(g.p), g.ld,
        static_cast<float*>(beta.p), beta.ld, s.scale(a[16]),
        bytes_of(a[5], "tape", s.q, bs_gdelta_tape(s.heads_v, s.dk, s.dv, s.batch, s.rows)), o.p, o.ld,
        f32(a[13], "dhT", s.q, s.states()), dq.p, dq.ld, dk.p, dk.ld, dv.p, dv.ld,
        static_cast<float*>(dg.p), dg.ld, static_cast<float*>(dbeta.p), dbeta.ld,
        f32(a[14], "dh0", s.q, s.states()), work, bytes, handle(a[17]));
  });
}

PyObject* gdelta_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("gdelta_step", n, 10, [&] {
    const Heads s(a[0], a[2], Py_None, true);
    const Row q = s.keys(a[0], "q"), k = s.keys(a[1], "k"), v = s.values(a[2], "v"),
              g = s.gates(a[3], "g"), beta = s.gates(a[4], "beta"), o = s.values(a[6], "o");
    const at::Tensor* state = tensor(a[5], "state");
    const int64_t want[] = {state && state->dim() ? state->size(0) : 0, s.heads_v, s.dk, s.dv};
    if (!state || state->sizes() != c10::IntArrayRef(want))
      value_error("state: shape " + (state ? text(state->sizes()) : std::string("None")) +
                  ", expected (num_slots, heads_v, dk, dv)");
    return enter(
        s.q, bs_gdelta_step_batched, s.q.code, static_cast<int>(s.heads_k),
        static_cast<int>(s.heads_v), static_cast<int>(s.dk), static_cast<int>(s.dv), s.batch, q.p,
        q.ld, k.p, k.ld, v.p, v.ld, static_cast<float*>(g.p), g.ld, static_cast<float*>(beta.p),
        beta.ld, s.scale(a[8]), f32(a[5], "state", s.q, state->numel()), want[0],
        vec<int32_t>(a[7], "slots", s.q, s.batch, at::kInt), o.p, o.ld, handle(a[9]));
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

PyObject* gdelta_workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return query(n, 3, [&] {
    return bs_gdelta_workspace(small(a[0]), integer(a[1]), integer(a[2]));
  });
}
PyObject* gdelta_tape(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return query(n, 5, [&] {
    return bs_gdelta_tape(small(a[0]), small(a[1]), small(a[2]), integer(a[3]), integer(a[4]));
  });
}

PyObject* gdelta_backward_workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return query(n, 5, [&] {
    return bs_gdelta_backward_workspace(small(a[0]), small(a[1]), small(a[2]), integer(a[3]),
                                        integer(a[4]));
  });
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
                         method<gnorm_q8>("gnorm_q8"), method<gemm_q8>("gemm_q8"),
                         method<gdelta>("gdelta"), method<gdelta_step>("gdelta_step"),
                         method<gdelta_backward>("gdelta_backward"),
                         method<gdelta_backward_workspace>("gdelta_backward_workspace"),
                         method<gdelta_workspace>("gdelta_workspace"),
                         method<gdelta_tape>("gdelta_tape"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rowcall", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rowcall() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "target", BSOLVE_ROWCALL_TARGET) != 0) Py_CLEAR(m);
  return m;
}
