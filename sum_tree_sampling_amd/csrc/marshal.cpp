// marshal.cpp -- Python binding of include/per_train.h and include/per_block.h: takes tensors, checks
// them, and passes pointers, sizes and strides to the C entry points.
//
// The smallest of these calls take 3 us on the device; the same checks written
// in Python over ctypes took 6 to 12 us per call on the host and set the pace.
// The C entry points are given by address (bind), so the extension links
// against no other library of this package; a loader set from Python binds them
// at the first call.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <c10/core/AutogradState.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/per_block.h"

namespace {

using at::Tensor;

#define ENTRY_POINTS(X)                                                                     \
  X(per_rows_write) X(per_rows_write_at) X(per_rows_read) X(per_scan_workspace_bytes)       \
  X(per_scan_forward) X(per_scan_backward) X(per_scan_step) X(per_distill_workspace_bytes)  \
  X(per_distill) X(per_distill_forward) X(per_distill_backward) X(per_embed_forward)        \
  X(per_embed_workspace_bytes) X(per_embed_backward) X(per_norm_forward)                    \
  X(per_norm_workspace_bytes) X(per_norm_backward) X(per_delta_workspace_bytes)             \
  X(per_delta_forward) X(per_delta_backward) X(per_delta_step) X(per_last_error)

struct Api {
#define MEMBER(name) decltype(&::name) name = nullptr;
  ENTRY_POINTS(MEMBER)
#undef MEMBER
} api;
PyObject* per_error = nullptr;
PyObject* loader = nullptr;  // called once, before the first call, to bind

// A failed check, and a status code of the library.
struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct Failed {
  int code;
};
[[noreturn]] void refuse(const std::string& what) { throw Refused(what); }
void check(int rc) {
  if (rc != PER_OK) throw Failed{rc};
}

// ------------------------------------------------------------------ arguments

constexpr int kMaxArgs = 18;

// Arguments of one call by position in `names`; NULL where not given or None.
struct Args {
  PyObject* v[kMaxArgs] = {};
  const char* const* names;

  Args(const char* fn, const char* const* names_, PyObject** interned, int n, int required,
       PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames)
      : names(names_) {
    if (nargs > n) refuse(std::string(fn) + " takes at most " + std::to_string(n) + " arguments");
    for (Py_ssize_t i = 0; i < nargs; ++i) v[i] = args[i];
    const Py_ssize_t nk = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t k = 0; k < nk; ++k) {
      PyObject* name = PyTuple_GET_ITEM(kwnames, k);
      int at = -1;
      for (int i = 0; i < n && at < 0; ++i)
        if (interned[i] == name) at = i;
      for (int i = 0; i < n && at < 0; ++i)
        if (PyUnicode_Compare(interned[i], name) == 0) at = i;
      if (at < 0)
        refuse(std::string(fn) + " has no argument " + (PyUnicode_AsUTF8(name) ? PyUnicode_AsUTF8(name) : "?"));
      if (at < nargs || v[at]) refuse(std::string(fn) + ": " + names[at] + " is given twice");
      v[at] = args[nargs + k];
    }
    for (int i = 0; i < n; ++i) {
      if (v[i] == Py_None) v[i] = nullptr;
      if (i < required && !v[i]) refuse(std::string(fn) + ": " + names[i] + " is required");
    }
  }

  // The tensor of argument i (which must be given).
  const Tensor& tensor(int i) const {
    if (!THPVariable_Check(v[i])) refuse(std::string(names[i]) + " must be a tensor");
    return THPVariable_Unpack(v[i]);
  }
  int64_t integer(int i, int64_t otherwise) const {
    if (!v[i]) return otherwise;
    PyObject* n = PyNumber_Index(v[i]);
    if (!n) {
      PyErr_Clear();
      refuse(std::string(names[i]) + " must be an integer");
    }
    int over = 0;
    const long long x = PyLong_AsLongLongAndOverflow(n, &over);
    Py_DECREF(n);
    if (over) refuse(std::string(names[i]) + " is out of range");
    return x;
  }
  double real(int i, double otherwise) const {
    if (!v[i]) return otherwise;
    const double x = PyFloat_AsDouble(v[i]);
    if (x == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse(std::string(names[i]) + " must be a number");
    }
    return x;
  }
};

// The device and stream a call runs on, and where its outputs are allocated.
struct Where {
  int device = -2;  // no tensor lies there
  hipStream_t stream = nullptr;
  c10::hip::OptionalHIPStreamGuard guard;

  explicit Where(PyObject* s, const Tensor& first, const char* name) {
    // A tensor on the host is refused before anything touches a device.
    if (!first.is_cuda()) refuse(std::string(name) + " must be a tensor on the current device");
    device = c10::hip::current_device();
    if (first.get_device() != device)
      refuse(std::string(name) + " must be a tensor on the current device");
    if (!s) {
      stream = c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
      return;
    }
    PyObject* raw = PyLong_Check(s) ? (Py_INCREF(s), s) : PyObject_GetAttrString(s, "cuda_stream");
    if (!raw) {
      PyErr_Clear();
      refuse("stream must be a stream or its address");
    }
    stream = static_cast<hipStream_t>(PyLong_AsVoidPtr(raw));
    Py_DECREF(raw);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      refuse("stream must be a stream or its address");
    }
    guard.reset_stream(stream ? c10::hip::getStreamFromExternal(stream, (c10::DeviceIndex)device)
                              : c10::hip::getDefaultHIPStream((c10::DeviceIndex)device));
  }
  Tensor empty(at::IntArrayRef shape, at::ScalarType dtype) const {
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(at::kCUDA, device));
  }
};

std::string text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

void expect(const Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape,
            const Where& w) {
  if (!t.is_cuda() || t.get_device() != w.device)
    refuse(std::string(name) + " must be a tensor on the current device");
  if (t.scalar_type() != dtype)
    refuse(std::string(name) + " has type " + c10::toString(t.scalar_type()) + ", expected " +
           c10::toString(dtype));
  if (t.sizes() != shape)
    refuse(std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(shape));
}

// A dense tensor's data.
template <typename P>
P* dense(const Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape,
         const Where& w) {
  expect(t, name, dtype, shape, w);
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return static_cast<P*>(t.data_ptr());
}
// The same of an argument that may be left out.
template <typename P>
P* dense(const Args& a, int i, at::ScalarType dtype, at::IntArrayRef shape, const Where& w) {
  return a.v[i] ? dense<P>(a.tensor(i), a.names[i], dtype, shape, w) : nullptr;
}
const uint8_t* flags(const Args& a, int i, at::IntArrayRef shape, const Where& w) {
  if (!a.v[i]) return nullptr;
  const bool byte = a.tensor(i).scalar_type() == at::kByte;
  return dense<const uint8_t>(a, i, byte ? at::kByte : at::kBool, shape, w);
}

int type_of(const Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kFloat: return PER_F32;
    case at::kBFloat16: return PER_BF16;
    case at::kHalf: return PER_F16;
    default: refuse(std::string(name) + " must be float32, bfloat16 or float16");
  }
}

// A matrix with unit column stride: data and stride between rows.
struct Matrix {
  void* p;
  int64_t stride;
};
Matrix matrix(const Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape,
              const Where& w) {
  expect(t, name, dtype, shape, w);
  if (shape[1] > 1 && t.stride(1) != 1)
    refuse(std::string(name) + " must have unit stride in its last dimension");
  return {t.data_ptr(), shape[0] > 1 ? t.stride(0) : std::max(shape[1], t.stride(0))};
}
// [B x T x D] with unit channel stride.
struct View {
  void* p;
  int64_t sb, st;
};
View view(const Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape,
          const Where& w) {
  expect(t, name, dtype, shape, w);
  if (shape[2] > 1 && t.stride(2) != 1)
    refuse(std::string(name) + " must have unit stride in its last dimension");
  return {t.data_ptr(), t.stride(0), t.stride(1)};
}

// An output: the tensor given, or a new one.
Tensor output(const Args& a, int i, at::IntArrayRef shape, at::ScalarType dtype, const Where& w) {
  return a.v[i] ? a.tensor(i) : w.empty(shape, dtype);
}

PyObject* pair(const Tensor& a, const Tensor& b) {
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
  return t;
}
PyObject* triple(const Tensor& a, const Tensor& b, const Tensor& c) {
  PyObject* t = PyTuple_New(3);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
  PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(c));
  return t;
}

// ------------------------------------------------------------ 8-bit row store

struct Store {
  int64_t capacity, dim;
  int format, group;
  Matrix codes, scales;
};
Store store(const Tensor& codes, const Tensor& scales, int64_t group, const Where& w) {
  Store s;
  const auto t = codes.scalar_type();
  if (codes.dim() != 2 || (t != at::kFloat8_e4m3fn && t != at::kChar))
    refuse("codes must be [capacity x dim], float8_e4m3fn or int8");
  if (group != 0 && group != 32 && group != 64 && group != 128)
    refuse("group is 0 (the row), 32, 64 or 128");
  s.capacity = codes.size(0);
  s.dim = codes.size(1);
  s.format = t == at::kChar ? PER_I8 : PER_E4M3;
  s.group = (int)group;
  s.codes = matrix(codes, "codes", t, codes.sizes(), w);
  const int64_t shape[] = {s.capacity, group ? (s.dim + group - 1) / group : 1};
  s.scales = matrix(scales, "scales", at::kFloat, shape, w);
  return s;
}
#define STORE(s)                                                                            \
  s.capacity, s.dim, s.format, s.group, static_cast<uint8_t*>(s.codes.p), s.codes.stride,  \
      static_cast<float*>(s.scales.p), s.scales.stride

Matrix source(const Tensor& src, int64_t dim, const Where& w) {
  if (src.dim() != 2) refuse("src must be [count x dim]");
  const int64_t shape[] = {src.size(0), dim};
  return matrix(src, "src", src.scalar_type(), shape, w);
}

// codes, scales, src, first = 0, group = 128, stream = None
PyObject* rows_write(const Args& a) {
  const Tensor &codes = a.tensor(0), &src = a.tensor(2);
  const Where w(a.v[5], codes, "codes");
  const Store s = store(codes, a.tensor(1), a.integer(4, 128), w);
  const int type = type_of(src, "src");
  const Matrix m = source(src, s.dim, w);
  check(api.per_rows_write(STORE(s), src.size(0), a.integer(3, 0), m.p, type, m.stride, w.stream));
  Py_RETURN_NONE;
}

// codes, scales, src, slots, claims, group = 128, stream = None
PyObject* rows_write_at(const Args& a) {
  const Tensor &codes = a.tensor(0), &src = a.tensor(2);
  const Where w(a.v[6], codes, "codes");
  const Store s = store(codes, a.tensor(1), a.integer(5, 128), w);
  const int type = type_of(src, "src");
  const Matrix m = source(src, s.dim, w);
  const int64_t n = src.size(0);
  check(api.per_rows_write_at(STORE(s), n, dense<const int64_t>(a, 3, at::kLong, {n}, w),
                              dense<uint32_t>(a, 4, at::kInt, {s.capacity}, w), m.p, type, m.stride,
                              w.stream));
  Py_RETURN_NONE;
}

// codes, scales, idx, window = 1, group = 128, out = None, dtype = float32, stream = None
PyObject* rows_read(const Args& a) {
  const Tensor &codes = a.tensor(0), &idx = a.tensor(2);
  const Where w(a.v[7], codes, "codes");
  const Store s = store(codes, a.tensor(1), a.integer(4, 128), w);
  if (idx.dim() != 1) refuse("idx must be [B]");
  const int64_t B = idx.size(0), window = a.integer(3, 1);
  if (window < 1) refuse("window is at least 1");
  at::ScalarType dtype = at::kFloat;
  if (a.v[6]) {
    if (!THPDtype_Check(a.v[6])) refuse("dtype must be a torch.dtype");
    dtype = reinterpret_cast<THPDtype*>(a.v[6])->scalar_type;
    if (dtype != at::kFloat && dtype != at::kBFloat16 && dtype != at::kHalf)
      refuse("dtype must be float32, bfloat16 or float16");
  }
  const int64_t shape[] = {B, window, s.dim};
  const Tensor out = output(a, 5, shape, dtype, w);
  const int type = type_of(out, "out");
  check(api.per_rows_read(STORE(s), B, dense<const int64_t>(idx, "idx", at::kLong, {B}, w), window,
                          dense<void>(out, "out", out.scalar_type(), shape, w), type, s.dim,
                          w.stream));
  return THPVariable_Wrap(out);
}

// ----------------------------------------------------- gated linear recurrence

int64_t scan_bytes(int64_t B, int64_t T, int64_t D) {
  size_t n = 0;
  check(api.per_scan_workspace_bytes(B, T, D, &n));
  return (int64_t)n;
}

struct Sequences {
  int64_t B, T, D, chunks;
  int type;
  at::ScalarType dtype;
  View x, g;
};
Sequences sequences(const Args& a, const Where& w) {
  const Tensor& x = a.tensor(0);
  if (x.dim() != 3) refuse("x must be [B x T x D]");
  Sequences s;
  s.type = type_of(x, "x");
  s.dtype = x.scalar_type();
  s.B = x.size(0);
  s.T = x.size(1);
  s.D = x.size(2);
  s.chunks = (s.T + PER_SCAN_CHUNK - 1) / PER_SCAN_CHUNK;
  s.x = view(x, "x", s.dtype, x.sizes(), w);
  s.g = view(a.tensor(1), "g", s.dtype, x.sizes(), w);
  return s;
}

// x, g, reset, length, h0, y, h_last, carries, stream
PyObject* scan_forward(const Args& a) {
  const Where w(a.v[8], a.tensor(0), "x");
  const Sequences s = sequences(a, w);
  const int64_t all[] = {s.B, s.T, s.D}, state[] = {s.B, s.D}, carry[] = {s.B, s.chunks, s.D};
  const uint8_t* reset = flags(a, 2, {s.B, s.T}, w);
  const auto* length = dense<const int64_t>(a, 3, at::kLong, {s.B}, w);
  const auto* h0 = dense<const float>(a, 4, at::kFloat, state, w);
  const Tensor y = output(a, 5, all, s.dtype, w), h = output(a, 6, state, at::kFloat, w),
               c = output(a, 7, carry, at::kFloat, w);
  const View vy = view(y, "y", s.dtype, all, w);
  float* ph = dense<float>(h, "h_last", at::kFloat, state, w);
  float* pc = dense<float>(c, "carries", at::kFloat, carry, w);
  const int64_t bytes = scan_bytes(s.B, s.T, s.D);
  Tensor ws;
  if (bytes) ws = w.empty({bytes}, at::kByte);
  check(api.per_scan_forward(s.B, s.T, s.D, s.type, s.x.p, s.x.sb, s.x.st, s.g.p, s.g.sb, s.g.st,
                             reset, length, h0, vy.p, vy.sb, vy.st, ph, pc,
                             bytes ? ws.data_ptr() : nullptr, (size_t)bytes, w.stream));
  return triple(y, h, c);
}

// x, g, carries, dy, reset, length, dh_last, dx, dg, dh0, stream
PyObject* scan_backward(const Args& a) {
  const Where w(a.v[10], a.tensor(0), "x");
  const Sequences s = sequences(a, w);
  const int64_t all[] = {s.B, s.T, s.D}, state[] = {s.B, s.D}, carry[] = {s.B, s.chunks, s.D};
  const auto* pc = dense<const float>(a, 2, at::kFloat, carry, w);
  const View dy = view(a.tensor(3), "dy", s.dtype, all, w);
  const uint8_t* reset = flags(a, 4, {s.B, s.T}, w);
  const auto* length = dense<const int64_t>(a, 5, at::kLong, {s.B}, w);
  const auto* dl = dense<const float>(a, 6, at::kFloat, state, w);
  const Tensor dx = output(a, 7, all, s.dtype, w), dg = output(a, 8, all, s.dtype, w),
               dh0 = output(a, 9, state, at::kFloat, w);
  const View vx = view(dx, "dx", s.dtype, all, w), vg = view(dg, "dg", s.dtype, all, w);
  float* p0 = dense<float>(dh0, "dh0", at::kFloat, state, w);
  const int64_t bytes = scan_bytes(s.B, s.T, s.D);
  Tensor ws;
  if (bytes) ws = w.empty({bytes}, at::kByte);
  check(api.per_scan_backward(s.B, s.T, s.D, s.type, s.x.p, s.x.sb, s.x.st, s.g.p, s.g.sb, s.g.st,
                              reset, length, pc, dy.p, dy.sb, dy.st, dl, vx.p, vx.sb, vx.st, vg.p,
                              vg.sb, vg.st, p0, bytes ? ws.data_ptr() : nullptr, (size_t)bytes,
                              w.stream));
  return triple(dx, dg, dh0);
}

// x, g, h, reset, h_out, y, stream
PyObject* scan_step(const Args& a) {
  const Tensor& x = a.tensor(0);
  const Where w(a.v[6], x, "x");
  if (x.dim() != 2) refuse("x must be [B x D]");
  const int type = type_of(x, "x");
  const auto dt = x.scalar_type();
  const int64_t shape[] = {x.size(0), x.size(1)};
  const Matrix mx = matrix(x, "x", dt, shape, w), mg = matrix(a.tensor(1), "g", dt, shape, w);
  const auto* h = dense<const float>(a, 2, at::kFloat, shape, w);
  const uint8_t* reset = flags(a, 3, {shape[0]}, w);
  const Tensor ho = a.v[4] ? a.tensor(4) : a.tensor(2);
  float* pho = dense<float>(ho, "h_out", at::kFloat, shape, w);
  const Tensor y = output(a, 5, shape, dt, w);
  const Matrix my = matrix(y, "y", dt, shape, w);
  check(api.per_scan_step(shape[0], shape[1], type, mx.p, mx.stride, mg.p, mg.stride, reset, h, pho,
                          my.p, my.stride, w.stream));
  if (!a.v[4] && !ho.is_inference()) ho.unsafeGetTensorImpl()->bump_version();
  return pair(y, ho);
}

PyObject* scan_workspace(const Args& a) {
  return PyLong_FromLongLong(scan_bytes(a.integer(0, 0), a.integer(1, 0), a.integer(2, 0)));
}

// ----------------------------------------------------------------- distillation

int64_t distill_bytes(int64_t N, int64_t V, int64_t K, int type) {
  size_t n = 0;
  check(api.per_distill_workspace_bytes(N, V, K, type, &n));
  return (int64_t)n;
}

struct Top {
  int64_t N, V, K;
  int type, t_type;
  at::ScalarType dtype;
  Matrix z;
  const int32_t* tidx;
  const void* t;
  const float* tlse;
  double tau;
};
// Arguments 0, 1, 2: logits, tidx, tlogit; tlse and temperature at `lse`, `lse` + 1.
Top top(const Args& a, int lse, const Where& w) {
  const Tensor &z = a.tensor(0), &tidx = a.tensor(1), &t = a.tensor(2);
  if (z.dim() != 2 || tidx.dim() != 2) refuse("logits must be [N x V], tidx [N x K]");
  Top o;
  o.type = type_of(z, "logits");
  o.t_type = type_of(t, "tlogit");
  o.dtype = z.scalar_type();
  o.N = z.size(0);
  o.V = z.size(1);
  o.K = tidx.size(1);
  const int64_t entries[] = {o.N, o.K};
  o.z = matrix(z, "logits", o.dtype, z.sizes(), w);
  o.tidx = dense<const int32_t>(tidx, "tidx", at::kInt, entries, w);
  o.t = dense<const void>(t, "tlogit", t.scalar_type(), entries, w);
  o.tlse = dense<const float>(a, lse, at::kFloat, {o.N}, w);
  o.tau = a.real(lse + 1, 1.0);
  return o;
}
#define TOP(o) o.N, o.V, o.K, o.type, o.z.p, o.z.stride, o.tidx, o.t, o.t_type, o.tlse, o.tau

// logits, tidx, tlogit, tlse, temperature, weight, loss, grad, stream
PyObject* distill(const Args& a) {
  const Where w(a.v[8], a.tensor(0), "logits");
  const Top o = top(a, 3, w);
  const int64_t all[] = {o.N, o.V};
  const auto* weight = dense<const float>(a, 5, at::kFloat, {o.N}, w);
  const Tensor loss = output(a, 6, {o.N}, at::kFloat, w), grad = output(a, 7, all, o.dtype, w);
  float* pl = dense<float>(loss, "loss", at::kFloat, {o.N}, w);
  const Matrix mg = matrix(grad, "grad", o.dtype, all, w);
  const int64_t bytes = distill_bytes(o.N, o.V, o.K, o.type);
  Tensor ws;
  if (bytes) ws = w.empty({bytes}, at::kByte);
  check(api.per_distill(TOP(o), weight, pl, mg.p, mg.stride, bytes ? ws.data_ptr() : nullptr,
                        (size_t)bytes, w.stream));
  return pair(loss, grad);
}

// logits, tidx, tlogit, tlse, temperature, loss, saved, stream
PyObject* distill_forward(const Args& a) {
  const Where w(a.v[7], a.tensor(0), "logits");
  const Top o = top(a, 3, w);
  const Tensor loss = output(a, 5, {o.N}, at::kFloat, w),
               saved = output(a, 6, {o.N, 4 + o.K}, at::kFloat, w);
  float* pl = dense<float>(loss, "loss", at::kFloat, {o.N}, w);
  float* ps = dense<float>(saved, "saved", at::kFloat, {o.N, 4 + o.K}, w);
  const int64_t bytes = distill_bytes(o.N, o.V, o.K, o.type);
  Tensor ws;
  if (bytes) ws = w.empty({bytes}, at::kByte);
  check(api.per_distill_forward(TOP(o), pl, ps, bytes ? ws.data_ptr() : nullptr, (size_t)bytes,
                                w.stream));
  return pair(loss, saved);
}

// logits, tidx, tlogit, saved, gloss, tlse, temperature, grad, stream
PyObject* distill_backward(const Args& a) {
  const Where w(a.v[8], a.tensor(0), "logits");
  const Top o = top(a, 5, w);
  const int64_t all[] = {o.N, o.V};
  const auto* saved = dense<const float>(a, 3, at::kFloat, {o.N, 4 + o.K}, w);
  const auto* gloss = dense<const float>(a, 4, at::kFloat, {o.N}, w);
  const Tensor grad = output(a, 7, all, o.dtype, w);
  const Matrix mg = matrix(grad, "grad", o.dtype, all, w);
  check(api.per_distill_backward(TOP(o), saved, gloss, mg.p, mg.stride, w.stream));
  return THPVariable_Wrap(grad);
}

PyObject* distill_workspace(const Args& a) {
  return PyLong_FromLongLong(
      distill_bytes(a.integer(0, 0), a.integer(1, 0), a.integer(2, 0), (int)a.integer(3, 0)));
}

// -------------------------------------------------------------------- embedding

// A dense array of int32 or int64 tokens.
struct Tokens {
  const void* p;
  int64_t N;
  int bytes;
};
Tokens tokens_of(const Tensor& t, const Where& w) {
  const bool wide = t.scalar_type() == at::kLong;
  if (t.dim() != 1 || (!wide && t.scalar_type() != at::kInt))
    refuse("tokens must be [N], int32 or int64");
  return {dense<const void>(t, "tokens", t.scalar_type(), t.sizes(), w), t.size(0), wide ? 8 : 4};
}
bool flag(const Args& a, int i, bool otherwise) {
  if (!a.v[i]) return otherwise;
  const int on = PyObject_IsTrue(a.v[i]);
  if (on < 0) {
    PyErr_Clear();
    refuse(std::string(a.names[i]) + " must be a truth value");
  }
  return on != 0;
}
at::ScalarType dtype_of(const Args& a, int i, at::ScalarType otherwise) {
  if (!a.v[i]) return otherwise;
  if (!THPDtype_Check(a.v[i])) refuse("dtype must be a torch.dtype");
  const at::ScalarType t = reinterpret_cast<THPDtype*>(a.v[i])->scalar_type;
  if (t != at::kFloat && t != at::kBFloat16 && t != at::kHalf)
    refuse("dtype must be float32, bfloat16 or float16");
  return t;
}
Tensor scratch(int64_t bytes, const Where& w) {
  return bytes ? w.empty({bytes}, at::kByte) : Tensor();
}
void* data(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// tokens, table, scale = 1, out, dtype, stream
PyObject* embed_forward(const Args& a) {
  const Tensor& table = a.tensor(1);
  const Where w(a.v[5], table, "table");
  if (table.dim() != 2) refuse("table must be [V x D]");
  const int from = type_of(table, "table");
  const Matrix mt = matrix(table, "table", table.scalar_type(), table.sizes(), w);
  const Tokens t = tokens_of(a.tensor(0), w);
  const int64_t shape[] = {t.N, table.size(1)};
  const Tensor out = output(a, 3, shape, dtype_of(a, 4, table.scalar_type()), w);
  const int to = type_of(out, "out");
  if (a.v[3] && a.v[4] && out.scalar_type() != dtype_of(a, 4, at::kFloat))
    refuse("out is not of the dtype given");
  const Matrix mo = matrix(out, "out", out.scalar_type(), shape, w);
  check(api.per_embed_forward(t.N, table.size(0), shape[1], t.p, t.bytes, mt.p, from, mt.stride,
                              a.real(2, 1.0), mo.p, to, mo.stride, w.stream));
  return THPVariable_Wrap(out);
}

int64_t embed_bytes(int64_t N, int64_t V, int64_t D) {
  size_t n = 0;
  check(api.per_embed_workspace_bytes(N, V, D, &n));
  return (int64_t)n;
}

// tokens, dout, vocab, scale = 1, grad, accumulate = False, stream
PyObject* embed_backward(const Args& a) {
  const Tensor& dout = a.tensor(1);
  const Where w(a.v[6], dout, "dout");
  const Tokens t = tokens_of(a.tensor(0), w);
  if (dout.dim() != 2) refuse("dout must be [N x D]");
  const int from = type_of(dout, "dout");
  const int64_t rows[] = {t.N, dout.size(1)}, V = a.integer(2, 0);
  const Matrix md = matrix(dout, "dout", dout.scalar_type(), rows, w);
  const bool add = flag(a, 5, false);
  if (add && !a.v[4]) refuse("accumulate needs the grad to add to");
  const int64_t bytes = embed_bytes(t.N, V, rows[1]);
  const int64_t shape[] = {V, rows[1]};
  const Tensor grad = output(a, 4, shape, at::kFloat, w);
  const int to = type_of(grad, "grad");
  const Matrix mg = matrix(grad, "grad", grad.scalar_type(), shape, w);
  const Tensor ws = scratch(bytes, w);
  check(api.per_embed_backward(t.N, V, rows[1], t.p, t.bytes, md.p, from, md.stride, a.real(3, 1.0),
                               add, mg.p, to, mg.stride, data(ws), (size_t)bytes, w.stream));
  return THPVariable_Wrap(grad);
}

PyObject* embed_workspace(const Args& a) {
  return PyLong_FromLongLong(embed_bytes(a.integer(0, 0), a.integer(1, 0), a.integer(2, 0)));
}

// ------------------------------------------------------------------- layer norm

// Weight and bias [D], both f32 or both of the rows' type.
struct Affine {
  const void* weight = nullptr;
  const void* bias = nullptr;
  int type = PER_F32;
};
Affine affine(const Args& a, int weight, int bias, int64_t D, at::ScalarType rows, const Where& w) {
  Affine f;
  bool known = false;
  for (int i : {weight, bias}) {
    if (i < 0 || !a.v[i]) continue;
    const Tensor& t = a.tensor(i);
    if (t.scalar_type() != at::kFloat && t.scalar_type() != rows)
      refuse(std::string(a.names[i]) + " must be float32 or of the type of x");
    const int type = type_of(t, a.names[i]);
    if (known && type != f.type) refuse("weight and bias must have one type");
    f.type = type;
    known = true;
    (i == weight ? f.weight : f.bias) = dense<const void>(t, a.names[i], t.scalar_type(), {D}, w);
  }
  return f;
}

// x, weight, bias, eps = 1e-5, y, stats, stream
PyObject* norm_forward(const Args& a) {
  const Tensor& x = a.tensor(0);
  const Where w(a.v[6], x, "x");
  if (x.dim() != 2) refuse("x must be [N x D]");
  const int type = type_of(x, "x");
  const int64_t N = x.size(0), D = x.size(1);
  const Matrix mx = matrix(x, "x", x.scalar_type(), x.sizes(), w);
  const Affine f = affine(a, 1, 2, D, x.scalar_type(), w);
  const Tensor y = output(a, 4, x.sizes(), x.scalar_type(), w),
               stats = output(a, 5, {N, 2}, at::kFloat, w);
  const Matrix my = matrix(y, "y", x.scalar_type(), x.sizes(), w);
  float* ps = dense<float>(stats, "stats", at::kFloat, {N, 2}, w);
  check(api.per_norm_forward(N, D, type, mx.p, mx.stride, f.weight, f.bias, f.type,
                             a.real(3, 1e-5), my.p, my.stride, ps, w.stream));
  return pair(y, stats);
}

int64_t norm_bytes(int64_t N, int64_t D, int type) {
  size_t n = 0;
  check(api.per_norm_workspace_bytes(N, D, type, &n));
  return (int64_t)n;
}

// x, stats, dy, weight, dx, dweight, dbias, sums = True, stream
PyObject* norm_backward(const Args& a) {
  const Tensor& x = a.tensor(0);
  const Where w(a.v[8], x, "x");
  if (x.dim() != 2) refuse("x must be [N x D]");
  const int type = type_of(x, "x");
  const auto dt = x.scalar_type();
  const int64_t N = x.size(0), D = x.size(1);
  const Matrix mx = matrix(x, "x", dt, x.sizes(), w),
               md = matrix(a.tensor(2), "dy", dt, x.sizes(), w);
  const auto* stats = dense<const float>(a, 1, at::kFloat, {N, 2}, w);
  const Affine f = affine(a, 3, -1, D, dt, w);
  const bool sums = flag(a, 7, true);
  if (!sums && (a.v[5] || a.v[6])) refuse("dweight and dbias are given, and sums is false");
  const Tensor dx = output(a, 4, x.sizes(), dt, w);
  const Matrix mo = matrix(dx, "dx", dt, x.sizes(), w);
  Tensor dw, db;
  float *pw = nullptr, *pb = nullptr;
  if (sums) {
    dw = output(a, 5, {D}, at::kFloat, w);
    db = output(a, 6, {D}, at::kFloat, w);
    pw = dense<float>(dw, "dweight", at::kFloat, {D}, w);
    pb = dense<float>(db, "dbias", at::kFloat, {D}, w);
  }
  const int64_t bytes = norm_bytes(N, D, type);
  const Tensor ws = scratch(bytes, w);
  check(api.per_norm_backward(N, D, type, mx.p, mx.stride, stats, md.p, md.stride, f.weight, f.type,
                              mo.p, mo.stride, pw, pb, data(ws), (size_t)bytes, w.stream));
  return triple(dx, dw, db);  // an undefined tensor is None
}

PyObject* norm_workspace(const Args& a) {
  return PyLong_FromLongLong(norm_bytes(a.integer(0, 0), a.integer(1, 0), (int)a.integer(2, 0)));
}

// ------------------------------------------------------------- gated delta rule

// [B x T x H x D], or without T; unit stride along D.
per_seq seq(const Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape,
            bool steps, const Where& w) {
  expect(t, name, dtype, shape, w);
  const int n = steps ? 3 : 2;  // dimensions before D
  if ((int)shape.size() > n && shape[n] > 1 && t.stride(n) != 1)
    refuse(std::string(name) + " must have unit stride in its last dimension");
  return {t.data_ptr(), t.stride(0), steps ? t.stride(1) : 0, t.stride(n - 1)};
}
struct Delta {
  int64_t B, T, H, HK, DK, DV;
  int type;
  at::ScalarType dtype;
  std::vector<int64_t> qk, vo, gate, state;  // shapes
  per_seq q, k, v, g, b;
};
// Arguments 0 to 4: q, k, v, g, b.
Delta delta(const Args& a, bool steps, const Where& w) {
  const Tensor &q = a.tensor(0), &v = a.tensor(2);
  const int n = steps ? 4 : 3;
  if (q.dim() != n || v.dim() != n)
    refuse(steps ? "q must be [B x T x HK x DK], v [B x T x H x DV]"
                 : "q must be [B x HK x DK], v [B x H x DV]");
  Delta d;
  d.type = type_of(q, "q");
  d.dtype = q.scalar_type();
  d.B = v.size(0);
  d.T = steps ? v.size(1) : 1;
  d.H = v.size(n - 2);
  d.DV = v.size(n - 1);
  d.HK = q.size(n - 2);
  d.DK = q.size(n - 1);
  d.vo = v.sizes().vec();
  d.qk = d.vo;
  d.qk[n - 2] = d.HK;
  d.qk[n - 1] = d.DK;
  d.gate = d.vo;
  d.gate.pop_back();
  d.state = {d.B, d.H, d.DK, d.DV};
  d.q = seq(q, "q", d.dtype, d.qk, steps, w);
  d.k = seq(a.tensor(1), "k", d.dtype, d.qk, steps, w);
  d.v = seq(v, "v", d.dtype, d.vo, steps, w);
  d.g = seq(a.tensor(3), "g", d.dtype, d.gate, steps, w);
  d.b = seq(a.tensor(4), "b", d.dtype, d.gate, steps, w);
  return d;
}
#define DELTA(d) d.H, d.HK, d.DK, d.DV, d.type, d.q, d.k, d.v, d.g, d.b

int64_t delta_bytes(int64_t B, int64_t T, int64_t H, int64_t HK, int64_t DK, int64_t DV, int type,
                    bool backward) {
  size_t n = 0;
  check(api.per_delta_workspace_bytes(B, T, H, HK, DK, DV, type, backward, &n));
  return (int64_t)n;
}
std::vector<int64_t> carry_shape(const Delta& d) {
  return {d.B, (d.T + PER_DELTA_CHUNK - 1) / PER_DELTA_CHUNK, d.H, d.DK + PER_DELTA_CHUNK, d.DV};
}

// q, k, v, g, b, reset, length, s0, scale = 1, save = True, out, s_last, carries, stream
PyObject* delta_forward(const Args& a) {
  const Where w(a.v[13], a.tensor(0), "q");
  const Delta d = delta(a, true, w);
  const uint8_t* reset = flags(a, 5, {d.B, d.T}, w);
  const auto* length = dense<const int64_t>(a, 6, at::kLong, {d.B}, w);
  const auto* s0 = dense<const float>(a, 7, at::kFloat, d.state, w);
  const bool save = flag(a, 9, true);
  if (!save && a.v[12]) refuse("carries are given, and save is false");
  const int64_t bytes = delta_bytes(d.B, d.T, d.H, d.HK, d.DK, d.DV, d.type, false);
  const Tensor o = output(a, 10, d.vo, d.dtype, w), s = output(a, 11, d.state, at::kFloat, w);
  const per_seq vo = seq(o, "out", d.dtype, d.vo, true, w);
  float* ps = dense<float>(s, "s_last", at::kFloat, d.state, w);
  Tensor c;
  float* pc = nullptr;
  if (save) {
    c = output(a, 12, carry_shape(d), at::kFloat, w);
    pc = dense<float>(c, "carries", at::kFloat, carry_shape(d), w);
  }
  const Tensor ws = scratch(bytes, w);
  check(api.per_delta_forward(d.B, d.T, DELTA(d), reset, length, s0, a.real(8, 1.0), vo, ps, pc,
                              data(ws), (size_t)bytes, w.stream));
  return triple(o, s, c);
}

// q, k, v, g, b, carries, do, reset, length, ds_last, scale = 1, dq, dk, dv, dg, db, ds0, stream
PyObject* delta_backward(const Args& a) {
  const Where w(a.v[17], a.tensor(0), "q");
  const Delta d = delta(a, true, w);
  const auto* pc = dense<const float>(a, 5, at::kFloat, carry_shape(d), w);
  const per_seq d_o = seq(a.tensor(6), "do", d.dtype, d.vo, true, w);
  const uint8_t* reset = flags(a, 7, {d.B, d.T}, w);
  const auto* length = dense<const int64_t>(a, 8, at::kLong, {d.B}, w);
  const auto* dl = dense<const float>(a, 9, at::kFloat, d.state, w);
  const int64_t bytes = delta_bytes(d.B, d.T, d.H, d.HK, d.DK, d.DV, d.type, true);
  const std::vector<int64_t>* shapes[] = {&d.qk, &d.qk, &d.vo, &d.gate, &d.gate};
  Tensor out[6];
  per_seq views[5];
  for (int i = 0; i < 5; ++i) {
    out[i] = output(a, 11 + i, *shapes[i], d.dtype, w);
    views[i] = seq(out[i], a.names[11 + i], d.dtype, *shapes[i], true, w);
  }
  out[5] = output(a, 16, d.state, at::kFloat, w);
  float* p0 = dense<float>(out[5], "ds0", at::kFloat, d.state, w);
  const Tensor ws = scratch(bytes, w);
  check(api.per_delta_backward(d.B, d.T, DELTA(d), reset, length, pc, d_o, dl, a.real(10, 1.0),
                               views[0], views[1], views[2], views[3], views[4], p0, data(ws),
                               (size_t)bytes, w.stream));
  PyObject* t = PyTuple_New(6);
  if (!t) return nullptr;
  for (int i = 0; i < 6; ++i) PyTuple_SET_ITEM(t, i, THPVariable_Wrap(out[i]));
  return t;
}

// q, k, v, g, b, s, reset, scale = 1, s_out, out, stream
PyObject* delta_step(const Args& a) {
  const Where w(a.v[10], a.tensor(0), "q");
  const Delta d = delta(a, false, w);
  const auto* s = dense<const float>(a, 5, at::kFloat, d.state, w);
  const uint8_t* reset = flags(a, 6, {d.B}, w);
  const Tensor so = a.v[8] ? a.tensor(8) : a.tensor(5);
  float* ps = dense<float>(so, "s_out", at::kFloat, d.state, w);
  const Tensor o = output(a, 9, d.vo, d.dtype, w);
  const per_seq vo = seq(o, "out", d.dtype, d.vo, false, w);
  check(api.per_delta_step(d.B, DELTA(d), reset, s, a.real(7, 1.0), ps, vo, w.stream));
  if (!a.v[8] && !so.is_inference()) so.unsafeGetTensorImpl()->bump_version();
  return pair(o, so);
}

PyObject* delta_workspace(const Args& a) {
  return PyLong_FromLongLong(delta_bytes(a.integer(0, 0), a.integer(1, 0), a.integer(2, 0),
                                         a.integer(3, 0), a.integer(4, 0), a.integer(5, 0),
                                         (int)a.integer(6, 0), flag(a, 7, false)));
}

// ----------------------------------------------------------------- the module

struct Function {
  const char* name;
  PyObject* (*run)(const Args&);
  int required;
  int n;
  unsigned written;  // bit i: argument i is written where it is given
  const char* names[kMaxArgs];
  const char* doc;
  PyObject* interned[kMaxArgs];
};
constexpr unsigned bits() { return 0; }
template <typename... I>
constexpr unsigned bits(int i, I... more) {
  return 1u << i | bits(more...);
}

// Nothing here is recorded for autograd: a call that would silently cut a graph, or
// drop a tangent, is refused, whichever argument it is.  (Inside an
// autograd.Function, and under no_grad, recording is off.)
void unrecorded(const Function& f, const Args& a) {
  const bool grad = at::GradMode::is_enabled();
  const bool tangent = c10::AutogradState::get_tls_state().get_fw_grad_mode();
  if (!grad && !tangent) return;
  for (int i = 0; i < f.n; ++i) {
    if (!a.v[i] || !THPVariable_Check(a.v[i])) continue;
    const Tensor& t = THPVariable_Unpack(a.v[i]);
    if (!t.unsafeGetTensorImpl()->autograd_meta()) continue;
    if (grad && t.requires_grad())
      refuse(std::string(f.names[i]) +
             " requires grad: call this under torch.no_grad() or from an autograd.Function; its "
             "gradients come from explicit calls");
    if (tangent && t._fw_grad(0).defined())
      refuse(std::string(f.names[i]) +
             " carries a forward-mode tangent, which this call would drop: pass its primal");
  }
}

// The tensors a call wrote count as changed in place, so that autograd notices where
// one of them had been saved.
void wrote(const Function& f, const Args& a) {
  for (int i = 0; i < f.n; ++i) {
    if (!(f.written >> i & 1u) || !a.v[i]) continue;
    const Tensor& t = THPVariable_Unpack(a.v[i]);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  }
}

Function functions[] = {
    {"per_rows_write", rows_write, 3, 6, bits(0, 1), {"codes", "scales", "src", "first", "group", "stream"},
     "per_rows_write(codes, scales, src, first=0, group=128, stream=None)\n\n"
     "Quantise the rows of src into the ring's slots first, first + 1, ...", {}},
    {"per_rows_write_at", rows_write_at, 5, 7, bits(0, 1, 4),
     {"codes", "scales", "src", "slots", "claims", "group", "stream"},
     "per_rows_write_at(codes, scales, src, slots, claims, group=128, stream=None)\n\n"
     "Quantise row j of src into slot slots[j]; of a repeated slot the last position wins.\n"
     "claims: [capacity] int32 zeros, zero again afterwards.", {}},
    {"per_rows_read", rows_read, 3, 8, bits(5),
     {"codes", "scales", "idx", "window", "group", "out", "dtype", "stream"},
     "per_rows_read(codes, scales, idx, window=1, group=128, out=None, dtype=torch.float32, "
     "stream=None)\n\n[B x window x dim]: the rows of slots idx[b], idx[b] + 1, ... of the ring.",
     {}},
    {"per_scan_workspace_bytes", scan_workspace, 3, 3, bits(), {"B", "T", "D"},
     "per_scan_workspace_bytes(B, T, D)", {}},
    {"per_scan_forward", scan_forward, 2, 9, bits(5, 6, 7),
     {"x", "g", "reset", "length", "h0", "y", "h_last", "carries", "stream"},
     "per_scan_forward(x, g, reset=None, length=None, h0=None, y=None, h_last=None, carries=None, "
     "stream=None)\n\nh_t = f h_{t-1} + (1 - f) x_t with f = sigmoid(g_t) along dim 1 of x, g\n"
     "[B x T x D].  Returns (y [B x T x D], h_last [B x D] f32, carries: the f32 states that\n"
     "per_scan_backward takes).", {}},
    {"per_scan_backward", scan_backward, 4, 11, bits(7, 8, 9),
     {"x", "g", "carries", "dy", "reset", "length", "dh_last", "dx", "dg", "dh0", "stream"},
     "per_scan_backward(x, g, carries, dy, reset=None, length=None, dh_last=None, dx=None, "
     "dg=None, dh0=None, stream=None)\n\n"
     "Gradients (dx, dg, dh0) of per_scan_forward from dy and dh_last.", {}},
    {"per_scan_step", scan_step, 3, 7, bits(4, 5), {"x", "g", "h", "reset", "h_out", "y", "stream"},
     "per_scan_step(x, g, h, reset=None, h_out=None, y=None, stream=None)\n\n"
     "One step of B sequences: x, g [B x D], h [B x D] f32 (updated in place without h_out).\n"
     "Returns (y, h_out).", {}},
    {"per_distill_workspace_bytes", distill_workspace, 4, 4, bits(), {"N", "V", "K", "type"},
     "per_distill_workspace_bytes(N, V, K, type)", {}},
    {"per_distill", distill, 3, 9, bits(6, 7),
     {"logits", "tidx", "tlogit", "tlse", "temperature", "weight", "loss", "grad", "stream"},
     "per_distill(logits, tidx, tlogit, tlse=None, temperature=1.0, weight=None, loss=None, "
     "grad=None, stream=None)\n\n"
     "Per-row distillation loss [N] (not weighted) and its gradient by the logits [N x V]\n"
     "(weighted), against the teacher's logits tlogit [N x K] at tokens tidx [N x K] int32.\n"
     "Temperatures lie in [2^-20, 64].\n"
     "grad may be logits.  Returns (loss, grad).", {}},
    {"per_distill_forward", distill_forward, 3, 8, bits(5, 6),
     {"logits", "tidx", "tlogit", "tlse", "temperature", "loss", "saved", "stream"},
     "per_distill_forward(logits, tidx, tlogit, tlse=None, temperature=1.0, loss=None, saved=None, "
     "stream=None)\n\n"
     "Per-row loss [N], and the row statistics per_distill_backward takes.", {}},
    {"per_distill_backward", distill_backward, 5, 9, bits(7),
     {"logits", "tidx", "tlogit", "saved", "gloss", "tlse", "temperature", "grad", "stream"},
     "per_distill_backward(logits, tidx, tlogit, saved, gloss, tlse=None, temperature=1.0, "
     "grad=None, stream=None)\n\n"
     "Gradient by the logits from the gradient by each row's loss.", {}},
    {"per_embed_forward", embed_forward, 2, 6, bits(3),
     {"tokens", "table", "scale", "out", "dtype", "stream"},
     "per_embed_forward(tokens, table, scale=1.0, out=None, dtype=None, stream=None)\n\n"
     "[N x D]: scale times the rows of table [V x D] that tokens [N] (int32 or int64) name, zeros\n"
     "for tokens outside [0, V); of dtype (the table's by default).", {}},
    {"per_embed_workspace_bytes", embed_workspace, 3, 3, bits(), {"N", "V", "D"},
     "per_embed_workspace_bytes(N, V, D)", {}},
    {"per_embed_backward", embed_backward, 3, 7, bits(4),
     {"tokens", "dout", "vocab", "scale", "grad", "accumulate", "stream"},
     "per_embed_backward(tokens, dout, vocab, scale=1.0, grad=None, accumulate=False, stream=None)"
     "\n\nGradient by the table [vocab x D] (float32 without grad): scale times the sum of each\n"
     "token's rows of dout, zeros for tokens that do not occur, or added to what grad holds.", {}},
    {"per_norm_forward", norm_forward, 1, 7, bits(4, 5),
     {"x", "weight", "bias", "eps", "y", "stats", "stream"},
     "per_norm_forward(x, weight=None, bias=None, eps=1e-5, y=None, stats=None, stream=None)\n\n"
     "Layer norm of the rows of x [N x D].  Returns (y, stats [N x 2] f32: mean and reciprocal\n"
     "deviation, which per_norm_backward takes).  y may be x.", {}},
    {"per_norm_workspace_bytes", norm_workspace, 3, 3, bits(), {"N", "D", "type"},
     "per_norm_workspace_bytes(N, D, type)", {}},
    {"per_norm_backward", norm_backward, 3, 9, bits(4, 5, 6),
     {"x", "stats", "dy", "weight", "dx", "dweight", "dbias", "sums", "stream"},
     "per_norm_backward(x, stats, dy, weight=None, dx=None, dweight=None, dbias=None, sums=True, "
     "stream=None)\n\n"
     "Gradients (dx, dweight [D] f32, dbias [D] f32) of per_norm_forward; without sums dx alone,\n"
     "and None for the others.  dx may be dy.", {}},
    {"per_delta_workspace_bytes", delta_workspace, 7, 8, bits(),
     {"B", "T", "H", "HK", "DK", "DV", "type", "backward"},
     "per_delta_workspace_bytes(B, T, H, HK, DK, DV, type, backward=False)", {}},
    {"per_delta_forward", delta_forward, 5, 14, bits(10, 11, 12),
     {"q", "k", "v", "g", "b", "reset", "length", "s0", "scale", "save", "out", "s_last", "carries",
      "stream"},
     "per_delta_forward(q, k, v, g, b, reset=None, length=None, s0=None, scale=1.0, save=True, "
     "out=None, s_last=None, carries=None, stream=None)\n\n"
     "The gated delta rule along dim 1 of q, k [B x T x HK x DK], v [B x T x H x DV] and the logits\n"
     "g, b [B x T x H] of gates and writing strengths.  Returns (out [B x T x H x DV], s_last\n"
     "[B x H x DK x DV] f32, carries: what per_delta_backward takes, None without save).", {}},
    {"per_delta_backward", delta_backward, 7, 18, bits(11, 12, 13, 14, 15, 16),
     {"q", "k", "v", "g", "b", "carries", "do", "reset", "length", "ds_last", "scale", "dq", "dk",
      "dv", "dg", "db", "ds0", "stream"},
     "per_delta_backward(q, k, v, g, b, carries, do, reset=None, length=None, ds_last=None, "
     "scale=1.0, dq=None, dk=None, dv=None, dg=None, db=None, ds0=None, stream=None)\n\n"
     "Gradients (dq, dk, dv, dg, db, ds0) of per_delta_forward from do and ds_last.", {}},
    {"per_delta_step", delta_step, 6, 11, bits(8, 9),
     {"q", "k", "v", "g", "b", "s", "reset", "scale", "s_out", "out", "stream"},
     "per_delta_step(q, k, v, g, b, s, reset=None, scale=1.0, s_out=None, out=None, stream=None)\n\n"
     "One step of B sequences: q, k [B x HK x DK], v [B x H x DV], g, b [B x H], s [B x H x DK x DV]\n"
     "f32 (updated in place without s_out).  Returns (out, s_out).", {}},
};
constexpr int kFunctions = sizeof functions / sizeof functions[0];

// No C++ exception leaves an entry point.
PyObject* call(Function& f, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  if (!api.per_rows_write) {
    PyObject* r = loader ? PyObject_CallNoArgs(loader) : nullptr;
    Py_XDECREF(r);
    if (!r || !api.per_rows_write) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ImportError, "the library is not bound");
      return nullptr;
    }
  }
  try {
    const Args a(f.name, f.names, f.interned, f.n, f.required, args, nargs, kwnames);
    unrecorded(f, a);
    PyObject* out = f.run(a);
    wrote(f, a);
    return out;
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Failed& e) {
    PyObject* err = PyObject_CallFunction(per_error, "is", e.code, api.per_last_error());
    if (err) {
      PyErr_SetObject(per_error, err);
      Py_DECREF(err);
    }
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    Py_XDECREF(torch);
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

template <int I>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return call(functions[I], args, nargs, kwnames);
}

// bind(addresses: dict of name to address, PerError)
PyObject* bind(PyObject*, PyObject* args) {
  PyObject *d, *err;
  if (!PyArg_ParseTuple(args, "O!O", &PyDict_Type, &d, &err)) return nullptr;
  Api got;
#define TAKE(name)                                                                    \
  {                                                                                   \
    PyObject* v = PyDict_GetItemString(d, #name);                                     \
    got.name = v ? reinterpret_cast<decltype(&::name)>(PyLong_AsVoidPtr(v)) : nullptr; \
    if (!got.name) {                                                                  \
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no address of " #name); \
      return nullptr;                                                                 \
    }                                                                                 \
  }
  ENTRY_POINTS(TAKE)
#undef TAKE
  api = got;
  Py_XDECREF(per_error);
  Py_INCREF(err);
  per_error = err;
  Py_RETURN_NONE;
}

// set_loader(function): it is to call bind().
PyObject* set_loader(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XDECREF(loader);
  loader = f;
  Py_RETURN_NONE;
}

PyMethodDef methods[kFunctions + 3];

template <int... I>
void fill(std::integer_sequence<int, I...>) {
  ((methods[I] = {functions[I].name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<I>)),
                  METH_FASTCALL | METH_KEYWORDS, functions[I].doc}),
   ...);
}

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "Binding of include/per_train.h and include/per_block.h.", -1,
                      methods,               nullptr,    nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  for (Function& f : functions)
    for (int i = 0; i < f.n; ++i) {
      f.interned[i] = PyUnicode_InternFromString(f.names[i]);
      if (!f.interned[i]) return nullptr;
    }
  fill(std::make_integer_sequence<int, kFunctions>{});
  methods[kFunctions] = {"bind", bind, METH_VARARGS, "bind(addresses, error): the C entry points."};
  methods[kFunctions + 1] = {"set_loader", set_loader, METH_O, "set_loader(function)"};
  methods[kFunctions + 2] = {nullptr, nullptr, 0, nullptr};
  return PyModule_Create(&module);
}
