// The calls of libnvq that take a few microseconds on the GPU, as Python
// functions: tensors in, their types, sizes and devices checked, the library's
// entry point called on the device's current stream.  A ctypes call with the
// same checks in Python costs more than such a kernel runs.  The entry points
// are bound by address from the library that the package has loaded (bind).
//
// Every function returns its outputs, or the status of a call that the library
// refused as an int; a tensor that does not fit is a ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>
#include <string>
#include <utility>

#include "../../include/nvq.h"

namespace {

struct Entry {
  decltype(&nvfp4_gemm_w4a4_epilogue) w4a4 = nullptr;
  decltype(&w4a16_gemm_epilogue) w4a16 = nullptr;
  decltype(&nvq_linear_epilogue) linear = nullptr;
  decltype(&nvq_linear_workspace_bytes) linear_bytes = nullptr;
  decltype(&moe_route) route = nullptr;
  decltype(&w4a16_moe_workspace_bytes) moe_bytes = nullptr;
  decltype(&w4a16_moe_experts) experts = nullptr;
  decltype(&w4a16_moe) moe = nullptr;
} g;

struct Bad {            // becomes a ValueError
  std::string what;
};
struct Raised {};       // Python's own error is set

std::string shown(c10::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Bad{std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

// A matrix whose rows share memory (a broadcast one has a row stride of 0, which the C
// calls take for "N") is no residual and no output.  Looked at before the device is, so
// that it can be without one.
void rows_apart(PyObject* o, const char* name) {
  if (o == Py_None) return;
  const at::Tensor& t = tensor(o, name);
  if (t.dim() == 2 && t.size(0) > 1 && t.stride(0) < t.size(1))
    throw Bad{std::string(name) + " must have a row stride of at least " + std::to_string(t.size(1)) + ", not " +
              std::to_string(t.stride(0)) + " (broadcast rows have to be copied)"};
}

// One call: the device of its first tensor, made current, and that device's stream.
struct Call {
  c10::cuda::OptionalCUDAGuard guard;
  c10::DeviceIndex dev;
  explicit Call(const at::Tensor& first) {
    if (!first.is_cuda()) throw Bad{"libnvq calls take CUDA tensors"};
    dev = first.get_device();
    guard.set_index(dev);
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
  void fits(const at::Tensor& t, const char* name, at::ScalarType type) const {
    if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev)
      throw Bad{std::string(name) + " must be a " + c10::toString(type) + " tensor on cuda:" + std::to_string(dev) +
                ", not " + c10::toString(t.scalar_type()) + " on " + t.device().str()};
  }
  // A contiguous tensor of at least n elements.
  void* flat(const at::Tensor& t, const char* name, at::ScalarType type, int64_t n) const {
    fits(t, name, type);
    if (!t.is_contiguous() || t.numel() < n)
      throw Bad{std::string(name) + " must be contiguous with at least " + std::to_string(n) + " elements"};
    return t.data_ptr();
  }
  // A contiguous tensor of this shape.
  void* exact(const at::Tensor& t, const char* name, at::ScalarType type, c10::IntArrayRef shape) const {
    fits(t, name, type);
    if (!t.is_contiguous() || t.sizes() != shape)
      throw Bad{std::string(name) + " must be contiguous of shape " + shown(shape) + ", not " + shown(t.sizes())};
    return t.data_ptr();
  }
  // A BF16 [M, N] matrix with contiguous rows that are apart (rows_apart); ld: its row stride (0, for one row: N).
  void* rows(const at::Tensor& t, const char* name, int64_t M, int64_t N, int64_t& ld) const {
    fits(t, name, at::kBFloat16);
    if (t.dim() != 2 || t.size(0) != M || t.size(1) != N)
      throw Bad{std::string(name) + " must have shape " + shown({M, N}) + ", not " + shown(t.sizes())};
    if (N > 1 && t.stride(1) != 1) throw Bad{std::string(name) + " must have contiguous rows"};
    ld = M > 1 ? t.stride(0) : 0;
    return t.data_ptr();
  }
  at::Tensor empty(c10::IntArrayRef shape, at::ScalarType type) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, dev)));
  }
  at::Tensor given_or(PyObject* o, const char* name, c10::IntArrayRef shape, at::ScalarType type) const {
    return o == Py_None ? empty(shape, type) : tensor(o, name);
  }
};

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Bad{"a size must be an integer"};
  }
  return v;
}

int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};                       // an object without a truth value
  return v;
}

// The library's call, without the interpreter's lock: a full launch queue makes it wait,
// and the other Python threads need not.
template <typename F>
nvq_status unlocked(F f) {
  struct Released {
    PyThreadState* state = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(state); }
  } released;
  return f();
}

// (codes, scales) or (codes, scales, t), held: they may come in a list that another thread changes meanwhile.
struct Pair {
  at::Tensor codes, scales, t;
  Pair() = default;
  Pair(PyObject* o, const char* name, Py_ssize_t n) {
    if (!(PyTuple_Check(o) || PyList_Check(o)) || PySequence_Fast_GET_SIZE(o) != n)
      throw Bad{std::string(name) + (n == 3 ? " must be (codes, scales, t)" : " must be (packed_codes, packed_scales)")};
    PyObject** v = PySequence_Fast_ITEMS(o);
    codes = tensor(v[0], name);
    scales = tensor(v[1], name);
    if (n == 3) t = tensor(v[2], name);
  }
};

int64_t tiled_scales(int64_t rows, int64_t K) { return (rows + 127) / 128 * 128 * (K / 16); }

struct Nvfp4 {
  Pair q;
  const uint8_t *codes = nullptr, *scales = nullptr;
  const float* t = nullptr;
  Nvfp4(const Call& c, Pair held, const char* name, int64_t rows, int64_t K) : q(std::move(held)) {
    codes = static_cast<uint8_t*>(c.flat(q.codes, name, at::kByte, rows * (K / 2)));
    scales = static_cast<uint8_t*>(c.flat(q.scales, name, at::kByte, tiled_scales(rows, K)));
    t = static_cast<float*>(c.flat(q.t, name, at::kFloat, 1));
  }
  Nvfp4(const Call& c, PyObject* o, const char* name, int64_t rows, int64_t K) : Nvfp4(c, Pair(o, name, 3), name, rows, K) {}
  Nvfp4() = default;      // none
};

struct Int4 {
  Pair q;
  const uint8_t* codes = nullptr;
  const void* scales = nullptr;
  Int4(const Call& c, PyObject* o, const char* name, int64_t rows, int64_t K) : q(o, name, 2) {
    codes = static_cast<uint8_t*>(c.flat(q.codes, name, at::kByte, rows * K / 2));
    scales = c.flat(q.scales, name, at::kByte, rows * (K / 128) * 2);
  }
  Int4() = default;       // none
};

nvq_epilogue epilogue(const Call& c, PyObject* bias, PyObject* act, PyObject* residual, const at::Tensor& y, int64_t M,
                      int64_t N, void** yp) {
  nvq_epilogue e = {};
  if (bias != Py_None) e.bias_bf16 = c.exact(tensor(bias, "bias"), "bias", at::kBFloat16, {N});
  if (residual != Py_None) e.residual_bf16 = c.rows(tensor(residual, "residual"), "residual", M, N, e.residual_stride);
  *yp = c.rows(y, "y", M, N, e.y_stride);
  e.activation = (int)integer(act);
  return e;
}

PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));   // takes the new reference
  return r;
}

PyObject* status(nvq_status s) { return PyLong_FromLong((long)s); }

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
  } catch (const Bad& b) {
    PyErr_SetString(PyExc_ValueError, b.what.c_str());
  } catch (...) {                                  // torch's own errors, out of memory among them
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// xq, wq, M, N, K, bias, activation, residual, y
PyObject* w4a4(PyObject* const* a) {
  rows_apart(a[7], "residual");
  rows_apart(a[8], "y");
  const int64_t M = integer(a[2]), N = integer(a[3]), K = integer(a[4]);
  Pair xq(a[0], "xq", 3);
  const Call c(xq.codes);
  const Nvfp4 x(c, std::move(xq), "xq", M, K), w(c, a[1], "wq", N, K);
  const at::Tensor y = c.given_or(a[8], "y", {M, N}, at::kBFloat16);
  void* yp;
  const nvq_epilogue e = epilogue(c, a[5], a[6], a[7], y, M, N, &yp);
  const nvq_status s = unlocked([&] { return g.w4a4(x.codes, x.scales, x.t, w.codes, w.scales, w.t, yp, M, N, K, &e, c.stream()); });
  return s == NVQ_OK ? THPVariable_Wrap(y) : status(s);
}

// x, (packed_codes, packed_scales), N, bias, activation, residual, y
PyObject* w4a16(PyObject* const* a) {
  rows_apart(a[5], "residual");
  rows_apart(a[6], "y");
  const at::Tensor& x = tensor(a[0], "x");
  const Call c(x);
  if (x.dim() != 2) throw Bad{"x must be [M, K]"};
  const int64_t M = x.size(0), K = x.size(1), N = integer(a[2]);
  const void* xp = c.flat(x, "x", at::kBFloat16, 0);
  const Int4 w(c, a[1], "packed weights", N, K);
  const at::Tensor y = c.given_or(a[6], "y", {M, N}, at::kBFloat16);
  void* yp;
  const nvq_epilogue e = epilogue(c, a[3], a[4], a[5], y, M, N, &yp);
  const nvq_status s = unlocked([&] { return g.w4a16(xp, w.codes, w.scales, yp, M, N, K, &e, c.stream()); });
  return s == NVQ_OK ? THPVariable_Wrap(y) : status(s);
}

// x, w4a4, w4a16, N, bias, activation, residual, crossover_m, y, workspace
PyObject* linear(PyObject* const* a) {
  rows_apart(a[6], "residual");
  rows_apart(a[8], "y");
  const at::Tensor& x = tensor(a[0], "x");
  const Call c(x);
  if (x.dim() != 2) throw Bad{"x must be [M, K]"};
  const int64_t M = x.size(0), K = x.size(1), N = integer(a[3]), crossover = integer(a[7]);
  const void* xp = c.flat(x, "x", at::kBFloat16, 0);
  const Nvfp4 w4a4 = a[1] == Py_None ? Nvfp4() : Nvfp4(c, a[1], "w4a4", N, K);
  const Int4 w4a16 = a[2] == Py_None ? Int4() : Int4(c, a[2], "w4a16", N, K);
  const at::Tensor y = c.given_or(a[8], "y", {M, N}, at::kBFloat16);
  const at::Tensor work = c.given_or(a[9], "workspace", {(int64_t)g.linear_bytes(M, N, K, crossover)}, at::kByte);
  void* wp = c.flat(work, "workspace", at::kByte, 0);
  void* yp;
  const nvq_epilogue e = epilogue(c, a[4], a[5], a[6], y, M, N, &yp);
  const nvq_status s = unlocked([&] {
    return g.linear(xp, M, N, K, w4a4.codes, w4a4.scales, w4a4.t, w4a16.codes, w4a16.scales, crossover, yp, &e, wp, work.numel(),
                    c.stream());
  });
  return s == NVQ_OK ? THPVariable_Wrap(y) : status(s);
}

struct Tokens {
  int64_t T, H;
  const void* x;
  Tokens(const Call& c, const at::Tensor& t) {
    if (t.dim() != 2) throw Bad{"x must be [T, H]"};
    T = t.size(0);
    H = t.size(1);
    x = c.flat(t, "x", at::kBFloat16, 0);
  }
};

struct Choices {
  at::Tensor ids, weights;
  int32_t* ip;
  float* wp;
  Choices(const Call& c, PyObject* i, PyObject* w, int64_t T, int64_t topk)
      : ids(c.given_or(i, "ids", {T, topk}, at::kInt)), weights(c.given_or(w, "weights", {T, topk}, at::kFloat)) {
    ip = static_cast<int32_t*>(c.exact(ids, "ids", at::kInt, {T, topk}));
    wp = static_cast<float*>(c.exact(weights, "weights", at::kFloat, {T, topk}));
  }
};

struct Layer {
  Int4 gate_up, down;
  at::Tensor y, work;
  void *yp, *rp = nullptr, *wp;
  Layer(const Call& c, PyObject* gu, PyObject* d, PyObject* residual, PyObject* out, PyObject* ws, int64_t T, int64_t E,
        int64_t H, int64_t I, int64_t topk)
      : gate_up(c, gu, "gate_up", E * 2 * I, H), down(c, d, "down", E * H, I), y(c.given_or(out, "y", {T, H}, at::kBFloat16)),
        work(c.given_or(ws, "workspace", {(int64_t)g.moe_bytes(T, H, I, (int)topk)}, at::kByte)) {
    yp = c.exact(y, "y", at::kBFloat16, {T, H});
    if (residual != Py_None) rp = c.exact(tensor(residual, "residual"), "residual", at::kBFloat16, {T, H});
    wp = c.flat(work, "workspace", at::kByte, 0);
  }
};

int64_t small_count(PyObject* o) {                 // topk: an int in the C call
  const int64_t v = integer(o);
  if (v < 0 || v > 1 << 20) throw Bad{"topk out of range"};
  return v;
}

// x, w_router, topk, renormalize, ids, weights
PyObject* route(PyObject* const* a) {
  const int renormalize = truth(a[3]);
  const at::Tensor &x = tensor(a[0], "x"), &wr = tensor(a[1], "w_router");
  const Call c(x);
  const Tokens t(c, x);
  if (wr.dim() != 2) throw Bad{"w_router must be [E, H]"};
  const int64_t E = wr.size(0), topk = small_count(a[2]);
  const void* rp = c.exact(wr, "w_router", at::kBFloat16, {E, t.H});
  const Choices k(c, a[4], a[5], t.T, topk);
  const nvq_status s = unlocked([&] { return g.route(t.x, rp, t.T, E, t.H, (int)topk, renormalize, k.ip, k.wp, c.stream()); });
  return s == NVQ_OK ? tuple_of({k.ids, k.weights}) : status(s);
}

// x, ids, weights, gate_up, down, E, I, residual, y, workspace
PyObject* experts(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "x"), &ids = tensor(a[1], "ids");
  tensor(a[2], "weights");                         // an input here: Choices would make one
  const Call c(x);
  const Tokens t(c, x);
  if (ids.dim() != 2) throw Bad{"ids must be [T, topk]"};
  const int64_t topk = ids.size(1), E = integer(a[5]), I = integer(a[6]);
  const Choices k(c, a[1], a[2], t.T, topk);
  if (topk > 1 << 20) throw Bad{"topk out of range"};
  const Layer l(c, a[3], a[4], a[7], a[8], a[9], t.T, E, t.H, I, topk);
  const nvq_status s = unlocked([&] {
    return g.experts(t.x, k.ip, k.wp, l.gate_up.codes, l.gate_up.scales, l.down.codes, l.down.scales, l.rp, l.yp, t.T, E, t.H, I,
                     (int)topk, l.wp, l.work.numel(), c.stream());
  });
  return s == NVQ_OK ? THPVariable_Wrap(l.y) : status(s);
}

// x, w_router, gate_up, down, I, topk, renormalize, residual, ids, weights, y, workspace
PyObject* moe(PyObject* const* a) {
  const int renormalize = truth(a[6]);
  const at::Tensor &x = tensor(a[0], "x"), &wr = tensor(a[1], "w_router");
  const Call c(x);
  const Tokens t(c, x);
  if (wr.dim() != 2) throw Bad{"w_router must be [E, H]"};
  const int64_t E = wr.size(0), I = integer(a[4]), topk = small_count(a[5]);
  const void* rp = c.exact(wr, "w_router", at::kBFloat16, {E, t.H});
  const Choices k(c, a[8], a[9], t.T, topk);
  const Layer l(c, a[2], a[3], a[7], a[10], a[11], t.T, E, t.H, I, topk);
  const nvq_status s = unlocked([&] {
    return g.moe(t.x, rp, l.gate_up.codes, l.gate_up.scales, l.down.codes, l.down.scales, l.rp, l.yp, k.ip, k.wp, t.T, E, t.H, I,
                 (int)topk, renormalize, l.wp, l.work.numel(), c.stream());
  });
  return s == NVQ_OK ? tuple_of({l.y, k.ids, k.weights}) : status(s);
}

// The addresses of the library's entry points, in the order of Entry.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void* p[8];
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "bind takes eight addresses");
    return nullptr;
  }
  for (int i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g.w4a4 = reinterpret_cast<decltype(g.w4a4)>(p[0]);
  g.w4a16 = reinterpret_cast<decltype(g.w4a16)>(p[1]);
  g.linear = reinterpret_cast<decltype(g.linear)>(p[2]);
  g.linear_bytes = reinterpret_cast<decltype(g.linear_bytes)>(p[3]);
  g.route = reinterpret_cast<decltype(g.route)>(p[4]);
  g.moe_bytes = reinterpret_cast<decltype(g.moe_bytes)>(p[5]);
  g.experts = reinterpret_cast<decltype(g.experts)>(p[6]);
  g.moe = reinterpret_cast<decltype(g.moe)>(p[7]);
  Py_RETURN_NONE;
}

#define FAST(name, fn, count) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<fn, count>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL, nullptr},
    FAST("nvfp4_gemm_w4a4_epilogue", w4a4, 9),
    FAST("w4a16_gemm_epilogue", w4a16, 7),
    FAST("nvq_linear_epilogue", linear, 10),
    FAST("moe_route", route, 6),
    FAST("w4a16_moe_experts", experts, 10),
    FAST("w4a16_moe", moe, 12),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", NVQ_BINDING_TAG) < 0) {   // the build looks for it in the file
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
