// Argument marshalling of the fine-tuning operators, as the Python binding does
// it for the layer's calls: types, shapes and devices are checked, outputs are
// allocated with PyTorch, the C entry point is called on the current stream.
// These calls are short (a kernel of under 5 us on a decode batch), so the
// marshalling is compiled: a call of combine_backward takes 4.5 us of host time
// here and 10.4 through ctypes and torch's Python functions; balance_loss, with
// its five allocations, 7.1 against 17.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <initializer_list>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe.h"

namespace {

struct Error {};   // a Python exception is set

PyObject* g_check = nullptr;   // the binding's status check: raises for a status that is not MOE_OK

template <typename... A>
[[noreturn]] void fail(PyObject* type, const char* format, A... a) {
  PyErr_Format(type, format, a...);
  throw Error();
}

using Type = at::ScalarType;
constexpr uint64_t bit(Type t) { return 1ull << static_cast<int>(t); }
constexpr uint64_t kF32 = bit(Type::Float), kI32 = bit(Type::Int), kBf16 = bit(Type::BFloat16), kByte = bit(Type::Byte);
constexpr uint64_t kAct = kBf16 | kF32, kLogits = kF32 | bit(Type::Half) | kBf16, kMask = kByte | bit(Type::Bool);

int code(Type t) { return t == Type::Float ? MOE_F32 : t == Type::Half ? MOE_F16 : MOE_BF16; }

const char* name_of(Type t) { return c10::toString(t); }

// A tensor argument; None is nullptr where it may be
const at::Tensor* tensor(PyObject* o, const char* what, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s: a tensor is wanted", what);
  return &THPVariable_Unpack(o);
}

int64_t dim(const at::Tensor& t, const char* what, int dims, int i) {
  if (t.dim() != dims) fail(PyExc_ValueError, "%s: %d dimensions where %d are wanted", what, static_cast<int>(t.dim()), dims);
  return t.size(i);
}

int as_int(int64_t v, const char* what) {
  if (v > INT32_MAX || v < INT32_MIN) fail(PyExc_ValueError, "%s: %lld is past 32 bits", what, static_cast<long long>(v));
  return static_cast<int>(v);
}

struct Call {
  c10::Device device;

  // on the device of the call's first tensor, which has to be the current one: kernels launch there
  explicit Call(const at::Tensor& first) : device(first.device()) {
    if (!first.is_cuda()) fail(PyExc_ValueError, "tensors must be contiguous CUDA tensors");
    if (device.index() != c10::cuda::current_device())
      fail(PyExc_ValueError, "tensors on cuda:%d, but the current device is cuda:%d", static_cast<int>(device.index()),
           static_cast<int>(c10::cuda::current_device()));
  }

  // The address of a tensor the call reads or writes (nullptr for none), checked: contiguous, on the
  // call's device, of one of these types and of this shape.
  void* at(const at::Tensor* t, const char* what, uint64_t types, std::initializer_list<int64_t> shape) const {
    if (!t) return nullptr;
    if (t->device() != device)
      fail(PyExc_ValueError, "%s: every tensor of a call must be a CUDA tensor on one device (cuda:%d)", what,
           static_cast<int>(device.index()));
    if (!(types >> static_cast<int>(t->scalar_type()) & 1))
      fail(PyExc_TypeError, "%s: unsupported dtype %s", what, name_of(t->scalar_type()));
    if (!t->sizes().equals(at::IntArrayRef(shape))) {
      const std::string has = c10::str(t->sizes()), wants = c10::str(at::IntArrayRef(shape));
      fail(PyExc_ValueError, "%s: shape %s where %s is wanted", what, has.c_str(), wants.c_str());
    }
    if (!t->is_contiguous()) fail(PyExc_ValueError, "%s: tensors must be contiguous CUDA tensors", what);
    return t->data_ptr();
  }

  at::Tensor empty(Type type, std::initializer_list<int64_t> shape) const {
    return at::detail::empty_cuda(at::IntArrayRef(shape), type, device, std::nullopt);
  }

  // the caller's workspace, or a new one of this size; `keep` holds it
  void* workspace(const at::Tensor* ws, size_t bytes, at::Tensor& keep, size_t& has) const {
    if (!ws) {
      keep = empty(Type::Byte, {static_cast<int64_t>(bytes < 256 ? 256 : bytes)});
      ws = &keep;
    } else if (ws->device() != device || ws->scalar_type() != Type::Byte || !ws->is_contiguous()) {
      fail(PyExc_ValueError, "ws: a contiguous uint8 tensor on the call's device is wanted");
    }
    has = ws->numel();
    return ws->data_ptr();
  }

  void* stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }
};

void check(int status, const char* what) {
  if (status == MOE_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "is", status, what);
  Py_XDECREF(r);
  throw Error();
}

Type dtype(PyObject* o, const char* what, uint64_t types) {
  if (!THPDtype_Check(o)) fail(PyExc_TypeError, "%s: a torch.dtype is wanted", what);
  const Type t = reinterpret_cast<THPDtype*>(o)->scalar_type;
  if (!(types >> static_cast<int>(t) & 1)) fail(PyExc_TypeError, "%s: unsupported dtype %s", what, name_of(t));
  return t;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Error();
  return v != 0;
}

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* wrap_or_none(const at::Tensor* t) {
  if (t) return THPVariable_Wrap(*t);
  Py_RETURN_NONE;
}
PyObject* tuple(std::initializer_list<PyObject*> items) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
  Py_ssize_t i = 0;
  for (PyObject* o : items) PyTuple_SET_ITEM(r, i++, o);
  return r;
}

template <typename F>
int unlocked(F call) {   // the C call without the interpreter's lock, as it may wait for the GPU's queue
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = call();
  Py_END_ALLOW_THREADS;
  return status;
}

// (dout, Y, token_to_row, topk_w, has_shared, offsets, want_dY, want_dw, dY)
PyObject* combine_backward(PyObject* const* a) {
  const at::Tensor &dout = *tensor(a[0], "dout"), &t2r = *tensor(a[2], "token_to_row"), &w = *tensor(a[3], "topk_w");
  const at::Tensor *Y = tensor(a[1], "Y", true), *offsets = tensor(a[5], "offsets", true), *into = tensor(a[8], "dY", true);
  const bool shared = truth(a[4]), want_dY = truth(a[6]), want_dw = truth(a[7]);
  const Call c(dout);
  const int64_t T = dim(t2r, "token_to_row", 2, 0), k = t2r.size(1), d = dim(dout, "dout", 2, 1);
  const int64_t rows = T * k + (shared ? T : 0), E = offsets ? offsets->numel() - 1 - shared : 0;
  const void* p_dout = c.at(&dout, "dout", kAct, {T, d});
  const int* p_t2r = static_cast<int*>(c.at(&t2r, "token_to_row", kI32, {T, k}));
  const float* p_w = static_cast<float*>(c.at(&w, "topk_w", kF32, {T, k}));
  const int* p_off = static_cast<int*>(c.at(offsets, "offsets", kI32, {E + 1 + shared}));
  const void* p_Y = c.at(Y, "Y", kBf16, {rows, d});
  at::Tensor dY, dw;
  void* p_dY = nullptr;
  if (want_dY) {
    if (into) dY = *into;
    else dY = c.empty(Type::BFloat16, {rows, d});
    if (!into && offsets) dY.zero_();   // rows of no token
    p_dY = c.at(&dY, "dY", kBf16, {rows, d});
  }
  if (want_dw) dw = c.empty(Type::Float, {T, k});
  const int nT = as_int(T, "tokens"), nd = as_int(d, "columns"), nk = as_int(k, "slots"), nE = as_int(E, "experts");
  float* p_dw = want_dw ? dw.data_ptr<float>() : nullptr;
  void* stream = c.stream();
  check(unlocked([&] {
          return moe_combine_backward(p_dout, code(dout.scalar_type()), p_Y, p_t2r, p_w, p_off, nE, shared, nT, nd, nk,
                                      p_dY, p_dw, stream);
        }), "moe_combine_backward");
  return tuple({wrap_or_none(want_dY ? &dY : nullptr), wrap_or_none(want_dw ? &dw : nullptr)});
}

int64_t sequences(const at::Tensor* offsets) {
  if (offsets && offsets->numel() < 2) fail(PyExc_ValueError, "seq_offsets: at least two entries are wanted");
  return offsets ? offsets->numel() - 1 : 1;
}

// (logits, topk_idx, alpha, seq_offsets, mask, want_prob, ws)
PyObject* balance_loss(PyObject* const* a) {
  const at::Tensor &logits = *tensor(a[0], "logits"), &idx = *tensor(a[1], "topk_idx");
  const double alpha = PyFloat_AsDouble(a[2]);
  if (alpha == -1.0 && PyErr_Occurred()) throw Error();
  const at::Tensor *offsets = tensor(a[3], "seq_offsets", true), *mask = tensor(a[4], "mask", true), *ws = tensor(a[6], "ws", true);
  const bool want_prob = truth(a[5]);
  const Call c(logits);
  const int64_t T = dim(logits, "logits", 2, 0), E = logits.size(1), k = dim(idx, "topk_idx", 2, 1), S = sequences(offsets);
  const void* p_l = c.at(&logits, "logits", kLogits, {T, E});
  const int* p_i = static_cast<int*>(c.at(&idx, "topk_idx", kI32, {T, k}));
  const int* p_o = static_cast<int*>(c.at(offsets, "seq_offsets", kI32, {S + 1}));
  const uint8_t* p_m = static_cast<uint8_t*>(c.at(mask, "mask", kMask, {T}));
  const int nT = as_int(T, "tokens"), nE = as_int(E, "experts"), nk = as_int(k, "slots"), nS = as_int(S, "sequences");
  at::Tensor keep, prob;
  size_t bytes;
  void* p_ws = c.workspace(ws, moe_balance_loss_workspace_size(nT, nE, nS), keep, bytes);
  at::Tensor counts = c.empty(Type::Int, {S, E}), loss = c.empty(Type::Float, {1}), coef = c.empty(Type::Float, {S});
  if (want_prob) prob = c.empty(Type::Float, {S, E});
  float *p_loss = loss.data_ptr<float>(), *p_prob = want_prob ? prob.data_ptr<float>() : nullptr, *p_coef = coef.data_ptr<float>();
  int* p_counts = counts.data_ptr<int>();
  void* stream = c.stream();
  check(unlocked([&] {
          return moe_balance_loss(p_l, code(logits.scalar_type()), p_i, nT, nE, nk, p_o, nS, p_m, static_cast<float>(alpha),
                                  p_loss, p_counts, p_prob, p_coef, p_ws, bytes, stream);
        }), "moe_balance_loss");
  return tuple({wrap(loss), wrap(counts), wrap_or_none(want_prob ? &prob : nullptr), wrap(coef)});
}

// (logits, topk_idx, d_topk_w, renormalize, counts, coef, d_loss, seq_offsets, mask, out_dtype, out)
PyObject* router_backward(PyObject* const* a) {
  const at::Tensor &logits = *tensor(a[0], "logits"), &idx = *tensor(a[1], "topk_idx");
  const at::Tensor *d_w = tensor(a[2], "d_topk_w", true), *counts = tensor(a[4], "counts", true), *coef = tensor(a[5], "coef", true);
  const at::Tensor *d_loss = tensor(a[6], "d_loss", true), *offsets = tensor(a[7], "seq_offsets", true);
  const at::Tensor *mask = tensor(a[8], "mask", true), *into = tensor(a[10], "out", true);
  const bool renorm = truth(a[3]);
  const Call c(logits);
  const int64_t T = dim(logits, "logits", 2, 0), E = logits.size(1), k = dim(idx, "topk_idx", 2, 1), S = sequences(offsets);
  const void* p_l = c.at(&logits, "logits", kLogits, {T, E});
  const int* p_i = static_cast<int*>(c.at(&idx, "topk_idx", kI32, {T, k}));
  const float* p_g = static_cast<float*>(c.at(d_w, "d_topk_w", kF32, {T, k}));
  const int* p_o = static_cast<int*>(c.at(offsets, "seq_offsets", kI32, {S + 1}));
  const uint8_t* p_m = static_cast<uint8_t*>(c.at(mask, "mask", kMask, {T}));
  const int* p_n = static_cast<int*>(c.at(counts, "counts", kI32, {S, E}));
  const float* p_c = static_cast<float*>(c.at(coef, "coef", kF32, {S}));
  if (d_loss && d_loss->numel() != 1) fail(PyExc_ValueError, "d_loss: one value is wanted");
  const at::Tensor one = d_loss ? d_loss->reshape({1}) : at::Tensor();
  const float* p_d = static_cast<float*>(c.at(d_loss ? &one : nullptr, "d_loss", kF32, {1}));
  const at::Tensor out = into ? *into : c.empty(dtype(a[9], "out_dtype", kLogits), {T, E});
  void* p_out = c.at(&out, "out", kLogits, {T, E});
  const int nT = as_int(T, "tokens"), nE = as_int(E, "experts"), nk = as_int(k, "slots"), nS = as_int(S, "sequences");
  void* stream = c.stream();
  check(unlocked([&] {
          return moe_router_backward(p_l, code(logits.scalar_type()), p_i, p_g, nT, nE, nk, renorm, p_o, nS, p_m, p_n, p_c,
                                     p_d, p_out, code(out.scalar_type()), stream);
        }), "moe_router_backward");
  return wrap(out);
}

// (row_adapter, n, ws)
PyObject* adapter_plan(PyObject* const* a) {
  const at::Tensor& row = *tensor(a[0], "row_adapter");
  const long n = PyLong_AsLong(a[1]);
  if (n == -1 && PyErr_Occurred()) throw Error();
  const at::Tensor* ws = tensor(a[2], "ws", true);
  const int nn = as_int(n, "adapters");   // first: offsets is made for n, the kernels write nn + 1 entries
  const Call c(row);
  const int64_t rows = row.numel();
  const int* p_r = static_cast<int*>(c.at(&row, "row_adapter", kI32, {rows}));
  const int nr = as_int(rows, "rows");
  at::Tensor keep;
  size_t bytes;
  void* p_ws = c.workspace(ws, moe_adapter_plan_workspace_size(nr, nn), keep, bytes);
  at::Tensor offsets = c.empty(Type::Int, {(n > 0 ? n : 0) + 1}), order = c.empty(Type::Int, {rows});
  int *p_off = offsets.data_ptr<int>(), *p_ord = order.data_ptr<int>();
  void* stream = c.stream();
  check(unlocked([&] { return moe_adapter_plan(p_r, nr, nn, p_off, p_ord, p_ws, bytes, stream); }), "moe_adapter_plan");
  return tuple({wrap(offsets), wrap(order)});
}

// what lora and its gradient share: x, A, B, the plan and the scales
struct Adapters {
  const at::Tensor &x, &A, &B;
  int64_t rows, d, n, R, N;
  const void *p_x, *p_A, *p_B;
  const int *p_off, *p_ord;
  const float* p_s;
  int nrows, nd, nn, nR, nN;

  Adapters(const Call& c, PyObject* ox, PyObject* oA, PyObject* oB, PyObject* off, PyObject* ord, PyObject* scale)
      : x(*tensor(ox, "x")), A(*tensor(oA, "A")), B(*tensor(oB, "B")) {
    rows = dim(x, "x", 2, 0), d = x.size(1), n = dim(A, "A", 3, 0), R = A.size(1), N = dim(B, "B", 3, 1);
    p_x = c.at(&x, "x", kBf16, {rows, d}), p_A = c.at(&A, "A", kBf16, {n, R, d}), p_B = c.at(&B, "B", kBf16, {n, N, R});
    p_off = static_cast<int*>(c.at(tensor(off, "offsets"), "offsets", kI32, {n + 1}));
    p_ord = static_cast<int*>(c.at(tensor(ord, "order"), "order", kI32, {rows}));
    p_s = static_cast<float*>(c.at(tensor(scale, "scale", true), "scale", kF32, {n}));
    nrows = as_int(rows, "rows"), nd = as_int(d, "columns"), nn = as_int(n, "adapters"), nR = as_int(R, "rank");
    nN = as_int(N, "columns");
  }
};

// (x, A, B, offsets, order, scale, base, out_dtype, out, want_h, ws)
PyObject* lora(PyObject* const* a) {
  const Call c(*tensor(a[0], "x"));
  const Adapters p(c, a[0], a[1], a[2], a[3], a[4], a[5]);
  const at::Tensor *base = tensor(a[6], "base", true), *into = tensor(a[8], "out", true), *ws = tensor(a[10], "ws", true);
  const bool want_h = truth(a[9]);
  const at::Tensor out = into ? *into : c.empty(base ? base->scalar_type() : dtype(a[7], "out_dtype", kAct), {p.rows, p.N});
  void* p_out = c.at(&out, "out", kAct, {p.rows, p.N});
  const void* p_base = c.at(base, "base", bit(out.scalar_type()), {p.rows, p.N});
  at::Tensor h, keep;
  if (want_h) h = c.empty(Type::Float, {p.rows, p.R});
  const size_t need = moe_lora_workspace_size(p.nrows, p.nn, p.nd, p.nN, p.nR);
  size_t bytes = 0;
  void* p_ws = need || ws ? c.workspace(ws, need, keep, bytes) : nullptr;
  float* p_h = want_h ? h.data_ptr<float>() : nullptr;
  void* stream = c.stream();
  check(unlocked([&] {
          return moe_lora(p.p_x, p.p_A, p.p_B, p.p_s, p.p_off, p.p_ord, p.nn, p.nrows, p.nd, p.nN, p.nR, p_base, p_out,
                          code(out.scalar_type()), p_h, p_ws, bytes, stream);
        }), "moe_lora");
  return want_h ? tuple({wrap(out), wrap(h)}) : wrap(out);
}

// (dC, x, h, A, B, offsets, order, scale, dx_base, want_dx, want_grads, dx_dtype, dx, grad_dtype, ws)
PyObject* lora_backward(PyObject* const* a) {
  const at::Tensor &dC = *tensor(a[0], "dC"), &h = *tensor(a[2], "h");
  const Call c(dC);
  const Adapters p(c, a[1], a[3], a[4], a[5], a[6], a[7]);
  const at::Tensor *base = tensor(a[8], "dx_base", true), *into = tensor(a[12], "dx", true), *ws = tensor(a[14], "ws", true);
  const bool want_dx = truth(a[9]), want_grads = truth(a[10]);
  const void* p_dC = c.at(&dC, "dC", kBf16, {p.rows, p.N});
  const float* p_h = static_cast<float*>(c.at(&h, "h", kF32, {p.rows, p.R}));
  at::Tensor dx, dA, dB, keep;
  void *p_dx = nullptr, *p_dA = nullptr, *p_dB = nullptr;
  const void* p_base = nullptr;
  int dx_code = MOE_BF16;
  if (want_dx) {
    if (into) dx = *into;
    else dx = c.empty(base ? base->scalar_type() : dtype(a[11], "dx_dtype", kAct), {p.rows, p.d});
    p_dx = c.at(&dx, "dx", kAct, {p.rows, p.d});
    p_base = c.at(base, "dx_base", bit(dx.scalar_type()), {p.rows, p.d});
    dx_code = code(dx.scalar_type());
  }
  const Type gt = dtype(a[13], "grad_dtype", kAct);
  if (want_grads) {
    dA = c.empty(gt, {p.n, p.R, p.d}), dB = c.empty(gt, {p.n, p.N, p.R});
    p_dA = dA.data_ptr(), p_dB = dB.data_ptr();
  }
  size_t bytes;
  void* p_ws = c.workspace(ws, moe_lora_backward_workspace_size(p.nrows, p.nn, p.nd, p.nN, p.nR), keep, bytes);
  void* stream = c.stream();
  check(unlocked([&] {
          return moe_lora_backward(p_dC, p.p_x, p_h, p.p_A, p.p_B, p.p_s, p.p_off, p.p_ord, p.nn, p.nrows, p.nd, p.nN, p.nR,
                                   p_base, p_dx, dx_code, p_dA, p_dB, code(gt), p_ws, bytes, stream);
        }), "moe_lora_backward");
  return tuple({wrap_or_none(want_dx ? &dx : nullptr), wrap_or_none(want_grads ? &dA : nullptr),
                wrap_or_none(want_grads ? &dB : nullptr)});
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments where %d are wanted", n, N);
    return nullptr;
  }
  HANDLE_TH_ERRORS   // C++ exceptions of the allocator (out of memory) become Python's
  try {
    return F(args);
  } catch (const Error&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_check(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_check, f);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<combine_backward, 9>("combine_backward"), method<balance_loss, 7>("balance_loss"),
                           method<router_backward, 11>("router_backward"),  method<adapter_plan, 3>("adapter_plan"),
                           method<lora, 11>("lora"),                        method<lora_backward, 15>("lora_backward"),
                           {"set_check", set_check, METH_O, nullptr},       {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops(void) { return PyModule_Create(&g_module); }
