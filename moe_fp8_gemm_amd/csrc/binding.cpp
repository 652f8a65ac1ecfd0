// Argument marshalling of the mixture-of-experts, layer and int8 operators for torch, in C++.
//
// A decoding step's calls work for a few microseconds, less than their arguments
// cost to check and their outputs to allocate from Python (8 to 11 us a call; 3 to
// 6 us from here).  Like the Python side of the binding this file only checks
// tensors, allocates the outputs that are not passed in and calls the C ABI of
// include/dgfp8.h with pointers, strides and the current stream of the tensors' device.
// Wrong types raise TypeError, wrong shapes or values ValueError, and a status other
// than DG_SUCCESS the package's DgError.
#include <Python.h>

#include <cmath>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include "../../include/dgfp8.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;            // DgError(status, where)
PyObject* g_auto_workspace = nullptr;   // (device, bytes) -> zero-filled tensor of the current stream

// ---- arguments

struct Args {
  PyObject* const* a;
  const char* call;

  bool none(int i) const { return a[i] == Py_None; }
  const Tensor& tensor(int i, const char* name) const {
    TORCH_CHECK_TYPE(THPVariable_Check(a[i]), call, ": ", name, " must be a tensor");
    return THPVariable_Unpack(a[i]);
  }
  int64_t integer(int i, const char* name) const {
    const long long v = PyLong_AsLongLong(a[i]);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      TORCH_CHECK_TYPE(false, call, ": ", name, " must be an integer");
    }
    return v;
  }
  // The C ABI's int parameters: a value outside int would change on its way.
  int small(int i, const char* name) const {
    const int64_t v = integer(i, name);
    TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, call, ": ", name, " is out of range: ", v);
    return (int)v;
  }
  double number(int i, const char* name) const {
    const double v = PyFloat_AsDouble(a[i]);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      TORCH_CHECK_TYPE(false, call, ": ", name, " must be a number");
    }
    return v;
  }
  bool truth(int i) const {
    const int v = PyObject_IsTrue(a[i]);
    if (v < 0) throw python_error();
    return v != 0;
  }
  int one_of(int i, const char* name, const char* zero, const char* one) const {
    TORCH_CHECK_TYPE(PyUnicode_Check(a[i]), call, ": ", name, " must be a string");
    if (PyUnicode_CompareWithASCIIString(a[i], zero) == 0) return 0;
    TORCH_CHECK_VALUE(PyUnicode_CompareWithASCIIString(a[i], one) == 0, call, ": ", name, " must be '", zero, "' or '",
                      one, "'");
    return 1;
  }
};

// ---- tensors

constexpr unsigned kF32 = 1, kBF16 = 2, kF16 = 4, kI32 = 8, kI8 = 16, kE4M3 = 32, kU8 = 64;

unsigned type_bit(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return kF32;
    case at::kBFloat16: return kBF16;
    case at::kHalf: return kF16;
    case at::kInt: return kI32;
    case at::kChar: return kI8;
    case at::kFloat8_e4m3fn: return kE4M3;
    case at::kByte: return kU8;
    default: return 0;
  }
}

int dtype_of(const Tensor& t) {
  return t.scalar_type() == at::kFloat ? DG_F32 : t.scalar_type() == at::kBFloat16 ? DG_BF16 : DG_F16;
}

// A device tensor of one of the types and of `dim` dimensions, the last of unit stride.
const Tensor& check(const Args& a, const Tensor& t, const char* name, unsigned types, int64_t dim) {
  TORCH_CHECK_TYPE(t.is_cuda() && (type_bit(t) & types) != 0, a.call, ": ", name, " is a ", t.scalar_type(),
                   " tensor on ", t.device(), ", which is not supported");
  TORCH_CHECK_VALUE(t.dim() == dim, a.call, ": ", name, " must have ", dim, " dimensions, got ", t.dim());
  TORCH_CHECK_VALUE(t.stride(dim - 1) == 1 || t.numel() <= 1 || t.size(dim - 1) <= 1, a.call, ": ", name,
                    " must have unit stride along its last dimension");
  return t;
}
const Tensor& check(const Args& a, int i, const char* name, unsigned types, int64_t dim) {
  return check(a, a.tensor(i, name), name, types, dim);
}

void shape(const Args& a, const Tensor& t, const char* name, at::IntArrayRef want) {
  TORCH_CHECK_VALUE(t.sizes() == want, a.call, ": ", name, " must have shape ", want, ", got ", t.sizes());
}

// A new contiguous tensor, without the dispatcher's share of at::empty (0.5 us of a
// call's 4 to 7 for each tensor); with a row stride, a matrix whose rows begin that far
// apart.
Tensor fresh(at::IntArrayRef size, at::ScalarType type, const Tensor& like, int64_t row_stride = 0) {
  if (row_stride > 0) return at::detail::empty_strided_cuda(size, {row_stride, 1}, type, like.device());
  return at::detail::empty_cuda(size, type, like.device(), std::nullopt);
}

// An output of this shape: the one passed in, or a new one.
Tensor output(const Args& a, int i, const char* name, at::IntArrayRef want, at::ScalarType type, unsigned types,
              const Tensor& like) {
  if (a.none(i)) return fresh(want, type, like);
  const Tensor& t = check(a, i, name, types, (int64_t)want.size());
  shape(a, t, name, want);
  return t;
}

void same_device(const Args& a, const Tensor& first, std::initializer_list<const Tensor*> others) {
  for (const Tensor* t : others)
    TORCH_CHECK_VALUE(!t || !t->defined() || t->get_device() == first.get_device(), a.call, ": tensors are on ",
                      t->device(), " and ", first.device());
}

// Row stride (dimension d of d + 2); a matrix of at most one row may carry any.
int64_t ld(const Tensor& t, int64_t d = 0) {
  const int64_t s = t.stride(d), cols = t.size(d + 1);
  return s >= cols || t.size(d) > 1 ? s : cols;
}

template <class T = void>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
const float* f32(const Tensor& t) { return ptr<float>(t); }
const int32_t* i32(const Tensor& t) { return ptr<int32_t>(t); }

// torch's current stream of a tensor's device, which is made the current device
// for the call.
struct On {
  c10::DeviceGuard guard;
  void* stream;
  explicit On(const Tensor& t)
      : guard(t.device()), stream(c10::hip::getCurrentHIPStream(t.device().index()).stream()) {}
};

// True for DG_SUCCESS; otherwise the Python error is set.
bool done(dg_status st, const char* where) {
  if (st == DG_SUCCESS) return true;
  PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", (int)st, where) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_SetString(PyExc_RuntimeError, where);
  }
  return false;
}

PyObject* pair(const Tensor& x, const Tensor& y) {
  return Py_BuildValue("(NN)", THPVariable_Wrap(x), THPVariable_Wrap(y));
}

// The workspace argument: "auto" (the binding's own for the current stream, where
// the problem can use one), None or a tensor.
struct Workspace {
  Tensor t;
  void* p = nullptr;
  size_t bytes = 0;
};
Workspace workspace(const Args& a, int i, const Tensor& like, size_t need) {
  Workspace w;
  if (a.none(i)) return w;
  if (PyUnicode_Check(a.a[i])) {
    TORCH_CHECK_VALUE(PyUnicode_CompareWithASCIIString(a.a[i], "auto") == 0, a.call,
                      ": workspace must be 'auto', None or a tensor");
    if (need == 0) return w;
    THPObjectPtr dev(PyObject_GetAttrString(THPObjectPtr(THPVariable_Wrap(like)).get(), "device"));
    THPObjectPtr made(dev ? PyObject_CallFunction(g_auto_workspace, "On", dev.get(), (Py_ssize_t)need) : nullptr);
    if (!made) throw python_error();
    TORCH_CHECK_TYPE(THPVariable_Check(made.get()), a.call, ": workspace must be a tensor");
    w.t = THPVariable_Unpack(made.get());
  } else {
    w.t = a.tensor(i, "workspace");
  }
  TORCH_CHECK_TYPE(w.t.is_cuda() && w.t.is_contiguous(), a.call, ": workspace must be a contiguous device tensor");
  w.p = w.t.data_ptr();
  w.bytes = (size_t)w.t.nbytes();
  return w;
}

// ---- routing

PyObject* route_topk(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Args a{args, "route_topk"};
  const Tensor& x = check(a, 0, "logits", kF32 | kBF16 | kF16, 2);
  const On on(x);
  const int topk = a.small(1, "topk");
  const int score = a.one_of(2, "score", "softmax", "sigmoid");
  const int64_t t = x.size(0), e = x.size(1);
  Tensor bias;
  if (!a.none(3)) {
    bias = check(a, 3, "bias", kF32, 1);
    shape(a, bias, "bias", {e});
  }
  TORCH_CHECK_VALUE(e <= INT32_MAX && topk >= 0, a.call, ": topk must not be negative");
  Tensor idx = output(a, 9, "indices", {t, topk}, at::kInt, kI32, x);
  Tensor w = output(a, 10, "weights", {t, topk}, at::kFloat, kF32, x);
  same_device(a, x, {&bias, &idx, &w});
  if (!done(dg_route_topk(ptr(x), dtype_of(x), ld(x), bias.defined() ? f32(bias) : nullptr, ptr<int32_t>(idx), ld(idx),
                          ptr<float>(w), ld(w), t, (int)e, topk, a.small(4, "num_expert_groups"),
                          a.small(5, "topk_groups"), a.one_of(6, "group_score", "max", "top2"), score, a.truth(7),
                          (float)a.number(8, "scale"), on.stream),
            "dg_route_topk"))
    return nullptr;
  return pair(idx, w);
  END_HANDLE_TH_ERRORS
}

PyObject* route_topk_grad(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Args a{args, "route_topk_grad"};
  const Tensor& x = check(a, 0, "logits", kF32 | kBF16 | kF16, 2);
  const On on(x);
  const Tensor& idx = check(a, 1, "indices", kI32, 2);
  const Tensor& g = check(a, 2, "dweights", kF32, 2);
  const int64_t t = x.size(0), e = x.size(1), topk = idx.size(1);
  shape(a, idx, "indices", {t, topk});
  shape(a, g, "dweights", {t, topk});
  TORCH_CHECK_VALUE(e <= INT32_MAX && topk <= INT32_MAX, a.call, ": too many columns");
  Tensor dx = output(a, 6, "dlogits", {t, e}, x.scalar_type(), type_bit(x), x);
  same_device(a, x, {&idx, &g, &dx});
  if (!done(dg_route_topk_grad(ptr(x), dtype_of(x), ld(x), i32(idx), ld(idx), f32(g), ld(g), ptr(dx), ld(dx), t, (int)e,
                               (int)topk, a.one_of(3, "score", "softmax", "sigmoid"), a.truth(4),
                               (float)a.number(5, "scale"), on.stream),
            "dg_route_topk_grad"))
    return nullptr;
  return THPVariable_Wrap(dx);
  END_HANDLE_TH_ERRORS
}

// ---- expert layout

// contiguous: rows (or None); masked: max_m
PyObject* layout(PyObject* const* args, bool masked) {
  const Args a{args, masked ? "expert_layout_masked" : "expert_layout_contiguous"};
  const Tensor& idx = check(a, 0, "indices", kI32, 2);
  const int64_t t = idx.size(0), k = idx.size(1);
  const int experts = a.small(1, "num_experts");
  TORCH_CHECK_VALUE(k <= INT32_MAX, a.call, ": too many columns");
  int64_t rows = 0, max_m = 0;
  if (masked) {
    max_m = a.integer(2, "max_m");
    rows = max_m > 0 && experts > 0 && max_m <= INT32_MAX ? experts * max_m : 0;
  } else {
    rows = a.none(2) ? dg_expert_layout_rows(t, (int)k, experts) : a.integer(2, "rows");
  }
  const On on(idx);
  const int64_t alloc = rows > 0 && rows <= INT32_MAX ? rows : 0;
  Tensor m = masked ? Tensor() : fresh({alloc}, at::kInt, idx);
  Tensor row_slot = fresh({alloc}, at::kInt, idx), slot_row = fresh({t, k}, at::kInt, idx);
  Tensor counts = fresh({experts > 0 ? experts : 0}, at::kInt, idx);
  const size_t need = dg_expert_layout_workspace_size(t, (int)k, experts);
  Tensor ws = need ? fresh({(int64_t)need}, at::kByte, idx) : Tensor();
  void* wp = need ? ws.data_ptr() : nullptr;
  const dg_status st =
      masked ? dg_expert_layout_masked(i32(idx), ld(idx), t, (int)k, experts, max_m, ptr<int32_t>(counts),
                                       ptr<int32_t>(row_slot), ptr<int32_t>(slot_row), wp, need, on.stream)
             : dg_expert_layout_contiguous(i32(idx), ld(idx), t, (int)k, experts, rows, ptr<int32_t>(m),
                                           ptr<int32_t>(row_slot), ptr<int32_t>(slot_row), ptr<int32_t>(counts), wp,
                                           need, on.stream);
  if (!done(st, masked ? "dg_expert_layout_masked" : "dg_expert_layout_contiguous")) return nullptr;
  PyObject* first = masked ? Py_NewRef(Py_None) : THPVariable_Wrap(m);
  return Py_BuildValue("(NNNN)", first, THPVariable_Wrap(row_slot), THPVariable_Wrap(slot_row),
                       THPVariable_Wrap(counts));
}

PyObject* expert_layout_contiguous(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  return layout(args, false);
  END_HANDLE_TH_ERRORS
}

PyObject* expert_layout_masked(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  return layout(args, true);
  END_HANDLE_TH_ERRORS
}

// ---- casts and dispatch

// int8 codes [rows, k]; new ones have rows that begin at 128-byte lines, which the
// GEMM reads up to a third faster than rows that straddle them.
Tensor int8_codes(const Args& a, int i, int64_t rows, int64_t k, const Tensor& like) {
  if (a.none(i)) return fresh({rows, k}, at::kChar, like, (k + 127) / 128 * 128);
  return output(a, i, "q", {rows, k}, at::kChar, kI8, like);
}

// fp32 scales of any strides
Tensor scales(const Args& a, int i, const char* name, at::IntArrayRef want) {
  const Tensor& t = a.tensor(i, name);
  TORCH_CHECK_TYPE(t.is_cuda() && t.scalar_type() == at::kFloat, a.call, ": ", name,
                   " must be a float32 device tensor");
  shape(a, t, name, want);
  return t;
}

// Rows of the target: `rows`, or q's
int64_t target_rows(const Args& a, int rows, int q) {
  int64_t r = -1;
  if (!a.none(q)) r = a.tensor(q, "q").dim() == 2 ? a.tensor(q, "q").size(0) : 0;
  if (!a.none(rows)) {
    const int64_t v = a.integer(rows, "rows");
    TORCH_CHECK_VALUE((r < 0 || r == v) && v >= 0, a.call, ": rows must be q's and not negative, got ", v);
    r = v;
  }
  TORCH_CHECK_VALUE(r >= 0, a.call, ": rows (or q) must be given");
  return r;
}

PyObject* dispatch_cast_fp8(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Args a{args, "dispatch_cast_fp8"};
  const Tensor& x = check(a, 0, "x", kF32 | kBF16, 2);
  const On on(x);
  const Tensor& map = check(a, 1, "slot_row", kI32, 2);
  const int64_t t = x.size(0), k = x.size(1), topk = map.size(1);
  shape(a, map, "slot_row", {t, topk});
  TORCH_CHECK_VALUE(topk <= INT32_MAX, a.call, ": too many columns");
  const int64_t rows = target_rows(a, 2, 4);
  Tensor q = output(a, 4, "q", {rows, k}, at::kFloat8_e4m3fn, kE4M3 | kU8, x);
  // new scales of one block lie beside each other along the rows, as the GEMM reads them best
  Tensor sf = a.none(5) ? fresh({k / 128, rows}, at::kFloat, x).t()
                        : scales(a, 5, "sf", {rows, k / 128});
  same_device(a, x, {&map, &q, &sf});
  if (!done(dg_dispatch_cast_fp8(ptr(x), dtype_of(x), ld(x), i32(map), ld(map), ptr(q), ld(q), ptr<float>(sf),
                                 sf.stride(0), sf.stride(1), t, (int)topk, rows, k, a.truth(3), on.stream),
            "dg_dispatch_cast_fp8"))
    return nullptr;
  return pair(q, sf);
  END_HANDLE_TH_ERRORS
}

PyObject* dispatch_cast_int8(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Args a{args, "dispatch_cast_int8"};
  const Tensor& x = check(a, 0, "x", kF32 | kBF16, 2);
  const On on(x);
  const Tensor& map = check(a, 1, "slot_row", kI32, 2);
  const int64_t t = x.size(0), k = x.size(1), topk = map.size(1);
  shape(a, map, "slot_row", {t, topk});
  TORCH_CHECK_VALUE(topk <= INT32_MAX, a.call, ": too many columns");
  const int64_t rows = target_rows(a, 2, 3);
  Tensor q = int8_codes(a, 3, rows, k, x);
  Tensor sf = a.none(4) ? fresh({rows}, at::kFloat, x)
                        : scales(a, 4, "sf", {rows});
  same_device(a, x, {&map, &q, &sf});
  if (!done(dg_dispatch_cast_int8(ptr(x), dtype_of(x), ld(x), i32(map), ld(map), ptr(q), ld(q), ptr<float>(sf),
                                  sf.stride(0), t, (int)topk, rows, k, on.stream),
            "dg_dispatch_cast_int8"))
    return nullptr;
  return pair(q, sf);
  END_HANDLE_TH_ERRORS
}

PyObject* per_token_cast_int8(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Args a{args, "per_token_cast_int8"};
  const Tensor& x = check(a, 0, "x", kF32 | kBF16, 2);
  const On on(x);
  const int64_t m = x.size(0), k = x.size(1);
  Tensor q = int8_codes(a, 1, m, k, x);
  Tensor sf = a.none(2) ? fresh({m}, at::kFloat, x)
                        : scales(a, 2, "sf", {m});
  same_device(a, x, {&q, &sf});
  if (!done(dg_per_token_cast_int8(ptr(x), dtype_of(x), ld(x), ptr(q), ld(q), ptr<float>(sf), sf.stride(0), m, k,
                                   on.stream),
            "dg_per_token_cast_int8"))
    return nullptr;
  return pair(q, sf);
  END_HANDLE_TH_ERRORS
}

// ---- combination

PyObject* combine(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Args a{args, "combine"};
  const Tensor& y = check(a, 0, "y", kBF16, 2);
  const On on(y);
  const Tensor& map = check(a, 1, "slot_row", kI32, 2);
  const int64_t t = map.size(0), k = map.size(1), rows = y.size(0), h = y.size(1);
  TORCH_CHECK_VALUE(k <= INT32_MAX, a.call, ": too many columns");
  Tensor w;
  if (!a.none(2)) {
    w = check(a, 2, "weights", kF32, 2);
    shape(a, w, "weights", {t, k});
  }
  Tensor out = output(a, 3, "out", {t, h}, at::kBFloat16, kBF16 | kF32, y);
  same_device(a, y, {&map, &w, &out});
  if (!done(dg_combine(ptr(y), ld(y), i32(map), ld(map), w.defined() ? f32(w) : nullptr, w.defined() ? ld(w) : 0,
                       ptr(out), dtype_of(out), ld(out), t, (int)k, rows, h, on.stream),
            "dg_combine"))
    return nullptr;
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

PyObject* combine_grad(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Args a{args, "combine_grad"};
  const Tensor& g = check(a, 0, "dout", kBF16, 2);
  const Tensor& y = check(a, 1, "y", kBF16, 2);
  const On on(y);
  const Tensor& map = check(a, 2, "slot_row", kI32, 2);
  const Tensor& back = check(a, 3, "row_slot", kI32, 1);
  const Tensor& w = check(a, 4, "weights", kF32, 2);
  const int64_t t = map.size(0), k = map.size(1), rows = y.size(0), h = y.size(1);
  TORCH_CHECK_VALUE(k <= INT32_MAX, a.call, ": too many columns");
  shape(a, g, "dout", {t, h});
  shape(a, w, "weights", {t, k});
  shape(a, back, "row_slot", {rows});
  Tensor dy = output(a, 5, "dy", {rows, h}, at::kBFloat16, kBF16, y);
  Tensor dw = output(a, 6, "dweights", {t, k}, at::kFloat, kF32, y);
  same_device(a, y, {&g, &map, &back, &w, &dy, &dw});
  if (!done(dg_combine_grad(ptr(g), ld(g), ptr(y), ld(y), i32(map), ld(map), i32(back), f32(w), ld(w), ptr(dy), ld(dy),
                            ptr<float>(dw), ld(dw), t, (int)k, rows, h, on.stream),
            "dg_combine_grad"))
    return nullptr;
  return pair(dy, dw);
  END_HANDLE_TH_ERRORS
}

// ---- norm

// Weight of a norm over rows of x: defined or not; its type is x's or fp32.
Tensor norm_weight(const Args& a, int i, const Tensor& x) {
  if (a.none(i)) return Tensor();
  const Tensor& w = check(a, i, "weight", type_bit(x) | kF32, 1);
  shape(a, w, "weight", {x.size(1)});
  return w;
}

// FP8 codes and scales [rows, k], [rows, k/128]: passed in, or new ones whose scales of one block
// lie beside each other along the rows, as the GEMM reads them best.
struct Codes {
  Tensor q, sf;
};
Codes fp8_out(const Args& a, int q, int sf, int64_t rows, int64_t k, const Tensor& like) {
  return {output(a, q, "q", {rows, k}, at::kFloat8_e4m3fn, kE4M3 | kU8, like),
          a.none(sf) ? at::detail::empty_strided_cuda({rows, k / 128}, {1, rows}, at::kFloat, like.device())
                     : scales(a, sf, "sf", {rows, k / 128})};
}

// kind 0: rows, 1: FP8, 2: int8.  (x, weight, residual, eps, [ue8m0, q, sf | q, sf], y, h, rstd)
template <int kKind>
PyObject* norm(PyObject* const* args, const char* name, const char* abi) {
  const Args a{args, name};
  const Tensor& x = check(a, 0, "x", kF32 | kBF16 | kF16, 2);
  const On on(x);
  const int64_t rows = x.size(0), k = x.size(1);
  const Tensor w = norm_weight(a, 1, x);
  Tensor r;
  if (!a.none(2)) {
    r = check(a, 2, "residual", type_bit(x), 2);
    shape(a, r, "residual", x.sizes());
  }
  const float eps = (float)a.number(3, "eps");
  constexpr int at = kKind == 1 ? 7 : kKind == 2 ? 6 : 4;   // y, h, rstd
  Codes c;
  if (kKind == 1) c = fp8_out(a, 5, 6, rows, k, x);
  if (kKind == 2) c = {int8_codes(a, 4, rows, k, x), a.none(5) ? fresh({rows}, at::kFloat, x) : scales(a, 5, "sf", {rows})};
  Tensor y;
  if (kKind == 0 || !a.none(at)) y = output(a, at, "y", {rows, k}, x.scalar_type(), type_bit(x), x);
  Tensor h;
  if (r.defined() || !a.none(at + 1)) h = output(a, at + 1, "h", {rows, k}, x.scalar_type(), type_bit(x), x);
  Tensor rstd = output(a, at + 2, "rstd", {rows}, at::kFloat, kF32, x);
  same_device(a, x, {&w, &r, &c.q, &c.sf, &y, &h, &rstd});
  TORCH_CHECK_VALUE(!y.defined() || !h.defined() || rows == 0 || k == 0 || y.data_ptr() != h.data_ptr(), a.call,
                    ": y and h must be different tensors");
  TORCH_CHECK_VALUE(!y.defined() || h.defined() || rows == 0 || k == 0 || y.data_ptr() != x.data_ptr(), a.call,
                    ": y would overwrite x, which is the h that is returned; give h, or another y");
  void* const rp = r.defined() ? ptr(r) : nullptr;
  void* const wp = w.defined() ? ptr(w) : nullptr;
  void* const hp = h.defined() ? ptr(h) : nullptr;
  void* const yp = y.defined() ? ptr(y) : nullptr;
  const int64_t ldr = r.defined() ? ld(r) : 0, ldh = h.defined() ? ld(h) : 0, ldy = y.defined() ? ld(y) : 0;
  const int wt = w.defined() ? dtype_of(w) : DG_F32;
  dg_status st;
  if constexpr (kKind == 0) {
    st = dg_rms_norm(ptr(x), dtype_of(x), ld(x), rp, ldr, wp, wt, eps, hp, ldh, yp, ldy, ptr<float>(rstd), rows, k,
                     on.stream);
  } else if constexpr (kKind == 1) {
    st = dg_rms_norm_cast_fp8(ptr(x), dtype_of(x), ld(x), rp, ldr, wp, wt, eps, hp, ldh, yp, ldy, ptr<float>(rstd),
                              ptr(c.q), ld(c.q), ptr<float>(c.sf), c.sf.stride(0), c.sf.stride(1), rows, k, a.truth(4),
                              on.stream);
  } else {
    st = dg_rms_norm_cast_int8(ptr(x), dtype_of(x), ld(x), rp, ldr, wp, wt, eps, hp, ldh, yp, ldy, ptr<float>(rstd),
                               ptr(c.q), ld(c.q), ptr<float>(c.sf), c.sf.stride(0), rows, k, on.stream);
  }
  if (!done(st, abi)) return nullptr;
  if (k == 0 && rows > 0) {   // nothing was launched: the mean of no squares, and the scale of a row without a maximum
    rstd.fill_(NAN);
    if (kKind == 2) c.sf.fill_(1e-4f / 127.0f);
  }
  PyObject* hr = h.defined() ? THPVariable_Wrap(h) : Py_NewRef(args[0]);
  if (kKind == 0) return Py_BuildValue("(NNN)", THPVariable_Wrap(y), hr, THPVariable_Wrap(rstd));
  return Py_BuildValue("(NNN)", pair(c.q, c.sf), hr, THPVariable_Wrap(rstd));
}

PyObject* rms_norm(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  return norm<0>(args, "rms_norm", "dg_rms_norm");
  END_HANDLE_TH_ERRORS
}
PyObject* rms_norm_cast_fp8(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  return norm<1>(args, "rms_norm_cast_fp8", "dg_rms_norm_cast_fp8");
  END_HANDLE_TH_ERRORS
}
PyObject* rms_norm_cast_int8(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  return norm<2>(args, "rms_norm_cast_int8", "dg_rms_norm_cast_int8");
  END_HANDLE_TH_ERRORS
}

PyObject* rms_norm_grad(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Args a{args, "rms_norm_grad"};
  const Tensor& dy = check(a, 0, "dy", kF32 | kBF16 | kF16, 2);
  const On on(dy);
  const int64_t rows = dy.size(0), k = dy.size(1);
  const Tensor& h = check(a, 1, "h", type_bit(dy), 2);
  shape(a, h, "h", {rows, k});
  const Tensor w = norm_weight(a, 2, dy);
  const Tensor& rstd = check(a, 3, "rstd", kF32, 1);
  shape(a, rstd, "rstd", {rows});
  Tensor dh;
  if (!a.none(4)) {
    dh = check(a, 4, "dh", type_bit(dy), 2);
    shape(a, dh, "dh", {rows, k});
  }
  Tensor dx = output(a, 5, "dx", {rows, k}, dy.scalar_type(), type_bit(dy), dy);
  Tensor dw;
  if (w.defined()) dw = output(a, 6, "dweight", {k}, at::kFloat, kF32, dy);
  TORCH_CHECK_VALUE(w.defined() || a.none(6), a.call, ": dweight needs a weight");
  same_device(a, dy, {&h, &w, &rstd, &dh, &dx, &dw});
  const size_t need = dw.defined() ? dg_rms_norm_grad_workspace_size(rows, k) : 0;
  Tensor ws = need ? fresh({(int64_t)need}, at::kByte, dy) : Tensor();
  if (!done(dg_rms_norm_grad(ptr(dy), dtype_of(dy), ld(dy), ptr(h), ld(h), w.defined() ? ptr(w) : nullptr,
                             w.defined() ? dtype_of(w) : DG_F32, f32(rstd), dh.defined() ? ptr(dh) : nullptr,
                             dh.defined() ? ld(dh) : 0, ptr(dx), ld(dx), dw.defined() ? ptr<float>(dw) : nullptr, rows, k,
                             need ? ptr(ws) : nullptr, need, on.stream),
            "dg_rms_norm_grad"))
    return nullptr;
  return Py_BuildValue("(NN)", THPVariable_Wrap(dx), dw.defined() ? THPVariable_Wrap(dw) : Py_NewRef(Py_None));
  END_HANDLE_TH_ERRORS
}

// ---- gated activation

// Rows of a layout: (m_indices or None, masked_m or None).
struct Where {
  Tensor m_indices, masked_m;
  const int32_t* mi = nullptr;
  const int32_t* mm = nullptr;
  int groups = 0;
};
Where rows_of(const Args& a, int i, int64_t rows) {
  Where w;
  TORCH_CHECK_VALUE(a.none(i) || a.none(i + 1), a.call, ": m_indices and masked_m cannot both be given");
  if (!a.none(i)) {
    w.m_indices = check(a, i, "m_indices", kI32, 1);
    shape(a, w.m_indices, "m_indices", {rows});
    w.mi = i32(w.m_indices);
  }
  if (!a.none(i + 1)) {
    w.masked_m = check(a, i + 1, "masked_m", kI32, 1);
    const int64_t g = w.masked_m.size(0);
    TORCH_CHECK_VALUE(g > 0 && g <= INT32_MAX && rows % g == 0, a.call, ": ", rows, " rows are no multiple of ", g,
                      " groups");
    w.groups = (int)g;
    w.mm = i32(w.masked_m);
  }
  return w;
}

int64_t inner_of(const Args& a, const Tensor& h) {
  TORCH_CHECK_VALUE(h.size(1) % 2 == 0, a.call, ": h must have an even number of columns, got ", h.size(1));
  return h.size(1) / 2;
}

// (h, m_indices, masked_m, ue8m0, q, sf[, hq, hsf])
PyObject* swiglu_fp8(PyObject* const* args, const char* name, bool keep) {
  const Args a{args, name};
  const Tensor& h = check(a, 0, "h", kF32 | kBF16 | kF16, 2);
  const On on(h);
  const int64_t rows = h.size(0), inner = inner_of(a, h);
  const Where w = rows_of(a, 1, rows);
  const Codes c = fp8_out(a, 4, 5, rows, inner, h);
  Codes kept;
  if (keep) kept = fp8_out(a, 6, 7, rows, 2 * inner, h);
  same_device(a, h, {&w.m_indices, &w.masked_m, &c.q, &c.sf, &kept.q, &kept.sf});
  if (!done(dg_swiglu_cast_fp8(ptr(h), dtype_of(h), ld(h), w.mi, w.mm, w.groups, ptr(c.q), ld(c.q), ptr<float>(c.sf),
                               c.sf.stride(0), c.sf.stride(1), keep ? ptr(kept.q) : nullptr, keep ? ld(kept.q) : 0,
                               keep ? ptr<float>(kept.sf) : nullptr, keep ? kept.sf.stride(0) : 0,
                               keep ? kept.sf.stride(1) : 0, rows, inner, a.truth(3), on.stream),
            "dg_swiglu_cast_fp8"))
    return nullptr;
  return keep ? Py_BuildValue("(NN)", pair(c.q, c.sf), pair(kept.q, kept.sf)) : pair(c.q, c.sf);
}

PyObject* swiglu_cast_fp8(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  return swiglu_fp8(args, "swiglu_cast_fp8", false);
  END_HANDLE_TH_ERRORS
}
PyObject* swiglu_checkpoint_fp8(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  return swiglu_fp8(args, "swiglu_checkpoint_fp8", true);
  END_HANDLE_TH_ERRORS
}

PyObject* swiglu_cast_int8(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Args a{args, "swiglu_cast_int8"};
  const Tensor& h = check(a, 0, "h", kF32 | kBF16 | kF16, 2);
  const On on(h);
  const int64_t rows = h.size(0), inner = inner_of(a, h);
  const Where w = rows_of(a, 1, rows);
  Tensor q = int8_codes(a, 3, rows, inner, h);
  Tensor sf = a.none(4) ? fresh({rows}, at::kFloat, h) : scales(a, 4, "sf", {rows});
  same_device(a, h, {&w.m_indices, &w.masked_m, &q, &sf});
  if (!done(dg_swiglu_cast_int8(ptr(h), dtype_of(h), ld(h), w.mi, w.mm, w.groups, ptr(q), ld(q), ptr<float>(sf),
                                sf.stride(0), rows, inner, on.stream),
            "dg_swiglu_cast_int8"))
    return nullptr;
  return pair(q, sf);
  END_HANDLE_TH_ERRORS
}

// (da, h, hq, hsf, m_indices, masked_m, [ue8m0,] dh[, q, sf]): h, or its checkpoint (hq, hsf)
PyObject* swiglu_back(PyObject* const* args, const char* name, bool cast) {
  const Args a{args, name};
  const Tensor& da = check(a, 0, "da", kF32 | kBF16 | kF16, 2);
  const On on(da);
  const int64_t rows = da.size(0), inner = da.size(1);
  Tensor h, hq, hsf;
  if (!a.none(1)) {
    h = check(a, 1, "h", type_bit(da), 2);
    shape(a, h, "h", {rows, 2 * inner});
  } else {
    hq = check(a, 2, "h's codes", kE4M3 | kU8, 2);
    shape(a, hq, "h's codes", {rows, 2 * inner});
    hsf = scales(a, 3, "h's scales", {rows, 2 * inner / 128});
  }
  const Where w = rows_of(a, 4, rows);
  Tensor dh = output(a, cast ? 7 : 6, "dh", {rows, 2 * inner}, da.scalar_type(), type_bit(da), da);
  Codes c;
  if (cast) c = fp8_out(a, 8, 9, rows, 2 * inner, da);
  same_device(a, da, {&h, &hq, &hsf, &w.m_indices, &w.masked_m, &dh, &c.q, &c.sf});
  const bool codes = hq.defined();
  if (!done(dg_swiglu_grad(ptr(da), dtype_of(da), ld(da), codes ? nullptr : ptr(h), codes ? 0 : ld(h),
                           codes ? ptr(hq) : nullptr, codes ? ld(hq) : 0, codes ? f32(hsf) : nullptr,
                           codes ? hsf.stride(0) : 0, codes ? hsf.stride(1) : 0, w.mi, w.mm, w.groups, ptr(dh), ld(dh),
                           cast ? ptr(c.q) : nullptr, cast ? ld(c.q) : 0, cast ? ptr<float>(c.sf) : nullptr,
                           cast ? c.sf.stride(0) : 0, cast ? c.sf.stride(1) : 0, rows, inner, cast && a.truth(6),
                           on.stream),
            "dg_swiglu_grad"))
    return nullptr;
  return cast ? Py_BuildValue("(NN)", THPVariable_Wrap(dh), pair(c.q, c.sf)) : THPVariable_Wrap(dh);
}

PyObject* swiglu_grad(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  return swiglu_back(args, "swiglu_grad", false);
  END_HANDLE_TH_ERRORS
}
PyObject* swiglu_grad_cast_fp8(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  return swiglu_back(args, "swiglu_grad_cast_fp8", true);
  END_HANDLE_TH_ERRORS
}

// ---- weights' gradients: (dy, x, sf or None, dw, ...)

enum Grouping { kDense, kContiguous, kMasked };

PyObject* weights_gradient(PyObject* const* args, const char* name, const char* abi, Grouping how) {
  const Args a{args, name};
  const Tensor& dy = check(a, 0, "dy", kBF16, 2);
  const On on(dy);
  const bool codes = !a.none(2);
  const Tensor& x = check(a, 1, "x", codes ? kE4M3 | kU8 : kBF16, 2);
  const int64_t rows = dy.size(0), n = dy.size(1), k = x.size(1);
  shape(a, x, "x", {rows, k});
  Tensor sf, counts;
  if (codes) sf = scales(a, 2, "x's scales", {rows, k / 128});
  const int64_t dim = how == kDense ? 2 : 3;
  const Tensor& dw = check(a, 3, "dw", kF32 | kBF16, dim);
  int64_t groups = 1;
  if (how == kDense) {
    shape(a, dw, "dw", {n, k});
  } else {
    counts = check(a, 4, how == kMasked ? "masked_m" : "counts", kI32, 1);
    groups = counts.size(0);
    shape(a, dw, "dw", {groups, n, k});
    TORCH_CHECK_VALUE(groups <= INT32_MAX, a.call, ": too many groups");
    TORCH_CHECK_VALUE(how == kContiguous || (groups > 0 ? rows % groups == 0 : rows == 0), a.call, ": ", rows,
                      " rows are no multiple of ", groups, " groups");
  }
  same_device(a, dy, {&x, &sf, &dw, &counts});
  const size_t need = dg_weight_grad_workspace_size(rows, n, k, (int)groups);
  Tensor ws = need ? fresh({(int64_t)need}, at::kByte, dy) : Tensor();
  void* const wp = need ? ptr(ws) : nullptr;
  const float* const sp = codes ? f32(sf) : nullptr;
  const int64_t s0 = codes ? sf.stride(0) : 0, s1 = codes ? sf.stride(1) : 0;
  dg_status st;
  if (how == kDense) {
    st = dg_weight_grad(ptr(dy), ld(dy), ptr(x), ld(x), sp, s0, s1, ptr(dw), dtype_of(dw), ld(dw), a.truth(4), rows, n,
                        k, wp, need, on.stream);
  } else if (how == kContiguous) {
    st = dg_m_grouped_weight_grad_contiguous(ptr(dy), ld(dy), ptr(x), ld(x), sp, s0, s1, ptr(dw), dtype_of(dw),
                                             ld(dw, 1), dw.stride(0), i32(counts), (int)groups,
                                             a.integer(5, "alignment"), a.truth(6), rows, n, k, wp, need, on.stream);
  } else {
    st = dg_m_grouped_weight_grad_masked(ptr(dy), ld(dy), ptr(x), ld(x), sp, s0, s1, ptr(dw), dtype_of(dw), ld(dw, 1),
                                         dw.stride(0), i32(counts), (int)groups, groups > 0 ? rows / groups : 0,
                                         a.truth(5), n, k, wp, need, on.stream);
  }
  if (!done(st, abi)) return nullptr;
  return Py_NewRef(args[3]);
}

PyObject* weight_grad(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  return weights_gradient(args, "weight_grad", "dg_weight_grad", kDense);
  END_HANDLE_TH_ERRORS
}
PyObject* weight_grad_contiguous(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  return weights_gradient(args, "m_grouped_weight_grad_contiguous", "dg_m_grouped_weight_grad_contiguous", kContiguous);
  END_HANDLE_TH_ERRORS
}
PyObject* weight_grad_masked(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  return weights_gradient(args, "m_grouped_weight_grad_masked", "dg_m_grouped_weight_grad_masked", kMasked);
  END_HANDLE_TH_ERRORS
}

// ---- int8 products: (qa, sa, qb, sb, d, ...)

PyObject* int8_gemm_nt(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Args a{args, "int8_gemm_nt"};
  const Tensor& qa = check(a, 0, "a", kI8, 2);
  const Tensor& qb = check(a, 2, "b", kI8, 2);
  const Tensor& d = check(a, 4, "d", kF32 | kBF16 | kF16, 2);
  const int64_t m = qa.size(0), k = qa.size(1), n = qb.size(0);
  shape(a, qb, "b", {n, k});
  shape(a, d, "d", {m, n});
  const Tensor sa = scales(a, 1, "sfa", {m}), sb = scales(a, 3, "sfb", {n});
  same_device(a, qa, {&sa, &qb, &sb, &d});
  const On on(qa);
  const Workspace w = workspace(a, 5, d, dg_int8_gemm_nt_workspace_size(m, n, k));
  if (!done(dg_int8_gemm_nt(ptr(qa), ld(qa), f32(sa), sa.stride(0), ptr(qb), ld(qb), f32(sb), sb.stride(0), ptr(d),
                            dtype_of(d), ld(d), m, n, k, w.p, w.bytes, on.stream),
            "dg_int8_gemm_nt"))
    return nullptr;
  return Py_NewRef(args[4]);
  END_HANDLE_TH_ERRORS
}

PyObject* int8_contiguous(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Args a{args, "m_grouped_int8_gemm_nt_contiguous"};
  const Tensor& qa = check(a, 0, "a", kI8, 2);
  const Tensor& qb = check(a, 2, "b", kI8, 3);
  const Tensor& d = check(a, 4, "d", kF32 | kBF16 | kF16, 2);
  const Tensor& idx = check(a, 5, "m_indices", kI32, 1);
  const int64_t m = qa.size(0), k = qa.size(1), g = qb.size(0), n = qb.size(1);
  TORCH_CHECK_VALUE(g <= INT32_MAX, a.call, ": too many groups");
  shape(a, qb, "b", {g, n, k});
  shape(a, d, "d", {m, n});
  shape(a, idx, "m_indices", {m});
  const Tensor sa = scales(a, 1, "sfa", {m}), sb = scales(a, 3, "sfb", {g, n});
  same_device(a, qa, {&sa, &qb, &sb, &d, &idx});
  const On on(qa);
  const Workspace w =
      workspace(a, 6, d, dg_m_grouped_int8_gemm_nt_contiguous_workspace_size(m, n, k, (int)g));
  if (!done(dg_m_grouped_int8_gemm_nt_contiguous(ptr(qa), ld(qa), f32(sa), sa.stride(0), ptr(qb), ld(qb, 1),
                                                 qb.stride(0), f32(sb), sb.stride(1), sb.stride(0), ptr(d),
                                                 dtype_of(d), ld(d), i32(idx), m, n, k, (int)g, w.p, w.bytes,
                                                 on.stream),
            "dg_m_grouped_int8_gemm_nt_contiguous"))
    return nullptr;
  return Py_NewRef(args[4]);
  END_HANDLE_TH_ERRORS
}

PyObject* int8_masked(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Args a{args, "m_grouped_int8_gemm_nt_masked"};
  const Tensor& qa = check(a, 0, "a", kI8, 3);
  const Tensor& qb = check(a, 2, "b", kI8, 3);
  const Tensor& d = check(a, 4, "d", kF32 | kBF16 | kF16, 3);
  const Tensor& mm = check(a, 5, "masked_m", kI32, 1);
  const int64_t g = qa.size(0), m = qa.size(1), k = qa.size(2), n = qb.size(1);
  TORCH_CHECK_VALUE(g <= INT32_MAX, a.call, ": too many groups");
  shape(a, qb, "b", {g, n, k});
  shape(a, d, "d", {g, m, n});
  shape(a, mm, "masked_m", {g});
  const Tensor sa = scales(a, 1, "sfa", {g, m}), sb = scales(a, 3, "sfb", {g, n});
  same_device(a, qa, {&sa, &qb, &sb, &d, &mm});
  const On on(qa);
  if (!done(dg_m_grouped_int8_gemm_nt_masked(ptr(qa), ld(qa, 1), qa.stride(0), f32(sa), sa.stride(1), sa.stride(0),
                                             ptr(qb), ld(qb, 1), qb.stride(0), f32(sb), sb.stride(1), sb.stride(0),
                                             ptr(d), dtype_of(d), ld(d, 1), d.stride(0), i32(mm), (int)g, m, n, k,
                                             a.integer(6, "expected_m"), on.stream),
            "dg_m_grouped_int8_gemm_nt_masked"))
    return nullptr;
  return Py_NewRef(args[4]);
  END_HANDLE_TH_ERRORS
}

// (DgError, auto workspace): set once, when the package is imported
PyObject* connect(PyObject*, PyObject* const* args, Py_ssize_t) {
  Py_XDECREF(g_error);
  Py_XDECREF(g_auto_workspace);
  g_error = Py_NewRef(args[0]);
  g_auto_workspace = Py_NewRef(args[1]);
  Py_RETURN_NONE;
}

// Every function takes a fixed number of positional arguments: the Python side
// names them and gives their defaults.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t), int N>
PyObject* exactly(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are needed, got %zd", N, n);
    return nullptr;
  }
  return F(self, args, n);
}

#define DG_METHOD(name, n) {#name, (PyCFunction)(void (*)(void))exactly<name, n>, METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    DG_METHOD(connect, 2),
    DG_METHOD(route_topk, 11),
    DG_METHOD(route_topk_grad, 7),
    DG_METHOD(expert_layout_contiguous, 3),
    DG_METHOD(expert_layout_masked, 3),
    DG_METHOD(dispatch_cast_fp8, 6),
    DG_METHOD(dispatch_cast_int8, 5),
    DG_METHOD(per_token_cast_int8, 3),
    DG_METHOD(combine, 4),
    DG_METHOD(combine_grad, 7),
    DG_METHOD(rms_norm, 7),
    DG_METHOD(rms_norm_cast_fp8, 10),
    DG_METHOD(rms_norm_cast_int8, 9),
    DG_METHOD(rms_norm_grad, 7),
    DG_METHOD(swiglu_cast_fp8, 6),
    DG_METHOD(swiglu_checkpoint_fp8, 8),
    DG_METHOD(swiglu_cast_int8, 5),
    DG_METHOD(swiglu_grad, 7),
    DG_METHOD(swiglu_grad_cast_fp8, 10),
    DG_METHOD(weight_grad, 5),
    DG_METHOD(weight_grad_contiguous, 7),
    DG_METHOD(weight_grad_masked, 6),
    DG_METHOD(int8_gemm_nt, 6),
    DG_METHOD(int8_contiguous, 7),
    DG_METHOD(int8_masked, 7),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
