// The feed-forward half's calls, marshalled in C++: what the binding's functions of the same names
// do in Python (checks, outputs, workspace, stream, the library's entry point) for the calls
// that programs make most, contiguous CUDA tensors on the current device. A call that is
// anything else, or that the library refuses, is answered with NotImplemented, and the Python
// function then does it, or says what is wrong with it. One token's call costs 3 us this way and
// 11 in Python, where its kernel takes 2. Outputs and workspaces come from torch's allocator without
// its dispatcher: the norm's backward pass costs 7.1 us and not 9.8, the projections' 11.9 and not 14.6.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "la.h"

namespace {

// The library's functions, by their places in `kNames`
const char* const kNames[] = {"la_checkpoint",           "la_checkpoint_restore",
                              "la_layer_norm",           "la_layer_norm_workspace_bytes",
                              "la_layer_norm_backward",  "la_ffn_gate_workspace_bytes",
                              "la_ffn_gate",             "la_ffn_gate_backward_workspace_bytes",
                              "la_ffn_gate_backward"};
struct Library {
  decltype(&la_checkpoint) checkpoint;
  decltype(&la_checkpoint_restore) restore;
  decltype(&la_layer_norm) norm;
  decltype(&la_layer_norm_workspace_bytes) norm_bytes;
  decltype(&la_layer_norm_backward) norm_backward;
  decltype(&la_ffn_gate_workspace_bytes) ffn_bytes;
  decltype(&la_ffn_gate) ffn;
  decltype(&la_ffn_gate_backward_workspace_bytes) ffn_backward_bytes;
  decltype(&la_ffn_gate_backward) ffn_backward;
};
Library lib;
static_assert(sizeof(Library) == sizeof(kNames), "one pointer for each name");

PyObject* other() { Py_RETURN_NOTIMPLEMENTED; }

// Allocations and the library's calls run without Python's lock: a launch waits while its stream's queue
// is full, an allocation may wait for the GPU, and other threads (which the GPU may wait for) go on.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// f() without the lock
template <typename F>
auto unlocked(F f) {
  Unlocked u;
  return f();
}

// A C int, -1 for what is none
int int_of(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) PyErr_Clear();
  return v < -1 || v > 0x7fffffff ? -1 : (int)v;
}

// What a call's tensors have in common
struct Call {
  c10::DeviceIndex device = -1;
  at::ScalarType type = at::kFloat;
  int dtype = LA_F32;
  bool ok = true;

  // A plain contiguous CUDA tensor on the current device, its dtype the call's
  const at::Tensor* first(PyObject* o) {
    const at::Tensor* t = plain(o);
    if (t == nullptr) return nullptr;
    type = t->scalar_type();
    dtype = type == at::kFloat ? LA_F32 : LA_BF16;
    device = t->get_device();
    ok = ok && (type == at::kFloat || type == at::kBFloat16) && t->is_cuda() && t->dim() >= 1 &&
         device == c10::cuda::current_device();
    return ok ? t : nullptr;
  }
  const at::Tensor* like(PyObject* o, at::IntArrayRef sizes) { return typed(o, sizes, type); }
  const at::Tensor* typed(PyObject* o, at::IntArrayRef sizes, at::ScalarType want) {
    const at::Tensor* t = plain(o);
    if (t != nullptr && (t->scalar_type() != want || !t->is_cuda() || t->get_device() != device || t->sizes() != sizes))
      ok = false;
    return t;
  }
  const at::Tensor* plain(PyObject* o) {
    if (!THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != at::kStrided || !t.is_contiguous()) ok = false;
    return ok ? &t : nullptr;
  }
  // codes and exps of a checkpoint of values of `sizes` (None: neither)
  void pair(PyObject* o, at::IntArrayRef sizes, const at::Tensor*& codes, const at::Tensor*& exps) {
    codes = exps = nullptr;
    if (o == Py_None) return;
    if (!PyTuple_CheckExact(o) || PyTuple_GET_SIZE(o) != 2) {
      ok = false;
      return;
    }
    c10::SmallVector<int64_t, 6> blocks(sizes.begin(), sizes.end());
    blocks.back() = (blocks.back() + 31) / 32;
    codes = typed(PyTuple_GET_ITEM(o, 0), sizes, at::kChar);
    if (ok) exps = typed(PyTuple_GET_ITEM(o, 1), blocks, at::kByte);
  }
  at::Tensor empty(at::IntArrayRef sizes, at::ScalarType t) const {
    return at::Tensor(at::detail::empty_cuda(sizes, t, at::Device(at::kCUDA, device), std::nullopt));
  }
  // what is given, or undefined for None
  at::Tensor given(PyObject* o, at::IntArrayRef sizes) {
    if (o == Py_None) return at::Tensor();
    const at::Tensor* t = like(o, sizes);
    return ok ? *t : at::Tensor();
  }
  // on the current device and stream, as `empty`
  c10::DataPtr scratch(size_t bytes) const {
    return bytes ? c10::cuda::CUDACachingAllocator::get()->allocate(bytes) : c10::DataPtr();
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
};

void* ptr(const at::Tensor* t) { return t != nullptr ? t->data_ptr() : nullptr; }
signed char* codes_of(const at::Tensor* t) { return static_cast<signed char*>(ptr(t)); }
unsigned char* exps_of(const at::Tensor* t) { return static_cast<unsigned char*>(ptr(t)); }

long long rows_of(const at::Tensor& t, int64_t C) { return C ? t.numel() / C : 0; }
bool fits(int64_t n) { return n >= 0 && n <= 0x7fffffff; }

PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  Py_ssize_t i = 0;
  if (r != nullptr)
    for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

// C++ exceptions of torch (no memory, say) become NotImplemented: the Python function meets the
// same and raises it in torch's own way.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::exception&) {
    PyErr_Clear();
    return other();
  }
}

// checkpoint(x, pair or None)
PyObject* checkpoint(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2) return other();
  return guarded([&]() -> PyObject* {
    Call c;
    const at::Tensor* x = c.first(a[0]);
    if (!c.ok || a[1] != Py_None) return other();
    const int64_t C = x->size(-1);
    c10::SmallVector<int64_t, 6> blocks(x->sizes().begin(), x->sizes().end());
    blocks.back() = (C + 31) / 32;
    if (!fits(C)) return other();
    at::Tensor codes, exps;
    const int status = unlocked([&] {
      codes = c.empty(x->sizes(), at::kChar), exps = c.empty(blocks, at::kByte);
      return lib.checkpoint(x->data_ptr(), C, codes_of(&codes), exps_of(&exps), rows_of(*x, C), (int)C, c.dtype, c.stream());
    });
    if (status != LA_OK) return other();
    return tuple({codes, exps});
  });
}

// checkpoint_restore(codes, exps, float32 or bfloat16 as 0 or 1)
PyObject* checkpoint_restore(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 3) return other();
  return guarded([&]() -> PyObject* {
    Call c;
    const at::Tensor* codes = c.plain(a[0]);
    if (!c.ok || !codes->is_cuda() || codes->dim() < 1 || codes->scalar_type() != at::kChar) return other();
    c.device = codes->get_device();
    c.dtype = int_of(a[2]);
    if (c.device != c10::cuda::current_device() || (c.dtype != LA_F32 && c.dtype != LA_BF16)) return other();
    const int64_t C = codes->size(-1);
    c10::SmallVector<int64_t, 6> blocks(codes->sizes().begin(), codes->sizes().end());
    blocks.back() = (C + 31) / 32;
    const at::Tensor* exps = c.typed(a[1], blocks, at::kByte);
    if (!c.ok || !fits(C)) return other();
    at::Tensor out;
    const int status = unlocked([&] {
      out = c.empty(codes->sizes(), c.dtype == LA_F32 ? at::kFloat : at::kBFloat16);
      return lib.restore(codes_of(codes), exps_of(exps), out.data_ptr(), C, rows_of(*codes, C), (int)C, c.dtype, c.stream());
    });
    if (status != LA_OK) return other();
    return THPVariable_Wrap(out);
  });
}

// layer_norm(x, w, b or None, eps, out or None, pair or None)
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6 || !PyFloat_CheckExact(a[3])) return other();
  return guarded([&]() -> PyObject* {
    Call c;
    const at::Tensor* x = c.first(a[0]);
    if (!c.ok) return other();
    const int64_t C = x->size(-1);
    const at::Tensor* w = c.like(a[1], {C});
    const at::Tensor *b = c.ok && a[2] != Py_None ? c.like(a[2], {C}) : nullptr, *codes = nullptr, *exps = nullptr;
    if (c.ok) c.pair(a[5], x->sizes(), codes, exps);
    if (!c.ok || !fits(C)) return other();
    at::Tensor out = c.given(a[4], x->sizes());
    if (!c.ok) return other();
    const float eps = (float)PyFloat_AS_DOUBLE(a[3]);
    const int status = unlocked([&] {
      if (!out.defined()) out = c.empty(x->sizes(), c.type);
      return lib.norm(x->data_ptr(), C, ptr(w), ptr(b), out.data_ptr(), C, codes_of(codes), exps_of(exps), rows_of(*x, C),
                      (int)C, eps, c.dtype, c.stream());
    });
    if (status != LA_OK) return other();
    return THPVariable_Wrap(out);
  });
}

// layer_norm_backward(x or pair, w, dy, eps), all outputs new
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4 || !PyFloat_CheckExact(a[3])) return other();
  return guarded([&]() -> PyObject* {
    Call c;
    const at::Tensor* dy = c.first(a[2]);
    if (!c.ok) return other();
    const int64_t C = dy->size(-1);
    const at::Tensor *w = c.like(a[1], {C}), *x = nullptr, *codes = nullptr, *exps = nullptr;
    if (c.ok && PyTuple_CheckExact(a[0]))
      c.pair(a[0], dy->sizes(), codes, exps);
    else if (c.ok)
      x = c.like(a[0], dy->sizes());
    const long long rows = rows_of(*dy, C);
    if (!c.ok || !fits(C)) return other();
    at::Tensor dx, dw, db;
    const float eps = (float)PyFloat_AS_DOUBLE(a[3]);
    const int status = unlocked([&] {
      dx = c.empty(dy->sizes(), c.type), dw = c.empty({C}, c.type), db = c.empty({C}, c.type);
      const size_t bytes = lib.norm_bytes(rows, (int)C);
      const c10::DataPtr ws = c.scratch(bytes);
      return lib.norm_backward(ptr(x), C, codes_of(codes), exps_of(exps), ptr(w), dy->data_ptr(), C, dx.data_ptr(), C,
                               dw.data_ptr(), db.data_ptr(), rows, (int)C, eps, c.dtype, ws.get(), bytes, c.stream());
    });
    if (status != LA_OK) return other();
    return tuple({dx, dw, db});
  });
}

// x [..., C], wg and wu [F, C]: their sizes, and [..., F] or [..., 2, F]
struct Ffn {
  const at::Tensor *x, *wg, *wu;
  int64_t C = 0, F = 0;
  long long rows = 0;
  Ffn(Call& c, PyObject* const* a) : x(c.first(a[0])), wg(nullptr), wu(nullptr) {
    if (!c.ok) return;
    C = x->size(-1);
    wg = c.plain(a[1]);
    if (!c.ok || wg->dim() != 2) {
      c.ok = false;
      return;
    }
    F = wg->size(0);
    wg = c.like(a[1], {F, C});
    if (c.ok) wu = c.like(a[2], {F, C});
    rows = rows_of(*x, C);
    c.ok = c.ok && fits(C) && fits(F) && fits(rows);
  }
  c10::SmallVector<int64_t, 6> hidden(bool two) const {
    c10::SmallVector<int64_t, 6> s(x->sizes().begin(), x->sizes().end());
    if (two) s.back() = 2, s.push_back(F);
    else s.back() = F;
    return s;
  }
};

// ffn_gate(x, wg, wu, activation's code, out or None, pair or None)
PyObject* ffn_gate(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return other();
  return guarded([&]() -> PyObject* {
    Call c;
    const Ffn f(c, a);
    const at::Tensor *codes = nullptr, *exps = nullptr;
    if (c.ok) c.pair(a[5], f.hidden(true), codes, exps);
    if (!c.ok) return other();
    const auto hidden = f.hidden(false);
    at::Tensor out = c.given(a[4], hidden);
    if (!c.ok) return other();
    const int act = int_of(a[3]);
    const int status = unlocked([&] {
      if (!out.defined()) out = c.empty(hidden, c.type);
      const size_t bytes = lib.ffn_bytes((int)f.rows, (int)f.C, (int)f.F, codes != nullptr, c.dtype);
      const c10::DataPtr ws = c.scratch(bytes);
      return lib.ffn(f.x->data_ptr(), f.C, ptr(f.wg), ptr(f.wu), out.data_ptr(), f.F, codes_of(codes), exps_of(exps),
                     (int)f.rows, (int)f.C, (int)f.F, act, c.dtype, ws.get(), bytes, c.stream());
    });
    if (status != LA_OK) return other();
    return THPVariable_Wrap(out);
  });
}

// ffn_gate_backward(x, wg, wu, activation's code, dh, pair or None), all outputs new
PyObject* ffn_gate_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return other();
  return guarded([&]() -> PyObject* {
    Call c;
    const Ffn f(c, a);
    const at::Tensor *codes = nullptr, *exps = nullptr, *dh = c.ok ? c.like(a[4], f.hidden(false)) : nullptr;
    if (c.ok) c.pair(a[5], f.hidden(true), codes, exps);
    if (!c.ok) return other();
    at::Tensor dx, dwg, dwu;
    const int act = int_of(a[3]);
    const int status = unlocked([&] {
      dx = c.empty(f.x->sizes(), c.type), dwg = c.empty({f.F, f.C}, c.type), dwu = c.empty({f.F, f.C}, c.type);
      const size_t bytes = lib.ffn_backward_bytes((int)f.rows, (int)f.C, (int)f.F, c.dtype);
      const c10::DataPtr ws = c.scratch(bytes);
      return lib.ffn_backward(f.x->data_ptr(), f.C, ptr(f.wg), ptr(f.wu), ptr(dh), f.F, codes_of(codes), exps_of(exps),
                              dx.data_ptr(), f.C, dwg.data_ptr(), dwu.data_ptr(), (int)f.rows, (int)f.C, (int)f.F, act,
                              c.dtype, ws.get(), bytes, c.stream());
    });
    if (status != LA_OK) return other();
    return tuple({dx, dwg, dwu});
  });
}

// connect(address of each function in names())
PyObject* connect(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != (Py_ssize_t)(sizeof(kNames) / sizeof(kNames[0]))) {
    PyErr_SetString(PyExc_ValueError, "connect: one address for each name");
    return nullptr;
  }
  void* p[sizeof(kNames) / sizeof(kNames[0])];
  for (Py_ssize_t i = 0; i < n; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "connect: a null address");
      return nullptr;
    }
  }
  static_assert(sizeof(p) == sizeof(lib), "");
  __builtin_memcpy(&lib, p, sizeof(lib));
  Py_RETURN_NONE;
}

PyObject* names(PyObject*, PyObject*) {
  PyObject* r = PyTuple_New(sizeof(kNames) / sizeof(kNames[0]));
  Py_ssize_t i = 0;
  if (r != nullptr)
    for (const char* s : kNames) PyTuple_SET_ITEM(r, i++, PyUnicode_FromString(s));
  return r;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"checkpoint", FAST(checkpoint)},
                         {"checkpoint_restore", FAST(checkpoint_restore)},
                         {"layer_norm", FAST(layer_norm)},
                         {"layer_norm_backward", FAST(layer_norm_backward)},
                         {"ffn_gate", FAST(ffn_gate)},
                         {"ffn_gate_backward", FAST(ffn_gate_backward)},
                         {"connect", FAST(connect)},
                         {"names", names, METH_NOARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "la_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_la_marshal() { return PyModule_Create(&module); }
