// kmip_host.cpp -- the host side of the operators around the attention, as a
// CPython module: checks of torch tensors, their outputs, the current stream,
// the call of libkmip's entry point.
//
// A call on one node or a small graph is bound by what happens before its
// launch.  With these steps in Python and ctypes a rotary call on one node took
// 11.9 us, a norm of 1,024 x 32 14.2 and one feed-forward row 13.5; here 5.3, 8.2
// and 8.4 (of which its two kernels take 7).  Nothing is computed here: libkmip's
// C ABI is the only thing called, at the addresses that binding.py hands over.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <initializer_list>
#include <string>

#include "kmip.h"

namespace {

using at::Tensor;

PyObject* g_error;  // binding.KmipError
decltype(&kmip_rotary) g_rotary;
decltype(&kmip_group_norm_fwd) g_norm_fwd;
decltype(&kmip_group_norm_bwd) g_norm_bwd;
decltype(&kmip_ffn_fwd) g_ffn_fwd;
decltype(&kmip_ffn_bwd) g_ffn_bwd;

struct Refused {
  PyObject* type;
  std::string text;
};
struct Failed {
  kmip_status_t status;
  const char* where;
};
struct Raised {};  // Python's error is set

// (Plain strings: the process may hold two copies of the stream classes, torch's
// and the system's, which do not mix.)
std::string text(at::IntArrayRef shape) {
  std::string s = "[";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + "]";
}
std::string text(at::ScalarType t) { return c10::toString(t); }

[[noreturn]] void refuse(const std::string& text) { throw Refused{PyExc_ValueError, text}; }

// ------------------------------------------------------------------ arguments
const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o))
    throw Refused{PyExc_TypeError, std::string(name) + ": expected a tensor"};
  return THPVariable_Unpack(o);
}
const Tensor* optional(PyObject* o, const char* name) {
  return o == Py_None ? nullptr : &tensor(o, name);
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
int narrow(int64_t v, const char* name) {
  if (v < 0 || v > INT_MAX) refuse(std::string(name) + ": out of range");
  return (int)v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v;
}

kmip_dtype_t dtype_of(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return KMIP_BF16;
  if (t.scalar_type() == at::kFloat) return KMIP_F32;
  throw Refused{PyExc_TypeError,
                "unsupported dtype " + text(t.scalar_type()) + " (bf16 or fp32)"};
}

// Every tensor (null: none) on x's CUDA device and contiguous; x itself may be
// strided.
void same_device(const Tensor& x, std::initializer_list<const Tensor*> others) {
  if (!x.is_cuda()) refuse("libkmip takes CUDA tensors");
  for (const Tensor* t : others)
    if (t && (t->device() != x.device() || !t->is_contiguous()))
      refuse("expected a contiguous tensor on " + x.device().str());
}

void expect(const Tensor* t, const char* name, at::IntArrayRef shape, at::ScalarType type) {
  if (t && (t->sizes() != shape || t->scalar_type() != type))
    refuse(std::string(name) + ": expected " + text(shape) + " " + text(type) + ", got " +
           text(t->sizes()) + " " + text(t->scalar_type()));
}

// Graphs of graph_offsets (int32 [G + 1], or null: one).
int graphs(const Tensor* offsets) {
  if (!offsets) return 1;
  if (offsets->scalar_type() != at::kInt || offsets->dim() != 1 || offsets->size(0) < 2)
    refuse("graph_offsets: expected int32 [G + 1] with G >= 1");
  return narrow(offsets->size(0) - 1, "graph_offsets");
}

const void* in(const Tensor& t) { return t.const_data_ptr(); }
const void* in(const Tensor* t) { return t ? t->const_data_ptr() : nullptr; }
void* out(const Tensor& t) { return t.mutable_data_ptr(); }

// ----------------------------------------------------------------- the call
struct Unlocked {
  PyThreadState* thread = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(thread); }
};
// Python's lock is free while this lives, and x's device the current one.
struct Launch {
  Unlocked unlocked;
  c10::cuda::CUDAGuard guard;
  explicit Launch(const Tensor& x) : guard(x.device()) {}
};

// The stream that is current on x's device.  Results come from the allocator's
// pool of that stream, so the stream that writes them has to be this one.
kmip_stream_t stream_of(const Tensor& x) {
  return c10::cuda::getCurrentCUDAStream(x.get_device()).stream();
}

void check(kmip_status_t status, const char* where) {
  if (status != KMIP_OK) throw Failed{status, where};
}

PyObject* tuple(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Raised{};
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));  // undefined: None
  return r;
}

template <int ARGS, typename F>
PyObject* guarded(Py_ssize_t n, F&& f) {
  HANDLE_TH_ERRORS
  try {
    if (n != ARGS) throw Refused{PyExc_TypeError, "wrong number of arguments"};
    if (!g_error) throw Refused{PyExc_RuntimeError, "setup() comes first"};
    return f();
  } catch (const Refused& e) {
    PyErr_SetString(e.type, e.text.c_str());
  } catch (const Failed& e) {
    PyObject* v = Py_BuildValue("(is)", (int)e.status, e.where);
    if (v) PyErr_SetObject(g_error, v);
    Py_XDECREF(v);
  } catch (const Raised&) {
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ operators
// rotary(x, pos, freq, axis, inverse, interleaved, out or None)
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<7>(n, [&] {
    const Tensor &x = tensor(a[0], "x"), &pos = tensor(a[1], "pos"), &freq = tensor(a[2], "freq"),
                 &axis = tensor(a[3], "axis");
    const bool inverse = truth(a[4]), interleaved = truth(a[5]);
    const Tensor* given = optional(a[6], "out");
    if (x.dim() != 3) refuse("x: expected [N, H, d]");
    const int64_t N = x.size(0), H = x.size(1), d = x.size(2), P = freq.numel();
    const bool any = d > 1 && N > 0 && H > 0;
    if (x.stride(2) != 1 && any) refuse("x: expected adjacent elements in a head");
    kmip_pos_t type;
    switch (pos.scalar_type()) {
      case at::kFloat: type = KMIP_POS_F32; break;
      case at::kInt: type = KMIP_POS_I32; break;
      case at::kLong: type = KMIP_POS_I64; break;
      default:
        throw Refused{PyExc_TypeError, "unsupported position dtype " + text(pos.scalar_type()) +
                                           " (fp32, int32 or int64)"};
    }
    if (pos.dim() != 2 || pos.size(0) != N)
      refuse("pos: expected [" + std::to_string(N) + ", axes], got " + text(pos.sizes()));
    expect(&freq, "freq", {P}, at::kDouble);
    expect(&axis, "axis", {P}, at::kInt);
    same_device(x, {&pos, &freq, &axis});
    if (given && (given->sizes() != x.sizes() || given->scalar_type() != x.scalar_type() ||
                  given->device() != x.device() || (given->stride(2) != 1 && any)))
      refuse("out: expected a tensor like x");
    const kmip_dtype_t dtype = dtype_of(x);
    const int h = narrow(H, "x"), width = narrow(d, "x"), pairs = narrow(P, "freq");
    const int axes = narrow(pos.size(1), "pos");
    Tensor y;
    {
      const Launch launch(x);
      y = given ? *given : at::empty(x.sizes(), x.options());
      check(g_rotary(in(x), x.stride(0), x.stride(1), in(pos), type, axes,
                     static_cast<const double*>(in(freq)), static_cast<const int32_t*>(in(axis)),
                     pairs, interleaved, inverse, N, h, width, out(y), y.stride(0), y.stride(1),
                     stream_of(x), dtype),
            "kmip_rotary");
      // autograd learns that what it may have saved has changed
      if (given && !given->is_inference()) given->unsafeGetTensorImpl()->bump_version();
    }
    return THPVariable_Wrap(y);
  });
}

// group_norm_fwd(x, weight, bias, groups, eps, act, graph_offsets)
PyObject* group_norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<7>(n, [&] {
    const Tensor& x = tensor(a[0], "x");
    const Tensor *w = optional(a[1], "weight"), *b = optional(a[2], "bias");
    const int groups = narrow(integer(a[3]), "groups");
    const double eps = PyFloat_AsDouble(a[4]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
    const int act = narrow(integer(a[5]), "act");
    const Tensor* off = optional(a[6], "graph_offsets");
    if (x.dim() != 2) refuse("x: expected [N, C]");
    const int64_t N = x.size(0), C = x.size(1);
    const int G = graphs(off);
    same_device(x, {&x, w, b, off});
    expect(w, "weight", {C}, x.scalar_type());
    expect(b, "bias", {C}, x.scalar_type());
    const kmip_dtype_t dtype = dtype_of(x);
    const int channels = narrow(C, "x");
    Tensor y, mean, rstd;
    {
      const Launch launch(x);
      y = at::empty(x.sizes(), x.options());
      mean = at::empty({G, groups}, x.options().dtype(at::kFloat));
      rstd = at::empty({G, groups}, x.options().dtype(at::kFloat));
      check(g_norm_fwd(in(x), in(w), in(b), static_cast<const int32_t*>(in(off)), N, channels,
                       groups, (float)eps, (kmip_act_t)act, out(y),
                       static_cast<float*>(out(mean)), static_cast<float*>(out(rstd)),
                       stream_of(x), G, dtype),
            "kmip_group_norm_fwd");
    }
    return tuple({y, mean, rstd});
  });
}

// group_norm_bwd(dy, x, weight, bias, mean, rstd, groups, act, graph_offsets)
PyObject* group_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<9>(n, [&] {
    const Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x");
    const Tensor *w = optional(a[2], "weight"), *b = optional(a[3], "bias");
    const Tensor &mean = tensor(a[4], "mean"), &rstd = tensor(a[5], "rstd");
    const int groups = narrow(integer(a[6]), "groups"), act = narrow(integer(a[7]), "act");
    const Tensor* off = optional(a[8], "graph_offsets");
    if (x.dim() != 2) refuse("x: expected [N, C]");
    const int64_t N = x.size(0), C = x.size(1);
    const int G = graphs(off);
    same_device(x, {&x, &dy, w, b, off, &mean, &rstd});
    expect(&dy, "dy", {N, C}, x.scalar_type());
    expect(w, "weight", {C}, x.scalar_type());
    expect(b, "bias", {C}, x.scalar_type());
    expect(&mean, "mean", {G, groups}, at::kFloat);
    expect(&rstd, "rstd", {G, groups}, at::kFloat);
    const kmip_dtype_t dtype = dtype_of(x);
    const int channels = narrow(C, "x");
    Tensor dx, dw, db;
    {
      const Launch launch(x);
      dx = at::empty(x.sizes(), x.options());
      if (w) {
        dw = at::empty(w->sizes(), x.options());
        db = at::empty(w->sizes(), x.options());
      }
      check(g_norm_bwd(in(dy), in(x), in(w), in(b), static_cast<const int32_t*>(in(off)),
                       static_cast<const float*>(in(mean)), static_cast<const float*>(in(rstd)), N,
                       channels, groups, (kmip_act_t)act, out(dx), w ? out(dw) : nullptr,
                       w ? out(db) : nullptr, stream_of(x), G, dtype),
            "kmip_group_norm_bwd");
    }
    return tuple({dx, dw, db});
  });
}

struct Ffn {
  const Tensor &x, &wg, &wu, &wd;
  int64_t N, C, F;
  int c, f;
  kmip_act_t act;
  kmip_dtype_t dtype;
  // a: x, wg, wu, wd, act
  explicit Ffn(PyObject* const* a)
      : x(tensor(a[0], "x")), wg(tensor(a[1], "wg")), wu(tensor(a[2], "wu")),
        wd(tensor(a[3], "wd")), act((kmip_act_t)narrow(integer(a[4]), "act")) {
    if (x.dim() != 2 || wg.dim() != 2) refuse("x: expected [N, C]; wg, wu: [F, C]; wd: [C, F]");
    N = x.size(0);
    C = x.size(1);
    F = wg.size(0);
    same_device(x, {&x, &wg, &wu, &wd});
    expect(&wg, "wg", {F, C}, x.scalar_type());
    expect(&wu, "wu", {F, C}, x.scalar_type());
    expect(&wd, "wd", {C, F}, x.scalar_type());
    dtype = dtype_of(x);
    c = narrow(C, "x");
    f = narrow(F, "wg");
  }
};

// ffn_fwd(x, wg, wu, wd, act)
PyObject* ffn_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<5>(n, [&] {
    const Ffn p(a);
    Tensor y;
    {
      const Launch launch(p.x);
      y = at::empty(p.x.sizes(), p.x.options());
      check(g_ffn_fwd(in(p.x), in(p.wg), in(p.wu), in(p.wd), p.N, p.c, p.f, p.act, out(y),
                      stream_of(p.x), p.dtype),
            "kmip_ffn_fwd");
    }
    return THPVariable_Wrap(y);
  });
}

// ffn_bwd(dy, x, wg, wu, wd, act)
PyObject* ffn_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<6>(n, [&] {
    const Tensor& dy = tensor(a[0], "dy");
    const Ffn p(a + 1);
    same_device(p.x, {&dy});
    expect(&dy, "dy", {p.N, p.C}, p.x.scalar_type());
    Tensor dx, dwg, dwu, dwd;
    {
      const Launch launch(p.x);
      dx = at::empty(p.x.sizes(), p.x.options());
      dwg = at::empty(p.wg.sizes(), p.x.options());
      dwu = at::empty(p.wu.sizes(), p.x.options());
      dwd = at::empty(p.wd.sizes(), p.x.options());
      check(g_ffn_bwd(in(dy), in(p.x), in(p.wg), in(p.wu), in(p.wd), p.N, p.c, p.f, p.act, out(dx),
                      out(dwg), out(dwu), out(dwd), stream_of(p.x), p.dtype),
            "kmip_ffn_bwd");
    }
    return tuple({dx, dwg, dwu, dwd});
  });
}

// setup(KmipError, addresses of the five entry points in the order above)
PyObject* setup(PyObject*, PyObject* args) {
  PyObject* error;
  unsigned long long p[5];
  if (!PyArg_ParseTuple(args, "OKKKKK", &error, &p[0], &p[1], &p[2], &p[3], &p[4])) return nullptr;
  g_rotary = reinterpret_cast<decltype(g_rotary)>(p[0]);
  g_norm_fwd = reinterpret_cast<decltype(g_norm_fwd)>(p[1]);
  g_norm_bwd = reinterpret_cast<decltype(g_norm_bwd)>(p[2]);
  g_ffn_fwd = reinterpret_cast<decltype(g_ffn_fwd)>(p[3]);
  g_ffn_bwd = reinterpret_cast<decltype(g_ffn_bwd)>(p[4]);
  Py_INCREF(error);
  Py_XSETREF(g_error, error);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef fast(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {{"setup", setup, METH_VARARGS, nullptr},
                           fast<rotary>("rotary"),
                           fast<group_norm_fwd>("group_norm_fwd"),
                           fast<group_norm_bwd>("group_norm_bwd"),
                           fast<ffn_fwd>("ffn_fwd"),
                           fast<ffn_bwd>("ffn_bwd"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_kmip_host", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__kmip_host() { return PyModule_Create(&g_module); }
