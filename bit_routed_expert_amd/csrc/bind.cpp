// Argument marshalling of the operators around the experts, for bit_routed_expert_amd/__init__.py: the
// checks of tensors, the allocation of outputs and the call into the C ABI. It does what the ctypes binding of
// the other entry points does in Python; compiled, because these calls are short and take up to seven tensors:
// a call of add_rmsnorm_mx takes the host 15 us that way and 7 us this way, mx_matmul 8.6 and 4.6.
//
// Every function takes its arguments by position, ending with the current device and its stream's handle, and
// returns its outputs, or the negative status of the C ABI. Host code only.
#include <Python.h>
#include <dlfcn.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <string>

#include "../../include/moe_w2.h"

namespace {

struct Raised {};   // a Python exception is set
PyObject* out_of_memory = nullptr;   // torch.OutOfMemoryError

[[noreturn]] void raise(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Raised();
}

std::string words(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

// The C ABI, from the library that the Python module names.
struct Abi {
  decltype(&::mx_quantize) mx_quantize;
  decltype(&::mx_dequantize) mx_dequantize;
  decltype(&::mx_matmul) mx_matmul;
  decltype(&::add_rmsnorm_mx) add_rmsnorm_mx;
  decltype(&::moe_w2_permute_workspace_bytes) moe_w2_permute_workspace_bytes;
  decltype(&::moe_w2_permute) moe_w2_permute;
  decltype(&::moe_w2_unpermute) moe_w2_unpermute;
  decltype(&::moe_w2_unpermute_backward) moe_w2_unpermute_backward;
  decltype(&::moe_w2_permute_backward) moe_w2_permute_backward;
} abi;

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a CUDA (HIP) tensor");
  return THPVariable_Unpack(o);
}

// A contiguous tensor of this type and shape on device `dev`; its address.
void* address(const at::Tensor& t, at::ScalarType dtype, at::IntArrayRef shape, int dev, const char* name) {
  if (!t.is_cuda()) raise(PyExc_TypeError, std::string(name) + " must be a CUDA (HIP) tensor");
  if (t.scalar_type() != dtype)
    raise(PyExc_TypeError, std::string(name) + " must be " + at::toString(dtype) + ", got " + at::toString(t.scalar_type()));
  if (t.sizes() != shape) raise(PyExc_ValueError, std::string(name) + " must have shape " + words(shape) + ", got " + words(t.sizes()));
  if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
  if (t.get_device() != dev)
    raise(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", the current device is cuda:" + std::to_string(dev));
  return t.data_ptr();
}
void* address(PyObject* o, at::ScalarType dtype, at::IntArrayRef shape, int dev, const char* name) {
  return address(tensor(o, name), dtype, shape, dev, name);
}

struct Rows { int64_t r, k; };
Rows rows_of(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) raise(PyExc_ValueError, std::string(name) + " must be a tensor of rows (2 dimensions)");
  if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX) raise(PyExc_ValueError, std::string(name) + " has a dimension above 2^31 - 1");
  return {t.size(0), t.size(1)};
}

int dtype_of(at::ScalarType t, const char* name) {
  switch (t) {
    case at::kBFloat16: return MOE_W2_BF16;
    case at::kFloat: return MOE_W2_F32;
    case at::kHalf: return MOE_W2_F16;
    default: raise(PyExc_TypeError, std::string(name) + " must be a bfloat16, float16 or float32 tensor");
  }
}

// An output: the caller's, checked, or one that make() allocates.
struct Out {
  at::Tensor t;
  void* p = nullptr;
  c10::SmallVector<int64_t, 6> shape;
  at::ScalarType dtype = at::kByte;
  int dev = -1;                          // of one to be allocated
  void make() {
    if (dev < 0) return;
    t = at::empty(shape, at::TensorOptions().dtype(dtype).device(at::Device(at::kCUDA, dev)));
    p = t.data_ptr();
  }
};
Out output(PyObject* o, at::ScalarType dtype, at::IntArrayRef shape, int dev, const char* name) {
  Out r;
  if (o == Py_None) {
    if (dev < 0) raise(PyExc_RuntimeError, "no GPU is in use");
    r.shape.assign(shape.begin(), shape.end());
    r.dtype = dtype;
    r.dev = dev;
  } else {
    r.t = tensor(o, name);
    r.p = address(r.t, dtype, shape, dev, name);
  }
  return r;
}

// Allocates the outputs and calls the C ABI. Both may wait (for memory, for room in the stream's queue), so
// other Python threads run meanwhile; once a call, as taking the interpreter back may wait for them.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <class F, class... Outs>
int call(F&& f, Outs&... outs) {
  const Unlocked unlocked;
  (outs.make(), ...);
  return f();
}

int integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (v > INT32_MAX || v < INT32_MIN) raise(PyExc_ValueError, "an integer argument is out of range");
  return (int)v;
}
void* handle(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Raised();
  return p;
}
int format_of(PyObject* o) {
  const int f = integer(o);
  if (f != MOE_MX_E2M1 && f != MOE_MX_E4M3) raise(PyExc_ValueError, "format must be MX_E2M1 or MX_E4M3");
  return f;
}
int64_t code_bytes(int64_t k, int fmt) { return fmt == MOE_MX_E2M1 ? k / 2 : k; }

PyObject* status(int st) { return PyLong_FromLong(st); }
PyObject* give(const at::Tensor& t) { return THPVariable_Wrap(t); }
template <class... T>
PyObject* give(const at::Tensor& a, const at::Tensor& b, const T&... more) {
  PyObject* r = PyTuple_New(2 + sizeof...(more));
  if (!r) return nullptr;
  int i = 0;
  for (const at::Tensor* t : {&a, &b, &more...}) {
    PyObject* o = t->defined() ? THPVariable_Wrap(*t) : (Py_INCREF(Py_None), Py_None);
    if (!o) { Py_DECREF(r); return nullptr; }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

typedef PyObject* const* Args;

PyObject* quantize(Args a) {   // x, format, codes, scales
  const at::Tensor& x = tensor(a[0], "x");
  const Rows s = rows_of(x, "x");
  const int dt = dtype_of(x.scalar_type(), "x"), fmt = format_of(a[1]), dev = integer(a[4]);
  const void* px = address(x, x.scalar_type(), x.sizes(), dev, "x");
  Out codes = output(a[2], at::kByte, {s.r, code_bytes(s.k, fmt)}, dev, "codes");
  Out scales = output(a[3], at::kByte, {s.r, s.k / 32}, dev, "scales");
  void* const stream = handle(a[5]);
  const int st = call([&] {
    return abi.mx_quantize((int)s.r, (int)s.k, dt, px, fmt, (uint8_t*)codes.p, (uint8_t*)scales.p, stream);
  }, codes, scales);
  return st ? status(st) : give(codes.t, scales.t);
}

PyObject* dequantize(Args a) {   // codes, scales, format, dtype (enum moe_w2_dtype), x
  const at::Tensor& codes = tensor(a[0], "codes");
  const Rows s = rows_of(codes, "codes");
  const int fmt = format_of(a[2]), dt = integer(a[3]), dev = integer(a[5]);
  const int64_t k = fmt == MOE_MX_E2M1 ? 2 * s.k : s.k;
  const void* pc = address(codes, at::kByte, codes.sizes(), dev, "codes");
  const void* ps = address(a[1], at::kByte, {s.r, k / 32}, dev, "scales");
  Out x = output(a[4], dt == MOE_W2_F32 ? at::kFloat : dt == MOE_W2_F16 ? at::kHalf : at::kBFloat16, {s.r, k}, dev, "x");
  if (k > INT32_MAX) raise(PyExc_ValueError, "codes has too long rows");
  void* const stream = handle(a[6]);
  const int st = call([&] {
    return abi.mx_dequantize((int)s.r, (int)k, fmt, (const uint8_t*)pc, (const uint8_t*)ps, dt, x.p, stream);
  }, x);
  return st ? status(st) : give(x.t);
}

PyObject* matmul(Args a) {   // a_codes, a_scales, w_codes, w_scales, a_format, out_dtype, y
  const at::Tensor& ac = tensor(a[0], "a_codes");
  const at::Tensor& wc = tensor(a[2], "w_codes");
  const Rows s = rows_of(ac, "a_codes");
  const int64_t n = rows_of(wc, "w_codes").r;
  const int fmt = format_of(a[4]), out = integer(a[5]), dev = integer(a[7]);
  const int64_t k = fmt == MOE_MX_E2M1 ? 2 * s.k : s.k;
  if (k > INT32_MAX) raise(PyExc_ValueError, "a_codes has too long rows");
  const void* pa = address(ac, at::kByte, ac.sizes(), dev, "a_codes");
  const void* psa = address(a[1], at::kByte, {s.r, k / 32}, dev, "a_scales");
  const void* pw = address(wc, at::kByte, {n, k / 2}, dev, "w_codes");
  const void* psw = address(a[3], at::kByte, {n, k / 32}, dev, "w_scales");
  Out y = output(a[6], out == MOE_W2_OUT_F32 ? at::kFloat : at::kBFloat16, {s.r, n}, dev, "y");
  void* const stream = handle(a[8]);
  const int st = call([&] {
    return abi.mx_matmul((int)s.r, (int)n, (int)k, fmt, (const uint8_t*)pa, (const uint8_t*)psa, (const uint8_t*)pw,
                         (const uint8_t*)psw, y.p, out, stream);
  }, y);
  return st ? status(st) : give(y.t);
}

PyObject* add_rmsnorm(Args a) {   // x, residual, gamma, eps, format, normed (tensor, True or None), residual_out, codes, scales
  const at::Tensor& x = tensor(a[0], "x");
  const at::Tensor& gamma = tensor(a[2], "gamma");
  const Rows s = rows_of(x, "x");
  const at::ScalarType t = x.scalar_type();
  const int dt = dtype_of(t, "x"), gdt = dtype_of(gamma.scalar_type(), "gamma"), fmt = format_of(a[4]), dev = integer(a[9]);
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) throw Raised();
  const void* px = address(x, t, x.sizes(), dev, "x");
  const void* pr = a[1] == Py_None ? nullptr : address(a[1], t, x.sizes(), dev, "residual");
  const void* pg = address(gamma, gamma.scalar_type(), {s.k}, dev, "gamma");
  Out h = output(a[6], t, x.sizes(), dev, "residual_out");
  Out n;
  if (a[5] != Py_None) n = output(a[5] == Py_True ? Py_None : a[5], t, x.sizes(), dev, "normed");
  Out codes = output(a[7], at::kByte, {s.r, code_bytes(s.k, fmt)}, dev, "codes");
  Out scales = output(a[8], at::kByte, {s.r, s.k / 32}, dev, "scales");
  void* const stream = handle(a[10]);
  const int st = call([&] {
    return abi.add_rmsnorm_mx((int)s.r, (int)s.k, dt, px, pr, pg, gdt, (float)eps, h.p, n.p, fmt, (uint8_t*)codes.p,
                              (uint8_t*)scales.p, stream);
  }, h, n, codes, scales);
  return st ? status(st) : give(codes.t, scales.t, h.t, n.t);
}

PyObject* permute(Args a) {   // x, topk_ids, E, rows, workspace
  const at::Tensor& x = tensor(a[0], "x");
  const at::Tensor& ids = tensor(a[1], "topk_ids");
  const Rows s = rows_of(ids, "topk_ids");
  const int E = integer(a[2]), dev = integer(a[5]);
  if (x.dim() < 1 || x.size(0) != s.r) raise(PyExc_ValueError, "x must be a tensor of " + std::to_string(s.r) + " rows");
  int64_t row_bytes = x.element_size();
  for (int64_t i = 1; i < x.dim(); ++i) row_bytes *= x.size(i);
  const int64_t P = s.r * s.k;
  const void* px = address(x, x.scalar_type(), x.sizes(), dev, "x");
  const void* pi = address(ids, at::kInt, ids.sizes(), dev, "topk_ids");
  const size_t need = abi.moe_w2_permute_workspace_bytes(E, (int)s.r, (int)s.k);
  if (!need) return status(E < 1 || s.k < 1 ? MOE_W2_EINVAL : MOE_W2_EUNSUPPORTED);   // before outputs of such sizes
  c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
  shape[0] = P;
  Out rows = output(a[3], x.scalar_type(), shape, dev, "rows");
  Out w;
  if (a[4] != Py_None) {
    w.t = tensor(a[4], "workspace");
    w.p = address(w.t, at::kByte, w.t.sizes(), dev, "workspace");
  } else if (P > MOE_W2_PERMUTE_SMALL_PAIRS) {
    w = output(Py_None, at::kByte, {(int64_t)need}, dev, "workspace");
  }
  Out offsets = output(Py_None, at::kInt, {E + 1LL}, dev, "offsets");
  Out perm = output(Py_None, at::kInt, {P}, dev, "perm");
  Out pos = output(Py_None, at::kInt, {s.r, s.k}, dev, "pos");
  void* const stream = handle(a[6]);
  const int st = call([&] {
    return abi.moe_w2_permute(E, (int)s.r, (int)s.k, (const int32_t*)pi, px, row_bytes, rows.p, (int32_t*)offsets.p,
                              (int32_t*)perm.p, (int32_t*)pos.p, w.p, w.p ? (size_t)w.t.numel() : 0, stream);
  }, rows, w, offsets, perm, pos);
  return st ? status(st) : give(rows.t, offsets.t, perm.t, pos.t);
}

// The rows and positions that the other three share.
struct Pairs {
  int T, top_k, K, dtype;
  at::ScalarType t;
  const void *rows, *w;
  const int32_t* pos;
};
Pairs pairs_of(PyObject* rows, const char* name, PyObject* pos, PyObject* w, int dev) {
  const at::Tensor& r = tensor(rows, name);
  const at::Tensor& p = tensor(pos, "pos");
  const Rows rs = rows_of(r, name), ps = rows_of(p, "pos");
  if (rs.r != ps.r * ps.k)
    raise(PyExc_ValueError, std::string(name) + " must have " + std::to_string(ps.r * ps.k) + " rows, got " + std::to_string(rs.r));
  Pairs o;
  o.T = (int)ps.r; o.top_k = (int)ps.k; o.K = (int)rs.k;
  o.t = r.scalar_type();
  o.dtype = dtype_of(o.t, name);
  o.rows = address(r, o.t, r.sizes(), dev, name);
  o.pos = (const int32_t*)address(p, at::kInt, p.sizes(), dev, "pos");
  o.w = !w || w == Py_None ? nullptr : address(w, at::kFloat, p.sizes(), dev, "topk_w");
  return o;
}

PyObject* unpermute(Args a) {   // rows, pos, topk_w, y
  const int dev = integer(a[4]);
  const Pairs p = pairs_of(a[0], "rows", a[1], a[2], dev);
  Out y = output(a[3], p.t, {p.T, p.K}, dev, "y");
  void* const stream = handle(a[5]);
  const int st = call([&] {
    return abi.moe_w2_unpermute(p.T, p.top_k, p.K, p.dtype, p.rows, p.pos, (const float*)p.w, y.p, stream);
  }, y);
  return st ? status(st) : give(y.t);
}

PyObject* permute_backward(Args a) {   // d_rows, pos, dx
  const int dev = integer(a[3]);
  const Pairs p = pairs_of(a[0], "d_rows", a[1], nullptr, dev);
  Out dx = output(a[2], p.t, {p.T, p.K}, dev, "dx");
  void* const stream = handle(a[4]);
  const int st = call([&] { return abi.moe_w2_permute_backward(p.T, p.top_k, p.K, p.dtype, p.rows, p.pos, dx.p, stream); }, dx);
  return st ? status(st) : give(dx.t);
}

PyObject* unpermute_backward(Args a) {   // dy, rows, pos, topk_w, d_rows, d_w
  const int dev = integer(a[6]);
  const Pairs p = pairs_of(a[1], "rows", a[2], a[3], dev);
  const void* dy = address(a[0], p.t, {p.T, p.K}, dev, "dy");
  Out d_rows = output(a[4], p.t, {(int64_t)p.T * p.top_k, p.K}, dev, "d_rows");
  Out d_w = output(a[5], at::kFloat, {p.T, p.top_k}, dev, "d_w");
  void* const stream = handle(a[7]);
  const int st = call([&] {
    return abi.moe_w2_unpermute_backward(p.T, p.top_k, p.K, p.dtype, dy, p.rows, p.pos, (const float*)p.w, d_rows.p,
                                         (float*)d_w.p, stream);
  }, d_rows, d_w);
  return st ? status(st) : give(d_rows.t, d_w.t);
}

PyObject* load(Args a) {   // path of the library
  const char* path = PyUnicode_AsUTF8(a[0]);
  if (!path) throw Raised();
  void* lib = dlopen(path, RTLD_NOW);
  if (!lib) raise(PyExc_ImportError, dlerror());
#define MOEW2_ENTRY(name) \
  if (!(abi.name = (decltype(abi.name))dlsym(lib, #name))) raise(PyExc_ImportError, #name " is not in the library");
  MOEW2_ENTRY(mx_quantize)
  MOEW2_ENTRY(mx_dequantize)
  MOEW2_ENTRY(mx_matmul)
  MOEW2_ENTRY(add_rmsnorm_mx)
  MOEW2_ENTRY(moe_w2_permute_workspace_bytes)
  MOEW2_ENTRY(moe_w2_permute)
  MOEW2_ENTRY(moe_w2_unpermute)
  MOEW2_ENTRY(moe_w2_unpermute_backward)
  MOEW2_ENTRY(moe_w2_permute_backward)
#undef MOEW2_ENTRY
  PyObject* torch = PyImport_ImportModule("torch");
  if (!torch || !(out_of_memory = PyObject_GetAttrString(torch, "OutOfMemoryError"))) throw Raised();
  Py_DECREF(torch);
  Py_RETURN_NONE;
}

// C++ exceptions (an allocation that failed, say) become Python's; a call before load() is refused.
template <PyObject* (*F)(Args), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  if (F != load && !out_of_memory) {
    PyErr_SetString(PyExc_ImportError, "the library is not loaded");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(out_of_memory, e.what_without_backtrace());
    return nullptr;
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

#define MOEW2_METHOD(name, f, n) {name, (PyCFunction)(void (*)(void))entry<f, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    MOEW2_METHOD("load", load, 1),
    MOEW2_METHOD("mx_quantize", quantize, 6),
    MOEW2_METHOD("mx_dequantize", dequantize, 7),
    MOEW2_METHOD("mx_matmul", matmul, 9),
    MOEW2_METHOD("add_rmsnorm_mx", add_rmsnorm, 11),
    MOEW2_METHOD("moe_w2_permute", permute, 7),
    MOEW2_METHOD("moe_w2_unpermute", unpermute, 6),
    MOEW2_METHOD("moe_w2_permute_backward", permute_backward, 5),
    MOEW2_METHOD("moe_w2_unpermute_backward", unpermute_backward, 8),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// Tensors are read through PyTorch's headers, whose layouts go with its version.
PyMODINIT_FUNC PyInit__bind(void) {
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
  const char* v = version ? PyUnicode_AsUTF8(version) : nullptr;
  const bool same = v && !strcmp(v, MOEW2_TORCH_VERSION);
  if (v && !same) PyErr_Format(PyExc_ImportError, "_bind was built for PyTorch " MOEW2_TORCH_VERSION ", this is %s", v);
  Py_XDECREF(version);
  Py_XDECREF(torch);
  return same ? PyModule_Create(&module) : nullptr;
}
