// binding.cpp -- the short way from Python into the library for the calls that
// decode steps make by the hundred (module _fast).
//
// The binding's checks in Python cost about as much as the launch they precede
// (one router call of 8 tokens: 6.2 us of host time, 3.6 of them below the
// checks).  Each function here looks at the tensors directly, and where all is as
// the call needs it (dense tensors of the right types and sizes on the current
// device, outputs given) makes the C call on the current stream and returns True.
// Anything else enqueues nothing and returns None, also arguments that the C call
// refuses: the binding in Python then goes its own way, which finds and words the
// error, or serves the less plain call.  A launch that fails raises at once, since
// the same call made again might succeed and hide it.
//
// Torch's and the interpreter's internals are compiled in: beside others than those
// it was built for (BUILT_FOR_TORCH, torch's version) the module refuses to load, and
// the binding does without it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <dlfcn.h>
#include <cstdio>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/core/grad_mode.h>
#include <ATen/core/Tensor.h>

#include "../../include/moe.h"

namespace {

constexpr int64_t kMost = 0x7FFFFFFF;

decltype(&moe_route_topk) f_route_topk;
decltype(&moe_route_topk_backward) f_route_topk_backward;
decltype(&moe_fp8_quant) f_fp8_quant;
decltype(&moe_fp8_quant_weights) f_fp8_quant_weights;
decltype(&moe_fp8_linear) f_fp8_linear;
decltype(&moe_fp8_linear_dw) f_fp8_linear_dw;
int (*f_get_device)(int*);  // hipGetDevice
PyObject* raw_stream;       // torch._C._cuda_getCurrentRawStream
PyObject* launch_failed;    // called with MOE_ERR_HIP, raises

// One call's arguments: whether all was plain so far, and the device.
struct Call {
  bool plain = true;
  int dev = -1;

  Call() { plain = f_get_device && raw_stream && f_get_device(&dev) == 0; }

  // The tensor, or null (and no plain call).
  const at::Tensor* tensor(PyObject* o) {
    if (!plain || !THPVariable_Check(o)) return plain = false, nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda() || t.device().index() != dev || !t.is_contiguous())
      return plain = false, nullptr;
    return &t;
  }

  template <size_t N>
  void* data(PyObject* o, at::ScalarType type, const int64_t (&shape)[N]) {
    const at::Tensor* t = tensor(o);
    if (!t) return nullptr;
    if (t->scalar_type() != type || t->dim() != (int64_t)N) return plain = false, nullptr;
    for (size_t i = 0; i < N; ++i)
      if (t->size(i) != shape[i]) return plain = false, nullptr;
    return t->data_ptr();
  }

  template <size_t N>
  void* optional(PyObject* o, at::ScalarType type, const int64_t (&shape)[N]) {
    return o == Py_None ? nullptr : data(o, type, shape);
  }

  int64_t integer(PyObject* o, int64_t least, int64_t most) {
    if (!plain || !PyLong_Check(o)) return plain = false, 0;
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &over);
    if (over || v < least || v > most) return plain = false, 0;
    return v;
  }

  double real(PyObject* o) {
    if (plain && PyFloat_Check(o)) return PyFloat_AS_DOUBLE(o);
    return (double)integer(o, -kMost, kMost);
  }

  // An input whose gradient would be lost.
  void outside_autograd(const at::Tensor* t) {
    if (t && t->requires_grad() && at::GradMode::is_enabled()) plain = false;
  }

  void* stream() {
    if (!plain) return nullptr;
    PyObject* index = PyLong_FromLong(dev);
    PyObject* s = index ? PyObject_CallOneArg(raw_stream, index) : nullptr;
    Py_XDECREF(index);
    void* p = s ? PyLong_AsVoidPtr(s) : nullptr;
    Py_XDECREF(s);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      plain = false;
    }
    return p;
  }
};

int elem_of(at::ScalarType t) {
  return t == at::kBFloat16 ? MOE_ELEM_BF16 : t == at::kHalf ? MOE_ELEM_F16 : t == at::kFloat ? MOE_ELEM_F32 : -1;
}
int scale_of(at::ScalarType t) { return t == at::kFloat ? MOE_SCALE_F32 : t == at::kByte ? MOE_SCALE_E8M0 : -1; }
at::ScalarType scale_type(int64_t code) { return code == MOE_SCALE_F32 ? at::kFloat : at::kByte; }
int64_t groups(int64_t n) { return (n + 127) / 128; }

PyObject* not_plain() { Py_RETURN_NONE; }

// The outcome of the C call.
PyObject* made(int status) {
  if (status == MOE_OK) Py_RETURN_TRUE;
  if (status != MOE_ERR_HIP) Py_RETURN_NONE;  // refused before anything was enqueued
  PyObject* code = launch_failed ? PyLong_FromLong(status) : nullptr;
  PyObject* r = code ? PyObject_CallOneArg(launch_failed, code) : nullptr;
  Py_XDECREF(code);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "a launch failed");
  return nullptr;
}

// No C++ exception leaves a function of the module.
template <PyObject* (*F)(PyObject* const*)>
PyObject* guarded(PyObject* const* a) {
  try {
    return F(a);
  } catch (...) {
    Py_RETURN_NONE;
  }
}
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) Py_RETURN_NONE;
  return guarded<F>(a);
}

// logits, bias, ids, weights, top_k, scoring, n_group, topk_group, group_top, renormalize, scale
PyObject* route_topk(PyObject* const* a) {
  Call c;
  const at::Tensor* l = c.tensor(a[0]);
  if (!l || l->dim() != 2) return not_plain();
  c.outside_autograd(l);
  const int64_t T = l->size(0), E = l->size(1), k = c.integer(a[4], 1, kMost);
  const int elem = elem_of(l->scalar_type());
  const void* bias = c.optional(a[1], at::kFloat, {E});
  void* ids = c.data(a[2], at::kInt, {T, k});
  void* w = c.data(a[3], at::kFloat, {T, k});
  const int64_t scoring = c.integer(a[5], 0, 1), ng = c.integer(a[6], 1, kMost), tg = c.integer(a[7], 1, kMost);
  const int64_t top = c.integer(a[8], 1, 2), renorm = c.integer(a[9], 0, 1);
  const double scale = c.real(a[10]);
  void* s = c.stream();
  if (!c.plain || elem < 0 || E > kMost) return not_plain();
  return made(f_route_topk(elem, l->data_ptr(), static_cast<const float*>(bias), T, (int)E, (int)k, (int)scoring, (int)ng,
                           (int)tg, (int)top, (int)renorm, (float)scale, static_cast<int32_t*>(ids),
                           static_cast<float*>(w), s));
}

// logits, ids, d_weights, scoring, renormalize, scale, d_logits
PyObject* route_topk_backward(PyObject* const* a) {
  Call c;
  const at::Tensor* l = c.tensor(a[0]);
  const at::Tensor* i = c.tensor(a[1]);
  const at::Tensor* d = c.tensor(a[2]);
  if (!c.plain || l->dim() != 2 || i->dim() != 2) return not_plain();
  c.outside_autograd(l);
  c.outside_autograd(d);
  const int64_t T = l->size(0), E = l->size(1), k = i->size(1);
  const int elem = elem_of(l->scalar_type());
  const void* ids = c.data(a[1], at::kInt, {T, k});
  const void* dw = c.data(a[2], at::kFloat, {T, k});
  const int64_t scoring = c.integer(a[3], 0, 1), renorm = c.integer(a[4], 0, 1);
  const double scale = c.real(a[5]);
  void* out = c.data(a[6], l->scalar_type(), {T, E});
  void* s = c.stream();
  if (!c.plain || elem < 0 || E > kMost || k > kMost) return not_plain();
  return made(f_route_topk_backward(elem, l->data_ptr(), static_cast<const int32_t*>(ids), static_cast<const float*>(dw), T,
                                    (int)E, (int)k, (int)scoring, (int)renorm, (float)scale, out, s));
}

// x, scale code, rows, columns, num_tokens_post_padded, q, q_scale, qt, qt_scale
PyObject* fp8_quant(PyObject* const* a) {
  Call c;
  const at::Tensor* x = c.tensor(a[0]);
  if (!x || x->dim() != 2) return not_plain();
  c.outside_autograd(x);
  const int64_t M = x->size(0), K = x->size(1), code = c.integer(a[1], 0, 1);
  const int elem = elem_of(x->scalar_type());
  const bool rows = c.integer(a[2], 0, 1), columns = c.integer(a[3], 0, 1);
  const void* ntp = c.optional(a[4], at::kInt, {1});
  void* q = rows ? c.data(a[5], at::kFloat8_e4m3fn, {M, K}) : nullptr;
  void* qs = rows ? c.data(a[6], scale_type(code), {M, groups(K)}) : nullptr;
  void* qt = columns ? c.data(a[7], at::kFloat8_e4m3fn, {K, 128 * groups(M)}) : nullptr;
  void* qts = columns ? c.data(a[8], scale_type(code), {K, groups(M)}) : nullptr;
  void* s = c.stream();
  if (!c.plain || elem < 0 || !(rows || columns)) return not_plain();
  return made(f_fp8_quant(elem, (int)code, x->data_ptr(), M, K, static_cast<const int32_t*>(ntp), q, qs, qt, qts, s));
}

// w, scale code, transposed, q, q_scale, qt, qt_scale
PyObject* fp8_quant_weights(PyObject* const* a) {
  Call c;
  const at::Tensor* w = c.tensor(a[0]);
  if (!w || w->dim() != 3) return not_plain();
  c.outside_autograd(w);
  const int64_t E = w->size(0), N = w->size(1), K = w->size(2), code = c.integer(a[1], 0, 1);
  const int elem = elem_of(w->scalar_type());
  const bool turned = c.integer(a[2], 0, 1);
  void* q = c.data(a[3], at::kFloat8_e4m3fn, {E, N, K});
  void* qs = c.data(a[4], scale_type(code), {E, groups(N), groups(K)});
  void* qt = turned ? c.data(a[5], at::kFloat8_e4m3fn, {E, K, N}) : nullptr;
  void* qts = turned ? c.data(a[6], scale_type(code), {E, groups(K), groups(N)}) : nullptr;
  void* s = c.stream();
  if (!c.plain || elem < 0) return not_plain();
  return made(f_fp8_quant_weights(elem, (int)code, w->data_ptr(), E, N, K, q, qs, qt, qts, s));
}

// x, x_scale, w, w_scale, expert_ids, num_tokens_post_padded, block_m, out
PyObject* fp8_linear(PyObject* const* a) {
  Call c;
  const at::Tensor* x = c.tensor(a[0]);
  const at::Tensor* xs = c.tensor(a[1]);
  const at::Tensor* w = c.tensor(a[2]);
  const at::Tensor* out = c.tensor(a[7]);
  if (!c.plain || x->dim() != 2 || w->dim() != 3) return not_plain();
  for (int i = 0; i < 4; ++i) c.outside_autograd(c.tensor(a[i]));
  const int64_t M = x->size(0), K = x->size(1), E = w->size(0), N = w->size(1);
  const int code = scale_of(xs->scalar_type()), elem = elem_of(out->scalar_type());
  if (code < 0 || elem < 0 || elem > MOE_ELEM_F16) return not_plain();
  const int64_t block_m = c.integer(a[6], 0, kMost);
  const void* ids = nullptr;
  const void* ntp = nullptr;
  if (a[4] == Py_None) {
    if (a[5] != Py_None || block_m) return not_plain();
  } else {
    const at::Tensor* e = c.tensor(a[4]);
    if (!c.plain || block_m < 1 || e->numel() < (M + block_m - 1) / block_m) return not_plain();
    ids = c.data(a[4], at::kInt, {e->numel()});
    ntp = c.data(a[5], at::kInt, {1});
  }
  const void* xp = c.data(a[0], at::kFloat8_e4m3fn, {M, K});
  const void* xsp = c.data(a[1], scale_type(code), {M, groups(K)});
  const void* wp = c.data(a[2], at::kFloat8_e4m3fn, {E, N, K});
  const void* wsp = c.data(a[3], scale_type(code), {E, groups(N), groups(K)});
  void* op = c.data(a[7], out->scalar_type(), {M, N});
  void* s = c.stream();
  if (!c.plain || E > kMost) return not_plain();
  return made(f_fp8_linear(elem, code, xp, xsp, wp, wsp, static_cast<const int32_t*>(ids),
                           static_cast<const int32_t*>(ntp), op, M, K, N, (int)E, (int)block_m, s));
}

// dyt, dyt_scale, xt, xt_scale, num_experts, expert_ids, num_tokens_post_padded, block_m, out
PyObject* fp8_linear_dw(PyObject* const* a) {
  Call c;
  const at::Tensor* dy = c.tensor(a[0]);
  const at::Tensor* dys = c.tensor(a[1]);
  const at::Tensor* x = c.tensor(a[2]);
  const at::Tensor* out = c.tensor(a[8]);
  if (!c.plain || dy->dim() != 2 || x->dim() != 2) return not_plain();
  for (int i = 0; i < 4; ++i) c.outside_autograd(c.tensor(a[i]));
  const int64_t N = dy->size(0), M = dy->size(1), K = x->size(0), E = c.integer(a[4], 1, kMost);
  const int code = scale_of(dys->scalar_type()), elem = elem_of(out->scalar_type());
  if (code < 0 || elem < 0 || elem > MOE_ELEM_F16 || M % 128) return not_plain();
  const int64_t block_m = c.integer(a[7], 0, kMost);
  const void* ids = nullptr;
  const void* ntp = nullptr;
  int64_t blocks = 0;
  if (a[5] == Py_None) {
    if (a[6] != Py_None || block_m) return not_plain();
  } else {
    const at::Tensor* e = c.tensor(a[5]);
    if (!c.plain || block_m < 1) return not_plain();
    blocks = e->numel();
    ids = c.data(a[5], at::kInt, {blocks});
    ntp = c.data(a[6], at::kInt, {1});
  }
  const void* dp = c.data(a[0], at::kFloat8_e4m3fn, {N, M});
  const void* dsp = c.data(a[1], scale_type(code), {N, M / 128});
  const void* xp = c.data(a[2], at::kFloat8_e4m3fn, {K, M});
  const void* xsp = c.data(a[3], scale_type(code), {K, M / 128});
  void* op = c.data(a[8], out->scalar_type(), {E, N, K});
  void* s = c.stream();
  if (!c.plain) return not_plain();
  return made(f_fp8_linear_dw(elem, code, dp, dsp, xp, xsp, static_cast<const int32_t*>(ids),
                              static_cast<const int32_t*>(ntp), op, M, N, K, (int)E, (int)block_m, blocks, s));
}

// The library's handle (as dlopen gave it), torch's function for the current stream, and
// one that raises the error of a status.
PyObject* init(PyObject*, PyObject* args) {
  PyObject *handle, *stream, *failed = nullptr;
  if (!PyArg_ParseTuple(args, "OO|O", &handle, &stream, &failed)) return nullptr;
  void* h = PyLong_AsVoidPtr(handle);
  if (PyErr_Occurred()) return nullptr;
  auto get = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, name));
    return f != nullptr;
  };
  if (!get(f_route_topk, "moe_route_topk") || !get(f_route_topk_backward, "moe_route_topk_backward") ||
      !get(f_fp8_quant, "moe_fp8_quant") || !get(f_fp8_quant_weights, "moe_fp8_quant_weights") ||
      !get(f_fp8_linear, "moe_fp8_linear") || !get(f_fp8_linear_dw, "moe_fp8_linear_dw") ||
      !get(f_get_device, "hipGetDevice")) {
    f_get_device = nullptr;  // no call is plain then
    PyErr_SetString(PyExc_RuntimeError, "the library lacks an entry point");
    return nullptr;
  }
  Py_INCREF(stream);
  Py_XSETREF(raw_stream, stream);
  Py_XINCREF(failed);
  Py_XSETREF(launch_failed, failed);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, nullptr},
    {"route_topk", (PyCFunction)(void (*)())entry<route_topk, 11>, METH_FASTCALL, nullptr},
    {"route_topk_backward", (PyCFunction)(void (*)())entry<route_topk_backward, 7>, METH_FASTCALL, nullptr},
    {"fp8_quant", (PyCFunction)(void (*)())entry<fp8_quant, 9>, METH_FASTCALL, nullptr},
    {"fp8_quant_weights", (PyCFunction)(void (*)())entry<fp8_quant_weights, 7>, METH_FASTCALL, nullptr},
    {"fp8_linear", (PyCFunction)(void (*)())entry<fp8_linear, 8>, METH_FASTCALL, nullptr},
    {"fp8_linear_dw", (PyCFunction)(void (*)())entry<fp8_linear_dw, 9>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

// Whether this interpreter and this torch are the ones built for; sets an error if not.
bool built_for_these() {
  int major = 0, minor = 0;
  const bool python = sscanf(Py_GetVersion(), "%d.%d", &major, &minor) == 2 && major == PY_MAJOR_VERSION &&
                      minor == PY_MINOR_VERSION;
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
  PyObject* text = version ? PyObject_Str(version) : nullptr;
  const bool ok = text && python && PyUnicode_CompareWithASCIIString(text, BUILT_FOR_TORCH) == 0;
  if (text && !ok)
    PyErr_Format(PyExc_ImportError, "built for torch %s and Python %d.%d, not torch %U and Python %d.%d",
                 BUILT_FOR_TORCH, PY_MAJOR_VERSION, PY_MINOR_VERSION, text, major, minor);
  Py_XDECREF(text);
  Py_XDECREF(version);
  Py_XDECREF(torch);
  return ok;
}

}  // namespace

PyMODINIT_FUNC PyInit__fast() { return built_for_these() ? PyModule_Create(&module) : nullptr; }
