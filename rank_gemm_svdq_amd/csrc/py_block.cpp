// Python entry of the block operators: argument checks and marshalling of
// torch tensors into the C ABI (include/svdq.h), nothing else.
//
// A short call is bound by what happens before its launch (about 2.5 us of
// it the launch itself).  The same checks through ctypes took 3 us more a
// call: each property of a tensor is a Python call there and a field here.
//
// The functions of the C ABI are handed over as addresses (bind), so the module
// works on whichever build of the library the package has loaded.

#include <ATen/core/Tensor.h>
#include <c10/hip/HIPCachingAllocator.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "../../include/svdq.h"

namespace {

PyObject* g_error = nullptr;                       // SvdqError(status, text)
decltype(&svdq_add_rmsnorm_quantize) g_norm = nullptr;
decltype(&svdq_fp8_linear_shared) g_linear = nullptr;
decltype(&svdq_fp8_linear_workspace_bytes) g_linear_bytes = nullptr;
decltype(&svdq_rope) g_rope = nullptr;
decltype(&svdq_attention) g_attention = nullptr;

// thrown inside a call once the Python error is set
struct Refused {};

[[noreturn]] void refuse(int status, const char* where, const char* format, ...) {
  char text[512];
  va_list a;
  va_start(a, format);
  std::vsnprintf(text, sizeof text, format, a);
  va_end(a);
  const std::string all = std::string(where) + ": " + text;
  if (PyObject* e = PyObject_CallFunction(g_error, "is", status, all.c_str())) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Refused();
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

// What a call asks of its tensors.  `where` names the call, `dev` the GPU.
struct Call {
  const char* where;
  int dev = -1;
  at::ScalarType own{};       // the values' type
  int32_t dtype = 0;          // and its svdq_dtype

  const at::Tensor& tensor(PyObject* o, const char* what) const {
    if (!THPVariable_Check(o)) refuse(SVDQ_ERR_ARG, where, "%s is a %s, expected a tensor", what, Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
  }
  // the tensor that the others go by
  const at::Tensor& first(PyObject* o, const char* what, int64_t dims) {
    const at::Tensor& t = tensor(o, what);
    if (!t.is_cuda()) refuse(SVDQ_ERR_ARG, where, "%s is not in GPU memory", what);
    dev = t.get_device();
    if (dev != c10::hip::current_device())
      refuse(SVDQ_ERR_ARG, where, "%s is on cuda:%d, the current device is cuda:%d", what, dev,
             (int)c10::hip::current_device());
    own = t.scalar_type();
    if (own != at::kBFloat16 && own != at::kHalf && own != at::kShort)
      refuse(SVDQ_ERR_ARG, where, "%s has dtype %s, expected bfloat16, float16 or int16 (bf16 bits)", what,
             c10::toString(own));
    dtype = own == at::kHalf ? SVDQ_FP16 : SVDQ_BF16;
    if (t.dim() != dims)
      refuse(SVDQ_ERR_SHAPE, where, "%s has shape %s, expected %d dimensions", what, shape_text(t.sizes()).c_str(),
             (int)dims);
    return t;
  }
  void here(const at::Tensor& t, const char* what) const {
    if (!t.is_cuda() || t.get_device() != dev)
      refuse(SVDQ_ERR_ARG, where, "%s is on %s, expected cuda:%d", what, t.device().str().c_str(), dev);
  }
  void of(const at::Tensor& t, const char* what, at::ScalarType type) const {
    if (t.scalar_type() != type)
      refuse(SVDQ_ERR_ARG, where, "%s has dtype %s, expected %s", what, c10::toString(t.scalar_type()),
             c10::toString(type));
  }
  void shaped(const at::Tensor& t, const char* what, at::IntArrayRef shape) const {
    if (t.sizes() != shape)
      refuse(SVDQ_ERR_SHAPE, where, "%s has shape %s, expected %s", what, shape_text(t.sizes()).c_str(),
             shape_text(shape).c_str());
  }
  void whole(const at::Tensor& t, const char* what) const {
    if (!t.is_contiguous()) refuse(SVDQ_ERR_ARG, where, "%s is not contiguous", what);
  }
  // contiguous, of this type and shape
  void* plain(PyObject* o, const char* what, at::ScalarType type, at::IntArrayRef shape) const {
    const at::Tensor& t = tensor(o, what);
    here(t, what);
    of(t, what, type);
    shaped(t, what, shape);
    whole(t, what);
    return t.data_ptr();
  }
  void* optional(PyObject* o, const char* what, at::ScalarType type, at::IntArrayRef shape) const {
    return o == Py_None ? nullptr : plain(o, what, type, shape);
  }
  // contiguous E4M3 codes
  uint8_t* codes(const at::Tensor& t, const char* what) const {
    here(t, what);
    if (t.scalar_type() != at::kFloat8_e4m3fn && t.scalar_type() != at::kByte)
      refuse(SVDQ_ERR_ARG, where, "%s has dtype %s, expected float8_e4m3fn or uint8", what,
             c10::toString(t.scalar_type()));
    whole(t, what);
    return static_cast<uint8_t*>(t.data_ptr());
  }
  // values of the call's type and this shape, last dimension contiguous
  uint16_t* values(const at::Tensor& t, const char* what, at::IntArrayRef shape) const {
    here(t, what);
    of(t, what, own);
    shaped(t, what, shape);
    if (t.size(-1) > 1 && t.stride(-1) != 1)
      refuse(SVDQ_ERR_ARG, where, "the last dimension of %s is not contiguous", what);
    return static_cast<uint16_t*>(t.data_ptr());
  }
  // a workspace: bytes, or None
  void* memory(PyObject* o, size_t* bytes) const {
    if (o == Py_None) return nullptr;
    const at::Tensor& w = tensor(o, "workspace");
    *bytes = (size_t)w.numel();
    return *bytes ? plain(o, "workspace", at::kByte, w.sizes()) : nullptr;
  }
  void* stream(PyObject* o) const {
    if (o == Py_None) return c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream();
    PyObject* a = PyObject_GetAttrString(o, "cuda_stream");
    if (!a) throw Refused();
    void* s = PyLong_AsVoidPtr(a);
    Py_DECREF(a);
    if (!s && PyErr_Occurred()) throw Refused();
    return s;
  }
  void done(svdq_status s) const {
    if (s == SVDQ_OK) return;
    if (PyObject* e = PyObject_CallFunction(g_error, "is", (int)s, where)) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
    throw Refused();
  }
};

// the stride of a dimension with one place addresses nothing: 0
int64_t step(const at::Tensor& t, int64_t d) { return t.size(d) > 1 ? t.stride(d) : 0; }

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();
  return v != 0;
}
int32_t small(const Call& c, const char* what, int64_t n) {
  if (n < 0 || n > INT32_MAX) refuse(SVDQ_ERR_SHAPE, c.where, "%s is %lld", what, (long long)n);
  return (int32_t)n;
}

template <class Fn>
svdq_status without_gil(Fn&& fn) {
  svdq_status s;
  Py_BEGIN_ALLOW_THREADS
  s = fn();
  Py_END_ALLOW_THREADS
  return s;
}

template <class Fn>
PyObject* guarded(const char* where, Py_ssize_t got, Py_ssize_t want, Fn&& fn) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%s: %zd arguments, expected %zd", where, got, want);
    return nullptr;
  }
  if (!g_error) {
    PyErr_SetString(PyExc_RuntimeError, "the block module is not bound to a library");
    return nullptr;
  }
  try {
    fn();
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_Format(PyExc_RuntimeError, "%s: %s", where, e.what());
    return nullptr;
  }
  Py_RETURN_NONE;
}

// (x, weight, eps, q, s, residual, h, stream)
PyObject* add_rmsnorm_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const char* where = "svdq_add_rmsnorm_quantize";
  return guarded(where, n, 8, [&] {
    Call c{where};
    const at::Tensor& x = c.first(a[0], "x", 2);
    const int32_t M = small(c, "M", x.size(0)), K = small(c, "K", x.size(1));
    const auto shape = x.sizes();
    auto rows = [&](PyObject* o, const char* what, uint16_t** p, int64_t* st) {
      *p = nullptr;
      *st = K;
      if (o == Py_None) return;
      const at::Tensor& t = c.tensor(o, what);
      *p = c.values(t, what, shape);
      if (M > 1) *st = t.stride(0);                // the stride of a single row addresses nothing
    };
    uint16_t *xp, *rp, *hp;
    int64_t xs, rs, hs;
    rows(a[0], "x", &xp, &xs);
    rows(a[5], "residual", &rp, &rs);
    rows(a[6], "h", &hp, &hs);
    const auto* w = static_cast<uint16_t*>(c.plain(a[1], "weight", c.own, {K}));
    const at::Tensor& q = c.tensor(a[3], "q");
    uint8_t* qp = c.codes(q, "q");
    c.shaped(q, "q", shape);
    auto* s = static_cast<float*>(c.plain(a[4], "s", at::kFloat, {M, (K + SVDQ_FP8_BLOCK - 1) / SVDQ_FP8_BLOCK}));
    const float eps = (float)number(a[2]);
    void* st = c.stream(a[7]);
    c.done(without_gil([&] { return g_norm(xp, xs, rp, rs, w, eps, M, K, c.dtype, hp, hs, qp, s, st); }));
  });
}

// Memory of torch's allocator for the length of a call: handed out and taken
// back in the order of the call's own stream, so later work there may reuse it.
struct Scratch {
  void* p = nullptr;
  Scratch(size_t bytes, void* stream) {
    if (bytes) p = c10::hip::HIPCachingAllocator::raw_alloc_with_stream(bytes, static_cast<hipStream_t>(stream));
  }
  ~Scratch() {
    if (p) c10::hip::HIPCachingAllocator::raw_delete(p);
  }
  Scratch(const Scratch&) = delete;
  Scratch& operator=(const Scratch&) = delete;
};

// (xq, xs, wq, ws, Y, bias, workspace, stream); workspace None: torch's, for the call
PyObject* fp8_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const char* where = "svdq_fp8_linear";
  return guarded(where, n, 8, [&] {
    Call c{where};
    const at::Tensor& Y = c.first(a[4], "Y", 2);
    const at::Tensor &xq = c.tensor(a[0], "xq"), &wq = c.tensor(a[2], "wq");
    if (xq.dim() != 2 || wq.dim() != 2 || xq.size(0) != Y.size(0) || wq.size(0) != Y.size(1) || wq.size(1) != xq.size(1))
      refuse(SVDQ_ERR_SHAPE, where, "xq %s, wq %s and Y %s, expected (M, K), (N, K) and (M, N)",
             shape_text(xq.sizes()).c_str(), shape_text(wq.sizes()).c_str(), shape_text(Y.sizes()).c_str());
    const int32_t M = small(c, "M", xq.size(0)), K = small(c, "K", xq.size(1)), N = small(c, "N", wq.size(0));
    const int64_t kb = K / SVDQ_FP8_BLOCK;
    const uint8_t *xp = c.codes(xq, "xq"), *wp = c.codes(wq, "wq");
    const auto* sp = static_cast<float*>(c.plain(a[1], "xs", at::kFloat, {M, kb}));
    const auto* tp =
        static_cast<float*>(c.plain(a[3], "ws", at::kFloat, {(N + SVDQ_FP8_BLOCK - 1) / SVDQ_FP8_BLOCK, kb}));
    const auto* bp = static_cast<uint16_t*>(c.optional(a[5], "bias", c.own, {N}));
    c.whole(Y, "Y");
    auto* yp = static_cast<uint16_t*>(Y.data_ptr());
    size_t bytes = 0;
    void *own = c.memory(a[6], &bytes), *st = c.stream(a[7]);
    if (a[6] == Py_None) bytes = g_linear_bytes(M, K, N);
    const Scratch scratch(a[6] == Py_None ? bytes : 0, st);
    c.done(without_gil([&] {
      return g_linear(xp, sp, wp, tp, bp, M, K, N, c.dtype, yp, scratch.p ? scratch.p : own, bytes, st);
    }));
  });
}

// (turns, axis, axes, pairs, interleaved, positions, x, y, x2, y2, stream)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const char* where = "svdq_rope";
  return guarded(where, n, 11, [&] {
    Call c{where};
    const at::Tensor& x = c.first(a[6], "x", 3);
    svdq_rope_args p{};
    p.M = small(c, "M", x.size(0));
    p.axes = small(c, "axes", PyLong_AsLongLong(a[2]));
    p.pairs = small(c, "pairs", PyLong_AsLongLong(a[3]));
    p.head_dim = small(c, "head_dim", x.size(2));
    p.interleaved = truth(a[4]);
    p.dtype = c.dtype;
    auto heads = [&](int g, const at::Tensor& t, const char* xn, PyObject* yo, const char* yn) {
      const at::Tensor& y = c.tensor(yo, yn);
      p.x[g] = c.values(t, xn, t.sizes());
      p.y[g] = c.values(y, yn, t.sizes());
      p.heads[g] = small(c, "heads", t.size(1));
      p.x_token[g] = step(t, 0);
      p.x_head[g] = step(t, 1);
      p.y_token[g] = step(y, 0);
      p.y_head[g] = step(y, 1);
    };
    heads(0, x, "x", a[7], "y");
    if ((a[8] == Py_None) != (a[9] == Py_None)) refuse(SVDQ_ERR_ARG, where, "x2 and y2 go together");
    if (a[8] != Py_None) {
      const at::Tensor& x2 = c.tensor(a[8], "x2");
      if (x2.dim() != 3 || x2.size(0) != p.M || x2.size(2) != p.head_dim)
        refuse(SVDQ_ERR_SHAPE, where, "x2 has shape %s, expected (%d, heads, %d)", shape_text(x2.sizes()).c_str(), p.M,
               p.head_dim);
      heads(1, x2, "x2", a[9], "y2");
    }
    p.positions = static_cast<int32_t*>(c.plain(a[5], "positions", at::kInt, {p.M, p.axes}));
    p.turns = static_cast<float*>(c.plain(a[0], "the plan's turns", at::kFloat, {p.pairs, 2}));
    p.axis = static_cast<int32_t*>(c.plain(a[1], "the plan's axis", at::kInt, {p.pairs}));
    void* st = c.stream(a[10]);
    c.done(without_gil([&] { return g_rope(&p, st); }));
  });
}

// (q, k, v, o, ws, scale, causal, softcap, slopes, kv_len, prefix, q_doc, k_doc, stream)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const char* where = "svdq_attention";
  return guarded(where, n, 14, [&] {
    Call c{where};
    const at::Tensor &q = c.first(a[0], "q", 4), &k = c.tensor(a[1], "k"), &v = c.tensor(a[2], "v"),
                     &o = c.tensor(a[3], "o");
    if (k.dim() != 4 || k.size(0) != q.size(0) || k.size(3) != q.size(3))
      refuse(SVDQ_ERR_SHAPE, where, "q %s and k %s, expected (B, Sq, Hq, D) and (B, Skv, Hkv, D)",
             shape_text(q.sizes()).c_str(), shape_text(k.sizes()).c_str());
    svdq_attention_args p{};
    p.B = small(c, "B", q.size(0));
    p.Sq = small(c, "Sq", q.size(1));
    p.Skv = small(c, "Skv", k.size(1));
    p.Hq = small(c, "Hq", q.size(2));
    p.Hkv = small(c, "Hkv", k.size(2));
    p.D = small(c, "D", q.size(3));
    p.dtype = c.dtype;
    p.causal = truth(a[6]);
    p.scale = a[5] == Py_None ? (float)(1.0 / std::sqrt((double)p.D)) : (float)number(a[5]);
    p.softcap = (float)number(a[7]);
    p.q = c.values(q, "q", q.sizes());
    p.k = c.values(k, "k", k.sizes());
    p.v = c.values(v, "v", k.sizes());
    p.o = c.values(o, "o", q.sizes());
    p.q_batch = step(q, 0), p.q_token = step(q, 1), p.q_head = step(q, 2);
    p.k_batch = step(k, 0), p.k_token = step(k, 1), p.k_head = step(k, 2);
    p.v_batch = step(v, 0), p.v_token = step(v, 1), p.v_head = step(v, 2);
    p.o_batch = step(o, 0), p.o_token = step(o, 1), p.o_head = step(o, 2);
    p.slopes = static_cast<float*>(c.optional(a[8], "slopes", at::kFloat, {p.Hq}));
    p.kv_len = static_cast<int32_t*>(c.optional(a[9], "kv_len", at::kInt, {p.B}));
    p.prefix = static_cast<int32_t*>(c.optional(a[10], "prefix", at::kInt, {p.B}));
    if ((a[11] == Py_None) != (a[12] == Py_None)) refuse(SVDQ_ERR_ARG, where, "q_doc and k_doc go together");
    p.q_doc = static_cast<int32_t*>(c.optional(a[11], "q_doc", at::kInt, {p.B, p.Sq}));
    p.k_doc = static_cast<int32_t*>(c.optional(a[12], "k_doc", at::kInt, {p.B, p.Skv}));
    size_t bytes = 0;
    void *ws = c.memory(a[4], &bytes), *st = c.stream(a[13]);
    c.done(without_gil([&] { return g_attention(&p, ws, bytes, st); }));
  });
}

// (SvdqError, addresses of svdq_add_rmsnorm_quantize, svdq_fp8_linear_shared, svdq_fp8_linear_workspace_bytes,
// svdq_rope, svdq_attention)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind: an exception type and five addresses");
    return nullptr;
  }
  void* at[5];
  for (int i = 0; i < 5; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (!at[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
      return nullptr;
    }
  }
  g_norm = reinterpret_cast<decltype(g_norm)>(at[0]);
  g_linear = reinterpret_cast<decltype(g_linear)>(at[1]);
  g_linear_bytes = reinterpret_cast<decltype(g_linear_bytes)>(at[2]);
  g_rope = reinterpret_cast<decltype(g_rope)>(at[3]);
  g_attention = reinterpret_cast<decltype(g_attention)>(at[4]);
  Py_INCREF(a[0]);
  Py_XSETREF(g_error, a[0]);
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(add_rmsnorm_quantize), FAST(fp8_linear), FAST(rope), FAST(attention),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", "argument marshalling of the block operators", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&module); }
