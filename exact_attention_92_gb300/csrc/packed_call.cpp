// Calls on rows with strides (rotary positions, packed sequences) from Python
// without ctypes, as kv4_call.cpp does for the 4-bit cache: the tensors are checked
// and their pointers and strides passed to the entry points of libfa.so, whose
// addresses bind() is given.  A call whose tensors are not as they should be
// returns -1, and the binding works out what to say.
#include <Python.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "fa.h"

namespace {

decltype(&fa_rope) g_rope = nullptr;
decltype(&fa_packed_fwd) g_packed = nullptr;
decltype(&fa_prefix_fwd) g_prefix = nullptr;
decltype(&fa_packed_bwd) g_backward = nullptr;

PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
    return nullptr;
  }
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_rope = reinterpret_cast<decltype(g_rope)>(p[0]);
  g_packed = reinterpret_cast<decltype(g_packed)>(p[1]);
  g_prefix = reinterpret_cast<decltype(g_prefix)>(p[2]);
  g_backward = reinterpret_cast<decltype(g_backward)>(p[3]);
  Py_RETURN_NONE;
}

// The current device, and a stream's handle: that given, or torch's current one.
struct Where {
  long device;
  void* stream;
  explicit Where(PyObject* given)
      : device(c10::cuda::current_device()),
        stream(given == Py_None ? c10::cuda::getCurrentCUDAStream().stream() : PyLong_AsVoidPtr(given)) {}
};

// A bf16 tensor [tokens, heads, d] or [B, heads, N, d] on the device as rows; of
// an output, the rows do not overlap.
struct Rows {
  const at::Tensor* t = nullptr;
  fa_rows_t r = {};
  int64_t batch = 1, tokens = 0, heads = 0, d = 0;
  bool good = false;

  Rows(PyObject* o, int dims, long device, bool output) {
    if (!THPVariable_Check(o)) return;
    const at::Tensor& x = THPVariable_Unpack(o);
    if (x.scalar_type() != at::kBFloat16 || x.dim() != dims || !x.is_cuda() || x.get_device() != device) return;
    const int token_axis = dims == 3 ? 0 : 2, head_axis = dims == 3 ? 1 : 1;
    d = x.size(dims - 1);
    tokens = x.size(token_axis);
    heads = x.size(head_axis);
    if (d < 1 || d > INT32_MAX || tokens > INT32_MAX || heads > INT32_MAX || (d > 1 && x.stride(dims - 1) != 1)) return;
    r.row_stride = tokens > 1 ? x.stride(token_axis) : 0;
    r.head_stride = heads > 1 ? x.stride(head_axis) : 0;
    if (dims == 4) {
      batch = x.size(0);
      if (batch > INT32_MAX) return;
      r.batch_stride = batch > 1 ? x.stride(0) : 0;
    }
    if (r.row_stride % 8 != 0 || r.head_stride % 8 != 0 || r.batch_stride % 8 != 0) return;
    if (output) {
      struct Axis {
        int64_t stride, n;
      } axes[3] = {{r.row_stride, tokens}, {r.head_stride, heads}, {r.batch_stride, batch}};
      std::sort(axes, axes + 3, [](const Axis& a, const Axis& b) { return a.stride < b.stride; });
      int64_t reach = d;
      for (const Axis& a : axes) {
        if (a.n <= 1) continue;
        if (a.stride < reach) return;
        reach += a.stride * (a.n - 1);
      }
    }
    r.ptr = x.data_ptr();
    t = &x;
    good = true;
  }
  bool like(const Rows& o) const { return good && o.good && t->sizes() == o.t->sizes(); }
};

// A contiguous array on the device, or null.
const at::Tensor* array(PyObject* o, at::ScalarType type, int dims, long device) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.scalar_type() == type && t.dim() == dims && t.is_cuda() && t.get_device() == device && t.is_contiguous()
             ? &t
             : nullptr;
}

// rope(q, k or None, q_out, k_out, phases, positions, start, interleaved, mscale, inverse, stream)
int do_rope(PyObject* const* a) {
  const double mscale = PyFloat_AsDouble(a[8]);
  const int interleaved = PyObject_IsTrue(a[7]), inverse = PyObject_IsTrue(a[9]);
  const Where where(a[10]);
  if (PyErr_Occurred()) return -2;
  if (!THPVariable_Check(a[0])) return -1;
  const int dims = (int)THPVariable_Unpack(a[0]).dim();
  if (dims != 3 && dims != 4) return -1;
  const Rows q(a[0], dims, where.device, false), q_out(a[2], dims, where.device, true);
  if (!q_out.like(q)) return -1;
  const bool keys = a[1] != Py_None;
  if (!keys && a[3] != Py_None) return -1;
  const Rows k(keys ? a[1] : a[0], dims, where.device, false), k_out(keys ? a[3] : a[2], dims, where.device, true);
  if (!k_out.like(k) || k.batch != q.batch || k.tokens != q.tokens || k.d != q.d) return -1;
  const at::Tensor* phases = array(a[4], at::kLong, 1, where.device);
  const at::Tensor* pos = a[5] == Py_None ? nullptr : array(a[5], at::kInt, dims == 3 ? 1 : 2, where.device);
  const at::Tensor* start = a[6] == Py_None ? nullptr : array(a[6], at::kInt, 1, where.device);
  if (!phases || phases->size(0) > INT32_MAX / 2 || (a[5] != Py_None && !pos) || (a[6] != Py_None && !start)) return -1;
  if (pos && (pos->size(0) != (dims == 3 ? q.tokens : q.batch) || (dims == 4 && pos->size(1) != q.tokens))) return -1;
  if (start && start->size(0) != q.batch) return -1;
  const uint64_t* ph = static_cast<const uint64_t*>(phases->data_ptr());
  const int* pp = pos ? static_cast<const int*>(pos->data_ptr()) : nullptr;
  const int* sp = start ? static_cast<const int*>(start->data_ptr()) : nullptr;
  const int rot = (int)(2 * phases->size(0));
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = g_rope(&q.r, keys ? &k.r : nullptr, &q_out.r, keys ? &k_out.r : nullptr, ph, pp, sp, (int)q.batch, (int)q.tokens,
                  (int)q.heads, keys ? (int)k.heads : 0, (int)q.d, rot, interleaved, (float)mscale, inverse, where.stream);
  Py_END_ALLOW_THREADS;
  return status;
}

// What the attention calls share.
struct Sequences {
  const int *cu_q, *cu_k, *used;
  int B;
  int causal;
  float scale;
  bool good = false;
  Sequences(PyObject* q, PyObject* k, PyObject* u, PyObject* mask, PyObject* s, int64_t d, long device) {
    const long code = PyLong_AsLong(mask);
    const double given = s == Py_None ? 0.0 : PyFloat_AsDouble(s);
    if (PyErr_Occurred()) return;
    const at::Tensor* tq = array(q, at::kInt, 1, device);
    const at::Tensor* tk = array(k, at::kInt, 1, device);
    const at::Tensor* tu = u == Py_None ? nullptr : array(u, at::kInt, 1, device);
    if (!tq || !tk || tq->size(0) < 2 || tq->size(0) > INT32_MAX || tk->size(0) != tq->size(0)) return;
    if (u != Py_None && (!tu || tu->size(0) != tq->size(0) - 1)) return;
    B = (int)tq->size(0) - 1;
    cu_q = static_cast<const int*>(tq->data_ptr());
    cu_k = static_cast<const int*>(tk->data_ptr());
    used = tu ? static_cast<const int*>(tu->data_ptr()) : nullptr;
    causal = code >= 0 && code <= INT32_MAX ? (int)code : -1;
    scale = (float)(s == Py_None ? 1.0 / std::sqrt((double)d) : given);
    good = true;
  }
};

float* logsumexp(PyObject* o, const Rows& q, long device) {
  const at::Tensor* t = array(o, at::kFloat, 2, device);
  return t && t->size(0) == q.heads && t->size(1) == q.tokens ? static_cast<float*>(t->data_ptr()) : nullptr;
}

// forward(q, k_prefix or None, v_prefix, k, v, o, lse, cu_q, cu_k, used_k or None, causal, scale or None, stream or None)
int do_forward(PyObject* const* a) {
  const Where where(a[12]);
  if (PyErr_Occurred()) return -2;
  const Rows q(a[0], 3, where.device, false), k(a[3], 3, where.device, false), v(a[4], 3, where.device, false);
  const Rows o(a[5], 3, where.device, true);
  if (!o.like(q) || !v.like(k) || k.d != q.d) return -1;
  const Sequences s(a[7], a[8], a[9], a[10], a[11], q.d, where.device);
  if (PyErr_Occurred()) return -2;
  float* lse = logsumexp(a[6], q, where.device);
  if (!s.good || !lse) return -1;
  const bool prefix = a[1] != Py_None;
  const Rows kp(prefix ? a[1] : a[3], 3, where.device, false), vp(prefix ? a[2] : a[4], 3, where.device, false);
  if (!vp.like(kp) || kp.heads != k.heads || kp.d != q.d) return -1;
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = prefix ? g_prefix(&q.r, &kp.r, &vp.r, &k.r, &v.r, &o.r, lse, s.cu_q, s.cu_k, s.used, s.B, (int)kp.tokens,
                             (int)q.tokens, (int)k.tokens, (int)q.heads, (int)k.heads, (int)q.d, s.causal, s.scale,
                             where.stream)
                  : g_packed(&q.r, &k.r, &v.r, &o.r, lse, s.cu_q, s.cu_k, s.used, s.B, (int)q.tokens, (int)k.tokens,
                             (int)q.heads, (int)k.heads, (int)q.d, s.causal, s.scale, where.stream);
  Py_END_ALLOW_THREADS;
  return status;
}

// backward(q, k, v, o, lse, dout, dq, dk, dv, cu_q, cu_k, causal, scale or None, stream or None)
int do_backward(PyObject* const* a) {
  const Where where(a[13]);
  if (PyErr_Occurred()) return -2;
  const Rows q(a[0], 3, where.device, false), k(a[1], 3, where.device, false), v(a[2], 3, where.device, false);
  const Rows o(a[3], 3, where.device, false), dout(a[5], 3, where.device, false), dq(a[6], 3, where.device, true);
  const Rows dk(a[7], 3, where.device, true), dv(a[8], 3, where.device, true);
  if (!o.like(q) || !dout.like(q) || !dq.like(q) || !v.like(k) || !dk.like(k) || !dv.like(k) || k.d != q.d) return -1;
  const Sequences s(a[9], a[10], Py_None, a[11], a[12], q.d, where.device);
  if (PyErr_Occurred()) return -2;
  const float* lse = logsumexp(a[4], q, where.device);
  if (!s.good || !lse) return -1;
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = g_backward(&q.r, &k.r, &v.r, &o.r, lse, &dout.r, &dq.r, &dk.r, &dv.r, s.cu_q, s.cu_k, s.B, (int)q.tokens,
                      (int)k.tokens, (int)q.heads, (int)k.heads, (int)q.d, s.causal, s.scale, where.stream);
  Py_END_ALLOW_THREADS;
  return status;
}

// The status as a number; a tensor that torch cannot look into (it throws), or
// no CUDA device, is refused like any other that will not do.
template <int (*F)(PyObject* const*), int COUNT>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != COUNT || g_rope == nullptr) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or called before bind");
    return nullptr;
  }
  int status = -1;
  try {
    status = F(args);
  } catch (...) {
    status = PyErr_Occurred() ? -2 : -1;
  }
  if (status == -2) return nullptr;
  return PyLong_FromLong(status);
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {
    {"bind", fast(bind), METH_FASTCALL, "addresses of fa_rope, fa_packed_fwd, fa_prefix_fwd, fa_packed_bwd"},
    {"rope", fast(call<do_rope, 11>), METH_FASTCALL, "fa_rope"},
    {"forward", fast(call<do_forward, 13>), METH_FASTCALL, "fa_packed_fwd or fa_prefix_fwd"},
    {"backward", fast(call<do_backward, 14>), METH_FASTCALL, "fa_packed_bwd"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_packed_call", "Calls on rows with strides.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: of the headers, for the binding to compare with torch's own.
PyMODINIT_FUNC PyInit__packed_call() {
  PyObject* m = PyModule_Create(&g_module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
