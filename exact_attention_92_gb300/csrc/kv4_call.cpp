// Calls over the 4-bit key/value cache from Python without ctypes: a decoding
// step makes one or two of them a layer, and there the marshalling shows (7.2 us
// a call through ctypes and checks in Python, 2.1 us like this, 1.5 of them the
// launch).
//
// Argument marshalling only: the tensors are checked and their pointers passed
// to the entry points of libfa.so, whose addresses bind() is given.  A call
// whose tensors are not as they should be returns -1, and the binding works out
// what to say.
#include <Python.h>

#include <cmath>
#include <cstdint>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

namespace {

using WriteFn = int (*)(const void*, const void*, void*, const int*, const int*, const int*, int, int, int, int, int, int,
                        int, void*);
using ReadFn = int (*)(const void*, const int*, const int*, const int*, void*, void*, int, int, int, int, int, int, int,
                       void*);
using FwdFn = int (*)(const void*, const void*, const int*, const int*, void*, float*, int, int, int, int, int, int, int,
                      int, int, float, void*);
WriteFn g_write = nullptr;
ReadFn g_read = nullptr;
FwdFn g_fwd = nullptr;

// A contiguous CUDA tensor of a type on the current device, or null.
const at::Tensor* tensor(PyObject* o, at::ScalarType type, int dims, long device) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.scalar_type() == type && t.dim() == dims && t.is_cuda() && t.get_device() == device && t.is_contiguous()
             ? &t
             : nullptr;
}

// Sizes fit an int (the library checks the rest).
bool fits(const at::Tensor& t) {
  for (const int64_t n : t.sizes())
    if (n > INT32_MAX) return false;
  return true;
}

// Tokens of a page, from its bytes; 0 if they are not a whole number.
int page_size(int64_t page_bytes, int64_t d) {
  return d > 0 && page_bytes * 8 % (9 * d) == 0 ? (int)(page_bytes * 8 / (9 * d)) : 0;
}

PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "bind takes three addresses");
    return nullptr;
  }
  void* p[3];
  for (int i = 0; i < 3; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_write = reinterpret_cast<WriteFn>(p[0]);
  g_read = reinterpret_cast<ReadFn>(p[1]);
  g_fwd = reinterpret_cast<FwdFn>(p[2]);
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

// move(write, k, v, cache, block_table, start, count or None, stream or None)
int do_move(PyObject* const* a) {
  const Where where(a[7]);
  const long device = where.device;
  void* const stream = where.stream;
  if (PyErr_Occurred()) return -2;
  const at::Tensor* k = tensor(a[1], at::kBFloat16, 4, device);
  const at::Tensor* v = tensor(a[2], at::kBFloat16, 4, device);
  const at::Tensor* cache = tensor(a[3], at::kByte, 3, device);
  const at::Tensor* table = tensor(a[4], at::kInt, 2, device);
  const at::Tensor* start = tensor(a[5], at::kInt, 1, device);
  const at::Tensor* count = a[6] == Py_None ? nullptr : tensor(a[6], at::kInt, 1, device);
  if (!k || !v || !cache || !table || !start || (a[6] != Py_None && !count)) return -1;
  const int64_t B = k->size(0), heads = k->size(1), N = k->size(2), d = k->size(3);
  const int page = page_size(cache->size(2), d);
  if (k->sizes() != v->sizes() || cache->size(1) != heads || table->size(0) != B || start->size(0) != B ||
      (count && count->size(0) != B) || page == 0 || !fits(*k) || !fits(*cache) || !fits(*table))
    return -1;
  void* const kp = k->data_ptr();
  void* const vp = v->data_ptr();
  void* const cp = cache->data_ptr();
  const int* const tp = static_cast<const int*>(table->data_ptr());
  const int* const sp = static_cast<const int*>(start->data_ptr());
  const int* const np = count ? static_cast<const int*>(count->data_ptr()) : nullptr;
  const int pages = (int)cache->size(0), max_pages = (int)table->size(1);
  const bool write = a[0] == Py_True;
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = write ? g_write(kp, vp, cp, tp, sp, np, (int)B, (int)heads, (int)N, (int)d, pages, page, max_pages, stream)
                 : g_read(cp, tp, sp, np, kp, vp, (int)B, (int)heads, (int)N, (int)d, pages, page, max_pages, stream);
  Py_END_ALLOW_THREADS;
  return status;
}

// fwd(q, cache, block_table, lens, o, lse, causal, scale or None, stream or None)
int do_fwd(PyObject* const* a) {
  const long causal = PyLong_AsLong(a[6]);
  const double scale = a[7] == Py_None ? 0.0 : PyFloat_AsDouble(a[7]);
  const Where where(a[8]);
  const long device = where.device;
  void* const stream = where.stream;
  if (PyErr_Occurred()) return -2;
  const at::Tensor* q = tensor(a[0], at::kBFloat16, 4, device);
  const at::Tensor* cache = tensor(a[1], at::kByte, 3, device);
  const at::Tensor* table = tensor(a[2], at::kInt, 2, device);
  const at::Tensor* lens = tensor(a[3], at::kInt, 1, device);
  const at::Tensor* o = tensor(a[4], at::kBFloat16, 4, device);
  const at::Tensor* lse = tensor(a[5], at::kFloat, 3, device);
  if (!q || !cache || !table || !lens || !o || !lse) return -1;
  const int64_t B = q->size(0), H = q->size(1), Nq = q->size(2), d = q->size(3);
  const int page = page_size(cache->size(2), d);
  if (o->sizes() != q->sizes() || lse->size(0) != B || lse->size(1) != H || lse->size(2) != Nq || table->size(0) != B ||
      lens->size(0) != B || page == 0 || !fits(*q) || !fits(*cache) || !fits(*table))
    return -1;
  const float s = (float)(a[7] == Py_None ? 1.0 / std::sqrt((double)d) : scale);
  const int mask = causal >= 0 && causal <= INT32_MAX ? (int)causal : -1;  // not cut to a code that it is not
  const void* const qp = q->data_ptr();
  const void* const cp = cache->data_ptr();
  const int* const tp = static_cast<const int*>(table->data_ptr());
  const int* const np = static_cast<const int*>(lens->data_ptr());
  void* const op = o->data_ptr();
  float* const lp = static_cast<float*>(lse->data_ptr());
  const int pages = (int)cache->size(0), heads = (int)cache->size(1), max_pages = (int)table->size(1);
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = g_fwd(qp, cp, tp, np, op, lp, (int)B, (int)H, heads, (int)Nq, (int)d, pages, page, max_pages, mask, s, stream);
  Py_END_ALLOW_THREADS;
  return status;
}

// The status as a number; a tensor that torch cannot look into (it throws), or
// no CUDA device, is refused like any other that will not do.
template <int (*F)(PyObject* const*), int COUNT>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != COUNT || g_fwd == nullptr) {
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

PyMethodDef g_methods[] = {{"bind", fast(bind), METH_FASTCALL, "addresses of fa_kv4_write, fa_kv4_read, fa_kv4_fwd"},
                           {"move", fast(call<do_move, 8>), METH_FASTCALL, "fa_kv4_write or fa_kv4_read"},
                           {"fwd", fast(call<do_fwd, 9>), METH_FASTCALL, "fa_kv4_fwd"},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_kv4_call", "Calls over the 4-bit key/value cache.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: of the headers, for the binding to compare with torch's own.
PyMODINIT_FUNC PyInit__kv4_call() {
  PyObject* m = PyModule_Create(&g_module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
