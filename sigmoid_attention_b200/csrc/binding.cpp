// binding.cpp -- the paged calls for Python, for torch tensors.
//
// A serving step makes a few calls per layer whose kernels take 3 to 10 us. Checked
// in Python and marshalled by ctypes such a call took 8 to 12 us on the host, so
// the host set the pace; here it takes about 3 us, most of it the launch. Each
// function checks its tensors (type, device, shape, strides), takes the current
// stream unless one is given, and calls the C function of the same name; the
// names and argument order are those of the package's Python functions.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <exception>

#include "../../include/sigattn.h"

namespace {

// Thrown with a Python error set.
struct Refused {};

[[noreturn]] void refuse(const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(PyExc_ValueError, format, args);
  va_end(args);
  throw Refused{};
}

struct Call {
  PyObject* const* arg;
  Py_ssize_t count, next = 0;
  c10::DeviceIndex device = -1;  // the current device, once a tensor asks for it

  PyObject* take() {
    if (next >= count) refuse("too few arguments");
    return arg[next++];
  }
  static bool none(PyObject* o) { return o == Py_None; }
  // A tensor on the current device, on which the library launches.
  const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType type) {
    if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.is_cuda() && device < 0) device = c10::cuda::current_device();
    if (!t.is_cuda() || t.get_device() != device)
      refuse("%s must be on the current CUDA device", name);
    if (t.scalar_type() != type) refuse("%s must be a CUDA %s tensor", name, c10::toString(type));
    return t;
  }
  const at::Tensor& packed(const char* name, at::ScalarType type) { return packed(take(), name, type); }
  const at::Tensor& packed(PyObject* o, const char* name, at::ScalarType type) {
    const at::Tensor& t = tensor(o, name, type);
    if (!t.is_contiguous()) refuse("%s must be a contiguous CUDA %s tensor", name, c10::toString(type));
    return t;
  }
  // `n` int32 values.
  int32_t* ints(const char* name, int64_t n) { return ints(take(), name, n); }
  int32_t* ints(PyObject* o, const char* name, int64_t n) {
    const at::Tensor& t = packed(o, name, at::kInt);
    if (t.numel() != n) refuse("%s has %lld elements, expected %lld", name, (long long)t.numel(), (long long)n);
    return static_cast<int32_t*>(t.data_ptr());
  }
  // [B][width] int32.
  int32_t* table(int64_t B, int* width) {
    const at::Tensor& t = packed("block_table", at::kInt);
    if (t.dim() != 2 || t.size(0) != B) refuse("block_table must be [%lld, max_pages]", (long long)B);
    *width = small(t.size(1), "max_pages");
    return static_cast<int32_t*>(t.data_ptr());
  }
  // [rows][heads][d] bf16 whose rows may be strided.
  void* rows(PyObject* o, const char* name, int64_t rows, int64_t heads, int64_t d, long long* stride) {
    const at::Tensor& t = tensor(o, name, at::kBFloat16);
    if (t.dim() != 3 || t.size(0) != rows || t.size(1) != heads || t.size(2) != d)
      refuse("%s must be [%lld, %lld, %lld]", name, (long long)rows, (long long)heads, (long long)d);
    if ((t.stride(2) != 1 && d > 1) || (t.stride(1) != d && heads > 1)) refuse("%s must be contiguous within each row", name);
    *stride = rows > 1 ? t.stride(0) : heads * d;
    return t.data_ptr();
  }
  static int small(int64_t v, const char* name) {
    if (v < INT_MIN || v > INT_MAX) refuse("%s is out of range", name);
    return static_cast<int>(v);
  }
  int integer(const char* name) { return integer(take(), name); }
  int integer(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return small(v, name);
  }
  int truth() {
    const int v = PyObject_IsTrue(take());
    if (v < 0) throw Refused{};
    return v;
  }
  // None: the current stream; otherwise a torch stream's handle.
  void* stream() {
    PyObject* o = take();
    if (none(o)) return c10::cuda::getCurrentCUDAStream(device).stream();
    void* s = PyLong_AsVoidPtr(o);
    if (s == nullptr && PyErr_Occurred()) throw Refused{};
    return s;
  }
};

// The C call without Python's lock: a launch may wait for room in the queue.
template <typename F, typename... Args>
int unlocked(F* f, Args... args) {
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = f(args...);
  Py_END_ALLOW_THREADS;
  return status;
}

struct Cache {
  void *k, *v;
  int pages, heads, page, d;
  Cache(Call& c) {
    const at::Tensor &kt = c.packed("k_cache", at::kBFloat16), &vt = c.packed("v_cache", at::kBFloat16);
    if (kt.dim() != 4 || kt.sizes() != vt.sizes())
      refuse("k_cache and v_cache must be [num_pages, Hkv, page_size, d] tensors of one shape");
    k = kt.data_ptr();
    v = vt.data_ptr();
    pages = Call::small(kt.size(0), "num_pages");
    heads = Call::small(kt.size(1), "Hkv");
    page = Call::small(kt.size(2), "page_size");
    d = Call::small(kt.size(3), "d");
  }
};

int64_t rows_of(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.dim() < 1) refuse("%s must have rows", name);
  return t.size(0);
}
int64_t numel_of(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
  return THPVariable_Unpack(o).numel();
}

int reserve(Call& c) {
  const int64_t B = numel_of(c.arg[0], "cached_lens");
  int32_t* cached = c.ints("cached_lens", B);
  int32_t* fresh = c.ints("new_lens", B);
  int width;
  int32_t* table = c.table(B, &width);
  const at::Tensor& pages = c.packed("free_pages", at::kInt);
  int32_t* count = c.ints("free_count", 1);
  int32_t* count_out = c.ints("free_count_out", 1);
  int32_t* cu = c.ints("cu_seqlens", B + 1);
  int32_t* kv = c.ints("kv_lens", B);
  const at::Tensor& slots = c.packed("slots", at::kInt);
  PyObject* at_ = c.take();
  int32_t* positions = Call::none(at_) ? nullptr : c.ints(at_, "positions", slots.numel());
  const int page = c.integer("page_size");
  const at::Tensor& ws = c.packed("workspace", at::kByte);
  PyObject* bound = c.take();
  const int max_new = Call::none(bound) ? INT_MAX : c.integer(bound, "max_new");
  return unlocked(sigattn_paged_reserve_bounded, cached, fresh, table, static_cast<int32_t*>(pages.data_ptr()), count, count_out, cu, kv,
                               static_cast<int32_t*>(slots.data_ptr()), positions, Call::small(B, "B"), width, page,
                               Call::small(pages.numel(), "num_pages"), Call::small(slots.numel(), "rows"),
                               max_new, ws.data_ptr(), ws.numel(), c.stream());
}

int release(Call& c) {
  const int64_t B = numel_of(c.arg[0], "kv_lens");
  int32_t* kv = c.ints("kv_lens", B);
  PyObject* keep = c.take();
  int32_t* keep_lens = Call::none(keep) ? nullptr : c.ints(keep, "keep_lens", B);
  int width;
  int32_t* table = c.table(B, &width);
  const at::Tensor& pages = c.packed("free_pages", at::kInt);
  int32_t* count = c.ints("free_count", 1);
  int32_t* count_out = c.ints("free_count_out", 1);
  const int page = c.integer("page_size");
  const at::Tensor& ws = c.packed("workspace", at::kByte);
  PyObject* after = c.take();
  int32_t* kv_out = Call::none(after) ? nullptr : c.ints(after, "kv_lens_out", B);
  return unlocked(sigattn_paged_release_lens, kv, keep_lens, table, static_cast<int32_t*>(pages.data_ptr()), count, count_out,
                               kv_out, Call::small(B, "B"), width, page, Call::small(pages.numel(), "num_pages"), ws.data_ptr(),
                               ws.numel(), c.stream());
}

int write(Call& c) {
  PyObject *k = c.take(), *v = c.take(), *slots = c.take();
  const Cache cache(c);
  const int64_t rows = rows_of(k, "k");
  long long ks, vs, qs = 0, qos = 0;
  void* kp = c.rows(k, "k", rows, cache.heads, cache.d, &ks);
  void* vp = c.rows(v, "v", rows, cache.heads, cache.d, &vs);
  int32_t* sp = c.ints(slots, "slots", rows);
  const at::Tensor& ws = c.packed("workspace", at::kByte);
  PyObject *q = c.take(), *q_out = c.take(), *positions = c.take(), *freq = c.take(), *axis = c.take();
  if (Call::none(q) != Call::none(q_out)) refuse("q and q_out go together");
  void *qp = nullptr, *qo = nullptr;
  int Hq = 0;
  if (!Call::none(q)) {
    const at::Tensor& qt = c.tensor(q, "q", at::kBFloat16);
    if (qt.dim() != 3) refuse("q must be [rows, Hq, d]");
    Hq = Call::small(qt.size(1), "Hq");
    qp = c.rows(q, "q", rows, Hq, cache.d, &qs);
    qo = c.rows(q_out, "q_out", rows, Hq, cache.d, &qos);
  }
  int pairs = 0, axes = 1;
  int32_t *pp = nullptr, *ap = nullptr;
  float* fp = nullptr;
  if (!Call::none(freq)) {
    if (Call::none(positions)) refuse("inv_freq needs positions");
    const at::Tensor &ft = c.packed(freq, "inv_freq", at::kFloat), &pt = c.packed(positions, "positions", at::kInt);
    pairs = Call::small(ft.numel(), "pairs");
    fp = static_cast<float*>(ft.data_ptr());
    if (pt.dim() > 1) axes = Call::small(pt.size(0), "axes");
    pp = c.ints(positions, "positions", axes * rows);
    if (!Call::none(axis)) ap = c.ints(axis, "pair_axis", pairs);
  }
  const int adjacent = c.truth();
  return unlocked(sigattn_paged_write, kp, ks, vp, vs, sp, cache.k, cache.v, qp, qs, qo, qos, pp, fp, ap, axes, pairs, adjacent,
                             Call::small(rows, "rows"), Hq, cache.heads, cache.d, cache.page, cache.pages, ws.data_ptr(),
                             ws.numel(), c.stream());
}

int attend(Call& c) {
  PyObject* q = c.take();
  const Cache cache(c);
  const at::Tensor& qt = c.tensor(q, "q", at::kBFloat16);
  if (qt.dim() != 3) refuse("q must be [total, Hq, d]");
  const int64_t total = qt.size(0), Hq = qt.size(1);
  long long qs;
  void* qp = c.rows(q, "q", total, Hq, cache.d, &qs);
  const at::Tensor& o = c.packed("o", at::kBFloat16);
  if (o.sizes() != qt.sizes()) refuse("o must have q's shape");
  PyObject* cu = c.take();
  PyObject* kv = c.take();
  const int64_t B = numel_of(kv, "kv_lens");
  int32_t *cup = c.ints(cu, "cu_seqlens", B + 1), *kvp = c.ints(kv, "kv_lens", B);
  int width;
  int32_t* table = c.table(B, &width);
  const int most = c.integer("max_seqlen_q"), causal = c.truth();
  const at::Tensor& ws = c.packed("workspace", at::kByte);
  return unlocked(sigattn_fwd_paged, qp, qs, cache.k, cache.v, o.data_ptr(), cup, kvp, table, Call::small(B, "B"),
                           Call::small(Hq, "Hq"), cache.heads, most, Call::small(total, "total"), width, cache.page,
                           cache.pages, cache.d, causal, ws.data_ptr(), ws.numel(), c.stream());
}

// The status of a call as a Python int; no C++ exception leaves.
template <int (*F)(Call&), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
  try {
    Call c{args, n};
    return PyLong_FromLong(F(c));
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <int (*F)(Call&), Py_ssize_t N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<reserve, 14>("paged_reserve"), method<release, 10>("paged_release"), method<write, 13>("paged_write"),
    method<attend, 11>("fwd_paged"),      {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
