// Tensor arguments of the Python binding, checked without the interpreter: a
// call on six tensors spends 3.4 us on the checks in Python, as much as a short
// kernel takes, and 0.6 us on these.  sized() and rows() return what the
// functions of the same names in _lib.py return where every check passes, and
// call those for all else (other kinds of arguments, and the errors).
//
// gemv_i4group() and its like make a whole call of a decode step on the current
// stream: every argument checked as in _lib.py, the library's function called, its
// status returned.  None, and nothing done, where a check does not pass or an
// argument is of another kind: the function in _lib.py then looks at it (a 4-bit
// mat-vec 4.2 -> 3.3 us of the host, 3.1 of them the launch, attention 5.0 -> 3.4).
#include <Python.h>
#include <pthread.h>

#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pesti.h"

namespace {

PyObject* slow_sized = nullptr;
PyObject* slow_rows = nullptr;

// The tensor, if it is one on device dev with elements of `dtype` (None: any).
const at::Tensor* tensor_on(PyObject* dev, PyObject* obj, PyObject* dtype) {
  if (!THPVariable_CheckExact(obj)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(obj);
  if (!t.is_cuda() || t.get_device() != PyLong_AsLong(dev)) return nullptr;
  if (dtype != Py_None && (!THPDtype_Check(dtype) || t.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type))
    return nullptr;
  return &t;
}

// sized(dev, obj, nbytes, what, dtype=None) -> pointer, int or None
PyObject* sized(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n >= 4 && PyLong_CheckExact(a[0]) && PyLong_CheckExact(a[2])) {
    if (a[1] == Py_None || PyLong_CheckExact(a[1])) {
      Py_INCREF(a[1]);
      return a[1];
    }
    const at::Tensor* t = tensor_on(a[0], a[1], n > 4 ? a[4] : Py_None);
    if (t && static_cast<long long>(t->nbytes()) >= PyLong_AsLongLong(a[2]) && t->is_contiguous() && !PyErr_Occurred())
      return PyLong_FromVoidPtr(t->data_ptr());
    PyErr_Clear();
  }
  return PyObject_Vectorcall(slow_sized, a, n, nullptr);
}

// Values of a two-dimensional tensor from its first to its last, within its memory.
int64_t values_held(const at::Tensor& t, int64_t size) {
  if (t.size(0) == 0 || t.size(1) == 0) return 0;
  const int64_t own = (t.size(0) - 1) * t.stride(0) + (t.size(1) - 1) * t.stride(1) + 1;
  const int64_t memory = static_cast<int64_t>(t.storage().nbytes()) / size - t.storage_offset();
  return own < memory ? own : memory;
}

// rows(dev, obj, rows, width, stride, size, what, dtype) -> (pointer, stride)
PyObject* rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n == 8 && PyLong_CheckExact(a[0]) && PyLong_CheckExact(a[2]) && PyLong_CheckExact(a[3]) &&
      (a[4] == Py_None || PyLong_CheckExact(a[4])) && PyLong_CheckExact(a[5]) && a[7] != Py_None) {
    const at::Tensor* t = tensor_on(a[0], a[1], a[7]);
    if (t && t->dim() == 2 && (t->size(1) == 1 || t->stride(1) == 1)) {
      const long long count = PyLong_AsLongLong(a[2]), width = PyLong_AsLongLong(a[3]), size = PyLong_AsLongLong(a[5]);
      const long long stride = a[4] != Py_None ? PyLong_AsLongLong(a[4]) : (t->size(0) > 1 ? t->stride(0) : width);
      const long long most = 1LL << 40;
      if (!PyErr_Occurred() && size > 0 && count >= 0 && count < most && stride >= 0 && stride < most && width >= 0 &&
          width < most && count * (stride / 1024 + 1) < most) {
        if (count == 0 || (count - 1) * stride + width <= values_held(*t, size))
          return Py_BuildValue("(NL)", PyLong_FromVoidPtr(t->data_ptr()), stride);
      }
      PyErr_Clear();
    }
  }
  return PyObject_Vectorcall(slow_rows, a, n, nullptr);
}

// Has torch been asked for the device in this process?  It sets itself up then, or refuses a child
// forked behind its back; the device is not asked for here before that.
bool permitted = false;

// permit(): torch has named the device
PyObject* permit(PyObject*, PyObject* const*, Py_ssize_t) {
  permitted = true;
  Py_RETURN_NONE;
}

// place() -> (current device, its current stream's handle), None where torch is to be asked
PyObject* place(PyObject*, PyObject* const*, Py_ssize_t) {
  if (!permitted) Py_RETURN_NONE;
  const auto dev = c10::hip::current_device();   // (throws)
  return Py_BuildValue("(iN)", static_cast<int>(dev), PyLong_FromVoidPtr(c10::hip::getCurrentHIPStream(dev).stream()));
}

struct Library {
  decltype(&pesti_gemv_i4group) gemv_i4group;
  decltype(&pesti_gemv_i4group_swiglu) gemv_i4group_swiglu;
  decltype(&pesti_cache_append) cache_append;
  decltype(&pesti_attn_paged) attn_paged;
  decltype(&pesti_cache_extend) cache_extend;
  decltype(&pesti_cache_free) cache_free;
  decltype(&pesti_cache_fork) cache_fork;
  decltype(&pesti_cache_compact) cache_compact;
} library{};
constexpr int kCalls = 8;

// The arguments of a call, read in turn; `ok` falls where one is of another kind or
// does not pass.
struct Reader {
  PyObject* const* a;
  bool ok;
  int dev = -1;
  void* stream = nullptr;

  explicit Reader(PyObject* const* args) : a(args), ok(permitted) {
    if (!ok) return;
    dev = c10::hip::current_device();
    stream = c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(dev)).stream();
  }
  bool none(int i) const { return a[i] == Py_None; }
  // An integer of 0 .. most.
  int64_t integer(int i, int64_t most = int64_t{1} << 31) {
    if (!PyLong_CheckExact(a[i])) return fail();
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(a[i], &overflow);
    return overflow || v < 0 || v > most ? fail() : v;
  }
  float number(int i) {
    if (PyFloat_CheckExact(a[i])) return static_cast<float>(PyFloat_AS_DOUBLE(a[i]));
    return static_cast<float>(fail());
  }
  void* address(int i) {
    void* p = PyLong_CheckExact(a[i]) ? PyLong_AsVoidPtr(a[i]) : nullptr;
    if (!p) {
      PyErr_Clear();
      fail();
    }
    return p;
  }
  const at::Tensor* tensor(int i) {
    if (ok && THPVariable_CheckExact(a[i])) {
      const at::Tensor& t = THPVariable_Unpack(a[i]);
      if (t.is_cuda() && t.get_device() == dev) return &t;
    }
    fail();
    return nullptr;
  }
  // A contiguous tensor of at least `bytes` bytes; type: any where not given.  None is NULL.
  template <typename T>
  T* array(int i, int64_t bytes, c10::optional<at::ScalarType> type) {
    if (!ok || none(i)) return nullptr;
    const at::Tensor* t = tensor(i);
    if (!t || (type && t->scalar_type() != *type) || static_cast<int64_t>(t->nbytes()) < bytes || !t->is_contiguous()) {
      fail();
      return nullptr;
    }
    return static_cast<T*>(t->data_ptr());
  }
  // [count][width] values whose rows may lie apart, of a value format; *stride: given, or to be read off the tensor (-1).
  void* values(int i, int64_t count, int64_t width, int64_t* stride, int32_t* format) {
    const at::Tensor* t = tensor(i);
    if (!t || t->dim() != 2 || (t->size(1) != 1 && t->stride(1) != 1)) {
      fail();
      return nullptr;
    }
    const bool f32 = t->scalar_type() == at::kFloat;
    if (!f32 && t->scalar_type() != at::kHalf) fail();
    *format = f32 ? PESTI_FMT_F32 : PESTI_FMT_F16;
    if (*stride < 0) *stride = t->size(0) > 1 ? t->stride(0) : width;
    if (*stride < 0 || *stride > int64_t{1} << 31 || (count > 0 && (count - 1) * *stride + width > values_held(*t, f32 ? 4 : 2))) fail();
    return t->data_ptr();
  }
  // A workspace and its size (None: the tensor's).
  void* workspace(int i, int64_t* bytes) {
    if (none(i)) {
      *bytes = none(i + 1) ? 0 : integer(i + 1, INT64_MAX);
      return nullptr;
    }
    const at::Tensor* t = tensor(i);
    *bytes = t && none(i + 1) ? static_cast<int64_t>(t->nbytes()) : integer(i + 1, INT64_MAX);
    return array<void>(i, *bytes, c10::nullopt);
  }
  int64_t fail() {
    ok = false;
    return 0;
  }
};

template <typename F>
PyObject* make(Reader& r, F call) {
  if (!r.ok) Py_RETURN_NONE;
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = call();
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(status);
}

// gemv_i4group(out, in, group, packed, scales, zeros, x, y, bias, batch)
PyObject* gemv_i4group(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 10 || !library.gemv_i4group) Py_RETURN_NONE;
  Reader r(a);
  const int64_t out = r.integer(0), in = r.integer(1), group = r.integer(2), batch = r.integer(9, 1 << 20);
  if (!r.ok || group == 0) Py_RETURN_NONE;
  const int64_t groups = out * ((in + group - 1) / group);
  const void* packed = r.array<void>(3, out * (in / 2), at::kByte);
  const uint16_t* scales = r.array<uint16_t>(4, 2 * groups, at::kHalf);
  const uint8_t* zeros = r.array<uint8_t>(5, groups, at::kByte);
  const float* x = r.array<float>(6, 4 * batch * in, at::kFloat);
  float* y = r.array<float>(7, 4 * batch * out, at::kFloat);
  const float* bias = r.array<float>(8, 4 * out, at::kFloat);
  return make(r, [&] {
    return library.gemv_i4group(out, in, group, packed, scales, zeros, x, y, bias, static_cast<int32_t>(batch), r.stream);
  });
}

// gemv_i4group_swiglu(out, in, group, gate and up: packed, scales, zeros, x, h, batch)
PyObject* gemv_i4group_swiglu(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 12 || !library.gemv_i4group_swiglu) Py_RETURN_NONE;
  Reader r(a);
  const int64_t out = r.integer(0), in = r.integer(1), group = r.integer(2), batch = r.integer(11, 1 << 20);
  if (!r.ok || group == 0) Py_RETURN_NONE;
  const int64_t groups = out * ((in + group - 1) / group);
  const void* packed[2];
  const uint16_t* scales[2];
  const uint8_t* zeros[2];
  for (int m = 0; m < 2; ++m) {
    packed[m] = r.array<void>(3 + 3 * m, out * (in / 2), at::kByte);
    scales[m] = r.array<uint16_t>(4 + 3 * m, 2 * groups, at::kHalf);
    zeros[m] = r.array<uint8_t>(5 + 3 * m, groups, at::kByte);
  }
  const float* x = r.array<float>(9, 4 * batch * in, at::kFloat);
  float* h = r.array<float>(10, 4 * batch * out, at::kFloat);
  return make(r, [&] {
    return library.gemv_i4group_swiglu(out, in, group, packed[0], scales[0], zeros[0], packed[1], scales[1], zeros[1], x, h,
                                       static_cast<int32_t>(batch), r.stream);
  });
}

// The structs of a cache call, built for the current device and each other: their
// addresses, the devices that they were built on, the pages that refs holds (or None).
bool structs(Reader& r, const pesti_kv_cache** cache, const pesti_kv_table** table) {
  *cache = static_cast<const pesti_kv_cache*>(r.address(0));
  *table = static_cast<const pesti_kv_table*>(r.address(1));
  if (r.integer(2) != r.dev || r.integer(3) != r.dev) r.fail();
  if (r.ok && !r.none(4) && r.integer(4, INT64_MAX) < (*cache)->pages) r.fail();
  const int64_t most = int64_t{1} << 20;   // (the library looks at the sizes themselves)
  return r.ok && (*cache)->kv_heads >= 0 && (*cache)->kv_heads < most && (*cache)->head_dim >= 0 && (*cache)->head_dim < most;
}

// cache_append(cache, table, their devices, refs held, layer, rows, k, v, stride, seq_ids, positions)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 12 || !library.cache_append) Py_RETURN_NONE;
  Reader r(a);
  const pesti_kv_cache* cache;
  const pesti_kv_table* table;
  if (!structs(r, &cache, &table)) Py_RETURN_NONE;
  const int64_t layer = r.integer(5), rows = r.integer(6), width = cache->kv_heads * cache->head_dim;
  int64_t k_stride = r.none(9) ? -1 : r.integer(9), v_stride = k_stride;
  int32_t format = 0, v_format = 0;
  const void* k = r.values(7, rows, width, &k_stride, &format);
  const void* v = r.values(8, rows, width, &v_stride, &v_format);
  if (format != v_format || k_stride != v_stride) r.fail();
  const int32_t* seq_ids = r.array<int32_t>(10, 4 * rows, at::kInt);
  const int32_t* positions = r.array<int32_t>(11, 4 * rows, at::kInt);
  return make(r, [&] { return library.cache_append(cache, table, layer, rows, format, k, v, k_stride, seq_ids, positions, r.stream); });
}

// attn_paged(cache, table, their devices, refs held, layer, rows, heads, q, y, scale, q_stride, max_length, seq_ids,
//            workspace, workspace_bytes)
PyObject* attn_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 16 || !library.attn_paged) Py_RETURN_NONE;
  Reader r(a);
  const pesti_kv_cache* cache;
  const pesti_kv_table* table;
  if (!structs(r, &cache, &table)) Py_RETURN_NONE;
  const int64_t layer = r.integer(5), rows = r.integer(6), heads = r.integer(7, 1 << 20), width = heads * cache->head_dim;
  int64_t stride = r.none(11) ? -1 : r.integer(11);
  int32_t q_format = 0;
  const void* q = r.values(8, rows, width, &stride, &q_format);
  const at::Tensor* y = r.tensor(9);
  const bool f32 = y && y->scalar_type() == at::kFloat;
  if (y && !f32 && y->scalar_type() != at::kHalf) r.fail();
  void* out = r.array<void>(9, rows * width * (f32 ? 4 : 2), c10::nullopt);
  const float scale = r.number(10);
  const int64_t longest = r.integer(12);
  const int32_t* seq_ids = r.array<int32_t>(13, 4 * rows, at::kInt);
  int64_t bytes = 0;
  void* workspace = r.workspace(14, &bytes);
  return make(r, [&] {
    return library.attn_paged(cache, table, layer, rows, heads, seq_ids, q_format, q, stride, f32 ? PESTI_FMT_F32 : PESTI_FMT_F16, out,
                              scale, longest, workspace, bytes, r.stream);
  });
}

// cache_extend(cache, table, their devices, refs held, n, seq_ids, counts, status)
PyObject* cache_extend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 9 || !library.cache_extend) Py_RETURN_NONE;
  Reader r(a);
  const pesti_kv_cache* cache;
  const pesti_kv_table* table;
  if (!structs(r, &cache, &table)) Py_RETURN_NONE;
  const int64_t count = r.integer(5);
  const int32_t* seq_ids = r.array<int32_t>(6, 4 * count, at::kInt);
  const int32_t* counts = r.array<int32_t>(7, 4 * count, at::kInt);
  int32_t* status = r.array<int32_t>(8, 4, at::kInt);
  return make(r, [&] { return library.cache_extend(cache, table, count, seq_ids, counts, status, r.stream); });
}

// cache_free(cache, table, their devices, refs held, n, seq_ids)
PyObject* cache_free(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7 || !library.cache_free) Py_RETURN_NONE;
  Reader r(a);
  const pesti_kv_cache* cache;
  const pesti_kv_table* table;
  if (!structs(r, &cache, &table)) Py_RETURN_NONE;
  const int64_t count = r.integer(5);
  const int32_t* seq_ids = r.array<int32_t>(6, 4 * count, at::kInt);
  return make(r, [&] { return library.cache_free(cache, table, count, seq_ids, r.stream); });
}

// cache_fork(cache, table, their devices, refs held, n, parents, children, status, workspace, workspace_bytes)
PyObject* cache_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 11 || !library.cache_fork) Py_RETURN_NONE;
  Reader r(a);
  const pesti_kv_cache* cache;
  const pesti_kv_table* table;
  if (!structs(r, &cache, &table)) Py_RETURN_NONE;
  const int64_t count = r.integer(5);
  const int32_t* parents = r.array<int32_t>(6, 4 * count, at::kInt);
  const int32_t* children = r.array<int32_t>(7, 4 * count, at::kInt);
  int32_t* status = r.array<int32_t>(8, 4, at::kInt);
  int64_t bytes = 0;
  void* workspace = r.workspace(9, &bytes);
  return make(r, [&] { return library.cache_fork(cache, table, count, parents, children, status, workspace, bytes, r.stream); });
}

// cache_compact(cache, table, their devices, refs held, live, workspace, workspace_bytes)
PyObject* cache_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8 || !library.cache_compact) Py_RETURN_NONE;
  Reader r(a);
  const pesti_kv_cache* cache;
  const pesti_kv_table* table;
  if (!structs(r, &cache, &table)) Py_RETURN_NONE;
  int32_t* live = r.array<int32_t>(5, 4, at::kInt);
  int64_t bytes = 0;
  void* workspace = r.workspace(6, &bytes);
  return make(r, [&] { return library.cache_compact(cache, table, live, workspace, bytes, r.stream); });
}

// link(addresses of the library's functions, in Library's order)
PyObject* link(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* f[kCalls];
  if (n != kCalls) {
    PyErr_SetString(PyExc_TypeError, "link takes eight addresses");
    return nullptr;
  }
  for (int i = 0; i < kCalls; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  library.gemv_i4group = reinterpret_cast<decltype(library.gemv_i4group)>(f[0]);
  library.gemv_i4group_swiglu = reinterpret_cast<decltype(library.gemv_i4group_swiglu)>(f[1]);
  library.cache_append = reinterpret_cast<decltype(library.cache_append)>(f[2]);
  library.attn_paged = reinterpret_cast<decltype(library.attn_paged)>(f[3]);
  library.cache_extend = reinterpret_cast<decltype(library.cache_extend)>(f[4]);
  library.cache_free = reinterpret_cast<decltype(library.cache_free)>(f[5]);
  library.cache_fork = reinterpret_cast<decltype(library.cache_fork)>(f[6]);
  library.cache_compact = reinterpret_cast<decltype(library.cache_compact)>(f[7]);
  Py_RETURN_NONE;
}

// bind(sized, rows): the Python functions behind the fast ones
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "bind takes two functions");
    return nullptr;
  }
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  Py_XSETREF(slow_sized, a[0]);
  Py_XSETREF(slow_rows, a[1]);
  Py_RETURN_NONE;
}

// A tensor's methods throw where it has no strides or no memory of its own (sparse ones, those of a
// torch.vmap), and an exception that left these functions would end the process: such a call is
// left to the function in _lib.py, which raises the error.
typedef PyObject* Method(PyObject*, PyObject* const*, Py_ssize_t);
template <Method* CALL>
PyObject* or_none(PyObject* self, PyObject* const* a, Py_ssize_t n) noexcept {
  try {
    return CALL(self, a, n);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}
template <Method* CALL, PyObject** SLOW>
PyObject* or_slow(PyObject* self, PyObject* const* a, Py_ssize_t n) noexcept {
  try {
    return CALL(self, a, n);
  } catch (...) {
    PyErr_Clear();
    return PyObject_Vectorcall(*SLOW, a, n, nullptr);
  }
}

// A method of the module.
PyMethodDef entry(const char* name, Method* call) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    entry("sized", or_slow<sized, &slow_sized>),
    entry("rows", or_slow<rows, &slow_rows>),
    entry("permit", permit),
    entry("place", or_none<place>),
    entry("gemv_i4group", or_none<gemv_i4group>),
    entry("gemv_i4group_swiglu", or_none<gemv_i4group_swiglu>),
    entry("cache_append", or_none<cache_append>),
    entry("attn_paged", or_none<attn_paged>),
    entry("cache_extend", or_none<cache_extend>),
    entry("cache_free", or_none<cache_free>),
    entry("cache_fork", or_none<cache_fork>),
    entry("cache_compact", or_none<cache_compact>),
    entry("link", link),
    entry("bind", bind),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__tensor_args() {
  if (pthread_atfork(nullptr, nullptr, [] { permitted = false; }) != 0) return PyErr_NoMemory();
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch", PESTI_TORCH) != 0) {   // the one whose tensors these functions know
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
