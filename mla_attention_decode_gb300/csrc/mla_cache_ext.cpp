// mla_cache_ext.cpp -- the Python side of mla_cache.h: checks of tensors and
// packing of arguments, compiled.
//
// A decode step makes several of these calls, and each launch takes the host
// about 1.5 us; checking and packing the arguments of one in Python took 6 to
// 10 us on the Grace cores, several times the kernel's own time at small
// batches.  Here it takes a few tenths.  The module knows nothing of CUDA
// kernels: it calls the entry points of libmla_decode.so by the addresses that
// `bind` gives it, and returns their status.
//
// Every function takes a pool's core first (a capsule made by `core`) and the
// stream last: None (torch's current stream of the pool's device), a handle, or
// an object with a cuda_stream.  What a tensor must be and is not is a
// ValueError; C++ exceptions become Python ones before they leave.
#include <Python.h>

#include <cstdarg>
#include <cstdio>
#include <exception>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mla_cache.h"

namespace {

struct Entry {
  decltype(&mla_cache_append) append;
  decltype(&mla_cache_gather) gather;
  decltype(&mla_cache_slots) slots;
  decltype(&mla_cache_copy_pages) copy_pages;
  decltype(&mla_cache_fork) fork;
  decltype(&mla_cache_resize) resize;
  decltype(&mla_cache_free) free_;
  decltype(&mla_cache_compact) compact;
} g_lib;

struct Core {
  mla_cache cache;
  int32_t* workspace;  // its first word is the error word
  size_t workspace_bytes;
  int device;
};

PyObject* s_address;
PyObject* s_num_axes;
PyObject* s_device_index;
PyObject* s_cuda_stream;

// Thrown after a Python exception has been set.
struct PyError {};

[[noreturn]] void refuse(const char* format, ...) {
  char text[256];
  va_list args;
  va_start(args, format);
  std::vsnprintf(text, sizeof text, format, args);
  va_end(args);
  PyErr_SetString(PyExc_ValueError, text);
  throw PyError{};
}

Core* core_of(PyObject* o) {
  auto* c = static_cast<Core*>(PyCapsule_GetPointer(o, "mla_cache_core"));
  if (!c) throw PyError{};
  return c;
}

long long whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError{};
  return v;
}

long long attr(PyObject* o, PyObject* name) {
  PyObject* a = PyObject_GetAttr(o, name);
  if (!a) throw PyError{};
  const long long v = PyLong_AsLongLong(a);
  Py_DECREF(a);
  if (v == -1 && PyErr_Occurred()) throw PyError{};
  return v;
}

// A CUDA tensor of the pool's device and the type.
const at::Tensor& tensor(const Core* c, PyObject* o, const char* what, at::ScalarType type, const char* type_name) {
  if (!THPVariable_Check(o)) refuse("%s is a tensor", what);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != c->device) refuse("%s is on cuda:%d, the cache's device", what, c->device);
  if (t.scalar_type() != type) refuse("%s is %s", what, type_name);
  return t;
}

// A vector of consecutive int32; size < 0: of any length.
int32_t* vec(const Core* c, PyObject* o, const char* what, int64_t size, int64_t* numel = nullptr) {
  const at::Tensor& t = tensor(c, o, what, at::kInt, "int32");
  if (t.dim() != 1 || (t.size(0) > 1 && t.stride(0) != 1)) refuse("%s is a contiguous vector", what);
  if (size >= 0 && t.size(0) != size)
    refuse("%s has %lld entries, not %lld", what, (long long)size, (long long)t.size(0));
  if (numel) *numel = t.size(0);
  return static_cast<int32_t*>(t.data_ptr());
}

// bf16 [tokens, (16,) columns], the last dimension consecutive.
const at::Tensor& part(const Core* c, PyObject* o, const char* what, int64_t tokens, bool heads, int64_t columns) {
  const at::Tensor& t = tensor(c, o, what, at::kBFloat16, "bf16");
  const int d = heads ? 3 : 2;
  if (t.dim() != d || t.size(0) != tokens || (heads && t.size(1) != MLA_NUM_HEADS) || t.size(d - 1) != columns ||
      t.stride(d - 1) != 1)
    refuse("%s is [%lld, %s%lld], its last dimension consecutive", what, (long long)tokens, heads ? "16, " : "",
           (long long)columns);
  return t;
}

int32_t count32(int64_t n, const char* what) {
  if (n > INT32_MAX) refuse("%s is too long", what);
  return static_cast<int32_t>(n);
}

// A layer's number; one that has no 32 bits is no layer of any cache.
int32_t layer_of(PyObject* o) {
  const long long v = whole(o);
  return v < 0 || v > INT32_MAX ? -1 : static_cast<int32_t>(v);
}

// (page_indptr, kv_indices, last_page_len), a tuple or a list.
mla_page_table table(const Core* c, PyObject* o, const char* what) {
  PyObject* seq = PySequence_Fast(o, "a page table is (page_indptr, kv_indices, last_page_len)");
  if (!seq) throw PyError{};
  struct Hold {
    PyObject* o;
    ~Hold() { Py_DECREF(o); }
  } hold{seq};
  if (PySequence_Fast_GET_SIZE(seq) != 3) refuse("%s is (page_indptr, kv_indices, last_page_len)", what);
  PyObject** item = PySequence_Fast_ITEMS(seq);
  mla_page_table t;
  int64_t n = 0, room = 0;
  t.page_indptr = vec(c, item[0], "page_indptr", -1, &n);
  if (n < 1) refuse("page_indptr has at least one entry");
  t.kv_indices = vec(c, item[1], "kv_indices", -1, &room);
  t.last_page_len = vec(c, item[2], "last_page_len", n - 1);
  t.batch = count32(n - 1, "page_indptr");
  t.num_indices = count32(room, "kv_indices");
  return t;
}

// The stream a call runs on, and the pool's device made current for as long.
struct Where {
  c10::cuda::OptionalCUDAGuard guard;
  c10::cuda::CUDAStream current;
  void* handle;
  bool given;
  Where(const Core* c, PyObject* stream)
      : current(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c->device))),
        given(stream != Py_None) {
    if (c10::cuda::current_device() != c->device) guard.set_index(static_cast<c10::DeviceIndex>(c->device));
    if (!given)
      handle = current.stream();
    else if (PyLong_Check(stream))
      handle = PyLong_AsVoidPtr(stream);
    else
      handle = reinterpret_cast<void*>(static_cast<intptr_t>(attr(stream, s_cuda_stream)));
    if (PyErr_Occurred()) throw PyError{};
  }
};

// New memory that belongs to the stream of the call.
at::Tensor fresh(const Core* c, const Where& w, at::IntArrayRef shape, at::ScalarType type) {
  const auto options = at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(c->device));
  if (!w.given) return at::empty(shape, options);
  const c10::cuda::CUDAStreamGuard on(c10::cuda::getStreamFromExternal(
      static_cast<cudaStream_t>(w.handle), static_cast<c10::DeviceIndex>(c->device)));
  return at::empty(shape, options);
}

#define ARGS(n)                                                                        \
  if (nargs != (n)) {                                                                  \
    PyErr_Format(PyExc_TypeError, "%d arguments, not %zd", (n), (Py_ssize_t)nargs);    \
    return nullptr;                                                                    \
  }
#define BEGIN try {
#define END                                                \
  }                                                        \
  catch (const PyError&) { return nullptr; }               \
  catch (const std::exception& e) {                        \
    PyErr_SetString(PyExc_RuntimeError, e.what());         \
    return nullptr;                                        \
  }

template <class F>
int without_gil(F f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return rc;
}

// append(core, kv_lat, kv_pe, slots, rope, positions, norm, q_pe, q_lat, q_out, layer, stream) -> status
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(12)
  BEGIN
  const Core* c = core_of(a[0]);
  PyObject *kv_lat = a[1], *kv_pe = a[2], *slots = a[3], *rope = a[4], *positions = a[5], *norm = a[6], *q_pe = a[7],
           *q_lat = a[8], *q_out = a[9];
  PyObject* first = kv_lat != Py_None ? kv_lat : q_pe;
  if (first == Py_None) refuse("append needs keys (kv_lat, kv_pe, slots) or queries (q_pe, q_out)");
  if (!THPVariable_Check(first) || THPVariable_Unpack(first).dim() < 1) refuse("keys and queries are tensors");
  const int64_t t = THPVariable_Unpack(first).size(0);
  mla_append_args args = {};
  args.num_tokens = count32(t, "the batch");
  args.layer = layer_of(a[10]);
  if (kv_lat != Py_None) {
    if (kv_pe == Py_None || slots == Py_None) refuse("keys come as kv_lat, kv_pe and slots");
    const at::Tensor& x = part(c, kv_lat, "kv_lat", t, false, MLA_V_DIM);
    const at::Tensor& y = part(c, kv_pe, "kv_pe", t, false, MLA_PE_DIM);
    args.kv_lat = x.data_ptr();
    args.kv_lat_stride = t > 1 ? x.stride(0) : 0;
    args.kv_pe = y.data_ptr();
    args.kv_pe_stride = t > 1 ? y.stride(0) : 0;
    args.slots = vec(c, slots, "slots", t);
  } else if (kv_pe != Py_None || slots != Py_None) {
    refuse("keys come as kv_lat, kv_pe and slots");
  }
  const mla_rope* r = nullptr;
  if (rope != Py_None) {
    r = reinterpret_cast<const mla_rope*>(static_cast<intptr_t>(attr(rope, s_address)));
    const long long axes = attr(rope, s_num_axes);
    if (positions == Py_None) refuse("a rotation needs positions");
    const at::Tensor& x = tensor(c, positions, "positions", at::kInt, "int32");
    if ((x.dim() != 1 && x.dim() != 2) || x.size(0) != t || (x.dim() == 2 ? x.size(1) : 1) < axes)
      refuse("positions is [%lld, %lld]", (long long)t, axes);
    if (x.dim() == 2 && x.size(1) > 1 && x.stride(1) != 1) refuse("a token's positions are consecutive");
    args.positions = static_cast<const int32_t*>(x.data_ptr());
    args.position_stride = x.stride(0);
  }
  const mla_norm* n = nullptr;
  if (norm != Py_None) {
    n = reinterpret_cast<const mla_norm*>(static_cast<intptr_t>(attr(norm, s_address)));
    const long long at = attr(norm, s_device_index);
    if (at >= 0 && at != c->device) refuse("the norm's weights are on cuda:%lld, not cuda:%d", at, c->device);
  }
  if (q_pe != Py_None) {
    if (q_out == Py_None) refuse("queries come as q_pe and q_out");
    const at::Tensor& x = part(c, q_pe, "q_pe", t, true, MLA_PE_DIM);
    const at::Tensor& o = part(c, q_out, "q_out", t, true, MLA_QK_DIM);
    if (!o.is_contiguous()) refuse("q_out is contiguous");
    args.q_pe = x.data_ptr();
    args.q_pe_token_stride = t > 1 ? x.stride(0) : 0;
    args.q_pe_head_stride = x.stride(1);
    args.q_out = o.data_ptr();
    if (q_lat != Py_None) {
      const at::Tensor& y = part(c, q_lat, "q_lat", t, true, MLA_V_DIM);
      args.q_lat = y.data_ptr();
      args.q_lat_token_stride = t > 1 ? y.stride(0) : 0;
      args.q_lat_head_stride = y.stride(1);
    }
  } else if (q_lat != Py_None || q_out != Py_None) {
    refuse("queries come as q_pe and q_out");
  }
  const Where w(c, a[11]);
  return PyLong_FromLong(
      without_gil([&] { return g_lib.append(&c->cache, r, n, &args, c->workspace, w.handle); }));
  END
}

// gather(core, slots, out, layer, stream) -> (status, out)
PyObject* py_gather(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(5)
  BEGIN
  const Core* c = core_of(a[0]);
  int64_t n = 0;
  const int32_t* slots = vec(c, a[1], "slots", -1, &n);
  const int32_t rows = count32(n, "slots"), layer = layer_of(a[3]);
  const Where w(c, a[4]);
  at::Tensor out = a[2] == Py_None ? fresh(c, w, {n, MLA_QK_DIM}, at::kBFloat16)
                                   : part(c, a[2], "out", n, false, MLA_QK_DIM);
  void* at = out.data_ptr();
  const int64_t stride = n > 1 ? out.stride(0) : MLA_QK_DIM;
  const int rc = without_gil(
      [&] { return g_lib.gather(&c->cache, layer, slots, rows, at, stride, c->workspace, w.handle); });
  PyObject* o = a[2] == Py_None ? THPVariable_Wrap(std::move(out)) : Py_NewRef(a[2]);
  return Py_BuildValue("(iN)", rc, o);
  END
}

// slots(core, table, qo_indptr, num_tokens, slots, rows, stream) -> (status, slots)
PyObject* py_slots(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(7)
  BEGIN
  const Core* c = core_of(a[0]);
  const mla_page_table t = table(c, a[1], "the table");
  const int32_t* qo = vec(c, a[2], "qo_indptr", (int64_t)t.batch + 1);
  const long long n = whole(a[3]);
  if (n < 0) refuse("num_tokens is at least 0");
  const int32_t tokens = count32(n, "num_tokens");
  int32_t* rows = nullptr;
  int64_t stride = 0;
  if (a[5] != Py_None) {
    const at::Tensor& x = tensor(c, a[5], "rows", at::kInt, "int32");
    if (x.dim() != 1 || x.size(0) != n) refuse("rows is [%lld]", n);
    rows = static_cast<int32_t*>(x.data_ptr());
    stride = x.stride(0);
  }
  const Where w(c, a[6]);
  at::Tensor made;
  int32_t* slots;
  if (a[4] == Py_None) {
    made = fresh(c, w, {n}, at::kInt);
    slots = static_cast<int32_t*>(made.data_ptr());
  } else {
    slots = vec(c, a[4], "slots", n);
  }
  const int rc = without_gil(
      [&] { return g_lib.slots(&c->cache, &t, qo, tokens, slots, rows, stride, c->workspace, w.handle); });
  PyObject* o = a[4] == Py_None ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[4]);
  return Py_BuildValue("(iN)", rc, o);
  END
}

// copy_pages(core, src, dst, stream) -> status
PyObject* py_copy_pages(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(4)
  BEGIN
  const Core* c = core_of(a[0]);
  int64_t n = 0;
  const int32_t* src = vec(c, a[1], "src", -1, &n);
  const int32_t* dst = vec(c, a[2], "dst", n);
  const int32_t count = count32(n, "src");
  const Where w(c, a[3]);
  return PyLong_FromLong(
      without_gil([&] { return g_lib.copy_pages(&c->cache, src, dst, count, c->workspace, w.handle); }));
  END
}

// fork / resize(core, refs, table, parents / lengths, out, stream) -> status
template <bool kForks>
PyObject* py_table(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(6)
  BEGIN
  const Core* c = core_of(a[0]);
  int32_t* refs = vec(c, a[1], "refs", c->cache.num_pages);
  const mla_page_table from = table(c, a[2], "the table"), to = table(c, a[4], "out");
  const int32_t* by = vec(c, a[3], kForks ? "parents" : "lengths", to.batch);
  const Where w(c, a[5]);
  return PyLong_FromLong(without_gil([&] {
    return (kForks ? g_lib.fork : g_lib.resize)(&c->cache, refs, &from, by, &to, c->workspace, c->workspace_bytes,
                                                w.handle);
  }));
  END
}

// free(core, refs, pages, stream) -> status
PyObject* py_free(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(4)
  BEGIN
  const Core* c = core_of(a[0]);
  int32_t* refs = vec(c, a[1], "refs", c->cache.num_pages);
  int64_t n = 0;
  const int32_t* pages = vec(c, a[2], "pages", -1, &n);
  const int32_t count = count32(n, "pages");
  const Where w(c, a[3]);
  return PyLong_FromLong(
      without_gil([&] { return g_lib.free_(&c->cache, refs, pages, count, c->workspace, w.handle); }));
  END
}

// compact(core, refs, kv_indices, out indices or None, out refs or None, live or None, stream)
//   -> (status, out indices, out refs, live)
PyObject* py_compact(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(7)
  BEGIN
  const Core* c = core_of(a[0]);
  const int32_t* refs = vec(c, a[1], "refs", c->cache.num_pages);
  int64_t n = 0;
  const int32_t* indices = vec(c, a[2], "kv_indices", -1, &n);
  const int32_t count = count32(n, "kv_indices");
  const Where w(c, a[6]);
  at::Tensor made_indices, made_live;
  int32_t *to, *live;
  int32_t* refs_out = a[4] == Py_None ? const_cast<int32_t*>(refs) : vec(c, a[4], "out refs", c->cache.num_pages);
  if (a[3] == Py_None) {
    made_indices = fresh(c, w, {n}, at::kInt);
    to = static_cast<int32_t*>(made_indices.data_ptr());
  } else {
    to = vec(c, a[3], "out kv_indices", n);
  }
  if (a[5] == Py_None) {
    made_live = fresh(c, w, {1}, at::kInt);
    live = static_cast<int32_t*>(made_live.data_ptr());
  } else {
    live = vec(c, a[5], "live", 1);
  }
  const int rc = without_gil([&] {
    return g_lib.compact(&c->cache, refs, refs_out, indices, to, count, live, c->workspace, c->workspace_bytes,
                         w.handle);
  });
  PyObject* i = a[3] == Py_None ? THPVariable_Wrap(std::move(made_indices)) : Py_NewRef(a[3]);
  PyObject* l = a[5] == Py_None ? THPVariable_Wrap(std::move(made_live)) : Py_NewRef(a[5]);
  return Py_BuildValue("(iNON)", rc, i, a[4] == Py_None ? a[1] : a[4], l);
  END
}

void drop_core(PyObject* o) { delete static_cast<Core*>(PyCapsule_GetPointer(o, "mla_cache_core")); }

// core(address of an mla_cache, workspace address, its bytes, device index) -> capsule
PyObject* py_core(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(4)
  BEGIN
  Core* c = new Core{*static_cast<const mla_cache*>(PyLong_AsVoidPtr(a[0])),
                     static_cast<int32_t*>(PyLong_AsVoidPtr(a[1])), static_cast<size_t>(whole(a[2])),
                     static_cast<int>(whole(a[3]))};
  PyObject* o = PyCapsule_New(c, "mla_cache_core", drop_core);
  if (!o) delete c;
  return o;
  END
}

// bind(addresses of append, gather, slots, copy_pages, fork, resize, free, compact)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(8)
  BEGIN
  void* at[8];
  for (int i = 0; i < 8; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (!at[i]) refuse("an entry point has no address");
  }
  g_lib = Entry{reinterpret_cast<decltype(g_lib.append)>(at[0]),     reinterpret_cast<decltype(g_lib.gather)>(at[1]),
                reinterpret_cast<decltype(g_lib.slots)>(at[2]),      reinterpret_cast<decltype(g_lib.copy_pages)>(at[3]),
                reinterpret_cast<decltype(g_lib.fork)>(at[4]),       reinterpret_cast<decltype(g_lib.resize)>(at[5]),
                reinterpret_cast<decltype(g_lib.free_)>(at[6]),      reinterpret_cast<decltype(g_lib.compact)>(at[7])};
  Py_RETURN_NONE;
  END
}

#define METHOD(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(fn)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD("append", py_append),
                         METHOD("gather", py_gather),
                         METHOD("slots", py_slots),
                         METHOD("copy_pages", py_copy_pages),
                         METHOD("fork", py_table<true>),
                         METHOD("resize", py_table<false>),
                         METHOD("free", py_free),
                         METHOD("compact", py_compact),
                         METHOD("core", py_core),
                         METHOD("bind", py_bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mla_cache", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// MLA_TORCH_VERSION (the build's): the full version of the torch it was compiled against.
PyMODINIT_FUNC PyInit__mla_cache(void) {
  s_address = PyUnicode_InternFromString("address");
  s_num_axes = PyUnicode_InternFromString("num_axes");
  s_device_index = PyUnicode_InternFromString("device_index");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  if (!s_address || !s_num_axes || !s_device_index || !s_cuda_stream) return nullptr;
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", MLA_TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
