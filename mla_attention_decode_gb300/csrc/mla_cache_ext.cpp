// mla_cache_ext.cpp -- the Python side of mla_cache.h, and of the calls of
// mla_decode.h and mla_prompt.h that a step makes: checks of tensors and packing
// of arguments, compiled.
//
// A decode step makes several of these calls, and each launch takes the host
// about 1.5 us; checking and packing the arguments of one in Python took 6 to
// 10 us on the Grace cores, several times the kernel's own time at small
// batches (a decode 15 to 20, a prompt call 40).  Here it takes a few tenths.  The module knows nothing of CUDA
// kernels: it calls the entry points of libmla_decode.so by the addresses that
// `bind` gives it, and returns their status.
//
// Every function takes a core first (a capsule: a pool's, made by `core`, a
// decoder's by `decode_core`, a prompt's by `prompt_core`) and the
// stream last: None (torch's current stream of the core's device), a handle, or
// an object with a cuda_stream.  What a tensor must be and is not is a
// ValueError; C++ exceptions become Python ones before they leave.
#include <Python.h>

#include <cstdarg>
#include <cstdio>
#include <exception>

#include <ATen/core/Tensor.h>
#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mla_cache.h"
#include "mla_prompt.h"

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

struct {
  decltype(&mla_decode_fwd) decode;
  decltype(&mla_decode_fwd_paged) decode_paged;
  decltype(&mla_prompt_fwd) prompt;
} g_attention;

struct Device {
  int device;
};
struct Core : Device {
  mla_cache cache;
  int32_t* workspace;  // its first word is the error word
  size_t workspace_bytes;
};
struct DecodeCore : Device {
  const mla_plan* plan;  // the decoder's own, which keeps it
  void* workspace;
  size_t workspace_bytes;
};
struct PromptCore : Device {
  void* workspace;
  size_t workspace_bytes;
  int64_t tokens, keys, batch;  // at most
  int32_t heads, causal;
  float sm_scale;
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

template <class C>
const char* name_of();
template <>
const char* name_of<Core>() { return "mla_cache_core"; }
template <>
const char* name_of<DecodeCore>() { return "mla_decode_core"; }
template <>
const char* name_of<PromptCore>() { return "mla_prompt_core"; }

template <class C = Core>
C* core_of(PyObject* o) {
  auto* c = static_cast<C*>(PyCapsule_GetPointer(o, name_of<C>()));
  if (!c) throw PyError{};
  return c;
}
template <class C>
void drop(PyObject* o) { delete static_cast<C*>(PyCapsule_GetPointer(o, name_of<C>())); }
template <class C>
PyObject* capsule(C* c) {
  PyObject* o = PyCapsule_New(c, name_of<C>(), drop<C>);
  if (!o) delete c;
  return o;
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

// A CUDA tensor of the core's device and the type.
const at::Tensor& tensor(const Device* c, PyObject* o, const char* what, at::ScalarType type, const char* type_name) {
  if (!THPVariable_Check(o)) refuse("%s is a tensor", what);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != c->device) refuse("%s is on cuda:%d, the call's device", what, c->device);
  if (t.scalar_type() != type) refuse("%s is %s", what, type_name);
  return t;
}

// A vector of consecutive int32; size < 0: of any length.
int32_t* vec(const Device* c, PyObject* o, const char* what, int64_t size, int64_t* numel = nullptr) {
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

// The stream a call runs on, and the core's device made current for as long.
struct Where {
  c10::cuda::OptionalCUDAGuard guard;
  c10::cuda::CUDAStream current;
  void* handle;
  bool given;
  Where(const Device* c, PyObject* stream)
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
// (Straight from the allocator: through the dispatcher a tensor took 1.7 us by itself and
// twice that between launches, whose code displaces it from the processor's caches.)
at::Tensor fresh(const Device* c, const Where& w, at::IntArrayRef shape, at::ScalarType type) {
  const auto make = [&] {
    return at::Tensor(at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(),
                                                c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt));
  };
  if (!w.given) return make();  // (the core's device is current)
  const c10::cuda::CUDAStreamGuard on(c10::cuda::getStreamFromExternal(
      static_cast<cudaStream_t>(w.handle), static_cast<c10::DeviceIndex>(c->device)));
  return make();
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

// core(address of an mla_cache, workspace address, its bytes, device index) -> capsule
PyObject* py_core(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(4)
  BEGIN
  const int device = static_cast<int>(whole(a[3]));
  const size_t bytes = static_cast<size_t>(whole(a[2]));
  return capsule(new Core{{device}, *static_cast<const mla_cache*>(PyLong_AsVoidPtr(a[0])),
                          static_cast<int32_t*>(PyLong_AsVoidPtr(a[1])), bytes});
  END
}

// decode_core(address of an mla_plan, workspace address, its bytes, device index) -> capsule
PyObject* py_decode_core(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(4)
  BEGIN
  const int device = static_cast<int>(whole(a[3]));
  const size_t bytes = static_cast<size_t>(whole(a[2]));
  return capsule(new DecodeCore{{device}, static_cast<const mla_plan*>(PyLong_AsVoidPtr(a[0])), PyLong_AsVoidPtr(a[1]), bytes});
  END
}

// What a decode takes by address (None: null), consecutive and of `least` elements or more: memory
// of the core's device or, where the header allows it, pinned host memory.
const at::Tensor* given(PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse("%s is a tensor", what);
  return &THPVariable_Unpack(o);
}
void reachable(const Device* c, const at::Tensor& t, const char* what, bool host) {
  if (t.is_cuda() ? t.get_device() != c->device : !host || t.numel() == 0 || !t.is_pinned())
    refuse("%s is on cuda:%d, the call's device%s", what, c->device, host ? ", or in pinned host memory" : "");
}
void* plain(const Device* c, const at::Tensor* t, const char* what, const char* type_name, bool type_fits, int64_t least,
            bool host) {
  if (!t) return nullptr;
  if (!type_fits) refuse("%s is %s", what, type_name);
  if (!t->is_contiguous()) refuse("%s is contiguous", what);
  if (t->numel() < least) refuse("%s has %lld elements, not %lld or more", what, (long long)t->numel(), (long long)least);
  if (t->numel() > 0) reachable(c, *t, what, host);
  return t->data_ptr();
}
void* plain(const Device* c, PyObject* o, const char* what, at::ScalarType type, const char* type_name, int64_t least, bool host) {
  const at::Tensor* t = given(o, what);
  return plain(c, t, what, type_name, t && t->scalar_type() == type, least, host);
}
const int32_t* indices(const Device* c, PyObject* o, const char* what, int64_t least) {
  return static_cast<int32_t*>(plain(c, o, what, at::kInt, "int32", least, true));
}

// decode(core, q, kv, kv_scale, indptr, kv_indices, last_page_len, qo_indptr, out, lse, sm_scale, stream)
//   -> (status, out, lse); kv_indices and last_page_len None: a contiguous cache
PyObject* py_decode(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(12)
  BEGIN
  const DecodeCore* c = core_of<DecodeCore>(a[0]);
  const mla_plan* plan = c->plan;
  const int32_t type = plan->kv_dtype;
  const int64_t rows = plan->page_size ? (int64_t)plan->num_pages * plan->page_size : plan->total_kv;
  const int64_t sequences = plan->q_len > 1 ? plan->batch / plan->q_len : plan->batch;
  const void* q = plain(c, a[1], "q", at::kBFloat16, "bf16", 0, type != MLA_KV_BF16);
  const at::Tensor* cache = given(a[2], "kv");
  const void* kv = plain(c, cache, "kv", type == MLA_KV_BF16 ? "bf16" : "of one byte an element",
                         cache && (type == MLA_KV_BF16 ? cache->scalar_type() == at::kBFloat16 : cache->element_size() == 1),
                         rows * (type == MLA_KV_MXFP4 ? MLA_QK_DIM / 2 : MLA_QK_DIM), false);
  const at::Tensor* scale = given(a[3], "kv_scale");
  int64_t stride = 0;
  if (scale && type == MLA_KV_MXFP4) {
    if (scale->element_size() != 1 || scale->dim() != 2 || scale->size(0) < rows || scale->size(1) < MLA_MX_SCALES_PER_ROW ||
        scale->stride(1) != 1)
      refuse("kv_scale is e8m0 bytes [rows, >= 18], rows >= %lld", (long long)rows);
    stride = scale->size(0) > 1 ? scale->stride(0) : scale->size(1);  // (one row has no stride)
  } else if (scale && type == MLA_KV_FP8_ROW) {
    if (scale->scalar_type() != at::kFloat || scale->dim() != 1 || scale->size(0) < rows)
      refuse("kv_scale is fp32 [rows], rows >= %lld", (long long)rows);
    stride = scale->size(0) > 1 ? 4 * scale->stride(0) : 4;  // (one scale has no stride)
  } else if (scale && type == MLA_KV_FP8_E4M3) {
    if (scale->scalar_type() != at::kFloat || scale->numel() < 1) refuse("kv_scale is fp32 [1]");
  }
  if (stride < 0 || stride > INT32_MAX) refuse("kv_scale's rows are too far apart");
  if (scale && type != MLA_KV_BF16 && scale->numel() > 0) reachable(c, *scale, "kv_scale", false);
  const void* scales = scale ? scale->data_ptr() : nullptr;
  const int32_t *indptr = indices(c, a[4], plan->page_size ? "kv_page_indptr" : "kv_indptr", sequences + 1),
                *pages = indices(c, a[5], "kv_indices", plan->page_size ? plan->total_kv / plan->page_size : 0),
                *last = indices(c, a[6], "kv_last_page_len", sequences), *qo = indices(c, a[7], "qo_indptr", sequences);
  void* out = plain(c, a[8], "out", at::kBFloat16, "bf16", (int64_t)plan->batch * MLA_NUM_HEADS * MLA_V_DIM, true);
  float* lse = static_cast<float*>(plain(c, a[9], "lse", at::kFloat, "fp32", (int64_t)plan->batch * MLA_NUM_HEADS, true));
  const double sm_scale = PyFloat_AsDouble(a[10]);
  if (sm_scale == -1.0 && PyErr_Occurred()) throw PyError{};
  const Where w(c, a[11]);
  at::Tensor made_out, made_lse;
  if (a[8] == Py_None) {
    made_out = fresh(c, w, {plan->batch, MLA_NUM_HEADS, MLA_V_DIM}, at::kBFloat16);
    out = made_out.data_ptr();
  }
  if (a[9] == Py_None) {
    made_lse = fresh(c, w, {plan->batch, MLA_NUM_HEADS}, at::kFloat);
    lse = static_cast<float*>(made_lse.data_ptr());
  }
  const int rc = without_gil([&] {
    return plan->page_size ? g_attention.decode_paged(q, kv, scales, (int32_t)stride, indptr, pages, last, qo, out, lse,
                                                      (float)sm_scale, plan, c->workspace, c->workspace_bytes, w.handle)
                           : g_attention.decode(q, kv, scales, (int32_t)stride, indptr, qo, out, lse, (float)sm_scale, plan,
                                                c->workspace, c->workspace_bytes, w.handle);
  });
  PyObject* o = a[8] == Py_None ? THPVariable_Wrap(std::move(made_out)) : Py_NewRef(a[8]);
  PyObject* l = a[9] == Py_None ? THPVariable_Wrap(std::move(made_lse)) : Py_NewRef(a[9]);
  return Py_BuildValue("(iNN)", rc, o, l);
  END
}

// prompt_core(workspace address, its bytes, device index, tokens, keys, batch, heads, causal, sm_scale) -> capsule
PyObject* py_prompt_core(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(9)
  BEGIN
  const size_t bytes = static_cast<size_t>(whole(a[1]));
  const int device = static_cast<int>(whole(a[2]));
  const int64_t tokens = whole(a[3]), keys = whole(a[4]), batch = whole(a[5]);
  const int32_t heads = static_cast<int32_t>(whole(a[6])), causal = static_cast<int32_t>(whole(a[7]));
  const double sm_scale = PyFloat_AsDouble(a[8]);
  if (sm_scale == -1.0 && PyErr_Occurred()) throw PyError{};
  return capsule(new PromptCore{{device}, PyLong_AsVoidPtr(a[0]), bytes, tokens, keys, batch, heads, causal, (float)sm_scale});
  END
}

// bf16 [rows, (heads,) columns], the last dimension consecutive; its strides.
const at::Tensor& rows_of(const PromptCore* c, PyObject* o, const char* what, int64_t rows, bool heads, int64_t columns,
                          int64_t& row_stride, int64_t* head_stride) {
  const at::Tensor& t = tensor(c, o, what, at::kBFloat16, "bf16");
  const int d = heads ? 3 : 2;
  if (t.dim() != d || t.size(0) != rows || (heads && t.size(1) != c->heads) || t.size(d - 1) != columns)
    refuse("%s is [%lld, %s%lld]", what, (long long)rows, heads ? "heads, " : "", (long long)columns);
  if (t.stride(d - 1) != 1) refuse("%s: the last dimension is consecutive", what);
  row_stride = t.stride(0);
  if (heads) *head_stride = t.stride(1);
  return t;
}
int64_t first_size(PyObject* o, const char* what) {
  if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() < 1) refuse("%s is a tensor", what);
  return THPVariable_Unpack(o).size(0);
}

// prompt(core, q_nope, q_pe, k_nope, k_pe, v, qo_indptr, kv_indptr, prefix, out, lse, stream) -> (status, out, lse)
PyObject* py_prompt(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(12)
  BEGIN
  const PromptCore* c = core_of<PromptCore>(a[0]);
  const int64_t t = first_size(a[1], "q_nope"), s = first_size(a[3], "k_nope"), b = first_size(a[6], "qo_indptr") - 1;
  if (t > c->tokens || s > c->keys || b < 0 || b > c->batch)
    refuse("made for %lld tokens, %lld keys and %lld documents: got %lld, %lld, %lld", (long long)c->tokens, (long long)c->keys,
           (long long)c->batch, (long long)t, (long long)s, (long long)b);
  mla_prompt_args g = {};
  g.q_nope = rows_of(c, a[1], "q_nope", t, true, MLA_PROMPT_NOPE, g.q_nope_token_stride, &g.q_nope_head_stride).data_ptr();
  g.q_pe = rows_of(c, a[2], "q_pe", t, true, MLA_PROMPT_PE, g.q_pe_token_stride, &g.q_pe_head_stride).data_ptr();
  g.k_nope = rows_of(c, a[3], "k_nope", s, true, MLA_PROMPT_NOPE, g.k_nope_token_stride, &g.k_nope_head_stride).data_ptr();
  g.k_pe = rows_of(c, a[4], "k_pe", s, false, MLA_PROMPT_PE, g.k_pe_token_stride, nullptr).data_ptr();
  g.v = rows_of(c, a[5], "v", s, true, MLA_PROMPT_V, g.v_token_stride, &g.v_head_stride).data_ptr();
  g.qo_indptr = vec(c, a[6], "qo_indptr", b + 1);
  g.kv_indptr = vec(c, a[7], "kv_indptr", b + 1);
  g.prefix = a[8] == Py_None ? nullptr : vec(c, a[8], "prefix", b);
  g.num_q = count32(t, "q_nope");
  g.num_kv = count32(s, "k_nope");
  g.batch = count32(b, "qo_indptr");
  g.heads = c->heads;
  g.causal = c->causal;
  g.sm_scale = c->sm_scale;
  const Where w(c, a[11]);
  at::Tensor made_out, made_lse;
  if (a[9] == Py_None) {
    made_out = fresh(c, w, {t, c->heads, MLA_PROMPT_V}, at::kBFloat16);
    g.out = made_out.data_ptr();
    g.out_token_stride = (int64_t)c->heads * MLA_PROMPT_V;
    g.out_head_stride = MLA_PROMPT_V;
  } else {
    g.out = rows_of(c, a[9], "out", t, true, MLA_PROMPT_V, g.out_token_stride, &g.out_head_stride).data_ptr();
  }
  if (a[10] == Py_None) {
    made_lse = fresh(c, w, {t, c->heads}, at::kFloat);
    g.lse = static_cast<float*>(made_lse.data_ptr());
  } else {
    const at::Tensor& l = tensor(c, a[10], "lse", at::kFloat, "fp32");
    if (l.dim() != 2 || l.size(0) != t || l.size(1) != c->heads || !l.is_contiguous())
      refuse("lse is [%lld, %d], contiguous", (long long)t, c->heads);
    g.lse = static_cast<float*>(l.data_ptr());
  }
  const int rc = without_gil([&] { return g_attention.prompt(&g, c->workspace, c->workspace_bytes, w.handle); });
  PyObject* o = a[9] == Py_None ? THPVariable_Wrap(std::move(made_out)) : Py_NewRef(a[9]);
  PyObject* l = a[10] == Py_None ? THPVariable_Wrap(std::move(made_lse)) : Py_NewRef(a[10]);
  return Py_BuildValue("(iNN)", rc, o, l);
  END
}

// bind_attention(addresses of mla_decode_fwd, mla_decode_fwd_paged, mla_prompt_fwd)
PyObject* py_bind_attention(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(3)
  BEGIN
  void* at[3];
  for (int i = 0; i < 3; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (!at[i]) refuse("an entry point has no address");
  }
  g_attention.decode = reinterpret_cast<decltype(g_attention.decode)>(at[0]);
  g_attention.decode_paged = reinterpret_cast<decltype(g_attention.decode_paged)>(at[1]);
  g_attention.prompt = reinterpret_cast<decltype(g_attention.prompt)>(at[2]);
  Py_RETURN_NONE;
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
                         METHOD("decode_core", py_decode_core),
                         METHOD("decode", py_decode),
                         METHOD("prompt_core", py_prompt_core),
                         METHOD("prompt", py_prompt),
                         METHOD("bind_attention", py_bind_attention),
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
