// ta_binding.cpp -- the calls of PagedCache and LatentCache as a Python extension module
// (_binding.so): it checks tensor arguments and passes their addresses to the C
// entry points of include/tree_attn.h, nothing else.
//
// These calls are made once per layer and token, and their smallest take 3 us
// on the GPU; checks in Python and ctypes' conversion of up to 22 arguments took
// 3 to 6 us per call (append 9.0 us of host time in all), here 0.3.
#include <Python.h>

#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAException.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Stream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>
#include <memory>
#include <sstream>
#include <stdexcept>
#include <vector>

#include "tree_attn.h"

namespace {

// What every call on one cache passes; the Python object keeps the tensors.
struct Base {
  void* pages;
  const int32_t *indptr, *values, *length;
  void* workspace;
  size_t workspace_bytes;
  int device;
  at::ScalarType dtype;
  std::vector<at::Tensor> held;                // pages, table, workspace
  mutable std::vector<cudaStream_t> streams;   // that the allocator knows they are used on
};

struct Handle : Base {                         // a PagedCache
  using Dims = ta_cache_dims;
  static constexpr const char* kCapsule = "tree_attention_gb300.cache";
  Dims dims;
};

struct Latent : Base {                         // a LatentCache
  using Dims = ta_latent_dims;
  static constexpr const char* kCapsule = "tree_attention_gb300.latent_cache";
  Dims dims;
};

// The tensor argument ``o``; throws unless it has this type and shape and is on
// the handle's device.
const at::Tensor& tensor(const Base& h, const char* name, PyObject* o, at::ScalarType type,
                         std::initializer_list<int64_t> shape) {
  if (!THPVariable_Check(o)) throw std::invalid_argument(std::string(name) + " must be a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape) || !t.is_cuda() ||
      t.get_device() != h.device) {
    std::ostringstream s;
    s << name << " must be " << type << " " << at::IntArrayRef(shape) << " on cuda:" << h.device
      << ", got " << t.scalar_type() << " " << t.sizes() << " on " << t.device();
    throw std::invalid_argument(s.str());
  }
  return t;
}

// Address of a contiguous tensor argument.
template <typename T = void>
T* address(const Base& h, const char* name, PyObject* o, at::ScalarType type,
           std::initializer_list<int64_t> shape) {
  const at::Tensor& t = tensor(h, name, o, type, shape);
  if (!t.is_contiguous()) throw std::invalid_argument(std::string(name) + " must be contiguous");
  return static_cast<T*>(t.data_ptr());
}

int32_t* ints(const Base& h, const char* name, PyObject* o, int64_t n) {
  return address<int32_t>(h, name, o, at::kInt, {n});
}

// A [tokens, heads, d] argument whose tokens may be apart.
const void* rows(const Handle& h, const char* name, PyObject* o, int64_t n, int64_t heads,
                 int64_t* stride) {
  const int64_t d = h.dims.head_dim;
  const at::Tensor& t = tensor(h, name, o, h.dtype, {n, heads, d});
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d))
    throw std::invalid_argument(std::string("the rows of one token must be contiguous in ") + name);
  *stride = n > 1 ? t.stride(0) : heads * d;
  return t.data_ptr();
}

int64_t length(const char* name, PyObject* o, int dim) {
  if (!THPVariable_Check(o)) throw std::invalid_argument(std::string(name) + " must be a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.dim() != dim) {
    std::ostringstream s;
    s << name << " must have " << dim << " dimensions, got " << t.sizes();
    throw std::invalid_argument(s.str());
  }
  return t.size(0);
}

struct PythonError {};   // a Python exception is set

// Keeps the memory of what the handle holds from being reused, after the handle
// is gone, before the work on ``stream`` is done: it may have had the last
// reference.  Not on streams that torch did not make (their id is their
// address): they may be destroyed before the memory is freed.
void hold_on(const Base& h, c10::cuda::CUDAStream stream) {
  cudaStream_t s = stream.stream();
  if (stream.id() != 0 && stream.id() == reinterpret_cast<int64_t>(s)) return;
  if (std::find(h.streams.begin(), h.streams.end(), s) != h.streams.end()) return;
  for (const at::Tensor& t : h.held)
    c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), stream);
  h.streams.push_back(s);
}

// The stream of a call: torch's current one, a stream object, or an address.
void* stream_of(const Base& h, PyObject* o) {
  if (c10::cuda::current_device() != h.device) {
    std::ostringstream s;
    s << "the cache is on cuda:" << h.device << ", which is not the current device";
    throw std::invalid_argument(s.str());
  }
  if (o == Py_None) {
    const c10::cuda::CUDAStream stream = c10::cuda::getCurrentCUDAStream(h.device);
    hold_on(h, stream);
    return stream.stream();
  }
  if (THPStream_Check(o)) {
    const THPStream* t = reinterpret_cast<const THPStream*>(o);
    const c10::cuda::CUDAStream stream = c10::cuda::CUDAStream::unpack3(
        t->stream_id, static_cast<c10::DeviceIndex>(t->device_index),
        static_cast<c10::DeviceType>(t->device_type));
    if (stream.device_index() != h.device)
      throw std::invalid_argument("stream must be on the device of the cache");
    hold_on(h, stream);
    return stream.stream();
  }
  PyObject* a = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream")
                                                         : PyNumber_Long(o);
  if (!a) throw PythonError();
  void* p = PyLong_AsVoidPtr(a);
  Py_DECREF(a);
  if (PyErr_Occurred()) throw PythonError();
  return p;
}

float number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw PythonError();
  return static_cast<float>(x);
}

template <typename H>
const H& handle_of(PyObject* o) {
  void* p = PyCapsule_GetPointer(o, H::kCapsule);
  if (!p) throw PythonError();
  return *static_cast<H*>(p);
}
const Handle& handle(PyObject* o) { return handle_of<Handle>(o); }

// Runs ``body`` on ``n`` arguments, of which there must be ``want``; it returns a
// Python object, and its exceptions become Python's.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F body) {
  try {
    if (n != want) throw std::invalid_argument("wrong number of arguments");
    return body();
  } catch (const PythonError&) {
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The same for a ``body`` that returns a status.
template <typename F>
PyObject* call(Py_ssize_t n, Py_ssize_t want, F body) {
  return guarded(n, want, [&] { return PyLong_FromLong(body()); });
}

bool given(PyObject* o) { return o != Py_None; }

// handle(dims address, pages, page_indptr, page_values, length_info, workspace),
// latent_handle(the same)
template <typename H>
PyObject* make_handle(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const void* dims = PyLong_AsVoidPtr(a[0]);
    if (PyErr_Occurred()) throw PythonError();
    if (!dims) throw std::invalid_argument("the address of the dims expected");
    std::vector<at::Tensor> t;
    for (int i = 1; i < 6; ++i) {
      if (!THPVariable_Check(a[i])) throw std::invalid_argument("tensors expected");
      t.push_back(THPVariable_Unpack(a[i]));
    }
    auto ints = [&](int i) { return static_cast<int32_t*>(t[i].data_ptr()); };
    std::unique_ptr<H> h(new H{
        {t[0].data_ptr(), ints(1), ints(2), ints(3), t[4].data_ptr(),
         static_cast<size_t>(t[4].nbytes()), static_cast<int>(t[0].get_device()),
         t[0].scalar_type(), t, {}},
        *static_cast<const typename H::Dims*>(dims)});
    PyObject* c = PyCapsule_New(h.get(), H::kCapsule, [](PyObject* o) {
      delete static_cast<H*>(PyCapsule_GetPointer(o, H::kCapsule));
    });
    if (c) h.release();
    return c;
  });
}

// append(handle, q, k, v, append_indptr, positions, rope address, q_weight,
//        k_weight, norm_eps, q_out, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 12, [&] {
    const Handle& h = handle(a[0]);
    const int64_t tokens = length("q", a[1], 3), d = h.dims.head_dim;
    int64_t qs, ks, vs;
    const void* q = rows(h, "q", a[1], tokens, h.dims.h_q, &qs);
    const void* k = rows(h, "k", a[2], tokens, h.dims.h_kv, &ks);
    const void* v = rows(h, "v", a[3], tokens, h.dims.h_kv, &vs);
    if (tokens > INT32_MAX) throw std::invalid_argument("too many tokens");
    const ta_rope* rope = given(a[6]) ? static_cast<const ta_rope*>(PyLong_AsVoidPtr(a[6])) : nullptr;
    if (PyErr_Occurred()) throw PythonError();
    const int32_t* indptr = ints(h, "append_indptr", a[4], h.dims.batch_size + 1);
    const int32_t* positions = given(a[5]) ? ints(h, "positions", a[5], tokens) : nullptr;
    const void* qw = given(a[7]) ? address(h, "q_weight", a[7], h.dtype, {d}) : nullptr;
    const void* kw = given(a[8]) ? address(h, "k_weight", a[8], h.dtype, {d}) : nullptr;
    const float eps = number(a[9]);
    void* q_out = address(h, "q_out", a[10], h.dtype, {tokens, h.dims.h_q, d});
    return (long)tree_attn_append_paged(q, qs, k, ks, v, vs, (int32_t)tokens, indptr, positions, qw,
                                        kw, eps, rope, h.pages, h.indptr, h.values, h.length, q_out,
                                        &h.dims, h.workspace, h.workspace_bytes, stream_of(h, a[11]));
  });
}

// decode(handle, q, sm_scale, out, lse, stream)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 6, [&] {
    const Handle& h = handle(a[0]);
    const int64_t b = h.dims.batch_size, hq = h.dims.h_q, d = h.dims.head_dim;
    const void* q = address(h, "q", a[1], h.dtype, {b, hq, d});
    const float sm_scale = number(a[2]);
    void* out = address(h, "out", a[3], h.dtype, {b, hq, d});
    float* lse = address<float>(h, "lse", a[4], at::kFloat, {b, hq});
    return (long)tree_attn_decode_paged(q, h.pages, h.indptr, h.values, h.length, out, lse, sm_scale,
                                        &h.dims, h.workspace, h.workspace_bytes, stream_of(h, a[5]));
  });
}

// compact(handle, mn_indptr, accept_indptr, accept_nodes, new_page_indptr,
//         new_page_values, new_length_info, freed_pages, num_freed, stream)
template <typename H, auto F>
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, [&] {
    const H& h = handle_of<H>(a[0]);
    const int64_t b = h.dims.batch_size, nnz = h.dims.nnz_pages;
    const int64_t accepted = length("accept_nodes", a[3], 1);
    if (accepted > INT32_MAX) throw std::invalid_argument("too many accepted nodes");
    const int32_t* mn = ints(h, "mn_indptr", a[1], b + 1);
    const int32_t* accept = ints(h, "accept_indptr", a[2], b + 1);
    const int32_t* nodes = ints(h, "accept_nodes", a[3], accepted);
    int32_t* indptr = ints(h, "new_page_indptr", a[4], b + 1);
    int32_t* values = ints(h, "new_page_values", a[5], nnz);
    int32_t* lengths = ints(h, "new_length_info", a[6], b);
    int32_t* freed = ints(h, "freed_pages", a[7], nnz);
    int32_t* num_freed = ints(h, "num_freed", a[8], 1);
    return (long)F(h.pages, h.indptr, h.values, h.length, mn, accept, nodes, (int32_t)accepted, indptr,
                   values, lengths, freed, num_freed, &h.dims, h.workspace, h.workspace_bytes,
                   stream_of(h, a[9]));
  });
}

// copy_pages(handle, src_pages, dst_pages, stream)
template <typename H, auto F>
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 4, [&] {
    const H& h = handle_of<H>(a[0]);
    const int64_t pairs = length("src_pages", a[1], 1);
    if (pairs > INT32_MAX) throw std::invalid_argument("too many pages");
    const int32_t* src = ints(h, "src_pages", a[1], pairs);
    const int32_t* dst = ints(h, "dst_pages", a[2], pairs);
    return (long)F(h.pages, src, dst, (int32_t)pairs, &h.dims, h.workspace, h.workspace_bytes,
                   stream_of(h, a[3]));
  });
}

// A [tokens, width] argument whose rows may be apart.
const void* token_rows(const Base& h, const char* name, PyObject* o, int64_t n, int64_t width,
                       int64_t* stride) {
  const at::Tensor& t = tensor(h, name, o, h.dtype, {n, width});
  if (t.stride(1) != 1)
    throw std::invalid_argument(std::string("the elements of one token must be contiguous in ") + name);
  *stride = n > 1 ? t.stride(0) : width;
  return t.data_ptr();
}

// A [tokens, heads, width] argument whose tokens and heads may be apart.
void* head_rows(const Base& h, const char* name, PyObject* o, int64_t n, int64_t heads, int64_t width,
                int64_t* token, int64_t* head) {
  const at::Tensor& t = tensor(h, name, o, h.dtype, {n, heads, width});
  if (t.stride(2) != 1)
    throw std::invalid_argument(std::string("the elements of one head must be contiguous in ") + name);
  *head = heads > 1 ? t.stride(1) : width;
  *token = n > 1 ? t.stride(0) : (heads - 1) * *head + width;
  return t.data_ptr();
}

// latent_append(handle, latent, k_rope, q_rope, append_indptr, positions, rope
//               address, weight, norm_eps, q_out, rows_out, stream)
PyObject* latent_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 12, [&] {
    const Latent& h = handle_of<Latent>(a[0]);
    const int64_t tokens = length("latent", a[1], 2), heads = h.dims.h_q, rd = h.dims.rope_dim;
    const int64_t width = h.dims.rank + rd;
    int64_t ls, ks, qt = 0, qh = 0, ot = 0, oh = 0;
    const void* latent = token_rows(h, "latent", a[1], tokens, h.dims.rank, &ls);
    const void* k = token_rows(h, "k_rope", a[2], tokens, rd, &ks);
    if (tokens > INT32_MAX) throw std::invalid_argument("too many tokens");
    const void* q = given(a[3]) ? head_rows(h, "q_rope", a[3], tokens, heads, rd, &qt, &qh) : nullptr;
    const int32_t* indptr = ints(h, "append_indptr", a[4], h.dims.batch_size + 1);
    const int32_t* positions = given(a[5]) ? ints(h, "positions", a[5], tokens) : nullptr;
    const ta_rope* rope = given(a[6]) ? static_cast<const ta_rope*>(PyLong_AsVoidPtr(a[6])) : nullptr;
    if (PyErr_Occurred()) throw PythonError();
    const void* w = given(a[7]) ? address(h, "weight", a[7], h.dtype, {h.dims.rank}) : nullptr;
    const float eps = number(a[8]);
    void* q_out = given(a[9]) ? head_rows(h, "q_out", a[9], tokens, heads, rd, &ot, &oh) : nullptr;
    void* rows_out = given(a[10]) ? address(h, "rows_out", a[10], h.dtype, {tokens, width}) : nullptr;
    return (long)tree_attn_append_latent(latent, ls, k, ks, q, qt, qh, (int32_t)tokens, indptr,
                                         positions, w, eps, rope, h.pages, h.indptr, h.values,
                                         h.length, q_out, ot, oh, rows_out, &h.dims, h.workspace,
                                         h.workspace_bytes, stream_of(h, a[11]));
  });
}

// latent_decode(handle, q, sm_scale, out, lse, stream)
PyObject* latent_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 6, [&] {
    const Latent& h = handle_of<Latent>(a[0]);
    const int64_t b = h.dims.batch_size, hq = h.dims.h_q, rank = h.dims.rank;
    const void* q = address(h, "q", a[1], h.dtype, {b, hq, rank + h.dims.rope_dim});
    const float sm_scale = number(a[2]);
    void* out = address(h, "out", a[3], h.dtype, {b, hq, rank});
    float* lse = address<float>(h, "lse", a[4], at::kFloat, {b, hq});
    return (long)tree_attn_decode_latent(q, h.pages, h.indptr, h.values, h.length, out, lse, sm_scale,
                                         &h.dims, h.workspace, h.workspace_bytes, stream_of(h, a[5]));
  });
}

// latent_tree(handle, q, q_indptr, mn_indptr, tree_order, sm_scale, out, lse, stream)
PyObject* latent_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, [&] {
    const Latent& h = handle_of<Latent>(a[0]);
    const int64_t rows = length("q", a[1], 3), nodes = length("tree_order", a[4], 2);
    const int64_t b = h.dims.batch_size, hq = h.dims.h_q, rank = h.dims.rank;
    if (rows > INT32_MAX || nodes > INT32_MAX) throw std::invalid_argument("too many rows");
    const void* q = address(h, "q", a[1], h.dtype, {rows, hq, rank + h.dims.rope_dim});
    const int32_t* q_indptr = ints(h, "q_indptr", a[2], b + 1);
    const int32_t* mn = ints(h, "mn_indptr", a[3], b + 1);
    const int32_t* order = address<int32_t>(h, "tree_order", a[4], at::kInt, {nodes, 2});
    const float sm_scale = number(a[5]);
    void* out = address(h, "out", a[6], h.dtype, {rows, hq, rank});
    float* lse = address<float>(h, "lse", a[7], at::kFloat, {rows, hq});
    return (long)tree_attn_latent(q, q_indptr, (int32_t)rows, h.pages, h.indptr, h.values, h.length, mn,
                                  order, (int32_t)nodes, out, lse, sm_scale, &h.dims, h.workspace,
                                  h.workspace_bytes, stream_of(h, a[8]));
  });
}

// zero_now(tensor): zero-fills a CUDA tensor before it returns, also while the
// current stream is captured into a graph.
PyObject* zero_now(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 1, [&] {
    if (!THPVariable_Check(a[0])) throw std::invalid_argument("a tensor expected");
    const at::Tensor& t = THPVariable_Unpack(a[0]);
    if (!t.is_cuda() || !t.is_contiguous()) throw std::invalid_argument("a contiguous CUDA tensor expected");
    c10::cuda::CUDAStreamCaptureModeGuard relaxed{cudaStreamCaptureModeRelaxed};
    const c10::cuda::CUDAStream stream = c10::cuda::getStreamFromPool(false, t.device().index());
    C10_CUDA_CHECK(cudaMemsetAsync(t.data_ptr(), 0, t.nbytes(), stream));
    C10_CUDA_CHECK(cudaStreamSynchronize(stream));
    return 0L;
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<make_handle<Handle>>("handle"),
    method<append>("append"),
    method<decode>("decode"),
    method<compact<Handle, tree_attn_compact_paged>>("compact"),
    method<copy_pages<Handle, tree_attn_copy_pages>>("copy_pages"),
    method<make_handle<Latent>>("latent_handle"),
    method<latent_append>("latent_append"),
    method<latent_decode>("latent_decode"),
    method<latent_tree>("latent_tree"),
    method<compact<Latent, tree_attn_compact_latent>>("latent_compact"),
    method<copy_pages<Latent, tree_attn_copy_pages_latent>>("latent_copy_pages"),
    method<zero_now>("zero_now"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
