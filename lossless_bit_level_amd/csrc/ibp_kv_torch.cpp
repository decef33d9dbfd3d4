// The binding of the calls of libibp_kv and libibp_kv_long to torch tensors: checks
// of the arguments, tensors for the results, and the call of the C ABI
// (include/ibp_kv.h, include/ibp_kv_long.h).  Its
// functions stand behind those of the same names in ibp_kv.py.  No step of an
// operator is computed here.  A call runs on the GPU of its tensors, whichever
// is current; going backward through its results raises.
//
// Marshalled by ctypes, and without the checks of GPU and gradients (0.2 us), a
// short call took the host longer than the kernel takes: an append 10.0 us back to
// back, 5.5 us so; attention over 291 tokens 12.9 and 7.1 us (the kernel's own
// time); an eviction 9.6 and 7.4 us.
#include <Python.h>

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/DeviceGuard.h>

#include <dlfcn.h>

#include <cmath>
#include <cstring>
#include <initializer_list>
#include <memory>
#include <vector>

#include "ibp_kv.h"
#include "ibp_kv_long.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* refuse(const char* format, const char* name) {
  PyErr_Format(PyExc_ValueError, format, name);
  return nullptr;
}

bool is_tensor(PyObject* o, const char* name) {
  if (THPVariable_Check(o)) return true;
  refuse("%s must be a tensor", name);
  return false;
}

// Contiguous GPU tensors only: the kernels take their addresses as they are (a
// CPU pointer there would fault the GPU).
bool check(const Tensor& t, ScalarType type, const char* name) {
  if (t.is_cuda() && t.scalar_type() == type && t.is_contiguous()) return true;
  PyErr_Format(PyExc_ValueError, "%s must be a contiguous %s GPU tensor", name,
               type == ScalarType::Int ? "int32" : type == ScalarType::Float ? "float32" : type == ScalarType::Char ? "int8" : "uint8");
  return false;
}

// The GPU of the arguments `o` that are GPU tensors, which has to be one: a
// kernel runs on one GPU, with their addresses as they are.  What is no GPU
// tensor is left to the checks that follow.
struct Argument {
  PyObject* o;
  const char* name;
};

bool same_gpu(std::initializer_list<Argument> arguments, c10::Device* gpu) {
  bool known = false;
  for (const Argument& x : arguments) {
    if (!x.o || !THPVariable_Check(x.o) || !THPVariable_Unpack(x.o).is_cuda()) continue;
    const c10::Device d = THPVariable_Unpack(x.o).device();
    if (known && d != *gpu) {
      refuse("%s must be on the same GPU as the call's other tensors", x.name);
      return false;
    }
    *gpu = d;
    known = true;
  }
  return true;
}

// Makes a GPU current for the call.  (Most often it is: asking costs less than
// setting it.)
struct OnGpu {
  explicit OnGpu(c10::Device gpu) {
    if (c10::impl::getDeviceGuardImpl(gpu.type())->getDevice() != gpu) guard_.reset_device(gpu);
  }
  c10::OptionalDeviceGuard guard_;
};

// The tensors that a cache holds on to, a tuple (a borrowed reference, good as
// long as the cache); null for a structure that was filled by hand.
PyObject* tensors_of_cache(PyObject* cache) {
  static PyObject* const name = PyUnicode_InternFromString("tensors");
  PyObject* held = PyObject_GetAttr(cache, name);
  if (!held) {
    PyErr_Clear();
    return nullptr;
  }
  Py_DECREF(held);
  return PyTuple_Check(held) ? held : nullptr;
}

// The first of them: they are all on one GPU.
PyObject* tensor_of_cache(PyObject* cache) {
  PyObject* held = tensors_of_cache(cache);
  return held && PyTuple_GET_SIZE(held) ? PyTuple_GET_ITEM(held, 0) : nullptr;
}

// ---- autograd: no call has a gradient ----

bool wants_gradient(PyObject* o) {
  return o && THPVariable_Check(o) && THPVariable_Unpack(o).requires_grad() && at::GradMode::is_enabled();
}

// Inputs that require a gradient give results whose backward pass raises, not
// results that count as constants.  Results written to a given tensor cannot say
// so; like torch's functions with out= the calls refuse them.
class Gradients {
 public:
  Gradients(const char* call, std::initializer_list<PyObject*> inputs) : call_(call) {
    for (PyObject* o : inputs)
      if (wants_gradient(o)) wanted_.push_back(THPVariable_Unpack(o));
  }

  bool check_given(std::initializer_list<Argument> outputs) const {
    for (const Argument& x : outputs) {
      if (x.o == Py_None || (wanted_.empty() && !wants_gradient(x.o))) continue;
      PyErr_Format(PyExc_ValueError, "%s: %s is given, but one of the tensors requires a gradient, which this call does not have", call_,
                   x.name);
      return false;
    }
    return true;
  }

  void mark(std::initializer_list<Tensor> outputs) const {
    if (wanted_.empty()) return;
    const auto raises = std::make_shared<torch::autograd::NotImplemented>(call_, torch::autograd::collect_next_edges(wanted_));
    for (const Tensor& t : outputs)
      if (t.defined()) torch::autograd::set_history(t, raises);
  }

 private:
  const char* call_;
  std::vector<Tensor> wanted_;
};

// A given tensor that a call writes has changed (tensors of inference mode keep
// no count of that).
void written(PyObject* o) {
  if (!o || !THPVariable_Check(o)) return;
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

bool check(PyObject* o, ScalarType type, const char* name) {
  return is_tensor(o, name) && check(THPVariable_Unpack(o), type, name);
}

bool check_like(PyObject* o, ScalarType type, const char* name, const Tensor& like) {
  if (!check(o, type, name)) return false;
  if (THPVariable_Unpack(o).sizes() == like.sizes()) return true;
  refuse("%s must have the shape of pages or of lengths", name);
  return false;
}

// Strides of the leading axes are free, the last axis is contiguous.
bool check_rows(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape, ibp_kv_tensor* out) {
  if (!is_tensor(o, name)) return false;
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.scalar_type() != type || t.sizes() != shape) {
    PyErr_Format(PyExc_ValueError, "%s must be a GPU tensor of the call's 16-bit type and of shape (%lld, %lld, %lld, %lld)",
                 name, (long long)shape[0], (long long)shape[1], (long long)shape[2], (long long)shape[3]);
    return false;
  }
  const auto s = t.strides();
  if (s[3] != 1) {
    refuse("the last axis of %s must be contiguous", name);
    return false;
  }
  *out = {t.data_ptr(), s[0], s[1], s[2]};
  return true;
}

bool check_type(PyObject* o, const char* name, uint32_t* dtype) {
  if (!is_tensor(o, name)) return false;
  const Tensor& t = THPVariable_Unpack(o);
  const bool bf16 = t.scalar_type() == ScalarType::BFloat16;
  if ((bf16 || t.scalar_type() == ScalarType::Half) && t.dim() == 4) {
    *dtype = bf16 ? IBP_KV_BF16 : IBP_KV_FP16;
    return true;
  }
  refuse("%s must be a bfloat16 or float16 tensor [n_seqs, n_new, heads, head_dim]", name);
  return false;
}

bool check_table(PyObject* pages, PyObject* lengths, ibp_kv_table* table) {
  if (!check(pages, ScalarType::Int, "pages") || !check(lengths, ScalarType::Int, "lengths")) return false;
  const Tensor &p = THPVariable_Unpack(pages), &n = THPVariable_Unpack(lengths);
  if (p.dim() != 3) {
    refuse("%s must be [n_seqs, kv_heads, max_pages]", "pages");
    return false;
  }
  if (n.dim() != 2 || n.size(0) != p.size(0) || n.size(1) != p.size(1)) {
    refuse("%s must be [n_seqs, kv_heads], as pages is", "lengths");
    return false;
  }
  *table = {(uint64_t)p.size(0), (uint64_t)p.size(1), (uint64_t)p.size(2), (const int32_t*)p.data_ptr(),
            (const int32_t*)n.data_ptr()};
  return true;
}

bool check_counts(PyObject* o, uint64_t n_seqs, const int32_t** counts) {
  *counts = nullptr;
  if (o == Py_None) return true;
  if (!check(o, ScalarType::Int, "counts")) return false;
  const Tensor& t = THPVariable_Unpack(o);
  if (t.dim() != 1 || (uint64_t)t.size(0) != n_seqs) {
    refuse("%s must be [n_seqs]", "counts");
    return false;
  }
  *counts = (const int32_t*)t.data_ptr();
  return true;
}

// The bytes of a ctypes structure.
template <class T>
bool from_structure(PyObject* o, T* out, bool write = false) {
  Py_buffer view;
  if (PyObject_GetBuffer(o, &view, write ? PyBUF_WRITABLE : PyBUF_SIMPLE)) return false;
  const bool fits = view.len == (Py_ssize_t)sizeof(T);
  if (fits) {
    if (write)
      std::memcpy(view.buf, out, sizeof(T));
    else
      std::memcpy(out, view.buf, sizeof(T));
  }
  PyBuffer_Release(&view);
  if (!fits) PyErr_SetString(PyExc_ValueError, "not an ibp_kv_cache");
  return fits;
}

bool number(PyObject* o, uint64_t* out) {
  *out = PyLong_AsUnsignedLongLong(o);
  return !PyErr_Occurred();
}

bool stream_of(PyObject* o, void** out) {
  *out = PyLong_AsVoidPtr(o);
  return !PyErr_Occurred();
}

bool arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
  return false;
}

// set_cache(structure, k_codes, k_scales, v_codes, v_scales, page_tokens, head_dim)
PyObject* set_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  uint64_t page_tokens, head_dim;
  c10::Device gpu(c10::kCUDA, 0);
  if (!arguments(n, 7) ||
      !same_gpu({{a[1], "k_codes"}, {a[2], "k_scales"}, {a[3], "v_codes"}, {a[4], "v_scales"}}, &gpu) ||
      !check(a[1], ScalarType::Byte, "k_codes") ||
      !check(a[2], ScalarType::Float, "k_scales") || !check(a[3], ScalarType::Byte, "v_codes") ||
      !check(a[4], ScalarType::Float, "v_scales") || !number(a[5], &page_tokens) || !number(a[6], &head_dim))
    return nullptr;
  const Tensor &kc = THPVariable_Unpack(a[1]), &ks = THPVariable_Unpack(a[2]);
  const Tensor &vc = THPVariable_Unpack(a[3]), &vs = THPVariable_Unpack(a[4]);
  const uint64_t pages = (uint64_t)ks.numel();
  if (page_tokens > 0xFFFF || head_dim > 0xFFFF || (uint64_t)vs.numel() != pages || kc.numel() != vc.numel() ||
      (uint64_t)kc.numel() != pages * page_tokens * head_dim) {
    PyErr_Format(PyExc_ValueError,
                 "%llu pages of %llu x %llu codes and as many scales expected, for keys and for values",
                 (unsigned long long)pages, (unsigned long long)page_tokens, (unsigned long long)head_dim);
    return nullptr;
  }
  ibp_kv_cache c = {pages, (uint32_t)page_tokens, (uint32_t)head_dim, (uint8_t*)kc.data_ptr(), (float*)ks.data_ptr(),
                    (uint8_t*)vc.data_ptr(), (float*)vs.data_ptr()};
  if (!from_structure(a[0], &c, true)) return nullptr;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// append(cache, pages, lengths, k, v, counts, stream) -> status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  ibp_kv_cache cache;
  ibp_kv_table table;
  ibp_kv_tensor k, v;
  uint32_t dtype;
  const int32_t* counts;
  void* stream;
  c10::Device gpu(c10::kCUDA, 0);
  if (!arguments(n, 7) ||
      !same_gpu({{tensor_of_cache(a[0]), "the cache"}, {a[1], "pages"}, {a[2], "lengths"}, {a[3], "k"}, {a[4], "v"},
                 {a[5], "counts"}}, &gpu) ||
      !check_type(a[3], "k", &dtype) || !from_structure(a[0], &cache) || !check_table(a[1], a[2], &table))
    return nullptr;
  const Tensor& x = THPVariable_Unpack(a[3]);
  const int64_t shape[4] = {(int64_t)table.n_seqs, x.size(1), (int64_t)table.kv_heads, cache.head_dim};
  if (!check_rows(a[3], "k", x.scalar_type(), shape, &k) || !check_rows(a[4], "v", x.scalar_type(), shape, &v) ||
      !check_counts(a[5], table.n_seqs, &counts) || !stream_of(a[6], &stream))
    return nullptr;
  const OnGpu on(gpu);
  if (PyObject* held = tensors_of_cache(a[0]))
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(held); ++i) written(PyTuple_GET_ITEM(held, i));
  return PyLong_FromLong(ibp_kv_append(&cache, &table, dtype, (uint64_t)shape[1], &k, &v, counts, stream));
  END_HANDLE_TH_ERRORS
}

// attention(cache, pages, lengths, q, scale, weights, weights_out, counts, out,
//           workspace, stream) -> (status, out, weights_out)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  ibp_kv_cache cache;
  ibp_kv_table table;
  ibp_kv_tensor q, o;
  uint32_t dtype;
  const int32_t* counts;
  void* stream;
  c10::Device gpu(c10::kCUDA, 0);
  if (!arguments(n, 11) ||
      !same_gpu({{tensor_of_cache(a[0]), "the cache"}, {a[1], "pages"}, {a[2], "lengths"}, {a[3], "q"}, {a[5], "weights"},
                 {a[6], "weights_out"}, {a[7], "counts"}, {a[8], "out"}, {a[9], "workspace"}}, &gpu))
    return nullptr;
  const Gradients gradients("ibp_kv_attention", {a[3], a[5]});
  if (!gradients.check_given({{a[8], "out"}, {a[6], "weights_out"}}) || !check_type(a[3], "q", &dtype) || !from_structure(a[0], &cache) || !check_table(a[1], a[2], &table))
    return nullptr;
  const Tensor& x = THPVariable_Unpack(a[3]);
  const Tensor& pages = THPVariable_Unpack(a[1]);
  const int64_t n_new = x.size(1), q_heads = x.size(2);
  if (table.kv_heads && (q_heads == 0 || q_heads % (int64_t)table.kv_heads)) {
    PyErr_SetString(PyExc_ValueError, "q_heads must be a multiple of kv_heads");
    return nullptr;
  }
  const int64_t shape[4] = {(int64_t)table.n_seqs, n_new, q_heads, cache.head_dim};
  if (!check_rows(a[3], "q", x.scalar_type(), shape, &q)) return nullptr;
  float scale = 1.f / std::sqrt((float)cache.head_dim);
  if (a[4] != Py_None) {
    scale = (float)PyFloat_AsDouble(a[4]);
    if (PyErr_Occurred()) return nullptr;
  }
  const bool weighted = a[5] != Py_None;
  if (weighted ? !check_like(a[5], ScalarType::Float, "weights", pages) ||
                     (a[6] != Py_None && !check_like(a[6], ScalarType::Float, "weights_out", pages))
               : a[6] != Py_None) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "weights_out without weights");
    return nullptr;
  }
  if (!check_counts(a[7], table.n_seqs, &counts) ||
      (a[8] != Py_None && !check_rows(a[8], "out", x.scalar_type(), shape, &o)) ||
      (a[9] != Py_None && !check(a[9], ScalarType::Byte, "workspace")) || !stream_of(a[10], &stream))
    return nullptr;

  const OnGpu on(gpu);
  const Tensor out = a[8] != Py_None ? THPVariable_Unpack(a[8]) : at::empty(shape, x.options());
  if (a[8] == Py_None) o = {out.data_ptr(), out.stride(0), out.stride(1), out.stride(2)};
  Tensor weights_out;
  if (weighted) weights_out = a[6] != Py_None ? THPVariable_Unpack(a[6]) : at::empty_like(THPVariable_Unpack(a[5]));
  Tensor workspace;
  if (a[9] != Py_None) {
    workspace = THPVariable_Unpack(a[9]);
  } else if (const uint64_t bytes = ibp_kv_attention_workspace_bytes(&cache, &table, (uint64_t)q_heads, (uint64_t)n_new, weighted)) {
    workspace = at::empty({(int64_t)bytes}, x.options().dtype(at::kByte));
  }
  written(a[8]);
  written(a[6]);
  const int status = ibp_kv_attention(
      &cache, &table, dtype, (uint64_t)q_heads, (uint64_t)n_new, &q, &o, counts, scale,
      weighted ? (const float*)THPVariable_Unpack(a[5]).data_ptr() : nullptr,
      weighted ? (float*)weights_out.data_ptr() : nullptr, workspace.defined() ? workspace.data_ptr() : nullptr,
      workspace.defined() ? (uint64_t)workspace.numel() : 0, stream);
  gradients.mark({out, weights_out});
  PyObject* w = Py_None;
  Py_INCREF(w);
  if (weighted) {
    Py_DECREF(w);
    w = THPVariable_Wrap(weights_out);
  }
  return Py_BuildValue("(iNN)", status, THPVariable_Wrap(out), w);
  END_HANDLE_TH_ERRORS
}

// evict(pages, weights, lengths, page_tokens, keep, sink, recent, pages_out,
//       weights_out, lengths_out, stream) -> (status, pages, weights, lengths)
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  ibp_kv_table table;
  uint64_t page_tokens, keep, sink, recent;
  void* stream;
  c10::Device gpu(c10::kCUDA, 0);
  if (!arguments(n, 11) ||
      !same_gpu({{a[0], "pages"}, {a[1], "weights"}, {a[2], "lengths"}, {a[7], "pages_out"}, {a[8], "weights_out"},
                 {a[9], "lengths_out"}}, &gpu))
    return nullptr;
  const Gradients gradients("ibp_kv_evict", {a[1]});
  if (!gradients.check_given({{a[8], "weights_out"}}) || !check_table(a[0], a[2], &table)) return nullptr;
  const Tensor &pages = THPVariable_Unpack(a[0]), &lengths = THPVariable_Unpack(a[2]);
  if (!check_like(a[1], ScalarType::Float, "weights", pages) || !number(a[3], &page_tokens) || !number(a[4], &keep) ||
      !number(a[5], &sink) || !number(a[6], &recent) ||
      (a[7] != Py_None && !check_like(a[7], ScalarType::Int, "pages_out", pages)) ||
      (a[8] != Py_None && !check_like(a[8], ScalarType::Float, "weights_out", pages)) ||
      (a[9] != Py_None && !check_like(a[9], ScalarType::Int, "lengths_out", lengths)) || !stream_of(a[10], &stream))
    return nullptr;
  const Tensor& weights = THPVariable_Unpack(a[1]);
  const OnGpu on(gpu);
  const Tensor p = a[7] != Py_None ? THPVariable_Unpack(a[7]) : at::empty_like(pages);
  const Tensor w = a[8] != Py_None ? THPVariable_Unpack(a[8]) : at::empty_like(weights);
  const Tensor l = a[9] != Py_None ? THPVariable_Unpack(a[9]) : at::empty_like(lengths);
  for (int i = 7; i < 10; ++i) written(a[i]);
  const int status = ibp_kv_evict(&table, (uint32_t)std::min<uint64_t>(page_tokens, 0xFFFFFFFFull), keep, sink, recent,
                                  (const float*)weights.data_ptr(), (int32_t*)p.data_ptr(), (float*)w.data_ptr(),
                                  (int32_t*)l.data_ptr(), stream);
  gradients.mark({w});
  return Py_BuildValue("(iNNN)", status, THPVariable_Wrap(p), THPVariable_Wrap(w), THPVariable_Wrap(l));
  END_HANDLE_TH_ERRORS
}

// ---- libibp_kv_long ----

// Its calls, found by load_long, so that those of libibp_kv do without the library.
struct Long {
  decltype(&ibp_kv_append_rotated) append_rotated;
  decltype(&ibp_kv_outline) outline;
  decltype(&ibp_kv_select) select;
  decltype(&ibp_kv_select_workspace_bytes) select_workspace_bytes;
  decltype(&ibp_kv_attention_shared) attention_shared;
  decltype(&ibp_kv_attention_shared_workspace_bytes) attention_shared_workspace_bytes;
  bool loaded;
};
Long g_long = {};

template <class F>
bool find(void* library, const char* name, F* out) {
  *out = reinterpret_cast<F>(dlsym(library, name));
  return *out != nullptr;
}

// load_long(path)
PyObject* load_long(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 1)) return nullptr;
  const char* path = PyUnicode_AsUTF8(a[0]);
  if (!path) return nullptr;
  void* library = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  Long x = {};
  if (!library || !find(library, "ibp_kv_append_rotated", &x.append_rotated) || !find(library, "ibp_kv_outline", &x.outline) ||
      !find(library, "ibp_kv_select", &x.select) || !find(library, "ibp_kv_select_workspace_bytes", &x.select_workspace_bytes) ||
      !find(library, "ibp_kv_attention_shared", &x.attention_shared) ||
      !find(library, "ibp_kv_attention_shared_workspace_bytes", &x.attention_shared_workspace_bytes)) {
    PyErr_Format(PyExc_RuntimeError, "%s does not load: build it with `python -m lossless_bit_level_amd.build` (%s)", path, dlerror());
    return nullptr;
  }
  x.loaded = true;
  g_long = x;
  Py_RETURN_NONE;
}

bool long_loaded() {
  if (g_long.loaded) return true;
  PyErr_SetString(PyExc_RuntimeError, "libibp_kv_long.so is missing: build it with `python -m lossless_bit_level_amd.build`");
  return false;
}

// The outlines of a cache's pages.
bool check_outlines(PyObject* codes, PyObject* scales, const ibp_kv_cache& cache, ibp_kv_outlines* out) {
  if (!check(codes, ScalarType::Char, "outline codes") || !check(scales, ScalarType::Float, "outline scales")) return false;
  const Tensor &c = THPVariable_Unpack(codes), &s = THPVariable_Unpack(scales);
  if (c.dim() != 3 || (uint64_t)c.size(0) != cache.n_pages || c.size(1) != 2 || (uint64_t)c.size(2) != cache.head_dim ||
      (uint64_t)s.numel() != cache.n_pages) {
    PyErr_Format(PyExc_ValueError, "outlines must be codes [%llu, 2, %u] and as many scales", (unsigned long long)cache.n_pages,
                 cache.head_dim);
    return false;
  }
  *out = {(int8_t*)c.data_ptr(), (float*)s.data_ptr()};
  return true;
}

// Queries [n_seqs, n_new, q_heads, head_dim] of the type of `like` (null: of their own).
bool check_queries(PyObject* o, const ibp_kv_cache& cache, const ibp_kv_table& table, const Tensor* like, int64_t* n_new,
                   int64_t* q_heads, uint32_t* dtype, ibp_kv_tensor* q) {
  if (!check_type(o, "q", dtype)) return false;
  const Tensor& x = THPVariable_Unpack(o);
  *q_heads = x.size(2);
  if (table.kv_heads && (*q_heads == 0 || *q_heads % (int64_t)table.kv_heads)) {
    PyErr_SetString(PyExc_ValueError, "q_heads must be a multiple of kv_heads");
    return false;
  }
  if (!like) *n_new = x.size(1);
  const int64_t shape[4] = {(int64_t)table.n_seqs, *n_new, *q_heads, cache.head_dim};
  return check_rows(o, "q", like ? like->scalar_type() : x.scalar_type(), shape, q);
}

void written_all(PyObject* tuple) {
  if (tuple)
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(tuple); ++i) written(PyTuple_GET_ITEM(tuple, i));
}

// append_rotated(cache, pages, lengths, k, v, cos, sin, positions, q, q_out, counts,
//                interleaved, outline_codes, outline_scales, stream) -> (status, q_out)
PyObject* append_rotated(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  ibp_kv_cache cache;
  ibp_kv_table table;
  ibp_kv_tensor k, v, q, q_out;
  ibp_kv_outlines outlines;
  ibp_kv_rotation rotation;
  uint32_t dtype;
  const int32_t* counts;
  void* stream;
  c10::Device gpu(c10::kCUDA, 0);
  if (!long_loaded() || !arguments(n, 15) ||
      !same_gpu({{tensor_of_cache(a[0]), "the cache"}, {a[1], "pages"}, {a[2], "lengths"}, {a[3], "k"}, {a[4], "v"}, {a[5], "cos"},
                 {a[6], "sin"}, {a[7], "positions"}, {a[8], "q"}, {a[9], "q_out"}, {a[10], "counts"}, {a[12], "outline codes"},
                 {a[13], "outline scales"}}, &gpu))
    return nullptr;
  const Gradients gradients("ibp_kv_append_rotated", {a[8], a[5], a[6]});
  const bool queries = a[8] != Py_None, outlined = a[12] != Py_None;
  if ((queries && !gradients.check_given({{a[9], "q_out"}})) || !check_type(a[3], "k", &dtype) || !from_structure(a[0], &cache) ||
      !check_table(a[1], a[2], &table))
    return nullptr;
  const Tensor& x = THPVariable_Unpack(a[3]);
  int64_t n_new = x.size(1), q_heads = 0;
  const int64_t shape[4] = {(int64_t)table.n_seqs, n_new, (int64_t)table.kv_heads, cache.head_dim};
  if (!check_rows(a[3], "k", x.scalar_type(), shape, &k) || !check_rows(a[4], "v", x.scalar_type(), shape, &v) ||
      !check(a[5], ScalarType::Float, "cos") || !check(a[6], ScalarType::Float, "sin"))
    return nullptr;
  const Tensor &cos = THPVariable_Unpack(a[5]), &sin = THPVariable_Unpack(a[6]);
  if (cos.dim() != 2 || cos.sizes() != sin.sizes()) {
    PyErr_SetString(PyExc_ValueError, "cos and sin must be [n_positions, rotary_dim / 2]");
    return nullptr;
  }
  rotation.n_positions = (uint64_t)cos.size(0);
  rotation.rotary_dim = (uint32_t)std::min<int64_t>(2 * cos.size(1), 0x7FFFFFF0);
  const int interleaved = PyObject_IsTrue(a[11]);
  if (interleaved < 0) return nullptr;
  rotation.interleaved = (uint32_t)interleaved;
  rotation.cos = (const float*)cos.data_ptr();
  rotation.sin = (const float*)sin.data_ptr();
  rotation.positions = nullptr;
  if (a[7] != Py_None) {
    if (!check(a[7], ScalarType::Int, "positions")) return nullptr;
    const Tensor& p = THPVariable_Unpack(a[7]);
    if (p.dim() != 2 || (uint64_t)p.size(0) != table.n_seqs || p.size(1) != n_new) {
      refuse("%s must be [n_seqs, n_new]", "positions");
      return nullptr;
    }
    rotation.positions = (const int32_t*)p.data_ptr();
  }
  uint32_t q_type;
  if ((queries && !check_queries(a[8], cache, table, &x, &n_new, &q_heads, &q_type, &q)) || !check_counts(a[10], table.n_seqs, &counts) ||
      (outlined && !check_outlines(a[12], a[13], cache, &outlines)) || !stream_of(a[14], &stream))
    return nullptr;
  const int64_t q_shape[4] = {(int64_t)table.n_seqs, n_new, q_heads, cache.head_dim};
  if (!queries && a[9] != Py_None) {
    PyErr_SetString(PyExc_ValueError, "q_out without q");
    return nullptr;
  }
  if (a[9] != Py_None && !check_rows(a[9], "q_out", x.scalar_type(), q_shape, &q_out)) return nullptr;
  const OnGpu on(gpu);
  Tensor turned;
  if (queries) {
    turned = a[9] != Py_None ? THPVariable_Unpack(a[9]) : at::empty(q_shape, x.options());
    q_out = {turned.data_ptr(), turned.stride(0), turned.stride(1), turned.stride(2)};
  }
  written_all(tensors_of_cache(a[0]));
  written(a[9]);
  written(a[12]);
  written(a[13]);
  const int status = g_long.append_rotated(&cache, &table, dtype, (uint64_t)n_new, &k, &v, counts, &rotation, (uint64_t)q_heads,
                                           queries ? &q : nullptr, queries ? &q_out : nullptr, outlined ? &outlines : nullptr, stream);
  gradients.mark({turned});
  PyObject* result = Py_None;
  if (queries)
    result = THPVariable_Wrap(turned);
  else
    Py_INCREF(result);
  return Py_BuildValue("(iN)", status, result);
  END_HANDLE_TH_ERRORS
}

// outline(cache, outline_codes, outline_scales, pages, lengths, n_new, counts, stream) -> status
PyObject* outline(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  ibp_kv_cache cache;
  ibp_kv_table table;
  ibp_kv_outlines outlines;
  uint64_t n_new = 0x7FFFFFFF;  // every page that holds tokens
  const int32_t* counts;
  void* stream;
  c10::Device gpu(c10::kCUDA, 0);
  if (!long_loaded() || !arguments(n, 8) ||
      !same_gpu({{tensor_of_cache(a[0]), "the cache"}, {a[1], "outline codes"}, {a[2], "outline scales"}, {a[3], "pages"},
                 {a[4], "lengths"}, {a[6], "counts"}}, &gpu) ||
      !from_structure(a[0], &cache) || !check_outlines(a[1], a[2], cache, &outlines) || !check_table(a[3], a[4], &table) ||
      (a[5] != Py_None && !number(a[5], &n_new)) || !check_counts(a[6], table.n_seqs, &counts) || !stream_of(a[7], &stream))
    return nullptr;
  const OnGpu on(gpu);
  written(a[1]);
  written(a[2]);
  return PyLong_FromLong(g_long.outline(&cache, &outlines, &table, n_new, counts, stream));
  END_HANDLE_TH_ERRORS
}

bool check_shape(PyObject* o, ScalarType type, const char* name, at::IntArrayRef shape) {
  if (!check(o, type, name)) return false;
  if (THPVariable_Unpack(o).sizes() == shape) return true;
  refuse("%s has the wrong shape", name);
  return false;
}

// select(cache, outline_codes, outline_scales, pages, lengths, q, keep, sink, recent, counts,
//        pages_out, lengths_out, places_out, workspace, stream) -> (status, pages, lengths, places)
PyObject* select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  ibp_kv_cache cache;
  ibp_kv_table table;
  ibp_kv_tensor q;
  ibp_kv_outlines outlines;
  uint32_t dtype;
  uint64_t keep, sink, recent;
  int64_t n_new, q_heads;
  const int32_t* counts;
  void* stream;
  c10::Device gpu(c10::kCUDA, 0);
  if (!long_loaded() || !arguments(n, 15) ||
      !same_gpu({{tensor_of_cache(a[0]), "the cache"}, {a[1], "outline codes"}, {a[2], "outline scales"}, {a[3], "pages"},
                 {a[4], "lengths"}, {a[5], "q"}, {a[9], "counts"}, {a[10], "pages_out"}, {a[11], "lengths_out"}, {a[12], "places_out"},
                 {a[13], "workspace"}}, &gpu) ||
      !from_structure(a[0], &cache) || !check_outlines(a[1], a[2], cache, &outlines) || !check_table(a[3], a[4], &table) ||
      !check_queries(a[5], cache, table, nullptr, &n_new, &q_heads, &dtype, &q) || !number(a[6], &keep) || !number(a[7], &sink) ||
      !number(a[8], &recent) || !check_counts(a[9], table.n_seqs, &counts))
    return nullptr;
  if (keep > 0x7FFFFFFF) {
    PyErr_SetString(PyExc_ValueError, "keep_pages is past 2^31");
    return nullptr;
  }
  const int64_t shape[3] = {(int64_t)table.n_seqs, (int64_t)table.kv_heads, (int64_t)keep};
  if ((a[10] != Py_None && !check_shape(a[10], ScalarType::Int, "pages_out", shape)) ||
      (a[11] != Py_None && !check_shape(a[11], ScalarType::Int, "lengths_out", at::IntArrayRef(shape, 2))) ||
      (a[12] != Py_None && !check_shape(a[12], ScalarType::Int, "places_out", shape)) ||
      (a[13] != Py_None && !check(a[13], ScalarType::Byte, "workspace")) || !stream_of(a[14], &stream))
    return nullptr;
  const OnGpu on(gpu);
  const auto options = THPVariable_Unpack(a[3]).options();
  const Tensor p = a[10] != Py_None ? THPVariable_Unpack(a[10]) : at::empty(shape, options);
  const Tensor l = a[11] != Py_None ? THPVariable_Unpack(a[11]) : at::empty(at::IntArrayRef(shape, 2), options);
  const Tensor w = a[12] != Py_None ? THPVariable_Unpack(a[12]) : at::empty(shape, options);
  Tensor workspace;
  if (a[13] != Py_None)
    workspace = THPVariable_Unpack(a[13]);
  else if (const uint64_t bytes = g_long.select_workspace_bytes(&cache, &table))
    workspace = at::empty({(int64_t)bytes}, options.dtype(at::kByte));
  for (int i = 10; i < 13; ++i) written(a[i]);
  const int status = g_long.select(&cache, &outlines, &table, dtype, (uint64_t)q_heads, (uint64_t)n_new, &q, counts, keep, sink, recent,
                                   (int32_t*)p.data_ptr(), (int32_t*)l.data_ptr(), (int32_t*)w.data_ptr(),
                                   workspace.defined() ? workspace.data_ptr() : nullptr,
                                   workspace.defined() ? (uint64_t)workspace.numel() : 0, stream);
  return Py_BuildValue("(iNNN)", status, THPVariable_Wrap(p), THPVariable_Wrap(l), THPVariable_Wrap(w));
  END_HANDLE_TH_ERRORS
}

// attention_shared(cache, prefix_pages, prefix_lengths, pages, lengths, q, scale, counts, out,
//                  workspace, stream) -> (status, out)
PyObject* attention_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  ibp_kv_cache cache;
  ibp_kv_table table;
  ibp_kv_tensor q, o;
  uint32_t dtype;
  int64_t n_new, q_heads;
  const int32_t* counts;
  void* stream;
  c10::Device gpu(c10::kCUDA, 0);
  if (!long_loaded() || !arguments(n, 11) ||
      !same_gpu({{tensor_of_cache(a[0]), "the cache"}, {a[1], "prefix_pages"}, {a[2], "prefix_lengths"}, {a[3], "pages"},
                 {a[4], "lengths"}, {a[5], "q"}, {a[7], "counts"}, {a[8], "out"}, {a[9], "workspace"}}, &gpu))
    return nullptr;
  const Gradients gradients("ibp_kv_attention_shared", {a[5]});
  if (!gradients.check_given({{a[8], "out"}}) || !from_structure(a[0], &cache) || !check_table(a[3], a[4], &table) ||
      !check(a[1], ScalarType::Int, "prefix_pages") || !check(a[2], ScalarType::Int, "prefix_lengths"))
    return nullptr;
  const Tensor &pp = THPVariable_Unpack(a[1]), &pl = THPVariable_Unpack(a[2]);
  if (pp.dim() != 2 || pl.dim() != 1 || (uint64_t)pp.size(0) != table.kv_heads || (uint64_t)pl.size(0) != table.kv_heads) {
    PyErr_SetString(PyExc_ValueError, "prefix_pages must be [kv_heads, max_pages] and prefix_lengths [kv_heads]");
    return nullptr;
  }
  const ibp_kv_table prefix = {1, table.kv_heads, (uint64_t)pp.size(1), (const int32_t*)pp.data_ptr(), (const int32_t*)pl.data_ptr()};
  if (!check_queries(a[5], cache, table, nullptr, &n_new, &q_heads, &dtype, &q)) return nullptr;
  const Tensor& x = THPVariable_Unpack(a[5]);
  float scale = 1.f / std::sqrt((float)cache.head_dim);
  if (a[6] != Py_None) {
    scale = (float)PyFloat_AsDouble(a[6]);
    if (PyErr_Occurred()) return nullptr;
  }
  if (!check_counts(a[7], table.n_seqs, &counts) || (a[8] != Py_None && !check_rows(a[8], "out", x.scalar_type(), x.sizes(), &o)) ||
      (a[9] != Py_None && !check(a[9], ScalarType::Byte, "workspace")) || !stream_of(a[10], &stream))
    return nullptr;
  const OnGpu on(gpu);
  const Tensor out = a[8] != Py_None ? THPVariable_Unpack(a[8]) : at::empty(x.sizes(), x.options());
  if (a[8] == Py_None) o = {out.data_ptr(), out.stride(0), out.stride(1), out.stride(2)};
  Tensor workspace;
  if (a[9] != Py_None)
    workspace = THPVariable_Unpack(a[9]);
  else if (const uint64_t bytes = g_long.attention_shared_workspace_bytes(&cache, &prefix, &table, (uint64_t)q_heads, (uint64_t)n_new))
    workspace = at::empty({(int64_t)bytes}, x.options().dtype(at::kByte));
  written(a[8]);
  const int status = g_long.attention_shared(&cache, &prefix, &table, dtype, (uint64_t)q_heads, (uint64_t)n_new, &q, &o, counts, scale,
                                             workspace.defined() ? workspace.data_ptr() : nullptr,
                                             workspace.defined() ? (uint64_t)workspace.numel() : 0, stream);
  gradients.mark({out});
  return Py_BuildValue("(iN)", status, THPVariable_Wrap(out));
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"set_cache", (PyCFunction)(void (*)(void))set_cache, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {"attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, nullptr},
    {"evict", (PyCFunction)(void (*)(void))evict, METH_FASTCALL, nullptr},
    {"load_long", (PyCFunction)(void (*)(void))load_long, METH_FASTCALL, nullptr},
    {"append_rotated", (PyCFunction)(void (*)(void))append_rotated, METH_FASTCALL, nullptr},
    {"outline", (PyCFunction)(void (*)(void))outline, METH_FASTCALL, nullptr},
    {"select", (PyCFunction)(void (*)(void))select, METH_FASTCALL, nullptr},
    {"attention_shared", (PyCFunction)(void (*)(void))attention_shared, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ibp_kv", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ibp_kv(void) { return PyModule_Create(&module); }
