// The binding of libibp_kv's calls to torch tensors: checks of the arguments,
// tensors for the results, and the call of the C ABI (include/ibp_kv.h).  Its
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

#include <cmath>
#include <cstring>
#include <initializer_list>
#include <memory>
#include <vector>

#include "ibp_kv.h"

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
               type == ScalarType::Int ? "int32" : type == ScalarType::Float ? "float32" : "uint8");
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

PyMethodDef methods[] = {
    {"set_cache", (PyCFunction)(void (*)(void))set_cache, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {"attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, nullptr},
    {"evict", (PyCFunction)(void (*)(void))evict, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ibp_kv", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ibp_kv(void) { return PyModule_Create(&module); }
