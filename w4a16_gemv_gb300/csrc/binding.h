// binding.h -- what the compiled entry points share (attention_binding.cpp,
// decoding_binding.cpp): arguments, checks of tensors, the call's device and
// stream, and errors.
#pragma once

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>
#include <string>

#include "nf4_decoding.h"

namespace nf4_binding {

extern PyObject* g_error;                 // the package's NF4Error(status, where)
extern PyObject* g_memory;                // torch.OutOfMemoryError
extern PyMethodDef kDecodingMethods[];    // decoding_binding.cpp

namespace {

struct TypeError : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct ValueError : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct PythonError {};  // a Python exception is already set

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

// Positional and keyword arguments into `out` (null where absent).
void parse(const char* fn, const char* const* names, int n, int required, PyObject* const* args, Py_ssize_t nargs,
           PyObject* kwnames, PyObject** out) {
  if (nargs > n) throw TypeError(std::string(fn) + "() takes at most " + std::to_string(n) + " arguments");
  for (int i = 0; i < n; ++i) out[i] = i < nargs ? args[i] : nullptr;
  const Py_ssize_t kw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
  for (Py_ssize_t k = 0; k < kw; ++k) {
    PyObject* key = PyTuple_GET_ITEM(kwnames, k);
    int at = 0;
    while (at < n && PyUnicode_CompareWithASCIIString(key, names[at]) != 0) ++at;
    if (at == n) {
      const char* s = PyUnicode_AsUTF8(key);
      if (!s) throw PythonError();
      throw TypeError(std::string(fn) + "() got an unexpected keyword argument '" + s + "'");
    }
    if (out[at]) throw TypeError(std::string(fn) + "() got multiple values for argument '" + names[at] + "'");
    out[at] = args[nargs + k];
  }
  for (int i = 0; i < required; ++i)
    if (!out[i]) throw TypeError(std::string(fn) + "() missing argument '" + names[i] + "'");
}

bool given(PyObject* o) { return o && o != Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw TypeError(std::string(name) + " must be a tensor, got " + Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw TypeError(std::string(name) + " must be an integer");
  }
  return v;
}

double real(PyObject* o, double otherwise, const char* name) {
  if (!given(o)) return otherwise;
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw TypeError(std::string(name) + " must be a number");
  }
  return v;
}

bool truth(PyObject* o) {
  if (!o) return false;
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError();
  return v != 0;
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat: return "torch.float32";
    case at::kLong: return "torch.int64";
    case at::kInt: return "torch.int32";
    default: return c10::toString(t);
  }
}

// A CUDA tensor of this type and shape on the call's device, contiguous in its
// last dimension (throughout, with `whole`).
void check(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::DeviceIndex dev,
           bool whole) {
  if (t.scalar_type() != type)
    throw TypeError(std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
  if (t.sizes() != shape) throw ValueError(std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
  if (!t.is_cuda()) throw ValueError(std::string(name) + " must be a CUDA tensor");
  if (t.get_device() != dev) throw ValueError(std::string(name) + " must be on the same device as the others");
  if (whole ? !t.is_contiguous() : t.stride(-1) != 1 && shape.back() > 1)
    throw ValueError(std::string(name) + (whole ? " must be contiguous" : " must be contiguous in its last dimension"));
}
void* flat(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::DeviceIndex dev) {
  const at::Tensor& t = tensor(o, name);
  check(t, name, type, shape, dev, true);
  return t.data_ptr();
}

int64_t dtype_code(at::ScalarType t, const char* message) {
  if (t == at::kBFloat16) return NF4_BF16;
  if (t == at::kHalf) return NF4_FP16;
  if (t == at::kFloat) return NF4_F32;
  throw TypeError(message);
}

// The call's device, made current, and its stream: the current one, or the
// `stream` argument (a torch.cuda.Stream or a handle). Memory that the call
// allocates for another stream than the current one is kept from reuse until
// that stream is done with it.
class Launch {
 public:
  Launch(const at::Tensor& t, PyObject* stream, const char* name) : dev_(0) {
    if (!t.is_cuda()) throw ValueError(std::string(name) + " must be a CUDA tensor");
    dev_ = t.get_device();
    guard_.set_index(dev_);
    if (given(stream)) {
      PyObject* handle = PyObject_HasAttrString(stream, "cuda_stream") ? PyObject_GetAttrString(stream, "cuda_stream")
                                                                       : Py_NewRef(stream);
      if (!handle) throw PythonError();
      stream_ = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(handle));
      Py_DECREF(handle);
      if (PyErr_Occurred()) throw PythonError();
      other_ = true;
    } else {
      stream_ = c10::cuda::getCurrentCUDAStream(dev_).stream();
    }
  }
  // (Through the dispatcher an allocation costs 1.3 us instead of 0.8.)
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    at::Tensor t = at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, dev_), std::nullopt);
    if (other_ && t.numel() > 0) t.record_stream(c10::cuda::getStreamFromExternal(stream_, dev_).unwrap());
    return t;
  }
  c10::DeviceIndex device() const { return dev_; }
  nf4_stream_t stream() const { return reinterpret_cast<nf4_stream_t>(stream_); }

 private:
  c10::DeviceIndex dev_;
  c10::cuda::OptionalCUDAGuard guard_;
  cudaStream_t stream_ = nullptr;
  bool other_ = false;
};

// A C call, without the interpreter's lock: a launch waits while its stream's queue
// is full, and what it waits for may need another Python thread.
template <typename F>
nf4_status unlocked(F&& call) {
  PyThreadState* const thread = PyEval_SaveThread();
  const nf4_status st = call();
  PyEval_RestoreThread(thread);
  return st;
}

void raise_status(nf4_status status, const char* where) {
  PyObject* e = PyObject_CallFunction(g_error, "is", int(status), where);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw PythonError();
}

// Runs an entry point; no C++ exception leaves it.
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const PythonError&) {
  } catch (const TypeError& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const ValueError& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::bad_alloc&) {
    PyErr_NoMemory();
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_memory ? g_memory : PyExc_MemoryError, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

struct AttentionInputs {
  PyObject *q, *k_cache, *v_cache, *prefix_pages, *prefix_len, *suffix_pages, *suffix_lens, *cu_q, *scale;
};

void fill_attention(const AttentionInputs& in, c10::DeviceIndex dev, nf4_prefix_attention_args* a) {
  const at::Tensor& q = tensor(in.q, "q");
  const at::Tensor& kc = tensor(in.k_cache, "k_cache");
  const at::Tensor& vc = tensor(in.v_cache, "v_cache");
  const at::Tensor& pp = tensor(in.prefix_pages, "prefix_pages");
  const at::Tensor& sp = tensor(in.suffix_pages, "suffix_pages");
  const at::ScalarType type = q.scalar_type();
  if (q.dim() != 3) throw ValueError("q must have shape [tokens, heads, head_dim], got " + text(q.sizes()));
  if (kc.dim() != 4 || kc.size(3) != q.size(2))
    throw ValueError("k_cache must have shape [pages, page_size, heads, " + std::to_string(q.size(2)) + "], got " +
                     text(kc.sizes()));
  if (sp.dim() != 2) throw ValueError("suffix_pages must have shape [batch, width], got " + text(sp.sizes()));
  *a = nf4_prefix_attention_args{};
  a->dtype = dtype_code(type, "q must be bf16 or fp16");
  a->tokens = q.size(0);
  a->q_heads = q.size(1);
  a->head_dim = q.size(2);
  a->num_pages = kc.size(0);
  a->page_size = kc.size(1);
  a->k_heads = kc.size(2);
  a->batch = sp.size(0);
  a->suffix_pages_width = sp.size(1);
  a->prefix_len = integer(in.prefix_len, "prefix_len");
  if (pp.dim() != 1 || a->prefix_len > pp.size(0) * a->page_size)
    throw ValueError("prefix_pages of shape " + text(pp.sizes()) + " with pages of " + std::to_string(a->page_size) +
                     " cannot hold prefix_len " + std::to_string(a->prefix_len));
  check(q, "q", type, q.sizes(), dev, false);
  check(kc, "k_cache", type, kc.sizes(), dev, false);
  check(vc, "v_cache", type, kc.sizes(), dev, false);
  check(sp, "suffix_pages", at::kInt, sp.sizes(), dev, false);
  a->q = q.data_ptr();
  a->q_token_stride = q.stride(0);
  a->q_head_stride = q.stride(1);
  a->k_cache = kc.data_ptr();
  a->k_page_stride = kc.stride(0);
  a->k_slot_stride = kc.stride(1);
  a->k_head_stride = kc.stride(2);
  a->v_cache = vc.data_ptr();
  a->v_page_stride = vc.stride(0);
  a->v_slot_stride = vc.stride(1);
  a->v_head_stride = vc.stride(2);
  a->prefix_pages = static_cast<const int32_t*>(flat(in.prefix_pages, "prefix_pages", at::kInt, pp.sizes(), dev));
  a->suffix_pages = static_cast<const int32_t*>(sp.data_ptr());
  a->suffix_pages_stride = sp.stride(0);
  a->suffix_lens = static_cast<const int32_t*>(flat(in.suffix_lens, "suffix_lens", at::kInt, {a->batch}, dev));
  if (given(in.cu_q)) a->cu_q = static_cast<const int32_t*>(flat(in.cu_q, "cu_q", at::kInt, {a->batch + 1}, dev));
  a->scale = given(in.scale) ? real(in.scale, 0.0, "scale") : 1.0 / std::sqrt(double(a->head_dim));
}

struct AttentionOutputs {
  PyObject *out, *return_lse, *lse, *workspace;
};

// The outputs and the workspace of an attention call (made unless given), the call, and what it returns.
template <typename Size, typename Call>
PyObject* attention_outputs(const char* where, const at::Tensor& q, const AttentionOutputs& o, const Launch& on,
                            nf4_prefix_attention_args* a, Size&& size, Call&& call) {
  at::Tensor out, lse, ws;
  if (given(o.out)) {
    out = tensor(o.out, "out");
    check(out, "out", q.scalar_type(), q.sizes(), on.device(), false);
  } else {
    out = on.empty(q.sizes(), q.scalar_type());
  }
  a->out = out.data_ptr();
  a->out_token_stride = out.stride(0);
  a->out_head_stride = out.stride(1);
  const bool want_lse = truth(o.return_lse);
  if (given(o.lse))
    a->lse = static_cast<float*>(flat(o.lse, "lse", at::kFloat, {a->tokens, a->q_heads}, on.device()));
  else if (want_lse) {
    lse = on.empty({a->tokens, a->q_heads}, at::kFloat);
    a->lse = lse.data_ptr<float>();
  }
  void* scratch = nullptr;
  size_t bytes = 0;
  if (given(o.workspace)) {
    ws = tensor(o.workspace, "workspace");
    if (!ws.is_cuda() || !ws.is_contiguous()) throw ValueError("workspace must be a contiguous CUDA tensor");
    if (ws.get_device() != on.device()) throw ValueError("workspace must be on the same device as the others");
    scratch = ws.data_ptr();
    bytes = ws.nbytes();
  } else if ((bytes = size()) > 0) {
    ws = on.empty({int64_t(bytes)}, at::kByte);
    scratch = ws.data_ptr();
  }
  const nf4_status st = unlocked([&] { return call(scratch, bytes); });
  if (st != NF4_OK) raise_status(st, where);
  PyObject* y = given(o.out) ? Py_NewRef(o.out) : THPVariable_Wrap(out);
  if (!want_lse) return y;
  PyObject* l = given(o.lse) ? Py_NewRef(o.lse) : THPVariable_Wrap(lse);
  PyObject* r = y && l ? PyTuple_Pack(2, y, l) : nullptr;
  Py_XDECREF(y);
  Py_XDECREF(l);
  return r;
}

}  // namespace
}  // namespace nf4_binding
