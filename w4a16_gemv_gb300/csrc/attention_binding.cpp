// attention_binding.cpp -- Python entry points of the calls that stand between
// two launches of a decode step (include/nf4_attention.h): argument checks,
// output allocation and the C call.
//
// Marshalling only, as in the ctypes half of the binding; compiled because
// these calls are made for every layer of every token: one call looks at ten
// tensors, which costs 10 us through Python attributes and well under 1 us
// here, next to a launch of 2 us and a kernel of 3 us.
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

#include "nf4_attention.h"

namespace {

PyObject* g_error = nullptr;   // the package's NF4Error(status, where)
PyObject* g_memory = nullptr;  // torch.OutOfMemoryError

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

// ---------------------------------------------------------------------------

struct QkInputs {
  PyObject *q, *k, *positions, *cos_sin, *q_weight, *k_weight, *eps, *interleaved, *q_out, *k_out;
};

// The fields of nf4_qk_norm_rope_args. Outputs that are not given are made.
// With `append` there is no k_out.
void fill_qk(const QkInputs& in, const Launch& on, bool append, nf4_qk_norm_rope_args* a, at::Tensor* q_out,
             at::Tensor* k_out) {
  const at::Tensor& k = tensor(in.k, "k");
  if (k.dim() != 3) throw ValueError("k must have shape [tokens, heads, head_dim], got " + text(k.sizes()));
  const at::ScalarType type = k.scalar_type();
  const int64_t tokens = k.size(0), k_heads = k.size(1), dim = k.size(2);
  const c10::DeviceIndex dev = on.device();
  *a = nf4_qk_norm_rope_args{};
  a->dtype = dtype_code(type, "q and k must be bf16, fp16 or fp32");
  a->tokens = tokens;
  a->head_dim = dim;
  if (given(in.q)) {
    const at::Tensor& q = tensor(in.q, "q");
    if (q.dim() != 3) throw ValueError("q must have shape [tokens, heads, head_dim], got " + text(q.sizes()));
    const int64_t shape[3] = {tokens, q.size(1), dim};
    check(q, "q", type, shape, dev, false);
    if (given(in.q_out)) {
      *q_out = tensor(in.q_out, "q_out");
      check(*q_out, "q_out", type, shape, dev, false);
    } else {
      *q_out = on.empty(shape, type);
    }
    a->q = q.data_ptr();
    a->q_token_stride = q.stride(0);
    a->q_head_stride = q.stride(1);
    a->q_out = q_out->data_ptr();
    a->q_out_token_stride = q_out->stride(0);
    a->q_out_head_stride = q_out->stride(1);
    a->q_heads = shape[1];
  }
  check(k, "k", type, k.sizes(), dev, false);
  a->k = k.data_ptr();
  a->k_token_stride = k.stride(0);
  a->k_head_stride = k.stride(1);
  a->k_heads = k_heads;
  if (!append) {
    if (given(in.k_out)) {
      *k_out = tensor(in.k_out, "k_out");
      check(*k_out, "k_out", type, k.sizes(), dev, false);
    } else {
      *k_out = on.empty(k.sizes(), type);
    }
    a->k_out = k_out->data_ptr();
    a->k_out_token_stride = k_out->stride(0);
    a->k_out_head_stride = k_out->stride(1);
  }
  const at::Tensor& cs = tensor(in.cos_sin, "cos_sin");
  if (cs.dim() != 3 || cs.size(2) != 2)
    throw ValueError("cos_sin must have shape [positions, rot_dim / 2, 2], got " + text(cs.sizes()));
  a->positions = static_cast<const int64_t*>(flat(in.positions, "positions", at::kLong, {tokens}, dev));
  a->cos_sin = static_cast<const float*>(flat(in.cos_sin, "cos_sin", at::kFloat, cs.sizes(), dev));
  a->max_positions = cs.size(0);
  a->rot_dim = 2 * cs.size(1);
  a->interleaved = truth(in.interleaved) ? 1 : 0;
  if (given(in.q_weight)) a->q_weight = flat(in.q_weight, "q_weight", type, {dim}, dev);
  if (given(in.k_weight)) a->k_weight = flat(in.k_weight, "k_weight", type, {dim}, dev);
  a->eps = real(in.eps, 1e-6, "eps");
}

PyObject* py_qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const kNames[] = {"q",   "k",           "positions", "cos_sin", "q_weight", "k_weight",
                                         "eps", "interleaved", "q_out",     "k_out",   "stream"};
    PyObject* v[11];
    parse("nf4_qk_norm_rope", kNames, 11, 4, args, nargs, kwnames, v);
    if (!given(v[0])) throw TypeError("q must be a tensor");
    const Launch on(tensor(v[1], "k"), v[10], "k");
    nf4_qk_norm_rope_args a;
    at::Tensor q_out, k_out;
    fill_qk(QkInputs{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8], v[9]}, on, false, &a, &q_out, &k_out);
    const nf4_status st = unlocked([&] { return nf4_qk_norm_rope(&a, on.stream()); });
    if (st != NF4_OK) raise_status(st, "nf4_qk_norm_rope");
    PyObject* q = given(v[8]) ? Py_NewRef(v[8]) : THPVariable_Wrap(q_out);
    PyObject* k = given(v[9]) ? Py_NewRef(v[9]) : THPVariable_Wrap(k_out);
    PyObject* r = q && k ? PyTuple_Pack(2, q, k) : nullptr;
    Py_XDECREF(q);
    Py_XDECREF(k);
    return r;
  });
}

PyObject* py_kv_append(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const kNames[] = {"k_cache", "v_cache",  "slots",    "k",   "v",           "positions", "cos_sin",
                                         "q",       "q_weight", "k_weight", "eps", "interleaved", "q_out",     "stream"};
    PyObject* v[14];
    parse("nf4_kv_append", kNames, 14, 7, args, nargs, kwnames, v);
    const at::Tensor& k = tensor(v[3], "k");
    const Launch on(k, v[13], "k");
    nf4_kv_append_args a;
    at::Tensor q_out, none;
    fill_qk(QkInputs{v[7], v[3], v[5], v[6], v[8], v[9], v[10], v[11], v[12], nullptr}, on, true, &a.qk, &q_out, &none);
    const at::ScalarType type = k.scalar_type();
    const c10::DeviceIndex dev = on.device();
    const at::Tensor& kc = tensor(v[0], "k_cache");
    const at::Tensor& vc = tensor(v[1], "v_cache");
    if (kc.dim() != 4) throw ValueError("k_cache must have shape [pages, page_size, heads, head_dim], got " + text(kc.sizes()));
    const int64_t shape[4] = {kc.size(0), kc.size(1), k.size(1), k.size(2)};
    check(kc, "k_cache", type, shape, dev, false);
    check(vc, "v_cache", type, shape, dev, false);
    const at::Tensor& val = tensor(v[4], "v");
    check(val, "v", type, k.sizes(), dev, false);
    a.v = val.data_ptr();
    a.v_token_stride = val.stride(0);
    a.v_head_stride = val.stride(1);
    a.slots = static_cast<const int64_t*>(flat(v[2], "slots", at::kLong, {k.size(0)}, dev));
    a.k_cache = kc.data_ptr();
    a.k_page_stride = kc.stride(0);
    a.k_slot_stride = kc.stride(1);
    a.k_head_stride = kc.stride(2);
    a.v_cache = vc.data_ptr();
    a.v_page_stride = vc.stride(0);
    a.v_slot_stride = vc.stride(1);
    a.v_cache_head_stride = vc.stride(2);
    a.num_pages = shape[0];
    a.page_size = shape[1];
    const nf4_status st = unlocked([&] { return nf4_kv_append(&a, on.stream()); });
    if (st != NF4_OK) raise_status(st, "nf4_kv_append");
    if (!given(v[7])) Py_RETURN_NONE;
    return given(v[12]) ? Py_NewRef(v[12]) : THPVariable_Wrap(q_out);
  });
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

PyObject* py_prefix_attention(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const kNames[] = {"q",           "k_cache", "v_cache", "prefix_pages", "prefix_len", "suffix_pages",
                                         "suffix_lens", "cu_q",    "scale",   "out",          "return_lse", "lse",
                                         "workspace",   "stream"};
    PyObject* v[14];
    parse("nf4_prefix_attention", kNames, 14, 7, args, nargs, kwnames, v);
    const at::Tensor& q = tensor(v[0], "q");
    const Launch on(q, v[13], "q");
    const c10::DeviceIndex dev = on.device();
    nf4_prefix_attention_args a;
    fill_attention(AttentionInputs{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8]}, dev, &a);
    at::Tensor out, lse, ws;
    if (given(v[9])) {
      out = tensor(v[9], "out");
      check(out, "out", q.scalar_type(), q.sizes(), dev, false);
    } else {
      out = on.empty(q.sizes(), q.scalar_type());
    }
    a.out = out.data_ptr();
    a.out_token_stride = out.stride(0);
    a.out_head_stride = out.stride(1);
    const bool want_lse = truth(v[10]);
    if (given(v[11]))
      a.lse = static_cast<float*>(flat(v[11], "lse", at::kFloat, {a.tokens, a.q_heads}, dev));
    else if (want_lse) {
      lse = on.empty({a.tokens, a.q_heads}, at::kFloat);
      a.lse = lse.data_ptr<float>();
    }
    void* scratch = nullptr;
    size_t bytes = 0;
    if (given(v[12])) {
      ws = tensor(v[12], "workspace");
      if (!ws.is_cuda() || !ws.is_contiguous()) throw ValueError("workspace must be a contiguous CUDA tensor");
      if (ws.get_device() != dev) throw ValueError("workspace must be on the same device as the others");
      scratch = ws.data_ptr();
      bytes = ws.nbytes();
    } else if ((bytes = nf4_prefix_attention_workspace_size(&a)) > 0) {
      ws = on.empty({int64_t(bytes)}, at::kByte);
      scratch = ws.data_ptr();
    }
    const nf4_status st = unlocked([&] { return nf4_prefix_attention(&a, scratch, bytes, on.stream()); });
    if (st != NF4_OK) raise_status(st, "nf4_prefix_attention");
    PyObject* o = given(v[9]) ? Py_NewRef(v[9]) : THPVariable_Wrap(out);
    if (!want_lse) return o;
    PyObject* l = given(v[11]) ? Py_NewRef(v[11]) : THPVariable_Wrap(lse);
    PyObject* r = o && l ? PyTuple_Pack(2, o, l) : nullptr;
    Py_XDECREF(o);
    Py_XDECREF(l);
    return r;
  });
}

PyObject* py_workspace_size(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const kNames[] = {"q",           "k_cache", "v_cache", "prefix_pages", "prefix_len", "suffix_pages",
                                         "suffix_lens", "cu_q",    "scale"};
    PyObject* v[9];
    parse("nf4_prefix_attention_workspace_size", kNames, 9, 7, args, nargs, kwnames, v);
    const Launch on(tensor(v[0], "q"), nullptr, "q");
    nf4_prefix_attention_args a;
    fill_attention(AttentionInputs{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8]}, on.device(), &a);
    return PyLong_FromSize_t(nf4_prefix_attention_workspace_size(&a));
  });
}

PyObject* py_set_errors(PyObject*, PyObject* classes) {
  PyObject *error, *memory;
  if (!PyArg_ParseTuple(classes, "OO", &error, &memory)) return nullptr;
  Py_XSETREF(g_error, Py_NewRef(error));
  Py_XSETREF(g_memory, Py_NewRef(memory));
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef kMethods[] = {
    {"nf4_qk_norm_rope", fast(py_qk_norm_rope), METH_FASTCALL | METH_KEYWORDS,
     "nf4_qk_norm_rope(q, k, positions, cos_sin, q_weight=None, k_weight=None, eps=1e-06, interleaved=False, q_out=None, "
     "k_out=None, stream=None)\n--\n\n"
     "Norm (where a weight is given) and rotation of q [tokens, q_heads, dim] and k [tokens, k_heads, dim];\n"
     "positions int64 [tokens], cos_sin as from nf4_rope_table. Returns (q_out, k_out), new tensors unless given\n"
     "(an output may be its input)."},
    {"nf4_kv_append", fast(py_kv_append), METH_FASTCALL | METH_KEYWORDS,
     "nf4_kv_append(k_cache, v_cache, slots, k, v, positions, cos_sin, q=None, q_weight=None, k_weight=None, eps=1e-06, "
     "interleaved=False, q_out=None, stream=None)\n--\n\n"
     "Writes the normed and rotated k and the v of each token to slot slots[token] (int64, page * page_size +\n"
     "offset; negative: nowhere) of the paged caches [pages, page_size, kv_heads, dim]. With q, its rows are normed\n"
     "and rotated in the same launch and returned."},
    {"nf4_prefix_attention", fast(py_prefix_attention), METH_FASTCALL | METH_KEYWORDS,
     "nf4_prefix_attention(q, k_cache, v_cache, prefix_pages, prefix_len, suffix_pages, suffix_lens, cu_q=None, scale=None, "
     "out=None, return_lse=False, lse=None, workspace=None, stream=None)\n--\n\n"
     "Attention of q [tokens, q_heads, dim] over a paged cache [pages, page_size, kv_heads, dim]: the prefix_len\n"
     "keys on prefix_pages (int32) that the whole batch shares, then each sequence's own suffix_lens (int32 [batch])\n"
     "keys on its row of suffix_pages (int32 [batch, width]), causal among the sequence's tokens cu_q[b] ..\n"
     "cu_q[b + 1] - 1 (int32 [batch + 1]; None: one token each). Returns out, or (out, lse) with return_lse. The\n"
     "scale defaults to 1 / sqrt(dim); the workspace is allocated unless given."},
    {"nf4_prefix_attention_workspace_size", fast(py_workspace_size), METH_FASTCALL | METH_KEYWORDS,
     "nf4_prefix_attention_workspace_size(q, k_cache, v_cache, prefix_pages, prefix_len, suffix_pages, suffix_lens, cu_q=None, "
     "scale=None)\n--\n\nBytes of workspace that nf4_prefix_attention needs for tensors of these shapes."},
    {"_set_errors", py_set_errors, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_attention", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attention(void) { return PyModule_Create(&kModule); }
