// attention_binding.cpp -- Python entry points of the calls that stand between
// two launches of a decode step (include/nf4_attention.h): argument checks,
// output allocation and the C call.
//
// Marshalling only, as in the ctypes half of the binding; compiled because
// these calls are made for every layer of every token: one call looks at ten
// tensors, which costs 10 us through Python attributes and well under 1 us
// here, next to a launch of 2 us and a kernel of 3 us.
#include "binding.h"

namespace nf4_binding {

PyObject* g_error = nullptr;
PyObject* g_memory = nullptr;

namespace {

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
    return attention_outputs(
        "nf4_prefix_attention", q, AttentionOutputs{v[9], v[10], v[11], v[12]}, on, &a,
        [&] { return nf4_prefix_attention_workspace_size(&a); },
        [&](void* scratch, size_t bytes) { return nf4_prefix_attention(&a, scratch, bytes, on.stream()); });
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
}  // namespace nf4_binding

PyMODINIT_FUNC PyInit__attention(void) {
  PyObject* const m = PyModule_Create(&nf4_binding::kModule);
  if (m && PyModule_AddFunctions(m, nf4_binding::kDecodingMethods) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
