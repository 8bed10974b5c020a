// decoding_binding.cpp -- Python entry points of include/nf4_decoding.h:
// argument checks, output allocation and the C call, as in
// attention_binding.cpp.
#include "binding.h"

namespace nf4_binding {
namespace {

// A tensor of this type and number of dimensions.
const at::Tensor& shaped(PyObject* o, const char* name, int64_t dims, const char* shape) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != dims) throw ValueError(std::string(name) + " must have shape " + shape + ", got " + text(t.sizes()));
  return t;
}

// Outputs: the given tensors, or new ones; those of one type share an allocation (one takes 0.8 us, a call of four
// or five small outputs 7 to 8). Two passes: add() for each, then get() in the same order.
class Outputs {
 public:
  explicit Outputs(const Launch& on) : on_(on) {}
  void add(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
    Part& p = parts_[n_++];
    p.type = type;
    for (const int64_t s : shape) p.shape[p.dims++] = s;
    if (given(o)) {
      p.given = tensor(o, name);
      check(p.given, name, type, shape, on_.device(), true);
    } else {
      p.at = total_[type == at::kLong];
      total_[type == at::kLong] += p.numel();
    }
  }
  at::Tensor get() {
    Part& p = parts_[next_++];
    if (p.given.defined()) return p.given;
    at::Tensor& whole = whole_[p.type == at::kLong];
    if (!whole.defined()) whole = on_.empty({total_[p.type == at::kLong]}, p.type);
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(), whole.dtype());
    t.unsafeGetTensorImpl()->set_sizes_contiguous(at::IntArrayRef(p.shape, size_t(p.dims)));
    t.unsafeGetTensorImpl()->set_storage_offset(p.at);
    return t;
  }

 private:
  struct Part {
    at::ScalarType type = at::kInt;
    int64_t shape[2] = {0, 0}, at = 0;
    int dims = 0;
    at::Tensor given;
    int64_t numel() const { return shape[0] * (dims > 1 ? shape[1] : 1); }
  };
  const Launch& on_;
  Part parts_[5];
  int n_ = 0, next_ = 0;
  int64_t total_[2] = {0, 0};
  at::Tensor whole_[2];
};
PyObject* result(PyObject* given_one, const at::Tensor& made) {
  return given(given_one) ? Py_NewRef(given_one) : THPVariable_Wrap(made);
}
// A tuple of new references (null: an exception is set).
PyObject* pack(std::initializer_list<PyObject*> items) {
  PyObject* r = PyTuple_New(Py_ssize_t(items.size()));
  Py_ssize_t i = 0;
  bool whole = r != nullptr;
  for (PyObject* o : items) {
    whole = whole && o;
    if (r && o)
      PyTuple_SET_ITEM(r, i, o);
    else
      Py_XDECREF(o);
    ++i;
  }
  if (whole) return r;
  Py_XDECREF(r);
  return nullptr;
}

// int64 [rows, words] words of bits, rows at any stride.
const uint64_t* bits(PyObject* o, const char* name, int64_t rows, c10::DeviceIndex dev, int64_t* stride, int64_t* words) {
  const at::Tensor& t = shaped(o, name, 2, "[tokens, words]");
  check(t, name, at::kLong, {rows, t.size(1)}, dev, false);
  *stride = t.stride(0);
  *words = t.size(1);
  return static_cast<const uint64_t*>(t.data_ptr());
}

// The dimensions of more than one element, the largest stride first.
struct Dims {
  int64_t stride[5], size[5], extent[5];  // extent: elements from the first to the last of this dimension and those behind it
  int n = 0;
  int64_t from(int i) const { return i < n ? extent[i] : 1; }
};
// False where two indices of the tensor may be one address: strides that do not nest.
bool nested(const at::Tensor& t, Dims* d) {
  for (int64_t i = 0; i < t.dim(); ++i) {
    if (t.size(i) <= 1) continue;
    int at = d->n++;
    for (; at > 0 && d->stride[at - 1] < t.stride(i); --at) {
      d->stride[at] = d->stride[at - 1];
      d->size[at] = d->size[at - 1];
    }
    d->stride[at] = t.stride(i);
    d->size[at] = t.size(i);
  }
  for (int i = d->n - 1; i >= 0; --i) {
    if (d->stride[i] < d->from(i + 1)) return false;
    d->extent[i] = d->stride[i] * (d->size[i] - 1) + d->from(i + 1);
  }
  return true;
}
// Whether elements of a, and of b `off` elements on, may meet. A dimension that both have (a stacked cache's layers) is taken
// apart; what is left meets where its ranges do.
bool may_meet(const Dims& a, const Dims& b, int i, int64_t off) {
  if (off >= a.from(i) || -off >= b.from(i)) return false;
  if (i >= a.n || i >= b.n || a.stride[i] != b.stride[i] || a.size[i] != b.size[i]) return true;
  const int64_t s = a.stride[i], low = off >= 0 ? off / s : -((s - 1 - off) / s);
  for (int64_t d = low; d <= low + 1; ++d)  // (what is inside is no longer than the stride)
    if (d < a.size[i] && -d < a.size[i] && may_meet(a, b, i + 1, off - d * s)) return true;
  return false;
}
void check_apart(const at::Tensor& k, const at::Tensor& v) {
  if (k.numel() == 0) return;
  Dims a, b;
  if (!nested(k, &a) || !nested(v, &b)) throw ValueError("k_cache and v_cache must not overlap themselves");
  const int64_t bytes = static_cast<char*>(v.data_ptr()) - static_cast<char*>(k.data_ptr()), size = int64_t(k.element_size());
  const int64_t off = bytes >= 0 ? bytes / size : -((size - 1 - bytes) / size);
  if (may_meet(a, b, 0, off) || (bytes % size != 0 && may_meet(a, b, 0, off + 1)))
    throw ValueError("k_cache and v_cache must not overlap");
}

PyObject* py_kv_pages(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const kNames[] = {"lens",      "page_table", "held",      "free_pages", "free_count",     "page_size",
                                         "cu_q",      "tokens",     "depths",    "first_position", "slots",      "positions",
                                         "new_lens",  "new_held",   "new_free_count", "stream"};
    PyObject* v[16];
    parse("nf4_kv_pages", kNames, 16, 6, args, nargs, kwnames, v);
    const at::Tensor& lens = shaped(v[0], "lens", 1, "[batch]");
    const Launch on(lens, v[15], "lens");
    const c10::DeviceIndex dev = on.device();
    nf4_kv_pages_args a = {};
    a.batch = lens.size(0);
    a.page_size = integer(v[5], "page_size");
    a.first_position = given(v[9]) ? integer(v[9], "first_position") : 0;
    if (given(v[7]))
      a.tokens = integer(v[7], "tokens");
    else if (given(v[8]))
      a.tokens = shaped(v[8], "depths", 1, "[tokens]").size(0);
    else if (given(v[6]))
      throw TypeError("nf4_kv_pages() needs tokens (or depths) with cu_q");
    else
      a.tokens = a.batch;
    if (a.tokens < 0 || a.tokens > int64_t(1) << 24) throw ValueError("tokens must be 0 .. 2^24");
    a.lens = static_cast<const int32_t*>(flat(v[0], "lens", at::kInt, {a.batch}, dev));
    const at::Tensor& table = shaped(v[1], "page_table", 2, "[batch, width]");
    check(table, "page_table", at::kInt, {a.batch, table.size(1)}, dev, false);
    a.page_table = static_cast<int32_t*>(table.data_ptr());
    a.page_table_stride = table.stride(0);
    a.width = table.size(1);
    a.held = static_cast<const int32_t*>(flat(v[2], "held", at::kInt, {a.batch}, dev));
    const at::Tensor& stack = shaped(v[3], "free_pages", 1, "[capacity]");
    a.capacity = stack.size(0);
    a.free_pages = static_cast<int32_t*>(flat(v[3], "free_pages", at::kInt, {a.capacity}, dev));
    a.free_count = static_cast<const int32_t*>(flat(v[4], "free_count", at::kInt, {1}, dev));
    if (given(v[6])) a.cu_q = static_cast<const int32_t*>(flat(v[6], "cu_q", at::kInt, {a.batch + 1}, dev));
    if (given(v[8])) a.depths = static_cast<const int32_t*>(flat(v[8], "depths", at::kInt, {a.tokens}, dev));
    Outputs outputs(on);
    outputs.add(v[10], "slots", at::kLong, {a.tokens});
    outputs.add(v[11], "positions", at::kLong, {a.tokens});
    outputs.add(v[12], "new_lens", at::kInt, {a.batch});
    outputs.add(v[13], "new_held", at::kInt, {a.batch});
    outputs.add(v[14], "new_free_count", at::kInt, {1});
    const at::Tensor slots = outputs.get(), positions = outputs.get(), new_lens = outputs.get(), new_held = outputs.get(),
                     left = outputs.get();
    a.slots = static_cast<int64_t*>(slots.data_ptr());
    a.positions = static_cast<int64_t*>(positions.data_ptr());
    a.new_lens = static_cast<int32_t*>(new_lens.data_ptr());
    a.new_held = static_cast<int32_t*>(new_held.data_ptr());
    a.new_free_count = static_cast<int32_t*>(left.data_ptr());
    const nf4_status st = unlocked([&] { return nf4_kv_pages(&a, on.stream()); });
    if (st != NF4_OK) raise_status(st, "nf4_kv_pages");
    return pack({result(v[10], slots), result(v[11], positions), result(v[12], new_lens), result(v[13], new_held),
                 result(v[14], left)});
  });
}

// The fields of nf4_tree_attention_args but for the outputs; v: q, k_cache, v_cache, prefix_pages, prefix_len,
// suffix_pages, suffix_lens, tree_mask, cu_q, scale.
void fill_tree(PyObject* const* v, c10::DeviceIndex dev, nf4_tree_attention_args* a) {
  *a = nf4_tree_attention_args{};
  fill_attention(AttentionInputs{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[8], v[9]}, dev, &a->attention);
  a->tree_mask = bits(v[7], "tree_mask", a->attention.tokens, dev, &a->tree_mask_stride, &a->tree_words);
}

PyObject* py_tree_attention(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const kNames[] = {"q",           "k_cache",   "v_cache", "prefix_pages", "prefix_len", "suffix_pages",
                                         "suffix_lens", "tree_mask", "cu_q",    "scale",        "out",        "return_lse",
                                         "lse",         "workspace", "stream"};
    PyObject* v[15];
    parse("nf4_tree_attention", kNames, 15, 8, args, nargs, kwnames, v);
    const at::Tensor& q = tensor(v[0], "q");
    const Launch on(q, v[14], "q");
    nf4_tree_attention_args a;
    fill_tree(v, on.device(), &a);
    return attention_outputs(
        "nf4_tree_attention", q, AttentionOutputs{v[10], v[11], v[12], v[13]}, on, &a.attention,
        [&] { return nf4_tree_attention_workspace_size(&a); },
        [&](void* scratch, size_t bytes) { return nf4_tree_attention(&a, scratch, bytes, on.stream()); });
  });
}

PyObject* py_tree_workspace_size(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const kNames[] = {"q",           "k_cache",   "v_cache", "prefix_pages", "prefix_len", "suffix_pages",
                                         "suffix_lens", "tree_mask", "cu_q",    "scale"};
    PyObject* v[10];
    parse("nf4_tree_attention_workspace_size", kNames, 10, 8, args, nargs, kwnames, v);
    const Launch on(tensor(v[0], "q"), nullptr, "q");
    nf4_tree_attention_args a;
    fill_tree(v, on.device(), &a);
    return PyLong_FromSize_t(nf4_tree_attention_workspace_size(&a));
  });
}

PyObject* py_adjust_logits(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const kNames[] = {"logits",      "history",   "history_lens", "prompt_lens",  "repetition", "frequency",
                                         "presence",    "bias_tokens", "bias_values", "mask",        "mask_rows",  "cu_rows",
                                         "draft_tokens", "tree_mask", "out",          "return_best", "best",       "stream"};
    PyObject* v[18];
    parse("nf4_adjust_logits", kNames, 18, 1, args, nargs, kwnames, v);
    const at::Tensor& x = shaped(v[0], "logits", 2, "[rows, vocab]");
    const Launch on(x, v[17], "logits");
    const c10::DeviceIndex dev = on.device();
    const at::ScalarType type = x.scalar_type();
    nf4_adjust_logits_args a = {};
    a.dtype = dtype_code(type, "logits must be bf16, fp16 or fp32");
    a.rows = x.size(0);
    a.vocab = x.size(1);
    check(x, "logits", type, x.sizes(), dev, false);
    a.logits = x.data_ptr();
    a.logits_stride = x.stride(0);
    a.requests = a.rows;
    if (given(v[11])) {
      const at::Tensor& cu = shaped(v[11], "cu_rows", 1, "[requests + 1]");
      if (cu.size(0) < 1) throw ValueError("cu_rows must have shape [requests + 1], got " + text(cu.sizes()));
      a.requests = cu.size(0) - 1;
      a.cu_rows = static_cast<const int32_t*>(flat(v[11], "cu_rows", at::kInt, {a.requests + 1}, dev));
    }
    if (given(v[1]) != given(v[2])) throw TypeError("history and history_lens go together");
    if (given(v[1])) {
      const at::Tensor& h = shaped(v[1], "history", 2, "[requests, width]");
      check(h, "history", at::kInt, {a.requests, h.size(1)}, dev, false);
      a.history = static_cast<const int32_t*>(h.data_ptr());
      a.history_stride = h.stride(0);
      a.history_width = h.size(1);
      a.history_lens = static_cast<const int32_t*>(flat(v[2], "history_lens", at::kInt, {a.requests}, dev));
    }
    if (given(v[3])) a.prompt_lens = static_cast<const int32_t*>(flat(v[3], "prompt_lens", at::kInt, {a.requests}, dev));
    const float** const scales[3] = {&a.repetition, &a.frequency, &a.presence};
    for (int i = 0; i < 3; ++i)
      if (given(v[4 + i])) *scales[i] = static_cast<const float*>(flat(v[4 + i], kNames[4 + i], at::kFloat, {a.requests}, dev));
    if (given(v[7]) != given(v[8])) throw TypeError("bias_tokens and bias_values go together");
    if (given(v[7])) {
      const at::Tensor& t = shaped(v[7], "bias_tokens", 2, "[requests, width]");
      const at::Tensor& b = shaped(v[8], "bias_values", 2, "[requests, width]");
      check(t, "bias_tokens", at::kInt, {a.requests, t.size(1)}, dev, false);
      check(b, "bias_values", at::kFloat, t.sizes(), dev, false);
      if (a.requests > 1 && t.stride(0) != b.stride(0)) throw ValueError("bias_tokens and bias_values must have the same strides");
      a.bias_tokens = static_cast<const int32_t*>(t.data_ptr());
      a.bias_values = static_cast<const float*>(b.data_ptr());
      a.bias_stride = t.stride(0);
      a.bias_width = t.size(1);
    }
    if (given(v[9])) {
      const at::Tensor& m = shaped(v[9], "mask", 2, "[masks, ceil(vocab / 32)]");
      check(m, "mask", at::kInt, {m.size(0), (a.vocab + 31) / 32}, dev, false);
      a.mask = static_cast<const uint32_t*>(m.data_ptr());
      a.mask_stride = m.stride(0);
      a.mask_count = m.size(0);
      if (given(v[10]))
        a.mask_rows = static_cast<const int32_t*>(flat(v[10], "mask_rows", at::kInt, {a.rows}, dev));
      else if (a.mask_count != a.rows)
        throw ValueError("mask must have a row for each row of logits where mask_rows is not given");
    } else if (given(v[10])) {
      throw TypeError("mask_rows without mask");
    }
    if (given(v[12]) != given(v[13])) throw TypeError("draft_tokens and tree_mask go together");
    if (given(v[12])) {
      a.draft_tokens = static_cast<const int32_t*>(flat(v[12], "draft_tokens", at::kInt, {a.rows}, dev));
      a.tree_mask = bits(v[13], "tree_mask", a.rows, dev, &a.tree_mask_stride, &a.tree_words);
    }
    at::Tensor out, best;
    if (given(v[14])) {
      out = tensor(v[14], "out");
      check(out, "out", type, x.sizes(), dev, false);
    } else {
      out = on.empty(x.sizes(), type);
    }
    a.out = out.data_ptr();
    a.out_stride = out.stride(0);
    const bool want = truth(v[15]);
    if (want || given(v[16])) {
      Outputs outputs(on);
      outputs.add(v[16], "best", at::kInt, {a.rows});
      best = outputs.get();
      a.best = static_cast<int32_t*>(best.data_ptr());
    }
    const nf4_status st = unlocked([&] { return nf4_adjust_logits(&a, on.stream()); });
    if (st != NF4_OK) raise_status(st, "nf4_adjust_logits");
    PyObject* const o = result(v[14], out);
    return want ? pack({o, result(v[16], best)}) : o;
  });
}

PyObject* py_tree_commit(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const kNames[] = {"parents", "draft_tokens", "targets", "cu_q",     "lens",   "max_path", "page_table",
                                         "k_cache", "v_cache",      "accepted", "path",    "chosen", "new_lens", "stream"};
    PyObject* v[14];
    parse("nf4_tree_commit", kNames, 14, 6, args, nargs, kwnames, v);
    const at::Tensor& parents = shaped(v[0], "parents", 1, "[tokens]");
    const Launch on(parents, v[13], "parents");
    const c10::DeviceIndex dev = on.device();
    nf4_tree_commit_args a = {};
    a.tokens = parents.size(0);
    a.batch = shaped(v[4], "lens", 1, "[batch]").size(0);
    a.max_path = integer(v[5], "max_path");
    if (a.max_path < 1 || a.max_path > 1024) throw ValueError("max_path must be 1 .. 1024");
    const int32_t** const lists[3] = {&a.parents, &a.draft_tokens, &a.targets};
    for (int i = 0; i < 3; ++i) *lists[i] = static_cast<const int32_t*>(flat(v[i], kNames[i], at::kInt, {a.tokens}, dev));
    if (given(v[3])) a.cu_q = static_cast<const int32_t*>(flat(v[3], "cu_q", at::kInt, {a.batch + 1}, dev));
    a.lens = static_cast<const int32_t*>(flat(v[4], "lens", at::kInt, {a.batch}, dev));
    if (given(v[7]) != given(v[8]) || given(v[7]) != given(v[6]))
      throw TypeError("page_table, k_cache and v_cache go together");
    if (given(v[7])) {
      const at::Tensor& kc = tensor(v[7], "k_cache");
      const at::Tensor& vc = tensor(v[8], "v_cache");
      const int64_t d = kc.dim();
      if (d != 4 && d != 5)
        throw ValueError("k_cache must have shape [pages, page_size, heads, head_dim] or [layers, ...], got " + text(kc.sizes()));
      const at::ScalarType type = kc.scalar_type();
      if (type != at::kBFloat16 && type != at::kHalf) throw TypeError("k_cache must be bf16 or fp16");
      check(kc, "k_cache", type, kc.sizes(), dev, false);
      check(vc, "v_cache", type, kc.sizes(), dev, false);
      check_apart(kc, vc);
      const int64_t o = d - 4;
      a.layers = d == 5 ? kc.size(0) : 1;
      a.num_pages = kc.size(o);
      a.page_size = kc.size(o + 1);
      a.k_heads = kc.size(o + 2);
      a.head_dim = kc.size(o + 3);
      a.k_cache = kc.data_ptr();
      a.k_layer_stride = d == 5 ? kc.stride(0) : 0;
      a.k_page_stride = kc.stride(o);
      a.k_slot_stride = kc.stride(o + 1);
      a.k_head_stride = kc.stride(o + 2);
      a.v_cache = vc.data_ptr();
      a.v_layer_stride = d == 5 ? vc.stride(0) : 0;
      a.v_page_stride = vc.stride(o);
      a.v_slot_stride = vc.stride(o + 1);
      a.v_head_stride = vc.stride(o + 2);
      const at::Tensor& table = shaped(v[6], "page_table", 2, "[batch, width]");
      check(table, "page_table", at::kInt, {a.batch, table.size(1)}, dev, false);
      a.page_table = static_cast<const int32_t*>(table.data_ptr());
      a.page_table_stride = table.stride(0);
      a.width = table.size(1);
    }
    Outputs outputs(on);
    outputs.add(v[9], "accepted", at::kInt, {a.batch});
    outputs.add(v[10], "path", at::kInt, {a.batch, a.max_path});
    outputs.add(v[11], "chosen", at::kInt, {a.batch, a.max_path});
    outputs.add(v[12], "new_lens", at::kInt, {a.batch});
    const at::Tensor accepted = outputs.get(), path = outputs.get(), chosen = outputs.get(), new_lens = outputs.get();
    a.accepted = static_cast<int32_t*>(accepted.data_ptr());
    a.path = static_cast<int32_t*>(path.data_ptr());
    a.chosen = static_cast<int32_t*>(chosen.data_ptr());
    a.new_lens = static_cast<int32_t*>(new_lens.data_ptr());
    const nf4_status st = unlocked([&] { return nf4_tree_commit(&a, on.stream()); });
    if (st != NF4_OK) raise_status(st, "nf4_tree_commit");
    return pack({result(v[9], accepted), result(v[10], path), result(v[11], chosen), result(v[12], new_lens)});
  });
}

}  // namespace

PyMethodDef kDecodingMethods[] = {
    {"nf4_kv_pages", fast(py_kv_pages), METH_FASTCALL | METH_KEYWORDS,
     "nf4_kv_pages(lens, page_table, held, free_pages, free_count, page_size, cu_q=None, tokens=None, depths=None, "
     "first_position=0, slots=None, positions=None, new_lens=None, new_held=None, new_free_count=None, stream=None)\n--\n\n"
     "Lays out a batch's new tokens in a paged cache: lens int32 [batch] keys are cached, request b brings the tokens\n"
     "cu_q[b] .. cu_q[b + 1] - 1 (int32 [batch + 1]; None: one token each) of `tokens` in all. Each row of page_table\n"
     "(int32 [batch, width], of which held[b] pages count) is made just long enough: what it has too many goes onto the\n"
     "stack free_pages (int32, of which free_count[0] count), what is missing comes from its top. Both are changed in\n"
     "place. Returns (slots, positions, new_lens, new_held, new_free_count); the last two may be given as held and\n"
     "free_count. Requests whose pages are not there keep lens and held, and their slots are -1."},
    {"nf4_tree_attention", fast(py_tree_attention), METH_FASTCALL | METH_KEYWORDS,
     "nf4_tree_attention(q, k_cache, v_cache, prefix_pages, prefix_len, suffix_pages, suffix_lens, tree_mask, cu_q=None, "
     "scale=None, out=None, return_lse=False, lse=None, workspace=None, stream=None)\n--\n\n"
     "nf4_prefix_attention where each sequence's tokens are the nodes of a tree, their keys its last own ones: a token\n"
     "sees node x of its sequence where bit x % 64 of word x // 64 of its row of tree_mask (int64 [tokens, words]) is set."},
    {"nf4_tree_attention_workspace_size", fast(py_tree_workspace_size), METH_FASTCALL | METH_KEYWORDS,
     "nf4_tree_attention_workspace_size(q, k_cache, v_cache, prefix_pages, prefix_len, suffix_pages, suffix_lens, tree_mask, "
     "cu_q=None, scale=None)\n--\n\nBytes of workspace that nf4_tree_attention needs for tensors of these shapes."},
    {"nf4_adjust_logits", fast(py_adjust_logits), METH_FASTCALL | METH_KEYWORDS,
     "nf4_adjust_logits(logits, history=None, history_lens=None, prompt_lens=None, repetition=None, frequency=None, "
     "presence=None, bias_tokens=None, bias_values=None, mask=None, mask_rows=None, cu_rows=None, draft_tokens=None, "
     "tree_mask=None, out=None, return_best=False, best=None, stream=None)\n--\n\n"
     "Penalties for tokens of the history (int32 [requests, width], history_lens of them, the first prompt_lens the\n"
     "prompt) and of each row's branch of the drafted tree (draft_tokens int32 [rows], tree_mask int64 [rows, words]),\n"
     "by float32 [requests] factors; biases (int32 and float32 [requests, width], negative tokens: none); then tokens\n"
     "whose bit of the mask (int32 [masks, ceil(vocab / 32)], row mask_rows[r] for row r, negative: no mask) is 0 become\n"
     "-infinity. Rows cu_rows[b] .. cu_rows[b + 1] - 1 are request b's (None: one each). Returns out (new unless given;\n"
     "may be logits), or with return_best (out, best): int32 [rows], the lowest index of each row's largest output. A new out\n"
     "is dense: for logits that are columns of a padded buffer, out=logits or an out padded alike is about twice as fast."},
    {"nf4_tree_commit", fast(py_tree_commit), METH_FASTCALL | METH_KEYWORDS,
     "nf4_tree_commit(parents, draft_tokens, targets, cu_q, lens, max_path, page_table=None, k_cache=None, v_cache=None, "
     "accepted=None, path=None, chosen=None, new_lens=None, stream=None)\n--\n\n"
     "Walks each sequence's drafted tree (parents, draft_tokens, the model's targets: int32 [tokens]) from node 0 along the\n"
     "nodes that hold the model's choice, and moves the accepted nodes' keys and values to their places behind the cached\n"
     "ones (caches [pages, page_size, kv_heads, dim], or [layers, ...] of them, that share no element; of one buffer where\n"
     "their views interleave alike). lens int32 [batch] counts the own keys with all nodes. Returns (accepted, path, chosen,\n"
     "new_lens): int32 [batch], [batch, max_path] twice (-1 behind the last), [batch]."},
    {nullptr, nullptr, 0, nullptr}};

}  // namespace nf4_binding
