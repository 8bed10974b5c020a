// nf4_decoding_api.cu -- the C ABI of include/nf4_decoding.h: host-side argument
// checks, then the launches on the caller's stream.
#include <stdint.h>

#include "nf4_decoding.cuh"

namespace {

constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxIndex = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxBatch = int64_t(1) << 20;
constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxKeys = int64_t(1) << 30;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
template <typename... P>
bool aligned4(const P*... p) {
  return (aligned(p, 4) && ...);
}
bool in(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }
// Rows of `width` elements that are written lie apart.
bool apart(int64_t rows, int64_t stride, int64_t width) { return rows <= 1 || stride >= width; }

// Rows of `width` elements read at `in` and written at `out` share no byte, or are the same rows.
bool apart_or_same(const void* in, int64_t in_stride, const void* out, int64_t out_stride, int64_t rows, int64_t width,
                   int64_t size) {
  const uintptr_t i = reinterpret_cast<uintptr_t>(in), o = reinterpret_cast<uintptr_t>(out);
  if (i == o && (rows <= 1 || in_stride == out_stride)) return true;
  const uintptr_t i_end = i + uintptr_t(((rows - 1) * in_stride + width) * size);
  const uintptr_t o_end = o + uintptr_t(((rows - 1) * out_stride + width) * size);
  if (i_end <= o || o_end <= i) return true;
  if (rows <= 1 || in_stride != out_stride) return false;
  const uintptr_t step = uintptr_t(in_stride * size), off = (o > i ? o - i : i - o) % step;  // columns of one buffer
  return off >= uintptr_t(width * size) && step - off >= uintptr_t(width * size);
}

// Two lists of `count` int32 share an entry.
bool meet(const int32_t* a, const int32_t* b, int64_t count) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return (x > y ? x - y : y - x) < uintptr_t(count * 4);
}

cudaStream_t on(nf4_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

nf4_status check_tree(const nf4_tree_attention_args& a) {
  if (!in(a.tree_words, 1, 1024) || !in(a.tree_mask_stride, 0, kMaxStride)) return NF4_ERR_INVALID_SIZE;
  return nf4::check_attention_sizes(a.attention);
}

}  // namespace

extern "C" {

nf4_status nf4_kv_pages(const nf4_kv_pages_args* args, nf4_stream_t stream) {
  if (!args) return NF4_ERR_NULL;
  const nf4_kv_pages_args& a = *args;
  if (!in(a.batch, 0, kMaxBatch) || !in(a.tokens, 0, kMaxTokens) || !in(a.page_size, 1, 65536) ||
      !in(a.width, 0, kMaxKeys / a.page_size) || !in(a.capacity, 0, kMaxIndex) || !in(a.first_position, 0, kMaxKeys) ||
      !in(a.page_table_stride, 0, kMaxStride) || !apart(a.batch, a.page_table_stride, a.width))
    return NF4_ERR_INVALID_SIZE;
  if (!a.cu_q && a.tokens != a.batch) return NF4_ERR_INVALID_SIZE;
  if (a.batch == 0 && a.tokens == 0 && a.new_free_count == a.free_count) return NF4_OK;
  if (!a.free_count || !a.new_free_count || (a.capacity > 0 && !a.free_pages) || (a.tokens > 0 && !a.slots))
    return NF4_ERR_NULL;
  if (a.batch > 0 && (!a.lens || !a.held || !a.new_lens || !a.new_held || (a.width > 0 && !a.page_table))) return NF4_ERR_NULL;
  if (!aligned4(a.lens, a.cu_q, a.depths, a.page_table, a.held, a.free_pages, a.free_count, a.new_lens, a.new_held,
                a.new_free_count) ||
      !aligned(a.slots, 8) || !aligned(a.positions, 8))
    return NF4_ERR_MISALIGNED;
  // Tokens read lens while new_lens is written; a request's held is read before its own new_held is.
  if (meet(a.new_lens, a.lens, a.batch) || (a.new_held != a.held && meet(a.new_held, a.held, a.batch))) return NF4_ERR_INVALID_SIZE;
  return nf4::status_of(nf4::launch_kv_pages(a, on(stream)));
}

size_t nf4_tree_attention_workspace_size(const nf4_tree_attention_args* args) {
  if (!args || check_tree(*args) != NF4_OK || args->attention.tokens == 0) return 0;
  return nf4::prefix_attention_workspace_bytes(args->attention, true);
}

nf4_status nf4_tree_attention(const nf4_tree_attention_args* args, void* workspace, size_t workspace_bytes,
                              nf4_stream_t stream) {
  if (!args) return NF4_ERR_NULL;
  const nf4_tree_attention_args& a = *args;
  nf4_status st = check_tree(a);
  if (st == NF4_OK) st = nf4::check_attention(a.attention);
  if (st != NF4_OK || a.attention.tokens == 0) return st;
  if (!a.tree_mask) return NF4_ERR_NULL;
  if (!aligned(a.tree_mask, 8)) return NF4_ERR_MISALIGNED;
  bool enough = false;
  const cudaError_t e =
      nf4::launch_prefix_attention(a.attention, &a, workspace, workspace_bytes, &enough, on(stream));
  return enough ? nf4::status_of(e) : NF4_ERR_WORKSPACE;
}

nf4_status nf4_adjust_logits(const nf4_adjust_logits_args* args, nf4_stream_t stream) {
  if (!args) return NF4_ERR_NULL;
  const nf4_adjust_logits_args& a = *args;
  if (!in(a.rows, 0, kMaxBatch) || !in(a.vocab, 1, kMaxTokens) || !in(a.requests, 0, kMaxBatch) ||
      !in(a.logits_stride, 0, kMaxStride) || !in(a.out_stride, 0, kMaxStride) || !apart(a.rows, a.out_stride, a.vocab))
    return NF4_ERR_INVALID_SIZE;
  if (a.dtype != NF4_BF16 && a.dtype != NF4_FP16 && a.dtype != NF4_F32) return NF4_ERR_UNSUPPORTED_DTYPE;
  if (a.history && (!in(a.history_width, 0, int64_t(1) << 28) || !in(a.history_stride, 0, kMaxStride)))
    return NF4_ERR_INVALID_SIZE;
  if (a.bias_tokens && (!in(a.bias_width, 0, 1024) || !in(a.bias_stride, 0, kMaxStride))) return NF4_ERR_INVALID_SIZE;
  if (a.mask && (!in(a.mask_count, 0, kMaxBatch) || !in(a.mask_stride, 0, kMaxStride) ||
                 (!a.mask_rows && a.mask_count < a.rows)))
    return NF4_ERR_INVALID_SIZE;
  if (a.draft_tokens && (!in(a.tree_words, 1, 1024) || !in(a.tree_mask_stride, 0, kMaxStride))) return NF4_ERR_INVALID_SIZE;
  if (!a.cu_rows && a.rows != a.requests) return NF4_ERR_INVALID_SIZE;
  if (a.rows == 0) return NF4_OK;
  if (!a.logits || !a.out || (a.history && !a.history_lens) || (a.bias_tokens && !a.bias_values) ||
      (a.draft_tokens && !a.tree_mask))
    return NF4_ERR_NULL;
  const uintptr_t size = a.dtype == NF4_F32 ? 4 : 2;
  if (!aligned(a.logits, size) || !aligned(a.out, size) ||
      !aligned4(a.best, a.cu_rows, a.history, a.history_lens, a.prompt_lens, a.repetition, a.frequency, a.presence,
                a.bias_tokens, a.bias_values, a.mask, a.mask_rows, a.draft_tokens) ||
      !aligned(a.tree_mask, 8))
    return NF4_ERR_MISALIGNED;
  if (!apart_or_same(a.logits, a.logits_stride, a.out, a.out_stride, a.rows, a.vocab, int64_t(size))) return NF4_ERR_INVALID_SIZE;
  return nf4::status_of(nf4::launch_adjust_logits(a, on(stream)));
}

nf4_status nf4_tree_commit(const nf4_tree_commit_args* args, nf4_stream_t stream) {
  if (!args) return NF4_ERR_NULL;
  const nf4_tree_commit_args& a = *args;
  if (!in(a.batch, 0, kMaxBatch) || !in(a.tokens, 0, kMaxTokens) || !in(a.max_path, 1, 1024)) return NF4_ERR_INVALID_SIZE;
  if (!a.cu_q && a.tokens != a.batch) return NF4_ERR_INVALID_SIZE;
  const bool moves = a.k_cache || a.v_cache;
  if (moves) {
    if (!in(a.layers, 0, 65535) || !in(a.num_pages, 0, kMaxIndex) || !in(a.page_size, 1, 65536) || !in(a.k_heads, 1, 65535) ||
        !in(a.head_dim, 1, 512) || !in(a.width, 0, kMaxKeys / a.page_size) || !in(a.page_table_stride, 0, kMaxStride))
      return NF4_ERR_INVALID_SIZE;
    for (const int64_t s : {a.k_layer_stride, a.k_page_stride, a.k_slot_stride, a.k_head_stride, a.v_layer_stride,
                            a.v_page_stride, a.v_slot_stride, a.v_head_stride})
      if (!in(s, 0, kMaxStride)) return NF4_ERR_INVALID_SIZE;
    // a row at two indices would be moved twice, beside itself
    const int64_t sizes[] = {a.layers, a.num_pages, a.page_size, a.k_heads};
    const int64_t strides[][4] = {{a.k_layer_stride, a.k_page_stride, a.k_slot_stride, a.k_head_stride},
                                  {a.v_layer_stride, a.v_page_stride, a.v_slot_stride, a.v_head_stride}};
    for (const auto& of : strides)
      for (int i = 0; i < 4; ++i)
        if (sizes[i] > 1 && of[i] == 0) return NF4_ERR_INVALID_SIZE;
    if (a.k_cache && a.k_cache == a.v_cache) return NF4_ERR_INVALID_SIZE;  // both would be moved, beside one another
  }
  if (a.batch == 0) return NF4_OK;
  if ((a.tokens > 0 && (!a.parents || !a.draft_tokens || !a.targets)) || !a.lens || !a.accepted || !a.path || !a.chosen ||
      !a.new_lens)
    return NF4_ERR_NULL;
  if (moves && (!a.k_cache || !a.v_cache || (a.width > 0 && !a.page_table))) return NF4_ERR_NULL;
  if (!aligned4(a.parents, a.draft_tokens, a.targets, a.cu_q, a.lens, a.accepted, a.path, a.chosen, a.new_lens, a.page_table) ||
      !aligned(a.k_cache, 2) || !aligned(a.v_cache, 2))
    return NF4_ERR_MISALIGNED;
  // Other blocks of a sequence, and of other ones, read lens while new_lens is written.
  if ((moves || a.new_lens != a.lens) && meet(a.new_lens, a.lens, a.batch)) return NF4_ERR_INVALID_SIZE;
  nf4_tree_commit_args c = a;
  if (!moves) c.layers = 0;  // (with no page, or a table of no columns, every row that would move is reported)
  return nf4::status_of(nf4::launch_tree_commit(c, on(stream)));
}

}  // extern "C"
