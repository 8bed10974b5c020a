// nf4_attn_api.cu -- the C ABI of include/nf4_attention.h: host-side argument
// checks, then the launches on the caller's stream.
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "nf4_attn.cuh"

namespace {

constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxIndex = (int64_t(1) << 31) - 1;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool in(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }
bool strides_ok(int64_t a, int64_t b, int64_t c = 0) {
  return in(a, 0, kMaxStride) && in(b, 0, kMaxStride) && in(c, 0, kMaxStride);
}

// Checks of nf4_qk_norm_rope; `append` leaves k_out out (the cache takes its place).
nf4_status check_qk(const nf4_qk_norm_rope_args& a, bool append) {
  if (!in(a.tokens, 0, kMaxIndex) || !in(a.head_dim, 1, 512) || !in(a.q_heads, 0, 65535) ||
      !in(a.k_heads, append ? 1 : 0, 65535))
    return NF4_ERR_INVALID_SIZE;
  if (!in(a.rot_dim, 0, a.head_dim) || (a.rot_dim & 1) != 0 || a.max_positions < 0) return NF4_ERR_INVALID_SIZE;
  if (!(a.eps >= 0.0) || !isfinite(a.eps)) return NF4_ERR_INVALID_SIZE;
  if (a.interleaved != 0 && a.interleaved != 1) return NF4_ERR_INVALID_SIZE;
  if (a.dtype != NF4_BF16 && a.dtype != NF4_FP16 && (a.dtype != NF4_F32 || append)) return NF4_ERR_UNSUPPORTED_DTYPE;
  const uintptr_t size = a.dtype == NF4_F32 ? 4 : 2;
  if (a.q_heads > 0 && (!strides_ok(a.q_token_stride, a.q_head_stride) ||
                        !strides_ok(a.q_out_token_stride, a.q_out_head_stride)))
    return NF4_ERR_INVALID_SIZE;
  if (a.k_heads > 0 && (!strides_ok(a.k_token_stride, a.k_head_stride) ||
                        (!append && !strides_ok(a.k_out_token_stride, a.k_out_head_stride))))
    return NF4_ERR_INVALID_SIZE;
  if (a.tokens == 0 || a.q_heads + a.k_heads == 0) return NF4_OK;
  if (a.q_heads > 0 && (!a.q || !a.q_out)) return NF4_ERR_NULL;
  if (a.k_heads > 0 && (!a.k || (!append && !a.k_out))) return NF4_ERR_NULL;
  if (a.rot_dim > 0 && (!a.positions || (!a.cos_sin && a.max_positions > 0))) return NF4_ERR_NULL;
  if (a.q_heads > 0 && (!aligned(a.q, size) || !aligned(a.q_out, size) || !aligned(a.q_weight, size)))
    return NF4_ERR_MISALIGNED;
  if (a.k_heads > 0 && (!aligned(a.k, size) || (!append && !aligned(a.k_out, size)) || !aligned(a.k_weight, size)))
    return NF4_ERR_MISALIGNED;
  if (a.rot_dim > 0 && (!aligned(a.positions, 8) || !aligned(a.cos_sin, 8))) return NF4_ERR_MISALIGNED;
  return NF4_OK;
}

nf4_status check_attention_sizes(const nf4_prefix_attention_args& a) {
  if (!in(a.batch, 0, int64_t(1) << 20) || !in(a.tokens, 0, int64_t(1) << 24) || !in(a.k_heads, 1, 65535) ||
      !in(a.q_heads, 1, 65535) || a.q_heads % a.k_heads != 0)
    return NF4_ERR_INVALID_SIZE;
  if (a.tokens * a.q_heads > int64_t(1) << 30) return NF4_ERR_INVALID_SIZE;
  if (!in(a.head_dim, 8, 128) || a.head_dim % 8 != 0) return NF4_ERR_INVALID_SIZE;
  if (!in(a.num_pages, 0, kMaxIndex) || !in(a.page_size, 1, 65536)) return NF4_ERR_INVALID_SIZE;
  if (!in(a.prefix_len, 0, int64_t(1) << 30) || !in(a.suffix_pages_width, 0, (int64_t(1) << 30) / a.page_size) ||
      !in(a.suffix_pages_stride, 0, kMaxStride))
    return NF4_ERR_INVALID_SIZE;
  if (!strides_ok(a.q_token_stride, a.q_head_stride) || !strides_ok(a.out_token_stride, a.out_head_stride) ||
      !strides_ok(a.k_page_stride, a.k_slot_stride, a.k_head_stride) ||
      !strides_ok(a.v_page_stride, a.v_slot_stride, a.v_head_stride))
    return NF4_ERR_INVALID_SIZE;
  // the kernels use it times log2 e in binary32: 0 there would make a masked score (-inf) NaN
  const double scale_log2 = a.scale * 1.4426950408889634;
  if (!(scale_log2 >= double(FLT_MIN) && scale_log2 <= double(FLT_MAX))) return NF4_ERR_INVALID_SIZE;
  if (a.dtype != NF4_BF16 && a.dtype != NF4_FP16) return NF4_ERR_UNSUPPORTED_DTYPE;
  return NF4_OK;
}

}  // namespace

extern "C" {

nf4_status nf4_rope_table(const nf4_rope_table_args* args, nf4_stream_t stream) {
  if (!args) return NF4_ERR_NULL;
  const nf4_rope_table_args& a = *args;
  if (!in(a.positions, 0, int64_t(1) << 30) || !in(a.rot_dim, 2, 512) || (a.rot_dim & 1) != 0)
    return NF4_ERR_INVALID_SIZE;
  if (!in(a.scaling, NF4_ROPE_PLAIN, NF4_ROPE_RAMP)) return NF4_ERR_INVALID_SIZE;
  if (!(a.base > 1.0) || !isfinite(a.base) || !(a.magnitude > 0.0) || !isfinite(a.magnitude))
    return NF4_ERR_INVALID_SIZE;
  if (a.scaling != NF4_ROPE_PLAIN && (!(a.factor >= 1.0) || !isfinite(a.factor))) return NF4_ERR_INVALID_SIZE;
  if ((a.scaling == NF4_ROPE_BANDS || a.scaling == NF4_ROPE_RAMP) &&
      (!(a.low > 0.0) || !(a.high > a.low) || !isfinite(a.high) || !(a.original_positions > 0.0) ||
       !isfinite(a.original_positions)))
    return NF4_ERR_INVALID_SIZE;
  if (a.positions == 0) return NF4_OK;
  if (!a.cos_sin) return NF4_ERR_NULL;
  if (!aligned(a.cos_sin, 8)) return NF4_ERR_MISALIGNED;
  return nf4::status_of(nf4::launch_rope_table(a, reinterpret_cast<cudaStream_t>(stream)));
}

nf4_status nf4_qk_norm_rope(const nf4_qk_norm_rope_args* args, nf4_stream_t stream) {
  if (!args) return NF4_ERR_NULL;
  const nf4_status st = check_qk(*args, false);
  if (st != NF4_OK || args->tokens == 0 || args->q_heads + args->k_heads == 0) return st;
  return nf4::status_of(nf4::launch_qk_rope(*args, nullptr, reinterpret_cast<cudaStream_t>(stream)));
}

nf4_status nf4_kv_append(const nf4_kv_append_args* args, nf4_stream_t stream) {
  if (!args) return NF4_ERR_NULL;
  const nf4_kv_append_args& a = *args;
  const nf4_status st = check_qk(a.qk, true);
  if (st != NF4_OK) return st;
  if (!in(a.num_pages, 0, kMaxIndex) || !in(a.page_size, 1, 65536)) return NF4_ERR_INVALID_SIZE;
  if (!strides_ok(a.v_token_stride, a.v_head_stride) ||
      !strides_ok(a.k_page_stride, a.k_slot_stride, a.k_head_stride) ||
      !strides_ok(a.v_page_stride, a.v_slot_stride, a.v_cache_head_stride))
    return NF4_ERR_INVALID_SIZE;
  if (a.qk.tokens == 0) return NF4_OK;
  if (!a.v || !a.slots || (a.num_pages > 0 && (!a.k_cache || !a.v_cache))) return NF4_ERR_NULL;
  if (!aligned(a.v, 2) || !aligned(a.slots, 8) || !aligned(a.k_cache, 2) || !aligned(a.v_cache, 2))
    return NF4_ERR_MISALIGNED;
  return nf4::status_of(nf4::launch_qk_rope(a.qk, &a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t nf4_prefix_attention_workspace_size(const nf4_prefix_attention_args* args) {
  if (!args || check_attention_sizes(*args) != NF4_OK || args->tokens == 0) return 0;
  return nf4::prefix_attention_workspace_bytes(*args);
}

nf4_status nf4_prefix_attention(const nf4_prefix_attention_args* args, void* workspace, size_t workspace_bytes,
                                nf4_stream_t stream) {
  if (!args) return NF4_ERR_NULL;
  const nf4_prefix_attention_args& a = *args;
  const nf4_status st = check_attention_sizes(a);
  if (st != NF4_OK) return st;
  if (!a.cu_q && a.tokens != a.batch) return NF4_ERR_INVALID_SIZE;
  if (a.tokens == 0) return NF4_OK;
  const bool own = a.batch > 0 && a.suffix_pages_width > 0;
  if (!a.q || !a.out || (a.prefix_len > 0 && !a.prefix_pages) || (own && (!a.suffix_pages || !a.suffix_lens)) ||
      (a.num_pages > 0 && (a.prefix_len > 0 || own) && (!a.k_cache || !a.v_cache)))
    return NF4_ERR_NULL;
  // the stride of a dimension of one is never used
  const int64_t sizes[] = {a.tokens, a.q_heads, a.num_pages, a.page_size, a.k_heads};
  const int64_t strides[][5] = {{a.q_token_stride, a.q_head_stride, 0, 0, 0},
                                {a.out_token_stride, a.out_head_stride, 0, 0, 0},
                                {0, 0, a.k_page_stride, a.k_slot_stride, a.k_head_stride},
                                {0, 0, a.v_page_stride, a.v_slot_stride, a.v_head_stride}};
  for (const auto& of : strides)
    for (int i = 0; i < 5; ++i)
      if (sizes[i] > 1 && of[i] % 8 != 0) return NF4_ERR_MISALIGNED;
  if (!aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) ||
      !aligned(a.lse, 4) || !aligned(a.prefix_pages, 4) || !aligned(a.suffix_pages, 4) ||
      !aligned(a.suffix_lens, 4) || !aligned(a.cu_q, 4))
    return NF4_ERR_MISALIGNED;
  bool enough = false;
  const cudaError_t e = nf4::launch_prefix_attention(a, workspace, workspace_bytes, &enough,
                                                     reinterpret_cast<cudaStream_t>(stream));
  return enough ? nf4::status_of(e) : NF4_ERR_WORKSPACE;
}

}  // extern "C"
