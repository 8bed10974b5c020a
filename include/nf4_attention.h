/*
 * nf4_attention.h -- C ABI of libnf4, attention side of a decoder layer: what
 * stands between the fused q/k/v GEMVs of nf4.h and the o GEMV. Rotary
 * position tables, the per-head norm and rotation of queries and keys, the
 * append of keys and values to a paged cache, and attention for a batch of
 * sequences that share a prefix of that cache.
 *
 * The conventions of nf4.h hold for every entry point here: device pointers
 * owned by the caller, work enqueued on `stream`, host-side argument checks
 * before any launch, status codes of nf4_status, no allocation, no
 * synchronisation. In addition:
 *   - Arguments that describe tensors come in one structure of 8-byte fields.
 *     The structure is read during the call and not kept.
 *   - Strides are in elements and may be any non-negative value (views of a
 *     fused q/k/v buffer, either order of the cache's heads and slots). The
 *     last dimension (head_dim) is contiguous. The stride of a dimension of
 *     size one is never used.
 *   - Positions, slots, pages, lengths and cu_q are device data and are
 *     checked by the kernels: a value out of range is never used as an index.
 *     It sets bit 1 of nf4_device_error_flags(), and the outputs that depend
 *     on it are as stated at each call.
 *
 * Paged cache: keys and values of every sequence live in pages of page_size
 * slots. Slot s of page p and key/value head h is the head_dim elements at
 *   k + p * k_page_stride + s * k_slot_stride + h * k_head_stride
 * (v likewise). A flat slot number is p * page_size + s. Slots that no call
 * reads may hold anything, NaN and infinities included.
 */
#ifndef NF4_ATTENTION_H_
#define NF4_ATTENTION_H_

#include "nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How nf4_rope_table stretches the frequencies f_i = base^(-2i/rot_dim) of a
 * model trained on `original_positions` positions to longer contexts. */
typedef enum {
  NF4_ROPE_PLAIN = 0,  /* f_i */
  NF4_ROPE_LINEAR = 1, /* f_i / factor */
  NF4_ROPE_BANDS = 2,  /* by wavelength: with r = original_positions f_i / (2 pi) turns over the original context,
                          f_i for r > high, f_i / factor for r < low, and between them the blend
                          (1 - s) f_i / factor + s f_i with s = (r - low) / (high - low) */
  NF4_ROPE_RAMP = 3    /* by index: with d(n) = rot_dim ln(original_positions / (2 pi n)) / (2 ln base) the (real)
                          index that turns n times, lo = max(floor(d(high)), 0), hi = min(ceil(d(low)), rot_dim - 1),
                          s = clamp((i - lo) / max(hi - lo, 1e-3), 0, 1): (1 - s) f_i + s f_i / factor */
} nf4_rope_scaling;

typedef struct nf4_rope_table_args {
  float* cos_sin;             /* [positions][rot_dim / 2][2], 8-byte aligned: (cos, sin) pairs */
  int64_t positions;          /* rows, 0 .. 2^30; row p holds position p */
  int64_t rot_dim;            /* even, 2 .. 512 */
  int64_t scaling;            /* nf4_rope_scaling */
  double base;                /* > 1 (10000 is the usual value) */
  double factor;              /* >= 1; ignored by NF4_ROPE_PLAIN */
  double low, high;           /* turns, 0 < low < high; NF4_ROPE_BANDS and NF4_ROPE_RAMP */
  double original_positions;  /* > 0; NF4_ROPE_BANDS and NF4_ROPE_RAMP */
  double magnitude;           /* > 0: both cos and sin are multiplied by it (1 leaves them) */
} nf4_rope_table_args;

/*
 * nf4_rope_table -- cos_sin[p][i] = (m cos(p g_i), m sin(p g_i)) with g_i the
 * scaled frequency above and m the magnitude. The angle is formed and reduced
 * in binary64, so that rows far into a long context are as exact as the first
 * ones: absolute error below 3e-7 m for p < 2^24.
 * Errors: NF4_ERR_NULL, NF4_ERR_INVALID_SIZE (a size or parameter outside the
 *   ranges above), NF4_ERR_MISALIGNED, NF4_ERR_CUDA.
 */
NF4_API nf4_status nf4_rope_table(const nf4_rope_table_args* args, nf4_stream_t stream);

typedef struct nf4_qk_norm_rope_args {
  const void* q;              /* [tokens][q_heads][head_dim] of dtype */
  int64_t q_token_stride, q_head_stride;
  void* q_out;
  int64_t q_out_token_stride, q_out_head_stride;
  int64_t q_heads;            /* >= 0; 0: no q (its pointers are ignored) */
  const void* k;              /* [tokens][k_heads][head_dim] of dtype */
  int64_t k_token_stride, k_head_stride;
  void* k_out;
  int64_t k_out_token_stride, k_out_head_stride;
  int64_t k_heads;            /* >= 0; 0: no k */
  const int64_t* positions;   /* [tokens], each 0 .. max_positions - 1 */
  const float* cos_sin;       /* [max_positions][rot_dim / 2][2], 8-byte aligned (nf4_rope_table's layout) */
  int64_t max_positions;
  int64_t rot_dim;            /* even, 0 .. head_dim: the first rot_dim elements of a head are rotated */
  int64_t interleaved;        /* 0: pairs (i, i + rot_dim / 2); 1: pairs (2i, 2i + 1) */
  const void* q_weight;       /* NULL: queries are not normed; else [head_dim] of dtype */
  const void* k_weight;       /* NULL: keys are not normed; else [head_dim] of dtype */
  double eps;                 /* >= 0 */
  int64_t tokens, head_dim;   /* tokens >= 0; head_dim 1 .. 512 */
  int64_t dtype;              /* NF4_BF16, NF4_FP16 or NF4_F32 */
} nf4_qk_norm_rope_args;

/*
 * nf4_qk_norm_rope -- each head row x of q and of k: with a weight w,
 * u = x * rsqrt(mean(x^2) + eps) * w over the whole head, else u = x; then
 * each pair (a, b) of the first rot_dim elements becomes
 * (a cos - b sin, b cos + a sin) with the row of the table that the token's
 * position names; the rest is u. Computed in binary32, rounded once into
 * dtype. One launch for q and k. An output may be its input (same pointer and
 * strides); any other overlap is undefined.
 * A position outside the table (device data): the token's rows become NaN and
 * bit 1 of the device error flags is set. rot_dim 0 reads neither.
 * Fastest (16-byte accesses) when head_dim and rot_dim are multiples of 16
 * (8 for NF4_F32), head_dim * sizeof(dtype) <= 1024 and all pointers and strides
 * are 16-byte aligned.
 * Errors: NF4_ERR_NULL, NF4_ERR_INVALID_SIZE (also negative strides, more than
 *   2^31 - 1 tokens or 65535 heads), NF4_ERR_UNSUPPORTED_DTYPE, NF4_ERR_MISALIGNED (a
 *   pointer not aligned to its element), NF4_ERR_CUDA.
 */
NF4_API nf4_status nf4_qk_norm_rope(const nf4_qk_norm_rope_args* args, nf4_stream_t stream);

typedef struct nf4_kv_append_args {
  nf4_qk_norm_rope_args qk;   /* k_out and its strides are ignored (the cache takes their place); k_heads >= 1;
                                 q_heads 0: keys and values alone; dtype is the cache's: NF4_BF16 or NF4_FP16 */
  const void* v;              /* [tokens][k_heads][head_dim] of dtype */
  int64_t v_token_stride, v_head_stride;
  const int64_t* slots;       /* [tokens]: flat slot of each token's key and value; negative: none is written */
  void* k_cache;
  int64_t k_page_stride, k_slot_stride, k_head_stride;
  void* v_cache;
  int64_t v_page_stride, v_slot_stride, v_cache_head_stride;
  int64_t num_pages;          /* 0 .. 2^31 - 1 */
  int64_t page_size;          /* 1 .. 65536 */
} nf4_kv_append_args;

/*
 * nf4_kv_append -- nf4_qk_norm_rope whose keys go to the paged cache, with the
 * values of the same tokens copied beside them, and (q_heads > 0) the queries
 * normed and rotated into q_out in the same launch. Tokens with a negative
 * slot write no key and no value; their queries are written. Two tokens with
 * the same slot are a race: the slot then holds parts of either.
 * A slot at or past num_pages * page_size (device data) writes nothing and
 * sets bit 1 of the device error flags. k and v must not overlap the cache.
 * Errors: as nf4_qk_norm_rope.
 */
NF4_API nf4_status nf4_kv_append(const nf4_kv_append_args* args, nf4_stream_t stream);

typedef struct nf4_prefix_attention_args {
  const void* q;              /* [tokens][q_heads][head_dim] of dtype */
  int64_t q_token_stride, q_head_stride;
  void* out;                  /* [tokens][q_heads][head_dim] of dtype */
  int64_t out_token_stride, out_head_stride;
  float* lse;                 /* NULL, or [tokens][q_heads] (contiguous): log-sum-exp of the scaled scores */
  const void* k_cache;
  int64_t k_page_stride, k_slot_stride, k_head_stride;
  const void* v_cache;
  int64_t v_page_stride, v_slot_stride, v_head_stride;
  int64_t num_pages;          /* 0 .. 2^31 - 1 */
  int64_t page_size;          /* 1 .. 65536 */
  const int32_t* prefix_pages; /* [ceil(prefix_len / page_size)] */
  int64_t prefix_len;         /* keys shared by every sequence, 0 .. 2^30 */
  const int32_t* suffix_pages; /* [batch][suffix_pages_width]: pages of each sequence's own keys */
  int64_t suffix_pages_stride; /* elements between the rows of two sequences */
  int64_t suffix_pages_width; /* width * page_size bounds the own keys of a sequence (at most 2^30) */
  const int32_t* suffix_lens; /* [batch]: own keys of each sequence, 0 .. width * page_size */
  const int32_t* cu_q;        /* [batch + 1], non-decreasing from 0 to tokens: sequence b has the tokens
                                 cu_q[b] .. cu_q[b + 1] - 1; NULL: one token each (tokens == batch) */
  int64_t batch;              /* 0 .. 2^20 */
  int64_t tokens;             /* 0 .. 2^24 */
  int64_t q_heads, k_heads;   /* k_heads >= 1 divides q_heads; query head h reads key/value head
                                 h / (q_heads / k_heads); tokens * q_heads at most 2^30 */
  int64_t head_dim;           /* a multiple of 8, 8 .. 128 */
  int64_t dtype;              /* NF4_BF16 or NF4_FP16: q, out and the cache */
  double scale;               /* of the scores, usually 1 / sqrt(head_dim); > 0, and scale * log2(e) a normal binary32
                                 number (about 8.2e-39 .. 2.3e38) */
} nf4_prefix_attention_args;

/* Bytes of device workspace that nf4_prefix_attention needs for these
 * arguments (their sizes only: pointers are not looked at); 0 where it needs
 * none or the sizes are not accepted. */
NF4_API size_t nf4_prefix_attention_workspace_size(const nf4_prefix_attention_args* args);

/*
 * nf4_prefix_attention -- softmax attention of each query token over the
 * prefix_len keys that the whole batch shares and then its sequence's own
 * keys. Token i of the n tokens of sequence b sees every prefix key and the
 * own keys j <= suffix_lens[b] - n + i (its own key is the last one that it
 * sees: append before attending). With s_j = scale * (q . k_j) over the keys
 * seen, out = sum_j exp(s_j - lse) v_j and lse = log sum_j exp(s_j). A row that
 * sees no key gives zeros and lse = -infinity.
 * The shared keys are read once for all rows of a key/value head together;
 * partial results of key ranges are joined in a fixed order, so that the
 * outputs of two identical calls are identical. Scores, the running maximum
 * and sum, and all partial outputs are binary32; the weights exp(s_j - m) are
 * rounded to dtype for the product with v (in fp16 times 2^7, so that those
 * down to 2^-31 of the largest count); ranges are of at most 2^17 keys, so that
 * binary32 sums lose at most 2^-8 of them to keys of no weight to speak of; the
 * result is rounded once.
 * A NaN or infinity in k or v reaches every row that sees it; one in v of an
 * own key may also reach rows of the same sequence that stand before it.
 * cu_q, lengths and pages are read on the device, so a recorded graph can be
 * replayed as sequences grow within suffix_pages_width. (The work is shared out
 * for sequences about that long: a table many times wider than the sequences
 * are long costs time, not exactness.) Lengths out of range
 * are clamped into it; rows that would read a page outside 0 .. num_pages - 1
 * are undefined; both set bit 1 of the device error flags. Tokens that no
 * sequence holds attend to the prefix alone.
 *   workspace  device scratch of at least nf4_prefix_attention_workspace_size()
 *              bytes, 16-byte aligned; contents on entry are ignored. Calls
 *              that overlap in time need workspaces of their own.
 * Errors: NF4_ERR_NULL, NF4_ERR_INVALID_SIZE, NF4_ERR_UNSUPPORTED_DTYPE,
 *   NF4_ERR_MISALIGNED (q, out or a cache not 16-byte aligned, a stride of
 *   theirs not a multiple of 8 elements, an index array not aligned to its element),
 *   NF4_ERR_WORKSPACE, NF4_ERR_CUDA.
 */
NF4_API nf4_status nf4_prefix_attention(const nf4_prefix_attention_args* args, void* workspace,
                                        size_t workspace_bytes, nf4_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* NF4_ATTENTION_H_ */
