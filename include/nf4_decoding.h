/*
 * nf4_decoding.h -- C ABI of libnf4, a step of decoding around its GEMVs: the
 * page tables and slots that nf4_kv_append and the attention calls read, made
 * on the device from the requests' lengths; attention for drafted tokens that
 * form a tree; penalties, biases and masks on logits, with the best token; and
 * taking the accepted branch of a tree into the cache.
 *
 * The conventions of nf4.h and nf4_attention.h hold for every entry point
 * here: device pointers owned by the caller, argument structures of 8-byte
 * fields that are read during the call, work enqueued on `stream`, host-side
 * checks before any launch, status codes of nf4_status, no allocation, no
 * synchronisation. Lengths, pages, tokens and offsets are device data and are
 * checked by the kernels: a value out of range is never used as an index and
 * sets bit 1 of nf4_device_error_flags(). A step of these calls can be
 * recorded into a graph and replayed; nothing is read back by the host.
 *
 * A drafted tree: each sequence brings n tokens (nodes), in an order in which
 * a parent stands before its children. Node 0 is the sequence's last token
 * that is certain; the others are guesses of what follows. Node i's context is
 * the sequence's cached keys and the nodes on the way from node 0 to node i.
 */
#ifndef NF4_DECODING_H_
#define NF4_DECODING_H_

#include "nf4_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct nf4_kv_pages_args {
  const int32_t* lens;        /* [batch]: keys that each request has in the cache (its own ones) */
  const int32_t* cu_q;        /* [batch + 1], non-decreasing from 0 to tokens: request b brings the tokens
                                 cu_q[b] .. cu_q[b + 1] - 1; NULL: one token each (tokens == batch) */
  const int32_t* depths;      /* NULL, or [tokens]: what takes the place of a token's number within its request in its
                                 position (the depth of a tree's node) */
  int32_t* page_table;        /* [batch][width], rows page_table_stride apart; read and written */
  int64_t page_table_stride;
  int64_t width;              /* 0 .. 2^30 / page_size */
  const int32_t* held;        /* [batch]: pages in each row of the table, 0 .. width */
  int32_t* free_pages;        /* [capacity]: the free pages, a stack of free_count[0]; read and written */
  int64_t capacity;           /* 0 .. 2^31 - 1 */
  const int32_t* free_count;  /* [1] */
  int64_t* slots;             /* [tokens]: flat slot of each token's key and value */
  int64_t* positions;         /* [tokens], or NULL */
  int32_t* new_lens;          /* [batch]: lens with the new tokens; shares no entry with lens */
  int32_t* new_held;          /* [batch]; may be held, else shares no entry with it */
  int32_t* new_free_count;    /* [1]; may be free_count */
  int64_t batch;              /* 0 .. 2^20 */
  int64_t tokens;             /* 0 .. 2^24 */
  int64_t page_size;          /* 1 .. 65536 */
  int64_t first_position;     /* position of a request's first own key (the length of a shared prefix), 0 .. 2^30 */
} nf4_kv_pages_args;

/*
 * nf4_kv_pages -- lays out the new tokens of a batch in the paged cache. A
 * request with L cached keys, n new tokens and h pages needs
 * p = ceil((L + n) / page_size) of them.
 *   - Where h > p (rejected drafts, a request that ended: L = n = 0), its last
 *     h - p pages go onto the free stack, in the order of the requests and,
 *     within one, of the table. The cells of the table keep them.
 *   - Then, where h < p, the missing pages come from the top of the stack, in
 *     the same order. What is taken stays in the array above the new top. Where
 *     a request asks for more pages than are left, it and the requests after it
 *     that need any get none and set bit 2 of the device error flags: their
 *     slots are -1, their new_lens and new_held are lens and held (to be called
 *     again with fewer requests, or once pages are back). So does a request that
 *     needs more than `width` pages (bit 1), without holding up the others.
 *   - Token i of request b gets slot table[b][(L + i) / page_size] * page_size +
 *     (L + i) % page_size and position first_position + L + (depths ? its depth : i).
 * Tokens that no request holds get slot -1 and position 0. The order of pages
 * is fixed, so that two identical calls give identical results.
 * Lengths, cu_q, held and free_count out of range are clamped into it, returned
 * pages past the capacity are dropped, a token on a negative page number gets
 * slot -1; all set bit 1 of the device error flags.
 * One launch of one thread-block cluster; a second one of the tokens where these are more than 4096 or the requests
 * more than 1024.
 * Errors: NF4_ERR_NULL, NF4_ERR_INVALID_SIZE, NF4_ERR_MISALIGNED, NF4_ERR_CUDA.
 */
NF4_API nf4_status nf4_kv_pages(const nf4_kv_pages_args* args, nf4_stream_t stream);

typedef struct nf4_tree_attention_args {
  nf4_prefix_attention_args attention; /* suffix_lens count the drafted keys, a sequence's last n own ones */
  const uint64_t* tree_mask;  /* [tokens][tree_words]: bit x % 64 of word x / 64 of a token's row is set where the token
                                 sees its sequence's node x; bits past the sequence's nodes are ignored */
  int64_t tree_mask_stride;   /* elements between the rows of two tokens */
  int64_t tree_words;         /* 1 .. 1024; nodes past 64 * tree_words are not seen */
} nf4_tree_attention_args;

/* Bytes of device workspace that nf4_tree_attention needs for these arguments
 * (their sizes only), as for nf4_prefix_attention. */
NF4_API size_t nf4_tree_attention_workspace_size(const nf4_tree_attention_args* args);

/*
 * nf4_tree_attention -- nf4_prefix_attention where the tokens of a sequence
 * form a tree. Token i of the n tokens of sequence b sees every prefix key, the
 * own keys j < suffix_lens[b] - n, and of the n keys after them (its
 * sequence's nodes, in order) key suffix_lens[b] - n + x where bit x of its row
 * of tree_mask is set. A row of ones up to bit i is nf4_prefix_attention's
 * causal order; a row without a bit and without other keys gives zeros and
 * lse = -infinity. Where suffix_lens[b] < n, the first n - suffix_lens[b]
 * nodes have no key.
 * Everything else is as stated there: rounding, joins in a fixed order,
 * workspaces, error flags; non-finite values in k stay with the rows that see
 * the key, those in v of an own key may also reach other rows of the sequence.
 * The work is cut up for own keys as many as a row of suffix_pages can hold: wider
 * tables give the same results, later. One tree of 25 nodes over 4000 keys (32 heads
 * over 8) takes 13.8 us with a table for 4000 keys, 14.9 for 8192, 25 for 32768 and 40
 * for 131072.
 * Errors: as nf4_prefix_attention; also NF4_ERR_NULL and NF4_ERR_MISALIGNED (8
 *   bytes) for tree_mask, NF4_ERR_INVALID_SIZE for its words and stride.
 */
NF4_API nf4_status nf4_tree_attention(const nf4_tree_attention_args* args, void* workspace,
                                      size_t workspace_bytes, nf4_stream_t stream);

typedef struct nf4_adjust_logits_args {
  const void* logits;          /* [rows][vocab] of dtype */
  int64_t logits_stride;       /* elements between rows */
  void* out;                   /* [rows][vocab] of dtype; may be logits (same stride), else shares no element with it */
  int64_t out_stride;
  int32_t* best;               /* NULL, or [rows]: index of each row's largest output */
  int64_t rows;                /* 0 .. 2^20 */
  int64_t vocab;               /* 1 .. 2^24 */
  int64_t dtype;               /* NF4_BF16, NF4_FP16 or NF4_F32 */
  int64_t requests;            /* 0 .. 2^20 */
  const int32_t* cu_rows;      /* [requests + 1], non-decreasing from 0 to rows: request b has the rows
                                  cu_rows[b] .. cu_rows[b + 1] - 1; NULL: one row each (rows == requests) */
  const int32_t* history;      /* NULL, or [requests][history_width]: tokens of each request, prompt first */
  int64_t history_stride;
  int64_t history_width;       /* 0 .. 2^28 */
  const int32_t* history_lens; /* [requests]: tokens that count, 0 .. history_width */
  const int32_t* prompt_lens;  /* NULL (0), or [requests]: how many of these are the prompt, from 0; past the last, all */
  const float* repetition;     /* NULL (1), or [requests] */
  const float* frequency;      /* NULL (0), or [requests] */
  const float* presence;       /* NULL (0), or [requests] */
  const int32_t* bias_tokens;  /* NULL, or [requests][bias_width]; negative: no entry */
  const float* bias_values;    /* [requests][bias_width] */
  int64_t bias_stride;         /* of both */
  int64_t bias_width;          /* 0 .. 1024 */
  const uint32_t* mask;        /* NULL, or [mask_count][ceil(vocab / 32)]: bit v % 32 of word v / 32 allows token v */
  int64_t mask_stride;
  int64_t mask_count;          /* 0 .. 2^20 */
  const int32_t* mask_rows;    /* NULL (row r has mask r; mask_count >= rows), or [rows]: each row's mask; negative: none */
  const int32_t* draft_tokens; /* NULL, or [rows]: the drafted tree's tokens, a request's rows being its nodes */
  const uint64_t* tree_mask;   /* [rows][tree_words], as nf4_tree_attention's; with draft_tokens */
  int64_t tree_mask_stride;
  int64_t tree_words;          /* 1 .. 1024 */
} nf4_adjust_logits_args;

/*
 * nf4_adjust_logits -- what stands between the last GEMV and the choice of a
 * token. For a row of request b, c counts the times that token v stands in
 * the part of the request's history after its prompt, and, with draft_tokens,
 * among the nodes x of the request whose bit x is set in the row's tree_mask;
 * v is known where it stands there or in the prompt. (A row's own node and node 0
 * count where their bits are set: a history then ends before node 0.) Then, in binary32 and in
 * this order,
 *   known:  x = x > 0 ? x / repetition : x * repetition
 *   c > 0:  x = (x - fl(frequency * c)) - presence
 *   bias:   x = x + (the sum of v's entries in the bias list, in its order), where it has any
 *   out = -infinity where v's bit in the row's mask is 0, whatever x is; else x rounded once.
 * best: the lowest index of the row's largest output as stored; NaN counts as
 * larger than any number, zeros are equal. A row without an allowed token is
 * -infinity throughout, best 0. Rows that no request holds get the mask only.
 * Tokens of histories and bias lists at or past vocab (a history's and a
 * drafted one's also below 0) are not counted; a mask row at or past mask_count
 * is no mask; lengths and cu_rows are clamped; all set bit 1 of the device error
 * flags.
 * One launch; one pass over the logits. Fastest when the rows of logits and out
 * are whole numbers of 16 bytes apart. Where rows of a tree differ in their distance from
 * a 16-byte boundary (rows of odd length one after another), each row goes through the
 * history again: 16 trees of up to 32 rows of 50257 in bf16 over 3000 words take 75 us,
 * 51 with rows of 50264. Where rows of out lie otherwise than those of logits (padded
 * logits, a dense out), elements are moved one by one: 105 us, 51 into an out that is
 * padded alike, 50 in place.
 * Errors: NF4_ERR_NULL, NF4_ERR_INVALID_SIZE, NF4_ERR_UNSUPPORTED_DTYPE,
 *   NF4_ERR_MISALIGNED (a pointer not aligned to its element), NF4_ERR_CUDA.
 */
NF4_API nf4_status nf4_adjust_logits(const nf4_adjust_logits_args* args, nf4_stream_t stream);

typedef struct nf4_tree_commit_args {
  const int32_t* parents;      /* [tokens]: each node's parent, a number within its sequence; node 0's is not looked at */
  const int32_t* draft_tokens; /* [tokens] */
  const int32_t* targets;      /* [tokens]: the token that the model chose after each node */
  const int32_t* cu_q;         /* [batch + 1], as nf4_prefix_attention's; NULL: one token each (tokens == batch) */
  const int32_t* lens;         /* [batch]: own keys of each sequence, its n nodes the last of them */
  int64_t batch;               /* 0 .. 2^20 */
  int64_t tokens;              /* 0 .. 2^24 */
  int64_t max_path;            /* 1 .. 1024: nodes that a path may have */
  int32_t* accepted;           /* [batch]: nodes of the accepted path */
  int32_t* path;               /* [batch][max_path]: the nodes, in order; -1 behind the last */
  int32_t* chosen;             /* [batch][max_path]: the model's choice after each of them; -1 behind the last */
  int32_t* new_lens;           /* [batch]: own keys with the accepted nodes only; may be lens where there is no cache,
                                  else shares no entry with it */
  void* k_cache;               /* NULL: nothing is moved; else `layers` caches of 16-bit elements */
  int64_t k_layer_stride, k_page_stride, k_slot_stride, k_head_stride;
  void* v_cache;
  int64_t v_layer_stride, v_page_stride, v_slot_stride, v_head_stride;
  int64_t layers;              /* 0 .. 65535 */
  int64_t num_pages, page_size, k_heads, head_dim; /* as nf4_kv_append's; head_dim 1 .. 512 */
  const int32_t* page_table;   /* [batch][width]: pages of each sequence's own keys */
  int64_t page_table_stride;
  int64_t width;
} nf4_tree_commit_args;

/*
 * nf4_tree_commit -- the accepted branch of each sequence's tree. The path
 * starts at node 0; after node x comes the lowest child y > x of x with
 * draft_tokens[y] == targets[x], until there is none or the path has max_path
 * nodes. accepted counts the path's nodes, chosen lists targets along it (the
 * sequence's new tokens, the last of which is the next tree's node 0), new_lens
 * is lens - n + accepted, or 0 where that is negative. With caches, the keys and
 * values of the path's node j (own key lens - n + path[j]) move to own key
 * lens - n + j, in every layer; the rejected nodes' slots then hold anything.
 * The two caches, and their layers, pages, slots and heads, must not overlap (nor may
 * two sequences share a page that is moved). Of such caches this call refuses equal
 * base pointers and strides of 0 of a dimension of more than one; the rest is the
 * caller's to see to. (The Python entry point sees how large its tensors are, and
 * refuses any that share an element.)
 * A sequence without nodes: accepted 0, path and chosen -1, new_lens = lens.
 * A node whose parent is not a node before it is on no path, nor is one past
 * the first 4096 of its sequence; a row whose slot
 * lies on a page out of range, or past the table's width, is not moved; nor is one of
 * a sequence's first nodes where lens is less than its nodes, so that these have no
 * own key; cu_q is clamped; all set bit 1 of the device error flags, and so does such
 * a lens where nothing would move.
 * Fastest when head_dim and the strides are multiples of 8 and the caches
 * 16-byte aligned. One launch.
 * Errors: NF4_ERR_NULL, NF4_ERR_INVALID_SIZE, NF4_ERR_MISALIGNED, NF4_ERR_CUDA.
 */
NF4_API nf4_status nf4_tree_commit(const nf4_tree_commit_args* args, nf4_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* NF4_DECODING_H_ */
