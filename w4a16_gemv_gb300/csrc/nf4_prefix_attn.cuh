// nf4_prefix_attn.cuh -- what the kernels of nf4_prefix_attention share: the
// arguments and the plan, the work items, and the paged rows of a cache.
#pragma once

#include "nf4_attn.cuh"

namespace nf4 {

// One call. A "row" of a key/value head is a (token, query head of its group)
// pair: row r of a segment of tokens is token r / group, query head
// k_head * group + r % group. A work item is a tile of rows against a range of
// keys; it leaves an unscaled partial output (binary32), the running maximum
// (of scores times log2 e) and the running sum, and a last kernel joins them,
// or, where a row has one item of own keys, that item.
struct PrefixArgs {
  const char* q;
  char* out;
  const char* k;
  const char* v;
  int64_t q_ts, q_hs, out_ts, out_hs;              // bytes
  int64_t k_ps, k_ss, k_hs, v_ps, v_ss, v_hs;      // bytes
  float* lse;
  const int32_t* prefix_pages;
  const int32_t* suffix_pages;
  const int32_t* suffix_lens;
  const int32_t* cu_q;
  int64_t suffix_pages_stride;
  int suffix_max;                                  // keys that the page table of a sequence can hold
  int prefix_len;
  int batch, tokens, q_heads, k_heads, group, dim;
  int page_size, page_shift, num_pages;            // page_shift: log2 of page_size, or -1
  float scale_log2;                                // scale * log2(e)
  // plan
  int prefix_rows, suffix_rows;                    // rows per tile: 16, 64 or 256
  int prefix_tiles, suffix_tiles;                  // tiles of a key/value head (suffix: the numbers they take)
  int tile_per_row;                                // 1: tiles of own rows are numbered by their first row
  int prefix_splits, suffix_splits;                // ranges of keys, of this many each:
  int prefix_chunk, suffix_chunk;
  int splits;                                      // prefix_splits + suffix_splits
  int direct;                                      // 1: the items write the output
  int fused;                                       // 1: one range of own keys, whose items write the output, with
                                                   // the one range of shared keys, if any, joined in
  int stream;                                      // 1: the shared keys leave L2 first
  int first;                                       // first item of the launch
  int beside;                                      // 1: runs beside the launch before it of the same call
  float* part;                                     // [splits][tokens * q_heads][dim]
  float2* ml;                                      // [tokens * q_heads][splits]: (maximum, sum)
};

// Keys of a tile of the tcgen05 kernel: 128, or the whole pages that nearly fill
// that (120 for pages of 24, 40 or 120, 112 for 56), whose largest power of two,
// eight, would make a tile of 16 or 32 copies (about 100 cycles each: 6 sequences
// of 160 tokens x 32 heads over 4188 keys in pages of 24 took 115 us, now 80; in
// pages of 32 71).
inline int prefix_tile_keys(int64_t page_size) {
  if (page_size % 16 != 8 || page_size > 128) return 128;
  const int keys = int(128 / page_size * page_size);
  return page_size > 8 && keys >= 112 ? keys : 128;
}

// The sizes and the plan of a call, and the bytes of its workspace.
void plan_prefix_attention(const nf4_prefix_attention_args& a, PrefixArgs* p, size_t* bytes);

// Items [p.first, p.first + items), tiles of 256 rows, on the tensor cores
// (nf4_prefix_attn_tc.cu).
cudaError_t launch_prefix_tc(const PrefixArgs& p, nf4_dtype dtype, unsigned items, cudaStream_t stream);

// One work item, the same in every thread.
struct PrefixItem {
  const int32_t* pages;
  int head;        // key/value head
  int split;       // its place among a row's partial results
  int t0;          // first token of the segment
  int n;           // tokens of the segment
  int r0;          // first row of the tile, within the segment
  int rows;        // rows of the tile (0: nothing to do)
  int k0, k1;      // keys of the item, within the segment's keys (k0 >= k1: none)
  int len;         // keys of the segment
  bool own;        // the sequence's own keys: token i sees the first len - n + i + 1
};

// Keys of the segment that token i (of n) sees.
__device__ __forceinline__ int visible_keys(const PrefixItem& it, int i) {
  return it.own ? min(max(it.len - it.n + i + 1, 0), it.len) : it.len;
}

// Tiles of own rows are numbered so that the sequence of a tile is found without
// counting the tiles of those before it: sequence b, with the rows [x, y) of a
// key/value head, has the numbers from x / suffix_rows + b on (rounded down; y / suffix_rows
// + b + 1 is the next one's first, which leaves room for its ceil((y - x) / suffix_rows)
// tiles), or from x on where that makes fewer numbers in all. Numbers past a
// sequence's rows are empty items. (8192 sequences x 2 heads over 200 own keys of 64:
// 120 us; with a scan of the batch for every tile 620.)
__device__ __forceinline__ int first_tile(const PrefixArgs& a, int t0, int b) {
  return a.tile_per_row ? t0 * a.group : ((t0 * a.group) >> (31 - __clz(a.suffix_rows))) + b;
}

// Item `index` of a launch that covers prefix items first (a key/value head's
// tiles of one key range side by side, so that they meet in L2), then suffix
// items. Called by whole warps.
__device__ __forceinline__ PrefixItem prefix_item(const PrefixArgs& a, unsigned index, unsigned int* flags) {
  PrefixItem it;
  const unsigned prefix_items = unsigned(a.prefix_tiles) * unsigned(a.k_heads) * unsigned(a.prefix_splits);
  if (index < prefix_items) {
    const unsigned rest = index / unsigned(a.prefix_tiles);
    const int tile = int(index - rest * unsigned(a.prefix_tiles));
    it.split = int(rest / unsigned(a.k_heads));
    it.head = int(rest) - it.split * a.k_heads;
    it.t0 = 0;
    it.n = a.tokens;
    it.r0 = tile * a.prefix_rows;
    it.rows = min(a.prefix_rows, a.tokens * a.group - it.r0);
    it.pages = a.prefix_pages;
    it.len = a.prefix_len;
    it.own = false;
    it.k0 = int(min(int64_t(it.split) * a.prefix_chunk, int64_t(it.len)));
    it.k1 = int(min(int64_t(it.k0) + a.prefix_chunk, int64_t(it.len)));
    return it;
  }
  index -= prefix_items;
  const unsigned rest = index / unsigned(a.suffix_tiles);
  const int tile = int(index - rest * unsigned(a.suffix_tiles));
  const int split = int(rest / unsigned(a.k_heads));
  it.head = int(rest) - split * a.k_heads;
  it.split = a.prefix_splits + split;
  it.own = true;
  it.rows = 0;
  it.r0 = it.t0 = it.n = it.len = it.k0 = it.k1 = 0;
  it.pages = a.suffix_pages;
  const int lane = threadIdx.x & 31;
  // The tile's sequence is the last whose first tile is at or before it. One
  // token each: b group / suffix_rows + b < tile + 1, solved for b (the product is at
  // most rows + batch * suffix_rows, below 2^31). Else a search of cu_q, 32 looks at a
  // time; whatever stands there, it ends at a sequence of the batch.
  int b0 = 0, span = a.batch;
  if (!a.cu_q) {
    const unsigned last =
        a.tile_per_row ? unsigned(tile) / unsigned(a.group)
                       : (unsigned(tile + 1) * unsigned(a.suffix_rows) - 1u) / unsigned(a.group + a.suffix_rows);
    b0 = min(int(last), a.batch - 1);
    span = 1;
  } else {
    while (span > 32) {
      const int step = (span + 31) >> 5, at = lane * step;
      const bool before = at < span && first_tile(a, min(max(a.cu_q[b0 + at], 0), a.tokens), b0 + at) <= tile;
      const int src = 31 - __clz(int(__ballot_sync(0xffffffffu, before) | 1u));
      b0 += src * step;
      span = min(step, span - src * step);
    }
  }
  int lo = 0, hi = 0, length = 0;
  if (lane < span) {
    length = a.suffix_lens[b0 + lane];  // with cu_q, not after it: one latency
    lo = a.cu_q ? a.cu_q[b0 + lane] : b0;
    hi = a.cu_q ? a.cu_q[b0 + lane + 1] : b0 + 1;
    const int l2 = min(max(lo, 0), a.tokens), h2 = min(max(hi, l2), a.tokens);
    if (l2 != lo || h2 != hi) atomicOr(flags, kFlagBadIndex);
    lo = l2;
    hi = h2;
  }
  const int mine = first_tile(a, lo, b0 + lane);
  const int src = 31 - __clz(int(__ballot_sync(0xffffffffu, lane < span && mine <= tile) | 1u));
  const int first = __shfl_sync(0xffffffffu, mine, src);
  it.t0 = __shfl_sync(0xffffffffu, lo, src);
  it.n = __shfl_sync(0xffffffffu, hi, src) - it.t0;
  const int len = __shfl_sync(0xffffffffu, length, src);
  if (tile < first || tile - first >= (it.n * a.group + a.suffix_rows - 1) >> (31 - __clz(a.suffix_rows))) return it;
  it.r0 = (tile - first) * a.suffix_rows;
  it.rows = min(a.suffix_rows, it.n * a.group - it.r0);
  it.len = min(max(len, 0), a.suffix_max);
  if (it.len != len && lane == 0) atomicOr(flags, kFlagBadIndex);
  it.pages = a.suffix_pages + int64_t(b0 + src) * a.suffix_pages_stride;
  const int sees = visible_keys(it, (it.r0 + it.rows - 1) / a.group);  // the tile's last row sees most
  it.k0 = int(min(int64_t(split) * a.suffix_chunk, int64_t(sees)));
  it.k1 = int(min(int64_t(it.k0) + a.suffix_chunk, int64_t(sees)));
  return it;
}

// Byte offsets of key j's rows in the two caches. A page out of range is
// reported; its keys are then taken as zeros (false).
struct KeyOffset {
  int64_t k, v;
};
__device__ __forceinline__ int key_page(const PrefixArgs& a, const PrefixItem& it, int j) {
  return it.pages[a.page_shift >= 0 ? j >> a.page_shift : j / a.page_size];
}
__device__ __forceinline__ bool key_offset(const PrefixArgs& a, const PrefixItem& it, int j, int page,
                                           unsigned int* flags, KeyOffset* off) {
  if (unsigned(page) >= unsigned(a.num_pages)) {
    atomicOr(flags, kFlagBadIndex);
    return false;
  }
  const int slot = a.page_shift >= 0 ? j & (a.page_size - 1) : j % a.page_size;
  off->k = int64_t(page) * a.k_ps + int64_t(slot) * a.k_ss + int64_t(it.head) * a.k_hs;
  off->v = int64_t(page) * a.v_ps + int64_t(slot) * a.v_ss + int64_t(it.head) * a.v_hs;
  return true;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrowth = 8.0f;  // log2 of the growth of a row's maximum that is let pass

// Weights are 2^(s - m + kLift<H>), s and m (the maximum) times log2 e. In
// binary16 a weight rounds to a multiple of 2^-24, so that without a lift all
// below 2^-25 would be lost to the product with v while the sum counts them.
// Lifted by 7 bits, a weight stays below 2^(7 + kGrowth) = 2^15.
template <typename H>
constexpr float kLift = H::kDtype == NF4_FP16 ? 7.0f : 0.0f;

// Keys of a range. Its sums are binary32, and one that holds a large weight loses
// what is added below 2^-25 of it (the tensor cores align every product with the
// accumulator and cut it off there): up to 2^17 x 2^-25 = 2^-8 of the range, one
// rounding of bf16, and with the lift 2^17 x 2^-32 more in binary16.
constexpr int64_t kMostKeys = int64_t(1) << 17;

// Where a finished row goes: the partial results, or the output itself.
struct RowOut {
  int64_t row;
  float* part;
  float2* ml;
  char* out;
  float* lse;
};
__device__ __forceinline__ RowOut row_out(const PrefixArgs& a, const PrefixItem& it, int r) {
  const int t = it.t0 + r / a.group;
  const int h = it.head * a.group + r % a.group;
  const int64_t row = int64_t(t) * a.q_heads + h;
  RowOut o;
  o.row = row;
  o.part = a.part + (int64_t(it.split) * a.tokens * a.q_heads + row) * a.dim;
  o.ml = a.ml + row * a.splits + it.split;
  o.out = a.out + int64_t(t) * a.out_ts + int64_t(h) * a.out_hs;
  o.lse = a.lse ? a.lse + row : nullptr;
  return o;
}

// Four columns of an output row from its sum l, its maximum m and v.
template <typename H>
__device__ __forceinline__ void write_row(char* out, float* lse, int col, float m, float l, const float4& v) {
  const bool any = l > 0.0f || l != l;
  const float inv = any ? 1.0f / l : 0.0f;
  *reinterpret_cast<uint2*>(out + col * 2) =
      make_uint2(H::down2(v.x * inv, v.y * inv), H::down2(v.z * inv, v.w * inv));
  if (col == 0 && lse) *lse = any ? fmaf(m, kLn2, logf(l)) : -INFINITY;
}

// Whether a part (maximum, sum) holds a key, and its weight when the row's
// maximum is m. (A maximum of -inf with a sum: of NaN.)
__device__ __forceinline__ bool part_holds(const float2& x) { return !(x.x == -INFINITY && x.y == 0.0f); }
__device__ __forceinline__ float part_weight(const float2& x, float m) {
  return x.x == -INFINITY ? 1.0f : ex2(x.x - m);
}

// Row `row` with shared keys only (one range of them, or none), by a whole warp.
template <typename H>
__device__ __forceinline__ void shared_row(const PrefixArgs& a, int64_t row) {
  const int col = int(threadIdx.x & 31u) * 4;
  if (col >= a.dim) return;
  float2 x = make_float2(-INFINITY, 0.0f);
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.splits > 0) {
    x = a.ml[row];
    if (part_holds(x)) v = *reinterpret_cast<const float4*>(a.part + row * a.dim + col);
  }
  const int64_t t = row / a.q_heads;
  char* const out = a.out + t * a.out_ts + (row - t * a.q_heads) * a.out_hs;
  write_row<H>(out, a.lse ? a.lse + row : nullptr, col, x.x, x.y, v);
}

// Reports entries of cu_q out of range, where an item's search does not look at
// all of them (more than 32 sequences). By the first `warps` warps of every CTA of
// a call's last launch, at its end.
__device__ __forceinline__ void check_cu_q(const PrefixArgs& a, int warps, unsigned int* flags) {
  if (!a.cu_q || a.suffix_splits == 0 || a.batch <= 32) return;
  for (int64_t b = int64_t(blockIdx.x) * warps * 32 + threadIdx.x; b < a.batch; b += int64_t(gridDim.x) * warps * 32) {
    const int lo = a.cu_q[b], hi = a.cu_q[b + 1];
    if (lo < 0 || hi < lo || hi > a.tokens) atomicOr(flags, kFlagBadIndex);
  }
}

// The rows of tokens that no sequence holds, dealt out to the first `warps`
// warps of every CTA of a launch of own items; and the check above.
template <typename H>
__device__ __forceinline__ void unheld_rows(const PrefixArgs& a, int warps, unsigned int* flags) {
  if (!a.cu_q) return;
  const int lo = min(max(a.cu_q[0], 0), a.tokens), hi = min(max(a.cu_q[a.batch], lo), a.tokens);
  const int64_t rows = int64_t(lo + a.tokens - hi) * a.q_heads;
  for (int64_t r = int64_t(blockIdx.x) * warps + (threadIdx.x >> 5); r < rows; r += int64_t(gridDim.x) * warps)
    shared_row<H>(a, r < int64_t(lo) * a.q_heads ? r : r + int64_t(hi - lo) * a.q_heads);
  check_cu_q(a, warps, flags);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace nf4
