// nf4_kv_pages.cu -- page tables and slots of a batch's new tokens, from the
// requests' lengths.
//
// Request b needs p_b = ceil((L_b + n_b) / page_size) pages. With back_b =
// max(h_b - p_b, 0), the pages past the need go to stack places
// F + sum_{c<b} back_c ..; with grow_b = max(p_b - h_b, 0) the missing ones are
// those at top - 1 - sum_{c<b} grow_c and below. Both are exclusive sums over the
// batch, so every request knows its places without waiting for the others.
//
// One cluster: every CTA forms the sums of the whole batch by itself (a few
// bytes per request), then the CTAs share the pages and the tokens. A token's page
// is looked up where it comes from (its row of the table, or the stack), not in
// the table after it has been written, so that both go on at once; a barrier of the
// cluster stands only where pages come back before any are taken, and in front of
// the results that may be the same arrays as inputs. Where there are many tokens,
// or more requests than a CTA has threads, a second launch lays them out on all SMs,
// from the tables as they are then (256 prompts, 115000 tokens: 8.0 us; by one
// cluster of eight CTAs 19).
// Latency bounds both: a chain of loads, sums, loads and stores.
#include "nf4_decoding.cuh"

namespace nf4 {
namespace {

__device__ unsigned int g_pages_flags = 0;

constexpr int kMostThreads = 1024;
constexpr int kNone = 0x7fffffff;
constexpr int kApart = 4096;  // more tokens than this have a launch of their own

struct PagesArgs {
  nf4_kv_pages_args a;
  int page_shift;  // log2 of page_size, or -1
  int apart;       // 1: the tokens have a launch of their own
};

// One request: L cached keys, n new tokens, h pages held, `need` needed.
struct Request {
  unsigned len, n, held, need;
  unsigned grow, back;
  bool wide;  // needs more pages than its row of the table has
};

__device__ __forceinline__ unsigned pages_of(const PagesArgs& p, unsigned keys) {
  const unsigned up = keys + unsigned(p.a.page_size) - 1u;  // below 2^31 + 2^24 + 2^16
  return p.page_shift >= 0 ? up >> p.page_shift : up / unsigned(p.a.page_size);
}

__device__ __forceinline__ Request request_of(const PagesArgs& p, int b, bool* bad) {
  Request r = {};
  if (b >= p.a.batch) return r;
  const int len = p.a.lens[b], held = p.a.held[b];
  int lo, hi;
  token_range(p.a.cu_q, b, int(p.a.tokens), &lo, &hi, bad);
  r.len = unsigned(max(len, 0));
  r.n = unsigned(hi - lo);
  r.held = unsigned(min(max(held, 0), int(p.a.width)));
  *bad = *bad || int(r.len) != len || int(r.held) != held;
  r.need = pages_of(p, r.len + r.n);
  r.wide = r.need > unsigned(p.a.width);
  *bad = *bad || r.wide;
  r.grow = !r.wide && r.need > r.held ? r.need - r.held : 0u;
  r.back = r.need < r.held ? r.held - r.need : 0u;
  return r;
}

// Exclusive sum over the block; *total in every thread.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* sums, uint64_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  uint64_t s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  __syncthreads();  // the sums of the last scan have been read
  if (lane == 31) sums[warp] = s;
  __syncthreads();
  uint64_t w = lane < warps ? sums[lane] : 0ull;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const uint64_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return s - v + (warp > 0 ? before : 0ull);
}

// Last of the n entries that is at most v (entry 0 is).
template <typename V>
__device__ __forceinline__ int last_at_most(const V* list, int n, V v) {
  int at = 0;
  for (int step = 1 << (31 - __clz(n)); step > 0; step >>= 1)
    if (at + step < n && list[at + step] <= v) at += step;
  return at;
}

// Where token t, the i-th of a request with len keys, goes.
__device__ __forceinline__ int64_t position_of(const PagesArgs& p, int t, unsigned len, int i) {
  return p.a.first_position + len + (p.a.depths ? p.a.depths[t] : i);
}
__device__ __forceinline__ unsigned page_number(const PagesArgs& p, unsigned key) {
  return p.page_shift >= 0 ? key >> p.page_shift : key / unsigned(p.a.page_size);
}
__device__ __forceinline__ int64_t slot_of(const PagesArgs& p, int page, unsigned key, unsigned at, bool* bad) {
  *bad = *bad || page < 0;
  return page < 0 ? -1 : int64_t(page) * p.a.page_size + (key - at * unsigned(p.a.page_size));
}

__global__ void __launch_bounds__(kMostThreads, 1) kv_pages_kernel(const __grid_constant__ PagesArgs p) {
  const nf4_kv_pages_args& a = p.a;
  // of a chunk of requests: its missing (or surplus) pages' first place in the chunk, and the first one's place in
  // its row; of a batch of one chunk also first tokens and lengths
  __shared__ uint64_t start[kMostThreads];
  __shared__ unsigned first[kMostThreads];
  __shared__ int s_cu[kMostThreads + 1];
  __shared__ unsigned s_len[kMostThreads];
  __shared__ uint64_t sums[32];
  __shared__ uint64_t s_limit;
  __shared__ int s_failed;
  pdl_wait_prior_grid();
  pdl_allow_dependents();
  const int tid = threadIdx.x, threads = blockDim.x;
  const unsigned rank = cluster_rank(), ctas = cluster_size();
  const int share = int(rank) * threads + tid, shares = int(ctas) * threads;
  const int batch = int(a.batch), tokens = int(a.tokens);
  const bool one_chunk = batch <= threads;
  bool bad = false;

  // Pages that come back.
  const int count = a.free_count[0], capacity = int(a.capacity);
  const int free0 = min(max(count, 0), capacity);
  bad = free0 != count;
  Request r = {};
  uint64_t back = 0;
  for (int b0 = 0; b0 < batch; b0 += threads) {
    r = request_of(p, b0 + tid, &bad);
    back += r.back;
  }
  if (tid == 0) s_failed = kNone;
  int top = free0;
  if (__syncthreads_or(back != 0)) {
    uint64_t done = 0;
    for (int b0 = 0; b0 < batch; b0 += threads) {
      if (!one_chunk) r = request_of(p, b0 + tid, &bad);
      uint64_t total;
      const uint64_t mine = block_scan(r.back, sums, &total);
      start[tid] = mine;
      first[tid] = r.need;
      __syncthreads();
      for (uint64_t e = share; e < total; e += shares) {
        const int i = last_at_most(start, threads, e);
        const int page = a.page_table[int64_t(b0 + i) * a.page_table_stride + first[i] + (e - start[i])];
        const uint64_t to = uint64_t(free0) + done + e;
        if (to < uint64_t(capacity)) a.free_pages[to] = page;
      }
      done += total;
    }
    bad = bad || uint64_t(free0) + done > uint64_t(capacity);
    top = int(min(uint64_t(free0) + done, uint64_t(capacity)));
    cluster_barrier();
  }

  // Pages that are taken. A request is served where the pages that it and those before it ask for are there;
  // `failed` is the first that is not.
  uint64_t taken = 0;
  int failed = kNone;
  for (int b0 = 0; b0 < batch; b0 += threads) {
    if (!one_chunk) r = request_of(p, b0 + tid, &bad);
    uint64_t total;
    const uint64_t mine = block_scan(r.grow, sums, &total);
    start[tid] = mine;
    first[tid] = r.held;
    if (tid == 0) s_limit = total;
    if (one_chunk && b0 + tid < batch) {
      int lo, hi;
      token_range(a.cu_q, tid, tokens, &lo, &hi, &bad);
      s_cu[tid] = lo;
      if (tid + 1 == batch) s_cu[batch] = hi;
      s_len[tid] = r.len;
    }
    if (taken + total > uint64_t(top)) {  // the same in every thread
      __syncthreads();
      if (r.grow > 0 && taken + mine + r.grow > uint64_t(top)) atomicMin(&s_failed, b0 + tid);
      __syncthreads();
      failed = s_failed;
      if (failed == b0 + tid) s_limit = mine;
    }
    __syncthreads();
    const uint64_t limit = s_limit;
    for (uint64_t e = share; e < limit; e += shares) {
      const int i = last_at_most(start, threads, e);
      a.page_table[int64_t(b0 + i) * a.page_table_stride + first[i] + (e - start[i])] =
          __ldcg(a.free_pages + (uint64_t(top) - 1 - taken - e));
    }
    taken += limit;
    if (failed != kNone) break;
  }
  auto served = [&](const Request& q, int b) { return !q.wide && (q.need <= q.held || b < failed); };

  // The tokens, of a batch of one chunk.
  if (!p.apart) {
#pragma unroll 1
    for (int t = share; t < tokens; t += shares) {
      int64_t slot = -1, position = 0;
      const int b = batch == 0 ? -1 : a.cu_q ? last_at_most(s_cu, batch, t) : t;
      const int lo = b < 0 ? 0 : s_cu[b], hi = b < 0 ? 0 : a.cu_q ? s_cu[b + 1] : t + 1;
      if (t >= lo && t < hi) {
        const unsigned len = s_len[b], held = first[b], need = pages_of(p, len + unsigned(hi - lo));
        const unsigned key = len + unsigned(t - lo), at = page_number(p, key);
        position = position_of(p, t, len, t - lo);
        if (need <= unsigned(a.width) && (need <= held || b < failed))
          slot = slot_of(p, __ldcg(at < held ? a.page_table + int64_t(b) * a.page_table_stride + at
                                             : a.free_pages + (uint64_t(top) - 1 - start[b] - (at - held))),
                         key, at, &bad);
      }
      a.slots[t] = slot;
      if (a.positions) a.positions[t] = position;
    }
  }

  // The requests' results, when nobody needs held and free_count as they were.
  cluster_barrier();
  for (int b = share; b < batch; b += shares) {
    if (!one_chunk) r = request_of(p, b, &bad);  // else this thread's own
    const bool yes = served(r, b);
    a.new_held[b] = int(yes ? r.need : r.held);
    a.new_lens[b] = int(yes ? r.len + r.n : r.len);
  }
  if (share == 0) {
    a.new_free_count[0] = top - int(taken);
    if (failed != kNone) atomicOr(&g_pages_flags, kFlagNoPages);
  }
  if (bad) atomicOr(&g_pages_flags, kFlagBadIndex);
}

// The tokens, from the tables, held pages and lengths that the launch before has written: a request whose pages
// are all there was served. Whole warps find the request of their first token, the lanes go on from there.
__global__ void __launch_bounds__(256) kv_slots_kernel(const __grid_constant__ PagesArgs p) {
  const nf4_kv_pages_args& a = p.a;
  pdl_wait_prior_grid();
  pdl_allow_dependents();
  const int tokens = int(a.tokens), batch = int(a.batch), t = int(blockIdx.x) * 256 + int(threadIdx.x);
  bool bad = false;
  int b = batch > 0 ? entry_of(a.cu_q, batch, tokens, t & ~31) : -1;
  if (t >= tokens) return;
  int64_t slot = -1, position = 0;
  if (b >= 0) {
    if (!a.cu_q) {
      b = t;
    } else {
      int steps = 0;
      while (b + 1 < batch && steps < 32 && offset_at(a.cu_q, b + 1, tokens) <= t) {
        ++b;
        ++steps;
      }
      for (int step = steps < 32 ? 0 : 1 << (31 - __clz(batch)); step > 0; step >>= 1)  // many empty requests
        if (b + step < batch && offset_at(a.cu_q, b + step, tokens) <= t) b += step;
    }
    int lo, hi;
    bool ignored = false;  // (reported by the launch before)
    token_range(a.cu_q, b, tokens, &lo, &hi, &ignored);
    if (t >= lo && t < hi) {
      const unsigned len = unsigned(max(a.lens[b], 0)), need = pages_of(p, len + unsigned(hi - lo));
      const unsigned key = len + unsigned(t - lo), at = page_number(p, key);
      position = position_of(p, t, len, t - lo);
      if (need <= unsigned(a.width) && need <= unsigned(max(a.new_held[b], 0)))
        slot = slot_of(p, a.page_table[int64_t(b) * a.page_table_stride + at], key, at, &bad);
    }
  }
  a.slots[t] = slot;
  if (a.positions) a.positions[t] = position;
  if (bad) atomicOr(&g_pages_flags, kFlagBadIndex);
}

}  // namespace

cudaError_t launch_kv_pages(const nf4_kv_pages_args& a, cudaStream_t stream) {
  PagesArgs p;
  p.a = a;
  p.page_shift = -1;
  for (int s = 0; s <= 16; ++s)
    if (a.page_size == int64_t(1) << s) p.page_shift = s;
  const unsigned threads = a.batch > 256 || a.tokens > 256 ? kMostThreads : 256;
  p.apart = a.tokens > kApart || (a.batch > kMostThreads && a.tokens > 0);
  unsigned ctas = 1;
  while (ctas < 4 && (p.apart || a.tokens > int64_t(ctas) * threads)) ctas *= 2;
  const cudaError_t e = launch_cluster(kv_pages_kernel, ctas, dim3(ctas), dim3(threads), 0, stream, p);
  if (e != cudaSuccess || !p.apart) return e;
  return launch_k(kv_slots_kernel, dim3(unsigned((a.tokens + 255) / 256)), dim3(256), 0, stream, p);
}

cudaError_t pages_flags(unsigned int** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_pages_flags);
}

}  // namespace nf4
