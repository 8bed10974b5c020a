// nf4_adjust_logits.cu -- penalties for repeated tokens, biases and masks on
// rows of logits, and each row's best token, in one pass.
//
// A cluster of CTAs takes a run of rows, each CTA every eighth (fourth, second) block
// of 256 tokens: frequent tokens often have low numbers, and in one piece the first
// part of a vocabulary would be most of the work. What a request's history, its
// bias list and a row's branch of the tree say about a token is one word in the
// shared memory of the token's CTA (how often it stands in the answer, whether it is
// known at all, whether it has a bias) and one bit that says that there is a word.
// These are made once per request and run of rows, by every CTA from the whole history
// (a warp picks what is in its CTA, about one in four, and counts that 32 at a time.
// Sharing the history among the CTAs and adding to one another's shared memory took
// longer: an SM does a remote addition every seven cycles).
// From one row to the next only the branch changes. Then each CTA streams its tokens, 16 bytes at a time, with the
// mask alone, and the tokens with a word are worked out and written over that, a thread
// each: a few in a hundred, and done where they lie every warp would go through the
// division and the bias list for each of its chunks.
// The logits are read and written once: memory bounds many rows, a chain of loads
// (offsets, lengths, history) a few. Without a context 64 rows of 128000 in bf16 take
// 5.6 us and 384 in binary32 66 (5.9 and 6.0 TB/s); with masks, best tokens and 8000 (3000)
// words of history each 24 and 108, bound by instructions (1200 of 3250 per warp are the
// history's) and by the latencies between a row's stream and its listed tokens.
#include "nf4_decoding.cuh"
#include "nf4_prefix_attn.cuh"  // 16-byte asynchronous copies

namespace nf4 {
namespace {

__device__ unsigned int g_logits_flags = 0;

constexpr int kThreads = 512;
constexpr int kResident = 2;  // CTAs on an SM: 64 registers a thread
constexpr int kMostRows = 64; // of a cluster
constexpr int kBlock = 256;   // tokens that lie in one CTA
constexpr int kList = 8192;   // listed tokens of a slice; where there are more, every word is looked at

constexpr int kSteps = 2;     // pieces of the history, of 128 words, that a warp has under way,
constexpr int kQueue = 256;   // and words that it has picked: together where the list will be
static_assert((kSteps * 128 + kQueue) * (kThreads / 32) <= kList, "");
constexpr uint32_t kOnlyKnown = 1u << 31;  // of a picked word: it stands in the prompt

struct LogitsArgs {
  nf4_adjust_logits_args a;
  int slice;   // tokens of a CTA at a time, whole blocks
  int passes;  // slices of a CTA, one after another
  int per;     // rows of a cluster
  int ctas_log2;
};

// What is known about a token: 16 bits, or 32 where a count may not fit.
struct Narrow {
  static constexpr uint32_t kBiased = 0x8000u, kKnown = 0x4000u, kCount = 0x3fffu;
  static constexpr int kPerWord = 2;
};
struct Wide {
  static constexpr uint32_t kBiased = 1u << 31, kKnown = 1u << 30, kCount = kKnown - 1;
  static constexpr int kPerWord = 1;
};

// Element types, 16 bytes (a chunk) at a time: the largest, NaN above all; a chunk with
// the elements whose bit is 0 replaced by -infinity; single ones.
struct F32 {
  using Store = float;
  static __device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
  }
  static __device__ __forceinline__ float largest(const uint4& r) {
    return max_nan(max_nan(__uint_as_float(r.x), __uint_as_float(r.y)), max_nan(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
  static __device__ __forceinline__ uint4 allow(uint4 r, uint32_t bits) {
    constexpr uint32_t kNone = 0xff800000u;
    return make_uint4(bits & 1u ? r.x : kNone, bits & 2u ? r.y : kNone, bits & 4u ? r.z : kNone, bits & 8u ? r.w : kNone);
  }
  static __device__ __forceinline__ float up1(float v) { return v; }
  static __device__ __forceinline__ float down1(float v) { return v; }
};
template <uint32_t kNone>  // -infinity, twice
struct Pairs {
  static __device__ __forceinline__ uint32_t pair(uint32_t r, uint32_t bits) {
    const uint32_t keep = (bits & 1u ? 0xffffu : 0u) | (bits & 2u ? 0xffff0000u : 0u);
    return (r & keep) | (kNone & ~keep);
  }
  static __device__ __forceinline__ uint4 allow(uint4 r, uint32_t bits) {
    return make_uint4(pair(r.x, bits), pair(r.y, bits >> 2), pair(r.z, bits >> 4), pair(r.w, bits >> 6));
  }
};
struct B16 : Pairs<0xff80ff80u> {
  using Store = __nv_bfloat16;
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float largest(const uint4& r) {
    const float2 f = Bf16::up2(max2(max2(r.x, r.y), max2(r.z, r.w)));
    return F32::max_nan(f.x, f.y);
  }
  static __device__ __forceinline__ float up1(Store v) { return __bfloat162float(v); }
  static __device__ __forceinline__ Store down1(float v) { return __float2bfloat16_rn(v); }
};
struct H16 : Pairs<0xfc00fc00u> {
  using Store = __half;
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float largest(const uint4& r) {
    const float2 f = Fp16::up2(max2(max2(r.x, r.y), max2(r.z, r.w)));
    return F32::max_nan(f.x, f.y);
  }
  static __device__ __forceinline__ float up1(Store v) { return __half2float(v); }
  static __device__ __forceinline__ Store down1(float v) { return __float2half_rn(v); }
};

// Larger values have larger keys; NaN the largest, zeros one key.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 + 0 = +0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// Where the tokens of a pass are: token v, as u = v + skew, in block u / kBlock; block x
// in CTA x % 2^log2, its blocks there being number `first` and on of all that it sees.
struct Places {
  int skew, rank, log2, first, blocks;
  __device__ __forceinline__ unsigned owner(int v) const { return unsigned((v + skew) / kBlock) & ((1u << log2) - 1u); }
  __device__ __forceinline__ int number(int v) const {  // within its CTA; -1: of another pass
    const int u = v + skew, nth = (u / kBlock >> log2) - first;
    return unsigned(nth) < unsigned(blocks) ? nth * kBlock + u % kBlock : -1;
  }
  __device__ __forceinline__ int here(int v) const {  // number(v) of a token of this CTA, else -1
    return owner(v) == unsigned(rank) ? number(v) : -1;
  }
  __device__ __forceinline__ int token(int at) const {  // may lie before or behind the vocabulary
    return ((((first + at / kBlock) << log2) + rank) * kBlock + at % kBlock) - skew;
  }
};
template <typename W>
__device__ __forceinline__ int shift_of(int at) {
  return W::kPerWord == 2 ? 16 * (at & 1) : 0;
}

__device__ __forceinline__ uint64_t best_key(float v, int at) { return uint64_t(order_key(v)) << 32 | uint32_t(~at); }

// kContext: there is a history, a branch or a bias list. kVector: rows of logits
// and out are alike modulo 16 bytes.
//
// Loads that do not depend on one another are asked for together (a request's
// lengths, factors, first words of history, bias and drafted tokens in one go), and
// the code is kept short: a few rows are a chain of memory latencies, and code that
// runs once per call is fetched once per call.
template <typename E, bool kVector, bool kContext, typename W>
__global__ void __launch_bounds__(kThreads, kResident) adjust_logits_kernel(const __grid_constant__ LogitsArgs p) {
  using S = typename E::Store;
  constexpr int V = kVector ? 16 / int(sizeof(S)) : 1;
  const nf4_adjust_logits_args& a = p.a;
  extern __shared__ __align__(16) uint32_t words[];  // of the CTA's tokens; then their bits, the listed tokens, the bias list
  __shared__ uint64_t s_best[kMostRows];             // of the rows, in this CTA,
  __shared__ uint64_t s_all[8][kMostRows];           // and (in the cluster's first) in all
  __shared__ int s_listed;
  uint32_t* const bits = words + p.slice / W::kPerWord;
  uint32_t* const s_list = bits + p.slice / 32;  // (16-byte aligned: slices are whole blocks; a bias list is any length)
  int* const s_bias = reinterpret_cast<int*>(s_list + kList);
  float* const s_value = reinterpret_cast<float*>(s_bias + a.bias_width);
  int* const s_stage = reinterpret_cast<int*>(s_list) + (threadIdx.x >> 5) * (kSteps * 128 + kQueue);
  uint32_t* const s_queue = reinterpret_cast<uint32_t*>(s_stage + kSteps * 128);
  const int tid = threadIdx.x;
  auto clear = [&]() {
    for (int i = tid; i < (p.slice / W::kPerWord + p.slice / 32) / 4; i += kThreads)
      reinterpret_cast<uint4*>(words)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) s_listed = 0;
  };
  if (kContext) clear();
  if (a.best) cluster_arrive();  // this CTA has begun
  pdl_wait_prior_grid();
  pdl_allow_dependents();
  // The CTA's part of the vocabulary: another one from cluster to cluster, since the CTAs of one rank often share an
  // SM, and the part with the most frequent words is the most work.
  const unsigned ctas = cluster_size(), part = (cluster_rank() + blockIdx.x / ctas) & (ctas - 1);
  const int vocab = int(a.vocab), rows = int(a.rows), mask_words = (vocab + 31) / 32;
  const int first_row = int(blockIdx.x / ctas) * p.per, end_row = min(first_row + p.per, rows);
  bool bad = false;
  if (a.best)
    for (int i = tid; i < p.per; i += kThreads) s_best[i] = 0;

  int b = -1, lo = 0, hi = 0;    // the row's request (-1: none) and its rows
  int built = -1, built_at = 0;  // what the words hold: a request, with the row's skew,
  int added = -1;                // and the branch of one of its rows
  int nodes = 0;
  float repetition = 1.0f, frequency = 0.0f, presence = 0.0f;

  for (int row = first_row; row < end_row; ++row) {
    const S* const in = reinterpret_cast<const S*>(a.logits) + int64_t(row) * a.logits_stride;
    S* const out = reinterpret_cast<S*>(a.out) + int64_t(row) * a.out_stride;
    // Tokens are numbered from the 16-byte boundary before the row: u = v + skew.
    const int skew = kVector ? int((reinterpret_cast<uintptr_t>(in) & 15u) / sizeof(S)) : 0;
    float most = 0.0f;
    int most_at = -1;    // the best that this thread streamed,
    uint64_t other = 0;  // and the best that it adjusted
    const uint32_t* mask = nullptr;
    if (a.mask) {
      const int m = a.mask_rows ? a.mask_rows[row] : row;
      bad = bad || m >= a.mask_count;
      if (m >= 0 && m < a.mask_count) mask = a.mask + int64_t(m) * a.mask_stride;
    }
    if (kContext && (row >= hi || row == first_row)) {
      b = -1;
      lo = row;
      hi = row + 1;
      if (a.requests > 0) {
        b = entry_of(a.cu_rows, int(a.requests), rows, row);
        int x0, x1;
        token_range(a.cu_rows, b, rows, &x0, &x1, &bad);
        if (row >= x0 && row < x1) {
          lo = x0;
          hi = x1;
        } else {
          b = -1;
        }
      }
    }
    const bool use = kContext && b >= 0;

    for (int pass = 0; pass < p.passes; ++pass) {
      const Places place{skew, int(part), p.ctas_log2, pass * (p.slice / kBlock), p.slice / kBlock};
      // Adds to (or ors into) a word of this CTA; true where the token was without a bit. (Most have theirs already:
      // a look is cheaper than an atomic operation on the few words that hold the bits of frequent tokens.)
      auto mark_at = [&](int at, uint32_t what, bool count) {
        uint32_t* const w = words + at / W::kPerWord;
        if (count)
          atomicAdd(w, what << shift_of<W>(at));
        else
          atomicOr(w, what << shift_of<W>(at));
        const uint32_t bit = 1u << (at & 31);
        return (bits[at / 32] & bit) == 0 && (atomicOr(bits + at / 32, bit) & bit) == 0;
      };
      auto exists = [&](int v) {
        bad = bad || unsigned(v) >= unsigned(vocab);
        return unsigned(v) < unsigned(vocab);
      };
      auto sees = [&](int r, int node) {
        return (a.tree_mask[int64_t(r) * a.tree_mask_stride + (node >> 6)] >> (node & 63) & 1ull) != 0;
      };
      const bool build = use && (b != built || skew != built_at || p.passes > 1);
      if (build) {
        if (built >= 0) {
          __syncthreads();  // the words have been read
          clear();
        }
        // What the request brings, asked for before any of it is looked at.
        const int width = a.history ? int(a.history_width) : 0;
        const int32_t* const h = a.history + int64_t(b) * a.history_stride;
        const int head = min(width, int((16u - (reinterpret_cast<uintptr_t>(h) & 15u)) % 16u / 4u));
        const int len = a.history ? a.history_lens[b] : 0;
        const int prompt = a.history && a.prompt_lens ? a.prompt_lens[b] : 0;
        repetition = a.repetition ? a.repetition[b] : 1.0f;
        frequency = a.frequency ? a.frequency[b] : 0.0f;
        presence = a.presence ? a.presence[b] : 0.0f;
        nodes = a.draft_tokens ? int(min(int64_t(hi - lo), a.tree_words * 64)) : 0;
        int draft = 0, biased = -1;
        bool on = false;
        if (tid < nodes) {
          draft = a.draft_tokens[lo + tid];
          on = sees(row, tid);
        }
        if (tid < int(a.bias_width)) {
          biased = a.bias_tokens[int64_t(b) * a.bias_stride + tid];
          s_value[tid] = a.bias_values[int64_t(b) * a.bias_stride + tid];
        }
        __syncthreads();  // all words are empty
        for (int i = tid; i < nodes; i += kThreads) {
          if (i > tid) {
            draft = a.draft_tokens[lo + i];
            on = sees(row, i);
          }
          if (on && exists(draft))
            if (const int at = place.here(draft); at >= 0) mark_at(at, 1u, true);
        }
        for (int j = tid; j < int(a.bias_width); j += kThreads) {
          if (j > tid) {
            biased = a.bias_tokens[int64_t(b) * a.bias_stride + j];
            s_value[j] = a.bias_values[int64_t(b) * a.bias_stride + j];
          }
          s_bias[j] = biased;
          if (biased >= 0 && exists(biased))
            if (const int at = place.here(biased); at >= 0) mark_at(at, W::kBiased, false);
        }
        // The history, 16 bytes at a time from its row's first boundary on. A warp copies its pieces ahead, picks the
        // words that are here into its queue and counts them from there, so that its lanes are all at work.
        const int n = min(max(len, 0), width), pieces = (max(n - head, 0) / 4 + 31) / 32;
        bad = bad || n != len || prompt < 0;
        const int lane = tid & 31, warp = tid >> 5, mine = (pieces - warp + kThreads / 32 - 1) / (kThreads / 32);
        const int whole_to = head + max(n - head, 0) / 4 * 4;  // the words of whole chunks end here
        auto copy = [&](int x) {                               // the warp's piece x
          const int j = head + ((x * (kThreads / 32) + warp) * 32 + lane) * 4;
          if (x < mine && j < whole_to) cp_async16(smem_u32(s_stage + x % kSteps * 128 + lane * 4), h + j, true);
          cp_async_commit();
        };
#pragma unroll 1
        for (int x = 0; x < kSteps; ++x) copy(x);
        if (tid < min(head, n) + max(n - whole_to, 0) && n > 0) {  // before the first chunk and behind the last
          const int j = tid < head ? tid : whole_to + tid - head, t = h[j];
          if (exists(t))
            if (const int at = place.here(t); at >= 0) mark_at(at, j < prompt ? W::kKnown : 1u, j >= prompt);
        }
        int held = 0;        // words in the queue
        unsigned worst = 0;  // the largest of the words
        // (u ^ first) & bits is 0 for the words of this CTA that are not negative
        const int first = int(part) * kBlock, bits_of = int(ctas - 1) * kBlock | int(0x80000000u);
#pragma unroll 1
        for (int x = 0; x <= mine; ++x) {
          const int j = head + ((x * (kThreads / 32) + warp) * 32 + lane) * 4;
          const bool real = x < mine && j < whole_to;
          cp_async_wait<kSteps - 1>();  // (this lane's words: no other's)
          int4 t = *reinterpret_cast<const int4*>(s_stage + x % kSteps * 128 + lane * 4);
          if (!real) t = make_int4(-1, -1, -1, -1);
          copy(x + kSteps);
          auto pick = [&](int v, int nth) {
            if (real) worst = max(worst, unsigned(v));
            const bool picked = ((int(unsigned(v) + unsigned(skew)) ^ first) & bits_of) == 0;
            const unsigned all = __ballot_sync(0xffffffffu, picked);
            if (picked) s_queue[held + __popc(all & ((1u << lane) - 1u))] = uint32_t(v) | (j + nth < prompt ? kOnlyKnown : 0u);
            held += __popc(all);
          };
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            pick(half ? t.z : t.x, 2 * half);
            pick(half ? t.w : t.y, 2 * half + 1);
          }
          if (held > kQueue - 128 || x == mine) {
            __syncwarp();
#pragma unroll 1
            for (int i = lane; i < held; i += 32) {
              const uint32_t w = s_queue[i];
              const int v = int(w & ~kOnlyKnown), at = v < vocab ? place.number(v) : -1;
              if (at >= 0) mark_at(at, w & kOnlyKnown ? W::kKnown : 1u, !(w & kOnlyKnown));
            }
            __syncwarp();
            held = 0;
          }
        }
        bad = bad || worst >= unsigned(vocab);
        cp_async_wait<0>();
      } else if (use) {
        __syncthreads();  // the words have been read
      }
      constexpr int kBatch = kContext ? 2 : 4;  // chunks of a thread under way (with four, registers spill)
      uint4 x[kBatch];
      uint32_t low[kBatch], high[kBatch];  // bits of the mask for these, from v0 & 31 on
      constexpr int kStep = kThreads * V;  // to the thread's next chunk: whole blocks,
      static_assert(!kVector || kStep % kBlock == 0, "");
      const int stride = kVector ? kStep << p.ctas_log2 : 0;  // so many tokens on
      auto next_token = [&](int v0, int at) { return kVector ? v0 + stride : place.token(at + kStep); };
      auto load = [&](int at, int v0) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k, v0 = next_token(v0, at), at += kStep) {
          low[k] = high[k] = 0xffffffffu;
          if (at >= p.slice || v0 < 0 || v0 + V > vocab) continue;
          if (kVector)
            x[k] = *reinterpret_cast<const uint4*>(in + v0);
          else
            *reinterpret_cast<S*>(&x[k]) = in[v0];
          if (mask) {
            low[k] = mask[v0 >> 5];
            if (kVector && skew != 0 && (v0 >> 5) + 1 < mask_words) high[k] = mask[(v0 >> 5) + 1];
          }
        }
      };
      const int token0 = place.token(tid * V);
      load(tid * V, token0);
      if (build) {
        __syncthreads();
        // The list: counted first, so that a warp takes its part at once.
        // (By bytes, so that the bits of frequent tokens, which lie side by side, are many lanes' work.)
        const uint8_t* const eight = reinterpret_cast<const uint8_t*>(bits);
        int mine = 0;
        for (int i = tid; i < p.slice / 8; i += kThreads) mine += __popc(eight[i]);
        int to = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, to, d);
          if ((tid & 31) >= d) to += y;
        }
        int start = 0;
        if ((tid & 31) == 31) start = atomicAdd(&s_listed, to);
        to += __shfl_sync(0xffffffffu, start, 31) - mine;
        for (int i = tid; i < p.slice / 8; i += kThreads)
          for (unsigned m = eight[i]; m; m &= m - 1, ++to)
            if (to < kList) s_list[to] = uint32_t(i * 8 + __ffs(int(m)) - 1);
        built = b;
        built_at = skew;
      } else if (use) {
        for (int i = tid; i < nodes; i += kThreads) {  // from the last row's branch to this one's
          const bool was = sees(added, i), is = sees(row, i);
          if (was == is) continue;
          const int v = a.draft_tokens[lo + i], at = exists(v) ? place.here(v) : -1;
          if (at >= 0 && mark_at(at, is ? 1u : ~0u, true)) {
            const int n = atomicAdd(&s_listed, 1);
            if (n < kList) s_list[n] = uint32_t(at);
          }
        }
        __syncthreads();
      }
      if (use) added = row;

      // The stream. Tokens with a word are left out of the choice of the best.
      for (int at = tid * V, v0 = token0; at < p.slice;) {
        if (at != tid * V) load(at, v0);
#pragma unroll
        for (int k = 0; k < kBatch; ++k, v0 = next_token(v0, at), at += kStep) {
          if (at >= p.slice || v0 < 0 || v0 + V > vocab) continue;
          const uint32_t allowed = __funnelshift_r(low[k], high[k], v0 & 31);
          if constexpr (kVector) {
            if ((~allowed & ((1u << V) - 1)) != 0) x[k] = E::allow(x[k], allowed);
            *reinterpret_cast<uint4*>(out + v0) = x[k];
          } else {
            if (!(allowed & 1u)) *reinterpret_cast<S*>(&x[k]) = E::down1(-INFINITY);
            out[v0] = *reinterpret_cast<const S*>(&x[k]);
          }
          if (!a.best) continue;
          const uint32_t has = use ? bits[at / 32] >> (at & 31) & ((1u << V) - 1) : 0u;
          float top;
          if constexpr (kVector) {  // (a token that is taken for -infinity here stands again among the listed ones)
            if (has != 0) x[k] = E::allow(x[k], ~has);
            top = E::largest(x[k]);
          } else {
            top = has ? -INFINITY : E::up1(*reinterpret_cast<const S*>(&x[k]));
          }
          if (most_at < 0 || (!(top <= most) && most == most)) {
            most = top;
            most_at = v0;
            if constexpr (kVector) {
#pragma unroll
              for (int i = V - 1; i > 0; --i) {  // the first that is the largest, or NaN
                const float y = E::up1(reinterpret_cast<const S*>(&x[k])[i]);
                const float y0 = E::up1(reinterpret_cast<const S*>(&x[k])[i - 1]);
                if (i == V - 1 && (y == top || y != y)) most_at = v0 + i;
                if (y0 == top || y0 != y0) most_at = v0 + i - 1;
              }
            }
          }
        }
      }

      // The listed tokens (where there are too many, every token with a word); and the tokens of the row's first and
      // last chunk, where these are not whole. Each once: out may be logits.
      if (use) __syncthreads();  // the stream has been written, and the list
      const int listed = use ? s_listed : 0;
      const int edges = kVector ? 2 * V : 0;
      const int start = kVector ? (V - skew) % V : 0, stop = kVector ? vocab - (vocab + skew) % V : vocab;
      const int count = edges + (listed > kList ? p.slice : listed);
      for (int e = tid; e < count; e += kThreads) {
        int v, at;
        if (e < edges) {
          v = e < V ? e : max(stop, start) + e - V;
          at = v < (e < V ? min(start, vocab) : vocab) ? place.here(v) : -1;
        } else {
          at = listed > kList ? e - edges : int(s_list[e - edges]);
          v = place.token(at);
          if (v < start || v >= stop || (listed > kList && (bits[at / 32] >> (at & 31) & 1u) == 0)) at = -1;
        }
        if (at < 0) continue;
        uint32_t w = use ? words[at / W::kPerWord] >> shift_of<W>(at) : 0u;
        if (W::kPerWord == 2) w &= 0xffffu;
        S y = in[v];
        if (mask && !(mask[v >> 5] >> (v & 31) & 1u)) {
          y = E::down1(-INFINITY);
        } else if (w != 0) {
          float z = E::up1(y);
          if (w & (W::kKnown | W::kCount)) z = z > 0.0f ? __fdiv_rn(z, repetition) : __fmul_rn(z, repetition);
          const uint32_t c = w & W::kCount;
          if (c) z = __fsub_rn(__fsub_rn(z, __fmul_rn(frequency, float(c))), presence);
          if (w & W::kBiased) {
            float sum = 0.0f;
#pragma unroll 4
            for (int j = 0; j < int(a.bias_width); ++j)
              if (s_bias[j] == v) sum = __fadd_rn(sum, s_value[j]);
            z = __fadd_rn(z, sum);
          }
          y = E::down1(z);
        }
        out[v] = y;
        if (a.best) {
          const uint64_t key = best_key(E::up1(y), v);
          other = key > other ? key : other;
        }
      }
    }
    if (a.best) {
      uint64_t key = most_at >= 0 ? best_key(most, most_at) : 0ull;
      key = other > key ? other : key;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        const uint64_t y = __shfl_xor_sync(0xffffffffu, key, d);
        key = y > key ? y : key;
      }
      if (row == first_row) __syncthreads();  // s_best is set
      if ((tid & 31) == 0) atomicMax(reinterpret_cast<unsigned long long*>(&s_best[row - first_row]), key);
    }
  }
  if (bad) atomicOr(&g_logits_flags, kFlagBadIndex);

  // Every CTA hands its rows' best to the cluster's first, and need not wait for it.
  if (a.best) {
    cluster_wait();  // the first has begun
    __syncthreads();
    const int n = end_row - first_row;
    for (int i = tid; i < n; i += kThreads) cluster_store64(cluster_address(smem_u32(&s_all[part][i]), 0), s_best[i]);
    cluster_arrive_release();
    if (cluster_rank() != 0) return;
    cluster_wait();
    for (int i = tid; i < n; i += kThreads) {
      uint64_t key = 0;
      for (unsigned r = 0; r < ctas; ++r) key = s_all[r][i] > key ? s_all[r][i] : key;
      a.best[first_row + i] = int(~uint32_t(key));
    }
  }
}

template <typename E, bool kVector, bool kContext, typename W>
cudaError_t launch(const LogitsArgs& p, unsigned ctas, cudaStream_t stream) {
  auto kern = adjust_logits_kernel<E, kVector, kContext, W>;
  const int64_t smem = kContext ? p.slice * 4 / W::kPerWord + p.slice / 8 + p.a.bias_width * 8 + kList * 4 : 0;
  static PerDeviceCache attr_set;
  const cudaError_t e = set_max_dynamic_smem_once(kern, kContext ? 216 * 1024 : 0, attr_set);
  if (e != cudaSuccess) return e;
  const int64_t clusters = (p.a.rows + p.per - 1) / p.per;
  return launch_cluster(kern, ctas, dim3(unsigned(clusters) * ctas), dim3(kThreads), size_t(smem), stream, p);
}
template <typename E, bool kVector>
cudaError_t launch_context(const LogitsArgs& p, bool context, bool wide, unsigned ctas, cudaStream_t stream) {
  return !context ? launch<E, kVector, false, Narrow>(p, ctas, stream)
         : wide   ? launch<E, kVector, true, Wide>(p, ctas, stream)
                  : launch<E, kVector, true, Narrow>(p, ctas, stream);
}
template <typename E>
cudaError_t launch_vector(const LogitsArgs& p, bool context, bool wide, unsigned ctas, cudaStream_t stream) {
  constexpr int V = 16 / int(sizeof(typename E::Store));
  // every row of logits and out the same distance from a 16-byte boundary
  const nf4_adjust_logits_args& a = p.a;
  const bool alike = ((reinterpret_cast<uintptr_t>(a.logits) - reinterpret_cast<uintptr_t>(a.out)) & 15u) == 0 &&
                     (a.rows <= 1 || (a.logits_stride - a.out_stride) % V == 0);
  return alike ? launch_context<E, true>(p, context, wide, ctas, stream)
               : launch_context<E, false>(p, context, wide, ctas, stream);
}

}  // namespace

cudaError_t launch_adjust_logits(const nf4_adjust_logits_args& a, cudaStream_t stream) {
  LogitsArgs p;
  p.a = a;
  if (!a.bias_tokens) p.a.bias_width = 0;
  const bool context = a.requests > 0 && ((a.history && a.history_width > 0) || a.draft_tokens || p.a.bias_width > 0);
  // the most that a count can become
  const int64_t count = (a.history ? a.history_width : 0) + (a.draft_tokens ? 64 * a.tree_words : 0);
  const bool wide = count > int64_t(Narrow::kCount);
  const int64_t most = context ? (wide ? 40 : 80) * 1024 : int64_t(1) << 24;  // tokens of a slice: 160 KB of words
  const int64_t all = a.vocab + 8;                                            // with the skew of any row
  unsigned ctas = 1;
  // Four CTAs a row, and eight where that is few CTAs or four would leave one an SM: every CTA reads the whole history.
  const unsigned cap = !context || a.rows * 8 <= 144 * kResident || all * (wide ? 4 : 2) > 4 * 64 * 1024 + 64 ? 8 : 4;
  while (ctas < cap && all > int64_t(ctas) * 4096) ctas *= 2;
  const int64_t per_pass = int64_t(ctas) * most;
  p.passes = int((all + per_pass - 1) / per_pass);
  const int64_t parts = int64_t(p.passes) * ctas;
  p.slice = int(((all + parts - 1) / parts + kBlock - 1) / kBlock * kBlock);
  p.ctas_log2 = ctas == 8 ? 3 : ctas == 4 ? 2 : ctas == 2 ? 1 : 0;
  // Rows of a cluster: so many that all clusters are there at once. (An SM takes two CTAs of up to 110 KB; the CTAs of a
  // cluster lie within a GPU processing cluster, whose last SMs may be left over: the numbers are the occupancy
  // calculator's. With 76 clusters of four where 74 are there, the last two ran alone: 384 rows 162 us, not 110.)
  const int64_t bytes = context ? int64_t(p.slice) * (wide ? 4 : 2) + p.slice / 8 + p.a.bias_width * 8 + kList * 4 : 0;
  const int per_sm = bytes <= 105 * 1024 ? kResident : 1;
  const int sms = ctas <= 2 ? 152 : ctas == 4 ? (per_sm > 1 ? 148 : 144) : per_sm > 1 ? 144 : 120;
  const int64_t resident = sms * per_sm / int(ctas), per = (a.rows + resident - 1) / resident;
  p.per = int(per < kMostRows ? per : kMostRows);
  switch (a.dtype) {
    case NF4_BF16: return launch_vector<B16>(p, context, wide, ctas, stream);
    case NF4_FP16: return launch_vector<H16>(p, context, wide, ctas, stream);
    default: return launch_vector<F32>(p, context, wide, ctas, stream);
  }
}

cudaError_t logits_flags(unsigned int** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_logits_flags);
}

}  // namespace nf4
