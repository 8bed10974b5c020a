// nf4_adjust_logits.cu -- penalties for repeated tokens, biases and masks on
// rows of logits, and each row's best token, in one pass.
//
// A cluster of CTAs per row, a slice of the vocabulary each. What the history and
// the row's branch of the tree say about a token is one 32-bit word in the shared
// memory of the token's CTA: how often it stands in the answer, whether it is known
// at all, whether it has a bias. The CTAs share the history and add to each other's
// words (distributed shared memory), so that it is read once per row and not once
// per slice; then every CTA streams its slice. The logits are read and written
// once: memory bounds it, for a single row the chain of loads and barriers.
#include "nf4_decoding.cuh"

namespace nf4 {
namespace {

__device__ unsigned int g_logits_flags = 0;

constexpr uint32_t kBiased = 1u << 31;   // has an entry in the bias list
constexpr uint32_t kKnown = 1u << 30;    // stands in the prompt
constexpr uint32_t kCount = kKnown - 1;  // times in the answer and the row's branch
constexpr int kMostBias = 1024;
constexpr int kThreads = 512;

struct LogitsArgs {
  nf4_adjust_logits_args a;
  int slice;   // tokens of a CTA, a multiple of 64
  int passes;  // slices of a CTA, one after another
};

struct F32 {
  using Store = float;
  static __device__ __forceinline__ float up(float v) { return v; }
  static __device__ __forceinline__ float down(float v) { return v; }
};
struct B16 {
  using Store = __nv_bfloat16;
  static __device__ __forceinline__ float up(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 down(float v) { return __float2bfloat16_rn(v); }
};
struct H16 {
  using Store = __half;
  static __device__ __forceinline__ float up(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half down(float v) { return __float2half_rn(v); }
};

// Larger values have larger keys; NaN the largest, zeros one key.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 + 0 = +0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Context: there is a history, a branch or a bias list. V elements of a row at a
// time: 16 bytes, or 1 where the rows of logits and out are not alike modulo 16
// bytes.
template <typename E, int V, bool kContext>
__global__ void __launch_bounds__(kThreads) adjust_logits_kernel(const __grid_constant__ LogitsArgs p) {
  using S = typename E::Store;
  const nf4_adjust_logits_args& a = p.a;
  extern __shared__ __align__(16) uint32_t words[];  // [slice]
  __shared__ int s_bias[kContext ? kMostBias : 1];
  __shared__ float s_value[kContext ? kMostBias : 1];
  __shared__ uint64_t s_best[8];
  __shared__ uint64_t s_warp[kThreads / 32];
  pdl_wait_prior_grid();
  pdl_allow_dependents();
  const int tid = threadIdx.x;
  const unsigned rank = cluster_rank(), ctas = cluster_size();
  const int row = int(blockIdx.x / ctas);
  const int vocab = int(a.vocab), share = int(rank) * kThreads + tid, shares = int(ctas) * kThreads;
  bool bad = false;

  // the row's request, or -1
  int b = -1, lo = 0, hi = 0;
  if (kContext) {
    if (a.cu_rows) {
      const int requests = int(a.requests), rows = int(a.rows);
      if (requests > 0) {
        b = 0;
        for (int step = 1 << (31 - __clz(requests)); step > 0; step >>= 1)
          if (b + step < requests && offset_at(a.cu_rows, b + step, rows) <= row) b += step;
        token_range(a.cu_rows, b, rows, &lo, &hi, &bad);
        if (row < lo || row >= hi) b = -1;
      }
    } else {
      b = lo = row;
      hi = row + 1;
    }
  }
  const float repetition = b >= 0 && a.repetition ? a.repetition[b] : 1.0f;
  const float frequency = b >= 0 && a.frequency ? a.frequency[b] : 0.0f;
  const float presence = b >= 0 && a.presence ? a.presence[b] : 0.0f;
  const uint32_t* mask = nullptr;
  if (a.mask) {
    const int m = a.mask_rows ? a.mask_rows[row] : row;
    if (m >= a.mask_count) bad = true;
    if (m >= 0 && m < a.mask_count) mask = a.mask + int64_t(m) * a.mask_stride;
  }
  const int mask_words = (vocab + 31) / 32;

  const S* const in = reinterpret_cast<const S*>(a.logits) + int64_t(row) * a.logits_stride;
  S* const out = reinterpret_cast<S*>(a.out) + int64_t(row) * a.out_stride;
  // Tokens are numbered from the 16-byte boundary before the row: u = v + skew.
  const int skew = V == 1 ? 0 : int((reinterpret_cast<uintptr_t>(in) & 15u) / sizeof(S));
  uint64_t best = 0;

  for (int pass = 0; pass < p.passes; ++pass) {
    const int base = pass * int(ctas) * p.slice;  // of the cluster, as u
    const int mine = base + int(rank) * p.slice;
    if (kContext) {
      if (pass > 0) cluster_barrier();  // the last pass's words have been read
      for (int i = tid; i < p.slice / 4; i += kThreads) reinterpret_cast<uint4*>(words)[i] = make_uint4(0, 0, 0, 0);
      cluster_barrier();
      if (b >= 0) {
        const uint32_t here = smem_u32(words);
        auto word = [&](int v, uint32_t* addr) {  // where token v's word is, if it is one of this pass
          const unsigned at = unsigned(v + skew - base), owner = at / unsigned(p.slice);
          if (v + skew < base || owner >= ctas) return false;
          *addr = cluster_address(here + (at - owner * unsigned(p.slice)) * 4u, owner);
          return true;
        };
        uint32_t addr;
        if (a.history) {
          const int len = a.history_lens[b], n = min(max(len, 0), int(a.history_width));
          const int prompt = a.prompt_lens ? a.prompt_lens[b] : 0;
          if (n != len || prompt < 0) bad = true;
          const int32_t* const h = a.history + int64_t(b) * a.history_stride;
          for (int j = share; j < n; j += shares) {
            const int v = h[j];
            if (unsigned(v) >= unsigned(vocab)) {
              bad = true;
            } else if (word(v, &addr)) {
              if (j < prompt)
                cluster_or(addr, kKnown);
              else
                cluster_add(addr, 1u);
            }
          }
        }
        if (a.draft_tokens) {
          const uint64_t* const seen = a.tree_mask + int64_t(row) * a.tree_mask_stride;
          const int nodes = int(min(int64_t(hi - lo), a.tree_words * 64));
          for (int x = share; x < nodes; x += shares) {
            if (!(seen[x >> 6] >> (x & 63) & 1ull)) continue;
            const int v = a.draft_tokens[lo + x];
            if (unsigned(v) >= unsigned(vocab))
              bad = true;
            else if (word(v, &addr))
              cluster_add(addr, 1u);
          }
        }
        if (a.bias_tokens) {
          const int64_t from = int64_t(b) * a.bias_stride;
          for (int j = tid; j < int(a.bias_width); j += kThreads) {
            const int v = a.bias_tokens[from + j];
            s_bias[j] = v;
            s_value[j] = a.bias_values[from + j];
            if (v >= vocab)
              bad = true;
            else if (v >= 0 && word(v, &addr) && int(unsigned(v + skew - mine) < unsigned(p.slice)))
              cluster_or(addr, kBiased);
          }
        }
      }
      cluster_barrier();
    }

    const int end = min(mine + p.slice, vocab + skew);
    for (int u = mine + tid * V; u < end; u += kThreads * V) {
      const int v0 = u - skew;
      alignas(16) S x[V];
      const bool whole = v0 >= 0 && v0 + V <= vocab;
      if (V > 1 && whole) {
        *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(in + v0);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = v0 + i >= 0 && v0 + i < vocab ? in[v0 + i] : E::down(0.0f);
      }
      uint32_t allowed = 0xffffffffu;
      if (mask) {
        const int w = v0 >> 5;  // -1 for the tokens before the row's first
        const uint32_t low = w >= 0 ? mask[w] : 0u, high = w + 1 < mask_words ? mask[w + 1] : 0u;
        allowed = __funnelshift_r(low, high, v0 & 31);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float y = E::up(x[i]);
        if (kContext) {
          const uint32_t w = words[u - mine + i];
          if (w != 0) {
            if (w & (kKnown | kCount)) y = y > 0.0f ? __fdiv_rn(y, repetition) : __fmul_rn(y, repetition);
            const uint32_t c = w & kCount;
            if (c) y = __fsub_rn(__fsub_rn(y, __fmul_rn(frequency, float(c))), presence);
            if (w & kBiased) {
              float sum = 0.0f;
              for (int j = 0; j < int(a.bias_width); ++j)
                if (s_bias[j] == v0 + i) sum = __fadd_rn(sum, s_value[j]);
              y = __fadd_rn(y, sum);
            }
            x[i] = E::down(y);
          }
        }
        if (!(allowed >> i & 1u)) x[i] = E::down(-INFINITY);
        if (a.best && v0 + i >= 0 && v0 + i < vocab) {
          const uint64_t key = uint64_t(order_key(E::up(x[i]))) << 32 | uint32_t(~(v0 + i));
          best = key > best ? key : best;
        }
      }
      if (V > 1 && whole) {
        *reinterpret_cast<uint4*>(out + v0) = *reinterpret_cast<const uint4*>(x);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (v0 + i >= 0 && v0 + i < vocab) out[v0 + i] = x[i];
      }
    }
  }
  if (bad) atomicOr(&g_logits_flags, kFlagBadIndex);

  if (a.best) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const uint64_t y = __shfl_xor_sync(0xffffffffu, best, d);
      best = y > best ? y : best;
    }
    if ((tid & 31) == 0) s_warp[tid >> 5] = best;
    __syncthreads();
    if (!kContext) cluster_barrier();  // every CTA has begun
    if (tid == 0) {
      for (int w = 1; w < kThreads / 32; ++w) best = s_warp[w] > best ? s_warp[w] : best;
      cluster_store64(cluster_address(smem_u32(&s_best[rank]), 0), best);
    }
    cluster_barrier();
    if (rank == 0 && tid == 0) {
      for (unsigned r = 0; r < ctas; ++r) best = s_best[r] > best ? s_best[r] : best;
      a.best[row] = int(~uint32_t(best));
    }
  }
}

template <typename E, int V, bool kContext>
cudaError_t launch(const LogitsArgs& p, unsigned ctas, cudaStream_t stream) {
  auto kern = adjust_logits_kernel<E, V, kContext>;
  const int smem = kContext ? p.slice * 4 : 0;
  static PerDeviceCache attr_set;
  const cudaError_t e = set_max_dynamic_smem_once(kern, kContext ? 200 * 1024 : 0, attr_set);
  if (e != cudaSuccess) return e;
  return launch_cluster(kern, ctas, dim3(unsigned(p.a.rows) * ctas), dim3(kThreads), size_t(smem), stream, p);
}
template <typename E, int V>
cudaError_t launch_context(const LogitsArgs& p, bool context, unsigned ctas, cudaStream_t stream) {
  return context ? launch<E, V, true>(p, ctas, stream) : launch<E, V, false>(p, ctas, stream);
}
template <typename E>
cudaError_t launch_vector(const LogitsArgs& p, bool context, unsigned ctas, cudaStream_t stream) {
  constexpr int V = 16 / int(sizeof(typename E::Store));
  // every row of logits and out the same distance from a 16-byte boundary
  const nf4_adjust_logits_args& a = p.a;
  const bool alike = ((reinterpret_cast<uintptr_t>(a.logits) - reinterpret_cast<uintptr_t>(a.out)) & 15u) == 0 &&
                     (a.rows <= 1 || (a.logits_stride - a.out_stride) % V == 0);
  return alike ? launch_context<E, V>(p, context, ctas, stream) : launch_context<E, 1>(p, context, ctas, stream);
}

}  // namespace

cudaError_t launch_adjust_logits(const nf4_adjust_logits_args& a, cudaStream_t stream) {
  LogitsArgs p;
  p.a = a;
  const bool context = a.requests > 0 && ((a.history && a.history_width > 0) || a.draft_tokens || (a.bias_tokens && a.bias_width > 0));
  const int64_t most = context ? 48 * 1024 : int64_t(1) << 24;  // tokens of a slice: 192 KB of words
  const int64_t all = a.vocab + 8;                              // with the skew of any row
  unsigned ctas = 1;
  while (ctas < 8 && all > int64_t(ctas) * 4096) ctas *= 2;
  const int64_t per_pass = int64_t(ctas) * most;
  p.passes = int((all + per_pass - 1) / per_pass);
  const int64_t parts = int64_t(p.passes) * ctas;
  p.slice = int(((all + parts - 1) / parts + 63) / 64 * 64);
  switch (a.dtype) {
    case NF4_BF16: return launch_vector<B16>(p, context, ctas, stream);
    case NF4_FP16: return launch_vector<H16>(p, context, ctas, stream);
    default: return launch_vector<F32>(p, context, ctas, stream);
  }
}

cudaError_t logits_flags(unsigned int** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_logits_flags);
}

}  // namespace nf4
