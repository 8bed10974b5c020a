// nf4_tree_commit.cu -- the accepted branch of each sequence's drafted tree, and
// its keys and values moved to their places in the paged cache.
//
// Every node asks at once whether it holds the model's choice at its parent, and the
// lowest such child becomes what follows the parent (a minimum in shared memory);
// the path is then a chain of looks there, one per accepted node. Own key
// base + path[j] moves to base + j, and path[j] >= j: a row's place was either
// read before or is no source at all. So a thread that owns the same few bytes of
// every row (16 of one head's key or value) moves them in order, eight rows under
// way, without waiting for anybody.
//
// A few rows per sequence, head and layer: latency bounds it (offsets, nodes,
// targets, pages and rows are loads that wait for one another). 4 trees of up to 8 nodes
// and one layer take 2.9 us; 64 of up to 32 with 28 layers of 8 heads 6.8 (4 layers a
// CTA, all there at once; a CTA per layer 12.5).
#include "nf4_decoding.cuh"

namespace nf4 {
namespace {

__device__ unsigned int g_commit_flags = 0;

constexpr int kThreads = 128;
constexpr int kMostNodes = 4096;
constexpr int kMostPath = 1024;
constexpr int kAhead = 8;  // rows under way

struct CommitArgs {
  nf4_tree_commit_args a;
  int units;       // per head row: of sizeof(U) bytes
  int blocks;      // CTAs that share a layer's units of a sequence
  int each;        // layers of a CTA
};

template <typename U>
__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const __grid_constant__ CommitArgs p) {
  const nf4_tree_commit_args& a = p.a;
  __shared__ int after[kMostNodes];           // the accepted child of each node
  __shared__ int path[kMostPath];
  __shared__ int2 from[kMostPath], to[kMostPath];  // (page, slot) of the rows that move, and of their places
  __shared__ int s_count;
  pdl_wait_prior_grid();
  pdl_allow_dependents();
  const int tid = threadIdx.x;
  const int b = int(blockIdx.x) / p.blocks, block = int(blockIdx.x) % p.blocks;
  const bool reports = block == 0 && blockIdx.y == 0;
  bool bad = false;
  int lo, hi;
  const int given_len = a.lens[b], len = max(given_len, 0), most = int(a.max_path);
  token_range(a.cu_q, b, int(a.tokens), &lo, &hi, &bad);
  const int nodes = min(hi - lo, kMostNodes);
  bad = bad || nodes != hi - lo;
  // The loads of a thread's first node are under way while the others are set.
  int up = -1, draft = 0;
  if (tid + 1 < nodes) {
    up = a.parents[lo + tid + 1];
    draft = a.draft_tokens[lo + tid + 1];
  }
  for (int x = tid; x < nodes; x += kThreads) after[x] = kMostNodes;
  __syncthreads();
  for (int x = tid + 1; x < nodes; x += kThreads) {
    if (x > tid + 1) {
      up = a.parents[lo + x];
      draft = a.draft_tokens[lo + x];
    }
    if (unsigned(up) >= unsigned(x))
      bad = true;
    else if (draft == a.targets[lo + up])
      atomicMin(&after[up], x);
  }
  __syncthreads();
  if (tid == 0) {
    int n = 0;
    for (int x = 0; n < most && x < nodes; x = after[x]) path[n++] = x;
    s_count = n;
  }
  __syncthreads();
  const int n = s_count;
  const int base = len - (hi - lo);
  if (reports) {
    for (int j = tid; j < most; j += kThreads) {
      a.path[int64_t(b) * most + j] = j < n ? path[j] : -1;
      a.chosen[int64_t(b) * most + j] = j < n ? a.targets[lo + path[j]] : -1;
    }
    if (tid == 0) {
      a.accepted[b] = n;
      a.new_lens[b] = max(base + n, 0);
      bad = bad || given_len < hi - lo;  // (also where it is negative)
    }
  }
  if (a.layers > 0 && n > 0) {
    // The rows that move, in the path's order: those behind the first node that is not in its place already.
    int still = 0;
    while (still < n && path[still] == still) ++still;
    const int moves = n - still;
    bool lost = false;
    for (int j = tid; j < moves; j += kThreads) {
      int2 at[2] = {make_int2(-1, 0), make_int2(-1, 0)};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = base + (i == 0 ? path[still + j] : still + j), nth = key >= 0 ? key / int(a.page_size) : -1;
        if (nth >= 0 && nth < a.width) at[i].x = a.page_table[int64_t(b) * a.page_table_stride + nth];
        at[i].y = key - nth * int(a.page_size);
      }
      if (unsigned(at[0].x) >= unsigned(a.num_pages) || unsigned(at[1].x) >= unsigned(a.num_pages)) {
        lost = true;
        at[0].x = -1;
      }
      from[j] = at[0];
      to[j] = at[1];
    }
    bad = bad || lost;
    const bool all = !__syncthreads_or(lost);
    const int columns = 2 * int(a.k_heads) * p.units;
    const int first = int(blockIdx.y) * p.each, layers = min(p.each, int(a.layers) - first);
    for (int c = block * kThreads + tid; c < columns; c += p.blocks * kThreads) {
      const bool value = c >= columns / 2;
      const int rest = value ? c - columns / 2 : c, head = rest / p.units;
      const int64_t layer_bytes = (value ? a.v_layer_stride : a.k_layer_stride) * 2;
      char* cache = static_cast<char*>(value ? a.v_cache : a.k_cache) + first * layer_bytes +
                    int64_t(head) * (value ? a.v_head_stride : a.k_head_stride) * 2 +
                    int64_t(rest - head * p.units) * int(sizeof(U));
      const int64_t page_bytes = (value ? a.v_page_stride : a.k_page_stride) * 2;
      const int64_t slot_bytes = (value ? a.v_slot_stride : a.k_slot_stride) * 2;
      // Rows of all layers in one run, a layer's in the path's order. (What a round writes, no later one of the
      // layer reads: a place is at or before the source of its own row.)
      int layer = 0, j = 0;
      while (layer < layers && moves > 0) {
        U row[kAhead];
        char* where[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          where[i] = nullptr;
          if (layer < layers) {
            const int2 f = from[j], t = to[j];
            if (all || f.x >= 0) {
              row[i] = *reinterpret_cast<const U*>(cache + f.x * page_bytes + f.y * slot_bytes);
              where[i] = cache + t.x * page_bytes + t.y * slot_bytes;
            }
            if (++j == moves) {
              j = 0;
              ++layer;
              cache += layer_bytes;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (where[i]) *reinterpret_cast<U*>(where[i]) = row[i];
      }
    }
  }
  if (bad) atomicOr(&g_commit_flags, kFlagBadIndex);
}

}  // namespace

cudaError_t launch_tree_commit(const nf4_tree_commit_args& a, cudaStream_t stream) {
  CommitArgs p;
  p.a = a;
  const auto wide = [&](const void* base, int64_t layer, int64_t page, int64_t slot, int64_t head) {
    return (reinterpret_cast<uintptr_t>(base) & 15u) == 0 && (a.layers <= 1 || layer % 8 == 0) &&
           (a.num_pages <= 1 || page % 8 == 0) && (a.page_size <= 1 || slot % 8 == 0) && (a.k_heads <= 1 || head % 8 == 0);
  };
  const bool chunks = a.head_dim % 8 == 0 &&
                      wide(a.k_cache, a.k_layer_stride, a.k_page_stride, a.k_slot_stride, a.k_head_stride) &&
                      wide(a.v_cache, a.v_layer_stride, a.v_page_stride, a.v_slot_stride, a.v_head_stride);
  p.units = int(chunks ? a.head_dim / 8 : a.head_dim);
  const int64_t layers = a.layers > 0 ? a.layers : 1;
  const int64_t columns = a.layers > 0 ? 2 * a.k_heads * p.units : 1;
  const int64_t blocks = (columns + kThreads - 1) / kThreads;
  p.blocks = int(blocks < 64 ? blocks : 64);
  // Six CTAs are on an SM (36 KB each): as many layers for each that all are there at once.
  const int64_t ctas = a.batch * p.blocks, room = 152 * 6 / ctas;
  const int64_t groups = room < 1 ? 1 : room < layers ? room : layers;
  p.each = int((layers + groups - 1) / groups);
  const dim3 grid(unsigned(ctas), unsigned((layers + p.each - 1) / p.each));
  return chunks ? launch_k(tree_commit_kernel<uint4>, grid, dim3(kThreads), 0, stream, p)
                : launch_k(tree_commit_kernel<uint16_t>, grid, dim3(kThreads), 0, stream, p);
}

cudaError_t commit_flags(unsigned int** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_commit_flags);
}

}  // namespace nf4
