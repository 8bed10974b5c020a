// nf4_decoding.cuh -- definitions shared by the translation units of
// include/nf4_decoding.h.
#pragma once

#include "nf4_attn.cuh"

namespace nf4 {

constexpr unsigned kFlagNoPages = 4u;  // a request asked for more pages than were free

cudaError_t pages_flags(unsigned int** word);
cudaError_t logits_flags(unsigned int** word);
cudaError_t commit_flags(unsigned int** word);

cudaError_t launch_kv_pages(const nf4_kv_pages_args& a, cudaStream_t stream);
cudaError_t launch_adjust_logits(const nf4_adjust_logits_args& a, cudaStream_t stream);
cudaError_t launch_tree_commit(const nf4_tree_commit_args& a, cudaStream_t stream);

// ---------------------------------------------------------------------------
// Thread-block clusters along x.

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// A barrier of all threads of the cluster in two halves; with the release, what they
// wrote to shared and device memory before is there for those that waited. (The wait
// is the hardware's: the CTAs of a cluster are on their SMs together, and one that
// has ended counts as arrived.)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_release() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_barrier() {
  cluster_arrive_release();
  cluster_wait();
}
// Address of `saddr` (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_address(uint32_t saddr, unsigned rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_store64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// Launch of clusters of `cluster` CTAs (1, 2, 4 or 8), with programmatic stream serialisation allowed.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), unsigned cluster, dim3 grid, dim3 block, size_t smem,
                           cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = NF4_USE_PDL;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ---------------------------------------------------------------------------
// Ragged batches: entry b of a list of offsets (cu_q, cu_rows), clamped so that
// whatever stands there stays in bounds. The offsets of a null list are 0, 1, 2, ..
__device__ __forceinline__ int offset_at(const int32_t* cu, int b, int total) {
  return cu ? min(max(cu[b], 0), total) : b;
}
// The tokens [lo, hi) of entry b; out-of-range offsets are reported by `bad`.
__device__ __forceinline__ void token_range(const int32_t* cu, int b, int total, int* lo, int* hi, bool* bad) {
  if (!cu) {
    *lo = b;
    *hi = b + 1;
    return;
  }
  const int x = cu[b], y = cu[b + 1];
  *lo = min(max(x, 0), total);
  *hi = min(max(y, *lo), total);
  *bad = *bad || *lo != x || *hi != y;
}

// The last of n entries whose first token is at most t (the first, where none is), by a whole warp, 32 looks at a time.
__device__ __forceinline__ int entry_of(const int32_t* cu, int n, int total, int t) {
  if (!cu) return min(t, n - 1);
  const int lane = threadIdx.x & 31;
  int b = 0, span = n;
  while (span > 1) {
    const int step = (span + 31) >> 5, at = lane * step;
    const bool before = at < span && offset_at(cu, b + at, total) <= t;
    const int src = 31 - __clz(int(__ballot_sync(0xffffffffu, before) | 1u));
    b += src * step;
    span = min(step, span - src * step);
  }
  return b;
}

}  // namespace nf4
