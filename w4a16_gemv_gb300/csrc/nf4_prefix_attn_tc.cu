// nf4_prefix_attn_tc.cu -- the many-row items of nf4_prefix_attention on the
// 5th-generation tensor cores: up to 256 rows of a key/value head (every query
// token of the batch times its group of query heads) against a range of keys.
//
// S = Q K^T and O += P V per 128 keys, as two tiles of 128 rows that take
// turns: while the softmax of one tile runs on the CUDA cores, the tensor
// cores do the other's products. Per 128 keys and tile of 128 rows the two
// products take 2 x 128 x 128 x 128 multiply-adds (about 1000 cycles of an
// SM's tensor cores at head_dim 128), the softmax 16384 exponentials, about
// half of that: with two full tiles the tensor cores bound it, with few rows the
// bytes of the keys and values do (32 KB each per 128 keys).
//
// One CTA of 16 warps per SM:
//   * warps 0-3 and 4-7: softmax of tile 0 and 1, one row per thread. Scores
//     come from tensor memory into registers, the weights exp2(s - m) (in binary16
//     lifted, see kLift) go back as 16-bit pairs, V's type, over the same columns,
//     where the second product reads them as its A operand. m is the maximum at the
//     time of the last rescale: O and l are rescaled only when a row's maximum has
//     grown past 2^8 (exact all the same, since O and l share m; binary32 and the
//     16-bit weights hold 2^8 times 1 with the same relative error), so that O is
//     rarely touched;
//   * warp 8: keys and values from their pages into a ring of 128-row tiles, by
//     tensor copies (TMA) of as many rows as are sure to lie in one page, one
//     lane per box; boxes past the range, or on a page that does not exist,
//     have their page coordinate past the end and arrive as zeros. Warp 9
//     zeroes what a last box brought from beyond the range, so that what lies in
//     unused slots never reaches a product. The copies' swizzle serves K as a
//     K-major and V as an N-major operand;
//   * page sizes without a factor of eight, and caches that no tensor map
//     describes: warps 8-11 bring the same tiles by 16-byte asynchronous copies
//     (about 1000 cycles of a warp per tile, where the tensor copies take 100);
//   * warp 12: issues the products. S of the next keys follows O += P V of a
//     tile in issue order, so P is read before S overwrites it, and the signal
//     that S is complete also says that O is at rest.
// In calls of trees, an item of up to 128 rows over two key tiles or more is a pair of
// halves: with one tile of rows a key tile's products and its softmax wait for one
// another (1.4 us per key tile), so tile 0 takes the even key tiles and tile 1 the odd
// ones, with Q, S and O as above, K and V by a warp each (small boxes are bound by
// their issue), and the ring one tile longer at 128 elements (the second tile of Q is
// not there). The halves' maxima, sums and outputs are joined on the way out. 16 trees
// of up to 32 nodes and 32 heads over 8 take 58 us over 4000 keys without, 44 with it
// (1.05 us per key tile; two key tiles 12.5 and 11.9), one of 25 over 50000 keys of 32
// heads 141 and 124. (tests/test_attention_barriers.py runs the barriers of this form as
// a model under random interleavings; whoever changes an arrival here changes it there.)
// An item leaves its partial result, or the output; an item of own keys of a call
// with one range of each joins the shared keys' part of its rows on the way out.
// Tensor memory: S (and P) of the tiles in columns 0 and 128, O in 256 and 384.
// Measured: 4864 tokens x 8 query heads over 16384 keys of 2 heads x 128 in
// bf16 take 195 us (1670 TFLOP/s, 88% of measured bf16 peak; head_dim 64: 170 us,
// 960); 12 heads of sixteen tokens stream 2^20 keys in 159 us (6.75 TB/s); a call over
// 8192 keys takes 8.5 us of start, two key tiles and partial results.
// Waits are bounded; one that runs out sets bit 0 of the device error flags.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "nf4_prefix_attn.cuh"

namespace nf4 {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace {

__device__ unsigned int g_prefix_tc_flags = 0;

constexpr int kTcThreads = 512;
constexpr int kTileRows = 128;
constexpr int kTileKeys = 128;
constexpr uint32_t kTmemCols = 512;
constexpr int kKeys = 4;  // barriers of K tiles where key tiles take turns
constexpr int kGo = 4;  // key tiles whose loads may be under way (a ring of 8 tiles holds less than 4 pairs)
// Registers: 512 threads launch with 128 each (65536); the two softmax
// warpgroups take 184, the others keep 72: 256 x 184 + 256 x 72 = 65536. (With
// 192 and 64 the loading and issuing warps spill, and a spill's reload behind
// streaming keys costs a microsecond per key tile.)
constexpr int kLaunchRegs = 128;

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// Waits for phase `parity` of `bar`: at most 1000 sleeps of up to a
// millisecond each. (Without a clock to read between them this wakes sooner
// than the shared bounded wait, and 512 threads poll here.)
__device__ __forceinline__ bool mbar_wait_counted(uint64_t* bar, uint32_t parity) {
  const uint32_t addr = smem_u32(bar);
  uint32_t done = 0;
#pragma unroll 1
  for (int k = 0; k < 1000 && !done; ++k)
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(addr), "r"(parity), "r"(1000000)
        : "memory");
  return done != 0;
}

// Shared-memory matrix descriptors, 128-byte swizzle: rows of 128 bytes in
// groups of eight (1024 bytes apart).
// K-major (rows along M or N, 64 elements of K per row; a further 64 elements
// of K lie in the next block, addressed by the caller).
__device__ __forceinline__ uint64_t desc_k_major(uint32_t saddr) {
  return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
// N-major (rows along K, 64 elements of N per row; the next 64 elements of N
// lie `block` bytes on).
__device__ __forceinline__ uint64_t desc_n_major(uint32_t saddr, uint32_t block) {
  return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(block >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// Instruction descriptor of kind::f16: binary32 accumulator, A and B of the
// same 16-bit type, M = 128.
template <typename H>
__device__ __forceinline__ constexpr uint32_t idesc(int n, bool b_n_major) {
  return (1u << 4) | (H::kDtype == NF4_BF16 ? (1u << 7) | (1u << 10) : 0u) | (b_n_major ? 1u << 16 : 0u) |
         (uint32_t(n >> 3) << 17) | (uint32_t(kTileRows >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(accumulate)
      : "memory");
}

// 32 columns of this warp's lanes (a thread's 32 values are one row's).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// The loaded values may be used after this (uses are tied to it by the
// compiler through the operands).
__device__ __forceinline__ void tmem_ld_wait(float* v, int n) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < n; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// The two caches as 4-D tensors: 64 elements x box_rows slots of one head and
// page. *_slot and *_head: which of the last three coordinates is the slot and
// the head; the other is the page (the tensor's dimensions are in the order of
// their strides).
struct CacheMaps {
  CUtensorMap k, v;
  int box_rows, tile_keys;
  int k_slot, k_head, v_slot, v_head;
};

// One box; `leave_first`: its lines leave L2 before others.
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* map, int x, int slot_at, int head_at,
                                             int slot, int head, int page, uint64_t* bar, bool leave_first) {
  const int c1 = slot_at == 0 ? slot : head_at == 0 ? head : page;
  const int c2 = slot_at == 1 ? slot : head_at == 1 ? head : page;
  const int c3 = slot_at == 2 ? slot : head_at == 2 ? head : page;
  if (leave_first)
    asm volatile(
        "{\n\t.reg .b64 p;\n\tcreatepolicy.fractional.L2::evict_first.b64 p, 1.0;\n\t"
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
        "[%1, {%2, %3, %4, %5}], [%6], p;\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

template <int DP>
struct Layout {
  static constexpr int kBlocks = DP / 64;                       // 128-byte columns blocks of a row
  static constexpr uint32_t kBlock = 128 * 128;                 // bytes of one block of 128 rows
  static constexpr uint32_t kTile = kBlocks * kBlock;           // 128 rows
  static constexpr int kStages = DP == 128 ? 5 : 8;             // ring of K and V tiles
  static constexpr int kLag = 3;                                // tiles that a loader leaves in flight
  static constexpr int kPairStages = DP == 128 ? 6 : 8;         // with the second tile of Q among them
  static constexpr uint32_t kRing = 2 * kTile;                  // after the two tiles of Q
  static constexpr uint32_t kBars = kRing + kStages * kTile;
  static constexpr uint32_t kBytes = kBars + 256 + 1024;        // + slack to align the base
};

// Address of ring tile `slot`; the one past a ring of kStages is the second tile of Q, in front of it.
template <int DP>
__device__ __forceinline__ uint32_t ring_tile(uint32_t sbase, int slot) {
  using L = Layout<DP>;
  return sbase + L::kRing + uint32_t(slot < L::kStages ? slot : -1) * L::kTile;
}
// The two softmax warps of the same 32 rows.
__device__ __forceinline__ void pair_sync(int quarter) {
  asm volatile("bar.sync %0, 64;" ::"r"(quarter + 2) : "memory");
}

template <typename H, int DP, bool kTma, bool T>
__global__ void __launch_bounds__(kTcThreads, 1)
    prefix_tc_kernel(const __grid_constant__ PrefixArgs a, const __grid_constant__ CacheMaps maps) {
  using L = Layout<DP>;
  constexpr int kLoaders = kTma ? 1 : 4;  // arrivals for a ring tile
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // go: all that the products of key tile i need besides P of the second tile
  // of rows: P of the first, V_i and K_{i+1}. One barrier, because a look at
  // a barrier costs the issuing thread some 250 cycles while the tensor cores
  // keep the shared memory busy, and their queue does not bridge that.
  uint64_t* const go = reinterpret_cast<uint64_t*>(smem + L::kBars);    // [kGo], key tile i: i % kGo
  uint64_t* const kfirst = go + kGo;                                    // K_0 landed; [kKeys], in a pair K_i: i % kKeys
  uint64_t* const empty = kfirst + kKeys;                               // a ring tile's products are done
  uint64_t* const sfull = empty + 8;                                    // S of a tile complete, O at rest
  uint64_t* const psecond = sfull + 2;                                  // P of the second tile written
  uint64_t* const qfull = psecond + 1;                                  // Q of a tile in place (4 softmax warps)
  uint64_t* const tail = qfull + 2;                                     // the last tile of V landed, to be cleaned
  uint32_t* const s_taddr = reinterpret_cast<uint32_t*>(tail + 1);

  // Keys of a tile; the rows of a ring tile past them stay zero.
  const int step = kTma ? maps.tile_keys : kTileKeys;
  if (kTma && step < kTileKeys) {
    const int past = (kTileKeys - step) * 8;  // 16 bytes each
    for (int block = T && L::kPairStages > L::kStages ? -L::kBlocks : 0; block < L::kStages * L::kBlocks; ++block)
      for (int e = tid; e < past; e += kTcThreads)
        *reinterpret_cast<uint4*>(smem + int(L::kRing) + block * int(L::kBlock) + step * 128 + e * 16) =
            make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
  }
  if (tid == 0) {
    for (int i = 0; i < kGo; ++i) mbar_init(&go[i], 4 + 2 * kLoaders);
    for (int i = 0; i < (T ? L::kPairStages : L::kStages); ++i) mbar_init(&empty[i], 1);
    for (int i = 0; i < (T ? kKeys : 1); ++i) mbar_init(&kfirst[i], kLoaders);
    mbar_init(psecond, 4);
    mbar_init(tail, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&qfull[i], 4);
    }
    fence_mbar_init();
  }
  if (kTma && tid == 32 * 8) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.v)) : "memory");
  }
  __syncthreads();  // the barriers exist; from here the warps start their parts as they can
  // Reads and writes of device memory, and the tensor memory, wait for the previous
  // grid (an allocation held by a grid that waits could starve the one waited
  // for); an item of shared keys is known before that, and each part waits when it
  // has worked out its addresses. (Own items that join the shared keys' parts run
  // beside the launch that makes these and wait for it at their end. That launch
  // let this one start when all its CTAs were on their SMs, and one of these, with
  // nearly all of an SM's shared memory, is never beside one of those.)
  auto begin = [&]() {
    if (!a.beside) pdl_wait_prior_grid();
  };
  if (unsigned(a.first) + blockIdx.x >= unsigned(a.prefix_tiles) * unsigned(a.k_heads) * unsigned(a.prefix_splits))
    begin();
  const PrefixItem it = prefix_item<T>(a, unsigned(a.first) + blockIdx.x, &g_prefix_tc_flags);
  const int n = (it.k1 - it.k0 + step - 1) / step;  // key tiles
  const bool works = it.rows > 0 && n > 0;          // the same in the whole CTA
  const int tiles = it.rows > kTileRows ? 2 : 1;
  const bool pair = T && kTma && tiles == 1 && n > 1 && !(a.fused && a.splits > 0);
  if (!works) {
    if (a.fused) {
      if (a.beside) pdl_wait_prior_grid();
      for (int r = warp; r < it.rows; r += kTcThreads / 32) shared_row<H>(a, row_out(a, it, it.r0 + r).row);
      if (warp < 8) unheld_rows<H>(a, 8, &g_prefix_tc_flags);
      return;
    }
    begin();
    for (int r = tid; r < it.rows; r += kTcThreads) {
      const RowOut ro = row_out(a, it, it.r0 + r);
      *ro.ml = make_float2(-INFINITY, 0.0f);  // (a plan with one range of shared keys has no empty range)
    }
    return;
  }
  // The softmax warps and the issuing warp meet here, when the tensor memory
  // is allocated.
  auto tmem_address = [&]() {
    tc_fence_before();
    asm volatile("bar.sync 1, 288;" ::: "memory");
    tc_fence_after();
    return *s_taddr;
  };
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = mbar_wait_counted(bar, parity);
  };

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int tile = warp >> 2;
    // Q: each warp asks for its 32 rows first
    if (tile >= tiles) {
      begin();
    } else {
      constexpr int kQChunks = DP / 8, kQStep = 32 / kQChunks;
      const int r = warp * 32 + lane, c = lane % kQChunks;
      int64_t off = 0;
      if (r < it.rows) {
        const int t = (it.r0 + r) / a.group;
        off = int64_t(it.t0 + t) * a.q_ts + int64_t(it.head * a.group + (it.r0 + r - t * a.group)) * a.q_hs;
      }
      const uint32_t dst = sbase + uint32_t(tile) * L::kTile + uint32_t(c >> 3) * L::kBlock;
      begin();
#pragma unroll
      for (int x = 0; x < 32 / kQStep; ++x) {
        const int rl = x * kQStep + lane / kQChunks, row = (warp & 3) * 32 + rl;
        const int64_t o = __shfl_sync(0xffffffffu, off, rl);
        const bool there = warp * 32 + rl < it.rows && c * 8 < a.dim;
        cp_async16(dst + uint32_t(row) * 128u + uint32_t(((c & 7) ^ (row & 7)) << 4),
                   there ? a.q + o + c * 16 : a.q, there);
      }
      cp_async_commit();
    }
    const uint32_t tbase = tmem_address();
    if (tile < tiles || pair) {
      cp_async_wait<0>();
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&qfull[tile]);
      const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
      const uint32_t s_col = tbase + lanes + uint32_t(tile) * 128u;
      const uint32_t o_col = tbase + lanes + 256u + uint32_t(tile) * 128u;
      // (a register, in place of what `pair` follows from: with that kept through the loop two registers spill, and
      // every key tile waits for them)
      int stride = pair ? 2 : 1;
      if constexpr (T && kTma) asm volatile("" : "+r"(stride));
      const int row0 = pair ? 0 : tile * kTileRows;  // in a pair this tile's keys are every second 128
      const int r = row0 + (warp & 3) * 32 + lane;
      const int limit = r < it.rows ? min(visible_keys<T>(it, (it.r0 + r) / a.group), it.k1) - it.k0 : 0;
      // key tiles below this one need no mask in this warp
      int free_tiles = T ? max(min(unmasked_keys<T>(it, 0), it.k1) - it.k0, 0) / step : limit / step;
      if (r >= it.rows) free_tiles = n;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) free_tiles = min(free_tiles, __shfl_xor_sync(0xffffffffu, free_tiles, d));
      float m = -INFINITY;
      float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
#pragma unroll 1
      for (int i = tile & (stride - 1); i < n; i += stride) {
        wait(&sfull[tile], uint32_t(i >> (stride - 1)) & 1u);
        __syncwarp();
        tc_fence_after();
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32u * c, s + 32 * c);
        tmem_ld_wait(s, 128);
        if (i >= free_tiles) {
#pragma unroll
          for (int j = 0; j < 128; ++j)
            if (i * step + j >= limit) s[j] = -INFINITY;
          if constexpr (T) {
            if (it.own && r < it.rows) {
              const int t = it.t0 + (it.r0 + r) / a.group;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint64_t seen = tree_window(a, it, t, it.k0 + i * step + 64 * h);
#pragma unroll
                for (int j = 0; j < 64; ++j)
                  if (!(seen >> j & 1ull)) s[64 * h + j] = -INFINITY;
              }
            }
          }
        }
        if (kTma && step < kTileKeys) {
#pragma unroll
          for (int j = 112; j < 128; ++j)
            if (j >= step) s[j] = -INFINITY;
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = s[c];
#pragma unroll
          for (int j = 1; j < 32; ++j) mx[c] = fmaxf(mx[c], s[4 * j + c]);
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
        if (i < stride) {
          m = top;
        } else if (__any_sync(0xffffffffu, top > m + kGrowth)) {
          const float nm = fmaxf(m, top);
          const float f = nm == -INFINITY ? 1.0f : ex2(m - nm);
          m = nm;
          l2[0].x *= f;
          l2[0].y *= f;
          l2[1].x *= f;
          l2[1].y *= f;
#pragma unroll 1
          for (int c = 0; c < DP / 32; ++c) {
            float o[32];
            tmem_ld32(o_col + 32u * c, o);
            tmem_ld_wait(o, 32);
            uint32_t w[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(o[j] * f);
            tmem_st32(o_col + 32u * c, w);
          }
        }
        const float base = m == -INFINITY ? 0.0f : m - kLift<H>;
        const float2 nb2 = make_float2(-base, -base);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float2 e = fma2(make_float2(s[64 * h + 2 * j], s[64 * h + 2 * j + 1]), scale2, nb2);
            const float2 w = make_float2(ex2(e.x), ex2(e.y));
            l2[j & 1] = add2(l2[j & 1], w);
            p[j] = H::down2(w.x, w.y);
          }
          tmem_st32(s_col + 32u * h, p);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tile == 0 || stride > 1 ? &go[i % kGo] : psecond);
      }
      m -= kLift<H>;  // from here what l and O are relative to
      const bool mine = r < it.rows;
      const RowOut ro = row_out(a, it, it.r0 + (mine ? r : 0));
      // 128 bytes of every row at a time go through this warp's part of the Q
      // tile (its products are done), so that rows leave in whole sectors:
      // 32 columns of partial results, or 64 of the 16-bit output.
      unsigned char* const stage = smem + tile * L::kTile + (warp & 3) * 4096;
      const int row_bytes = a.dim * (a.direct ? 2 : 4);
      const int ch = lane & 7;  // this lane's 16 bytes of rows lane / 8, lane / 8 + 4, ..
      char* dst[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int rl = 4 * j + (lane >> 3);
        dst[j] = reinterpret_cast<char*>(__shfl_sync(
            0xffffffffu, reinterpret_cast<uint64_t>(a.direct ? ro.out : reinterpret_cast<char*>(ro.part)), rl));
        if (row0 + (warp & 3) * 32 + rl >= it.rows) dst[j] = nullptr;
      }
      if constexpr (T && kTma) {
        if (stride > 1) {
          // Both halves of the keys of this thread's row are in its lane of tensor memory; maxima and sums change
          // hands through the stages, and each warp writes every second piece of the columns.
          // (Both stand in the first tile of Q: the second's place may still hold the other half's last keys.)
          wait(&sfull[tile], uint32_t(tile == 0 ? (n + 1) >> 1 : n >> 1) & 1u);  // this half's last product is in O
          __syncwarp();
          const float sum = l2[0].x + l2[0].y + (l2[1].x + l2[1].y);
          const float2 here = make_float2(m, ok ? sum : __uint_as_float(0x7fc00000u));
          float2* const exchange = reinterpret_cast<float2*>(smem + (warp & 3) * 4096) + lane;
          exchange[tile * 32] = here;
          tc_fence_before();
          pair_sync(warp & 3);  // and so is the other half's
          tc_fence_after();
          const float2 there = exchange[(tile ^ 1) * 32];
          pair_sync(warp & 3);  // it has been read
          const float top = fmaxf(here.x, there.x);
          const float f_here = part_holds(here) ? part_weight(here, top) : 0.0f;
          const float f_there = part_holds(there) ? part_weight(there, top) : 0.0f;
          const float l = here.y * f_here + there.y * f_there;
          const bool any = l > 0.0f || l != l;
          const float bad = here.y == here.y && there.y == there.y ? 0.0f : __uint_as_float(0x7fc00000u);
          const float by = a.direct ? (any ? 1.0f / l : 0.0f) : 1.0f;
          const float f0 = (tile == 0 ? f_here : f_there) * by, f1 = (tile == 0 ? f_there : f_here) * by;
          const uint32_t o_at = o_col - uint32_t(tile) * 128u;
          auto columns = [&](uint32_t at, float* o) {  // 32 joined columns
            float x[32];
            tmem_ld32(o_at + at, o);
            tmem_ld32(o_at + 128u + at, x);
            tmem_ld_wait(o, 32);
            tmem_ld_wait(x, 32);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float v = f0 != 0.0f ? o[j] * f0 : 0.0f;
              o[j] = (f1 != 0.0f ? fmaf(x[j], f1, v) : v) + bad;
            }
          };
#pragma unroll 1
          for (int c = tile; c < (a.direct ? DP / 64 : DP / 32); c += 2) {
            uint32_t w[32];
            float o[32];
            if (!a.direct) {
              columns(32u * c, o);
#pragma unroll
              for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(o[j]);
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                columns(64u * c + 32u * h, o);
#pragma unroll
                for (int j = 0; j < 16; ++j) w[16 * h + j] = H::down2(o[2 * j], o[2 * j + 1]);
              }
            }
            __syncwarp();  // the stage's last pass has been read
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                  make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            __syncwarp();
            const int at = c * 128 + ch * 16;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int rl = 4 * j + (lane >> 3);
              const uint4 y = *reinterpret_cast<const uint4*>(stage + rl * 128 + ((ch ^ (rl & 7)) << 4));
              if (dst[j] && at < row_bytes) *reinterpret_cast<uint4*>(dst[j] + at) = y;
            }
          }
          if (mine && tile == 0) {
            if (!a.direct)
              *ro.ml = make_float2(top, l);
            else if (ro.lse)
              *ro.lse = any ? fmaf(top, kLn2, logf(l)) : -INFINITY;
          }
        }
      }
      if (stride == 1) {
        const bool joins = !T && a.fused && a.splits > 0;  // (trees' own items never do)
        float2 shared = make_float2(-INFINITY, 0.0f);  // the row's shared keys: maximum and sum,
        float4 z[8];                                   // and 32 columns of their output, of the rows in dst
        auto shared_part = [&](int c) {
          const int row = int(ro.row);  // below 2^30
          const bool there = part_holds(shared);
          const float* src = a.part + c * 32 + ch * 4;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int rl = 4 * j + (lane >> 3);
            const int at = __shfl_sync(0xffffffffu, row, rl);
            const bool here = __shfl_sync(0xffffffffu, int(there), rl) && dst[j] && c * 32 + ch * 4 < a.dim;
            z[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (here) z[j] = *reinterpret_cast<const float4*>(src + int64_t(at) * a.dim);
          }
        };
        if (joins) {
          if (a.beside) pdl_wait_prior_grid();
          shared = a.ml[ro.row];
          shared_part(0);
        }
        wait(&sfull[tile], uint32_t(n) & 1u);  // the last product is in O
        __syncwarp();
        tc_fence_after();
        float l = l2[0].x + l2[0].y + (l2[1].x + l2[1].y);
        float own = 1.0f, other = 0.0f;  // weights of this item and of the shared keys
        const bool holds = part_holds(make_float2(m, l));
        if (joins) {
          const float top = fmaxf(m, shared.x);
          own = part_weight(make_float2(m, l), top);
          l *= own;
          if (part_holds(shared)) {
            other = part_weight(shared, top);
            l = fmaf(shared.y, other, l);
          }
          m = top;
        }
        const bool any = l > 0.0f || l != l;
        const float inv = any ? 1.0f / l : 0.0f;
        const float bad = ok ? 0.0f : __uint_as_float(0x7fc00000u);
        if (!T && a.fused) {
          own *= inv;
          other *= inv;
#pragma unroll 1
          for (int c = 0; c < DP / 32; ++c) {
            float o[32];
            tmem_ld32(o_col + 32u * c, o);
            tmem_ld_wait(o, 32);
            __syncwarp();  // the stage's last pass has been read
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float4 w = make_float4(bad, bad, bad, bad);
              if (holds)
                w = make_float4(o[4 * j] * own + bad, o[4 * j + 1] * own + bad, o[4 * j + 2] * own + bad,
                                o[4 * j + 3] * own + bad);
              *reinterpret_cast<float4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) = w;
            }
            __syncwarp();
            uint2 y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int rl = 4 * j + (lane >> 3);
              const float4 w = *reinterpret_cast<const float4*>(stage + rl * 128 + ((ch ^ (rl & 7)) << 4));
              const float f = __shfl_sync(0xffffffffu, other, rl);
              y[j] = joins ? make_uint2(H::down2(fmaf(z[j].x, f, w.x), fmaf(z[j].y, f, w.y)),
                                        H::down2(fmaf(z[j].z, f, w.z), fmaf(z[j].w, f, w.w)))
                           : make_uint2(H::down2(w.x, w.y), H::down2(w.z, w.w));
            }
            if (joins && c + 1 < DP / 32) shared_part(c + 1);
            const int col = c * 32 + ch * 4;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (dst[j] && col < a.dim) *reinterpret_cast<uint2*>(dst[j] + col * 2) = y[j];
          }
        }
        const int passes = !T && a.fused ? 0 : a.direct ? DP / 64 : DP / 32;
        float o[32];
        if (!a.direct) tmem_ld32(o_col, o);
#pragma unroll 1
        for (int c = 0; c < passes; ++c) {
          uint32_t w[32];
          if (!a.direct) {
            tmem_ld_wait(o, 32);
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(o[j] + bad);
            if (c + 1 < passes) tmem_ld32(o_col + 32u * (c + 1), o);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              tmem_ld32(o_col + 64u * c + 32u * h, o);
              tmem_ld_wait(o, 32);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                w[16 * h + j] = T && !any ? H::down2(bad, bad)
                                          : H::down2(o[2 * j] * inv + bad, o[2 * j + 1] * inv + bad);
            }
          }
          __syncwarp();  // the stage's last pass has been read
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
          __syncwarp();
          uint4 y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int rl = 4 * j + (lane >> 3);
            y[j] = *reinterpret_cast<const uint4*>(stage + rl * 128 + ((ch ^ (rl & 7)) << 4));
          }
          const int at = c * 128 + ch * 16;
          if (at < row_bytes) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (dst[j]) *reinterpret_cast<uint4*>(dst[j] + at) = y[j];
          }
        }
        if (mine) {
          if (!a.direct)
            *ro.ml = make_float2(m, l);
          else if (ro.lse)
            *ro.lse = any ? fmaf(m, kLn2, logf(l)) : -INFINITY;
        }
      }
    }
    if (a.fused) {
      if (a.beside) pdl_wait_prior_grid();
      unheld_rows<H>(a, 8, &g_prefix_tc_flags);
    }
  } else if (kTma && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int rows = maps.box_rows;
    const int valid = it.k1 - it.k0 - (n - 1) * step;  // keys of the last tile
    const bool clean = valid % rows != 0;                   // its last box reaches past them
    // Copies tiles kFirst (0: K) to kLast (1: V) of every key tile; in a pair K and V have a warp each.
    auto copy_tiles = [&](auto paired, auto first, auto last) {
      constexpr bool kPair = decltype(paired)::value;
      constexpr int kFirst = decltype(first)::value, kLast = decltype(last)::value;
      constexpr int kStages = kPair ? L::kPairStages : L::kStages;
      const int per_tile = (step / rows) * L::kBlocks;  // boxes of a tile: up to 32
      const int box = lane / L::kBlocks, block = lane % L::kBlocks;
      const bool mine = lane < per_tile;
      const bool leave_first = !it.own && a.stream;
      // (page, first slot) of this lane's box of key tile i; past the range, or
      // on a page that does not exist, the first page past the end
      int page = a.num_pages, slot0 = 0;
      auto fetch = [&](int i, int* pg, int* sl) {
        const int j = it.k0 + i * step + box * rows;
        *pg = a.num_pages;
        *sl = 0;
        if (mine && j < it.k1) {
          *pg = key_page(a, it, j);
          *sl = a.page_shift >= 0 ? j & (a.page_size - 1) : j % a.page_size;
        }
      };
      begin();
      fetch(0, &page, &slot0);
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const bool used = mine && it.k0 + i * step + box * rows < it.k1;
        if (used && unsigned(page) >= unsigned(a.num_pages)) {
          atomicOr(&g_prefix_tc_flags, kFlagBadIndex);
          page = a.num_pages;
        }
        int next_page, next_slot;
        fetch(i + 1, &next_page, &next_slot);
#pragma unroll
        for (int kv = kFirst; kv <= kLast; ++kv) {
          const int u = 2 * i + kv, slot = u % kStages;
          if (u >= kStages) wait(&empty[slot], uint32_t(u / kStages - 1) & 1u);
          uint64_t* const bar = kv == 0 ? (kPair ? &kfirst[i % kKeys] : i == 0 ? kfirst : &go[(i - 1) % kGo])
                                : clean && i + 1 == n ? tail : &go[i % kGo];
          if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(step * L::kBlocks) * 128u);
          __syncwarp();
          if (kPair && kv == 1 && i + 1 < n && lane == 0) mbar_arrive(&go[i % kGo]);  // in the place of the next K's
          const uint32_t dst = ring_tile<DP>(sbase, slot) + uint32_t(block) * L::kBlock + uint32_t(box * rows) * 128u;
          if (mine) {
            if (kv == 0)
              tma_load_box(dst, &maps.k, block * 64, maps.k_slot, maps.k_head, slot0, it.head, page, bar,
                           leave_first);
            else
              tma_load_box(dst, &maps.v, block * 64, maps.v_slot, maps.v_head, slot0, it.head, page, bar,
                           leave_first);
          }
        }
        page = next_page;
        slot0 = next_slot;
      }
      // There is no K after the last V. (In a pair the warp of V says so: that of K is ahead, and the barrier may still
      // be that of key tile n - 1 - kGo.)
      if (kLast == 1 && lane == 0) mbar_arrive(&go[(n - 1) % kGo]);
    };
    using Is = std::true_type;
    using No = std::false_type;
    using K = std::integral_constant<int, 0>;
    using V = std::integral_constant<int, 1>;
    if (warp == 8) {
      if constexpr (T) {
        if (pair)
          copy_tiles(Is(), K(), K());
        else
          copy_tiles(No(), K(), V());
      } else {
        copy_tiles(No(), K(), V());
      }
    } else if (T && pair && warp == 10) {
      copy_tiles(Is(), V(), V());
    } else if (warp == 9 && clean) {
      wait(tail, 0u);
      __syncwarp();
      const int u = 2 * n - 1, to = (valid + rows - 1) / rows * rows;
      unsigned char* const tile = smem + (ring_tile<DP>(sbase, pair ? u % L::kPairStages : u % L::kStages) - sbase);
      for (int e = valid * 8 + lane; e < to * 8; e += 32)
#pragma unroll
        for (int b = 0; b < L::kBlocks; ++b)
          *reinterpret_cast<uint4*>(tile + b * L::kBlock + e * 16) = make_uint4(0u, 0u, 0u, 0u);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&go[(n - 1) % kGo]);
    }
    __syncwarp();
  } else if (!kTma && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    constexpr int CPR = DP / 8, RPI = 32 / CPR;
    const int w = warp - 8;
    const int c = lane % CPR;
    const bool col = c * 8 < a.dim;
    const uint32_t col_off = uint32_t(c >> 3) * L::kBlock;
    KeyOffset off{0, 0};
    bool real = false;
    int page = 0;
    auto fetch_page = [&](int i) {
      const int j = it.k0 + i * kTileKeys + w * 32 + lane;
      if (j < it.k1) page = key_page(a, it, j);
    };
    auto landed = [&](int u) { return u == 0 ? kfirst : &go[((u - 1) >> 1) % kGo]; };
    begin();
    fetch_page(0);
#pragma unroll 1
    for (int u = 0; u < 2 * n; ++u) {
      const int slot = u % L::kStages;
      if (u >= L::kStages) wait(&empty[slot], uint32_t(u / L::kStages - 1) & 1u);
      if ((u & 1) == 0) {
        const int j = it.k0 + (u >> 1) * kTileKeys + w * 32 + lane;
        real = j < it.k1 && key_offset(a, it, j, page, &g_prefix_tc_flags, &off);
        if (u + 2 < 2 * n) fetch_page((u >> 1) + 1);
      }
      const char* src = (u & 1) == 0 ? a.k : a.v;
      const int64_t mine = (u & 1) == 0 ? off.k : off.v;
      const uint32_t dst = sbase + L::kRing + uint32_t(slot) * L::kTile + col_off;
#pragma unroll
      for (int x = 0; x < 32 / RPI; ++x) {
        const int rl = x * RPI + lane / CPR;
        const int64_t o = __shfl_sync(0xffffffffu, mine, rl);
        const bool there = __shfl_sync(0xffffffffu, int(real), rl) && col;
        const int row = w * 32 + rl;
        cp_async16(dst + uint32_t(row) * 128u + uint32_t(((c & 7) ^ (row & 7)) << 4),
                   there ? src + o + c * 16 : a.q, there);
      }
      cp_async_commit();
      if (u >= L::kLag) {
        cp_async_wait<L::kLag>();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(landed(u - L::kLag));
      }
    }
    cp_async_wait<0>();
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      for (int u = 2 * n > L::kLag ? 2 * n - L::kLag : 0; u < 2 * n; ++u) mbar_arrive(landed(u));
      mbar_arrive(&go[(n - 1) % kGo]);  // there is no K after the last V
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 12) {
      begin();
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_taddr)),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
      // Only now may what follows start: it lets its own followers start in turn, and
      // one of these that allocates ahead of its wait (the tensor-core GEMV) must not
      // hold what a CTA of this grid still waits for.
      pdl_allow_dependents();
      tmem_address();
    }
    if (warp == 12 && lane == 0) {
      const uint32_t tbase = *s_taddr;
      constexpr uint32_t kIdS = idesc<H>(kTileKeys, false);
      constexpr uint32_t kIdO = idesc<H>(DP, true);
      const uint32_t ring = sbase + L::kRing;
      auto product_s = [&](int t, int u) {  // S_t = Q_t K^T, K in ring tile u
        const uint64_t qd = desc_k_major(sbase + uint32_t(t) * L::kTile);
        const uint64_t kd = desc_k_major(ring + uint32_t(u % L::kStages) * L::kTile);
#pragma unroll
        for (int s = 0; s < DP / 16; ++s) {
          const uint64_t step = uint64_t((s >> 2) * (L::kBlock >> 4) + (s & 3) * 2);
          mma_ss(tbase + uint32_t(t) * 128u, qd + step, kd + step, kIdS, s > 0 ? 1u : 0u);
        }
        tc_commit(&sfull[t]);
      };
      // Key tiles that take turns: S of the next but one follows O += P V of one.
      if constexpr (T && kTma) {
        if (pair) {
          constexpr int kStages = L::kPairStages;
          auto pair_s = [&](int i) {
            const int slot = 2 * i % kStages;
            wait(&kfirst[i % kKeys], uint32_t(i / kKeys) & 1u);
            tc_fence_after();
            const uint64_t qd = desc_k_major(sbase), kd = desc_k_major(ring_tile<DP>(sbase, slot));
#pragma unroll
            for (int s = 0; s < DP / 16; ++s) {
              const uint64_t step = uint64_t((s >> 2) * (L::kBlock >> 4) + (s & 3) * 2);
              mma_ss(tbase + uint32_t(i & 1) * 128u, qd + step, kd + step, kIdS, s > 0 ? 1u : 0u);
            }
            tc_commit(&sfull[i & 1]);
            tc_commit(&empty[slot]);
          };
          wait(&qfull[0], 0u);
          pair_s(0);
          pair_s(1);
#pragma unroll 1
          for (int i = 0; i < n; ++i) {
            const int slot = (2 * i + 1) % kStages;
            const uint32_t t = uint32_t(i & 1) * 128u;
            const uint64_t vd = desc_n_major(ring_tile<DP>(sbase, slot), L::kBlock);
            wait(&go[i % kGo], uint32_t(i / kGo) & 1u);
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < kTileKeys / 16; ++s)
              mma_ts(tbase + 256u + t, tbase + t + 8u * s, vd + uint64_t(s * (2048 >> 4)), kIdO,
                     (i > 1 || s > 0) ? 1u : 0u);
            tc_commit(&empty[slot]);
            if (i + 2 < n)
              pair_s(i + 2);
            else
              tc_commit(&sfull[i & 1]);
          }
          const int end = 2 * n - 1;
          ok = mbar_wait_counted(&empty[end % kStages], uint32_t(end / kStages) & 1u) && ok;
        }
      }
      if (!pair) {
        wait(kfirst, 0u);
        for (int t = 0; t < tiles; ++t) {
          wait(&qfull[t], 0u);
          product_s(t, 0);
        }
        tc_commit(&empty[0]);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const int uv = 2 * i + 1, uk = 2 * i + 2;
          const uint64_t vd = desc_n_major(ring + uint32_t(uv % L::kStages) * L::kTile, L::kBlock);
          for (int t = 0; t < tiles; ++t) {
            if (t == 0)
              wait(&go[i % kGo], uint32_t(i / kGo) & 1u);
            else
              wait(psecond, uint32_t(i) & 1u);
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < kTileKeys / 16; ++s)  // 16 keys: two groups of eight rows
              mma_ts(tbase + 256u + uint32_t(t) * 128u, tbase + uint32_t(t) * 128u + 8u * s,
                     vd + uint64_t(s * (2048 >> 4)), kIdO, (i > 0 || s > 0) ? 1u : 0u);
            const bool end = t + 1 == tiles;
            if (end) tc_commit(&empty[uv % L::kStages]);
            if (i + 1 < n) {
              product_s(t, uk);
              if (end) tc_commit(&empty[uk % L::kStages]);
            } else {
              tc_commit(&sfull[t]);
            }
          }
        }
        // The ring's last tiles: every product is done before the memory is given back.
        const int last = 2 * n - 1;
        ok = mbar_wait_counted(&empty[last % L::kStages], uint32_t(last / L::kStages) & 1u) && ok;
      }
    }
    __syncwarp();
  }
  if (!ok) atomicOr(&g_prefix_tc_flags, kFlagWaitRanOut);
  // After a wait that ran out, tensor copies may still be in flight: wait for
  // them, with the same bound, before the shared memory is given back.
  if (__syncthreads_or(!ok) && kTma && tid == 0)
    for (int i = n > kGo ? n - kGo : 0; i < n; ++i) {
      mbar_wait_counted(&go[i % kGo], uint32_t(i / kGo) & 1u);
      if (pair) mbar_wait_counted(&kfirst[i % kKeys], uint32_t(i / kKeys) & 1u);
    }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(*s_taddr), "r"(kTmemCols) : "memory");
  }
}

template <typename H, int DP, bool kTma, bool T>
cudaError_t launch_one(const PrefixArgs& p, const CacheMaps& maps, unsigned items, cudaStream_t stream) {
  auto kern = prefix_tc_kernel<H, DP, kTma, T>;
  static PerDeviceCache attr_set, regs;
  cudaError_t e = set_max_dynamic_smem_once(kern, int(Layout<DP>::kBytes), attr_set);
  if (e != cudaSuccess) return e;
  // The register split above only adds up for exactly this launch size.
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int r = regs.get(dev, [&] {
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kern);
    return e == cudaSuccess ? attr.numRegs : -1;
  });
  if (e != cudaSuccess) return e;
  if (r != kLaunchRegs) return cudaErrorInvalidKernelImage;
  return launch_k(kern, dim3(items), dim3(kTcThreads), Layout<DP>::kBytes, stream, p, maps);
}

// One cache as a tensor map; false: no map describes it.
bool encode_cache(const PrefixArgs& p, nf4_dtype dtype, const char* base, int64_t page_stride, int64_t slot_stride,
                  int64_t head_stride, int box_rows, CUtensorMap* map, int* slot_at, int* head_at) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (!encode) return false;
  struct Dim {
    int64_t size, stride;
    int box;
    int* at;
  } d[3] = {{p.page_size, slot_stride, box_rows, slot_at}, {p.k_heads, head_stride, 1, head_at},
            {p.num_pages, page_stride, 1, nullptr}};
  for (Dim& x : d) {
    if (x.size == 1) x.stride = 256;  // never used, but a valid stride
    if (x.stride <= 0) return false;
  }
  for (int i = 0; i < 2; ++i)  // in the order of their strides
    for (int j = 0; j < 2 - i; ++j)
      if (d[j].stride > d[j + 1].stride) {
        const Dim t = d[j];
        d[j] = d[j + 1];
        d[j + 1] = t;
      }
  cuuint64_t dims[4] = {cuuint64_t(p.dim), 0, 0, 0}, strides[3];
  cuuint32_t box[4] = {64u, 0u, 0u, 0u};
  const cuuint32_t elem[4] = {1u, 1u, 1u, 1u};
  for (int i = 0; i < 3; ++i) {
    dims[i + 1] = cuuint64_t(d[i].size);
    strides[i] = cuuint64_t(d[i].stride);
    box[i + 1] = cuuint32_t(d[i].box);
    if (d[i].at) *d[i].at = i;
  }
  return encode(map, dtype == NF4_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                const_cast<char*>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kTma, bool T>
cudaError_t launch_typed(const PrefixArgs& p, const CacheMaps& maps, nf4_dtype dtype, unsigned items,
                         cudaStream_t stream) {
  if (dtype == NF4_BF16)
    return p.dim <= 64 ? launch_one<Bf16, 64, kTma, T>(p, maps, items, stream)
                       : launch_one<Bf16, 128, kTma, T>(p, maps, items, stream);
  return p.dim <= 64 ? launch_one<Fp16, 64, kTma, T>(p, maps, items, stream)
                     : launch_one<Fp16, 128, kTma, T>(p, maps, items, stream);
}
template <bool T>
cudaError_t launch_maps(const PrefixArgs& p, nf4_dtype dtype, unsigned items, cudaStream_t stream) {
  CacheMaps maps = {};
  // Rows of a box: the largest power of two that divides the page (a box that
  // starts at a multiple of it stays in one page), 8 to 128.
  maps.box_rows = p.page_size & -p.page_size;
  if (maps.box_rows > kTileKeys) maps.box_rows = kTileKeys;
  // Or whole pages, where a tile is made of these.
  maps.tile_keys = prefix_tile_keys(p.page_size);
  if (maps.tile_keys < kTileKeys) maps.box_rows = p.page_size;
  if (maps.box_rows >= 8 && p.num_pages > 0 &&
      encode_cache(p, dtype, p.k, p.k_ps, p.k_ss, p.k_hs, maps.box_rows, &maps.k, &maps.k_slot,
                   &maps.k_head) &&
      encode_cache(p, dtype, p.v, p.v_ps, p.v_ss, p.v_hs, maps.box_rows, &maps.v, &maps.v_slot,
                   &maps.v_head))
    return launch_typed<true, T>(p, maps, dtype, items, stream);
  return launch_typed<false, T>(p, maps, dtype, items, stream);
}

}  // namespace

cudaError_t launch_prefix_tc(const PrefixArgs& p, nf4_dtype dtype, bool tree, unsigned items, cudaStream_t stream) {
  return tree ? launch_maps<true>(p, dtype, items, stream) : launch_maps<false>(p, dtype, items, stream);
}

cudaError_t prefix_tc_flags(unsigned int** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_prefix_tc_flags);
}

}  // namespace nf4
