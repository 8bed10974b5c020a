// nf4_prefix_attn.cu -- attention of a batch over a paged cache whose first
// keys are shared by every sequence.
//
// out = sum_j exp(s_j - lse) v_j over the shared keys and then the sequence's
// own ones. A softmax over a union of key ranges joins from the ranges'
// (maximum m_x, sum l_x, unscaled output o_x): with m = max m_x,
// out = sum_x e^(m_x - m) o_x / sum_x e^(m_x - m) l_x. So the shared keys are
// treated once for all rows of a key/value head together (every query token
// of the batch times its group of query heads: a matrix product instead of
// one matrix-vector product per sequence), each sequence's own keys apart,
// both cut into ranges of keys so that a few rows over a long axis still fill
// the SMs, and a last kernel joins the ranges in order.
//
// Here: the plan, the kernel for items of few rows and the join. Few rows (a
// token and its group of query heads) make every key and value used by a
// handful of rows only: the bytes of the cache bound them, and the 16 x 8 x 16
// tensor instruction does the arithmetic, since the 128 rows of the
// 5th-generation ones would be empty. Own keys alone, 32 heads of 128: 128
// sequences of 187 keys take 66 us (6.0 TB/s, 89% of measured copy
// bandwidth), 64 of 750 keys 128 us (93%). Short sequences are bound by a
// warp's instructions (start, addresses, epilogue: 2200 of them for 75 keys before
// the addresses were made cheaper): 128 x 75 keys 37 us (64%).
//
// The weights e^(s - m) are rounded to the caches' 16-bit type for the product
// with v: a tensor instruction takes both operands in one type, and a second
// product with the remainders would double that work. One rounding per key
// (2^-8 of its weight in bf16, 2^-11 in fp16), independent from key to key, adds
// about what the output's own rounding does.
#include "nf4_prefix_attn.cuh"

namespace nf4 {
namespace {

__device__ unsigned int g_prefix_flags = 0;

constexpr int kSms = 152;
constexpr int kUnit = 64;    // granularity of the ranges of keys of the few-row kernel
constexpr int kStages = 2;

// R rows per tile, W warps. R = 64: a warp has 16 rows and all keys of a stage
// of 64. R = 16: the warps share the rows and have 16 keys of a stage each.
// Where there are enough items, two warps: small CTAs (34 KB at 128 elements), so
// that six are on an SM and the start of one (three dependent loads before its
// first keys) hides behind the keys of the others. Where all items fit on the
// SMs at once, four: a short range is one stage (two sequences over 300 keys
// 6.9 -> 5.8 us; 32 over 500 own keys each would take 12 instead of 10.4).
template <int R, int W>
struct Shape {
  static constexpr int kThreads = 32 * W;
  static constexpr int kKeys = R == 64 ? 64 : 16 * W;  // keys per stage
};
// A row of a stage in shared memory: 16 bytes on, so that eight rows' chunks lie in different banks.
template <int DP>
constexpr uint32_t kPitch = DP * 2 + 16;
constexpr int64_t kFewItems = kSms * 3;  // CTAs of four warps that fit on the SMs

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <typename H>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (H::kDtype == NF4_BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One item with tiles of R rows. The warps' key shares of R = 16 are joined
// through shared memory at the end.
template <typename H, int DP, int R, int W, bool T>
__device__ __forceinline__ void attend(const PrefixArgs& a, const PrefixItem& it, unsigned char* smem) {
  constexpr int kWarps = W, kThreads = Shape<R, W>::kThreads, kKeys = Shape<R, W>::kKeys;
  constexpr int KW = R == 64 ? kKeys : kKeys / kWarps;  // keys of a stage per warp
  constexpr int NB = KW / 8;                            // score blocks of 8 keys
  constexpr int CPR = DP / 8;                           // 16-byte chunks per row
  constexpr int RPI = 32 / CPR;                         // rows per copy instruction of a warp
  constexpr uint32_t kTile = kKeys * kPitch<DP>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem);
  const int ntiles = (it.k1 - it.k0 + kKeys - 1) / kKeys;

  // Copies of tile i: warp w brings rows 16 w .. 16 w + 15, lane l chunk l % CPR
  // of rows l / CPR, l / CPR + RPI, .. What is not there is filled with zeros,
  // from no address of the cache. Where 16 rows are sure to lie in one page, a
  // lane's addresses are a slot's stride apart; otherwise lane l looks up row
  // l & 15 and hands out its offsets. (Instructions bound items of few keys.
  // One bulk copy per row, no addresses to speak of, is slower all the same: 256
  // bytes at a time, 64 sequences x 32 heads x 187 keys took 47 us instead of 37.)
  const bool whole = a.page_size % 16 == 0;  // (ranges of keys begin at multiples of 64)
  const int copy_row = lane / CPR, copy_chunk = lane % CPR;
  const bool column = copy_chunk < a.dim / 8;
  const uint32_t copy_to = sbase + uint32_t(warp * 16 + copy_row) * kPitch<DP> + uint32_t(copy_chunk) * 16u;
  const char* const k_head = a.k + int64_t(it.head) * a.k_hs + copy_chunk * 16;
  const char* const v_head = a.v + int64_t(it.head) * a.v_hs + copy_chunk * 16;
  auto fetch_page = [&](int i) {
    const int j = it.k0 + i * kKeys + warp * 16 + (whole ? 0 : lane & 15);
    return j < it.k1 ? key_page(a, it, j) : 0;
  };
  auto copy_tile = [&](int i, int page) {
    const int j0 = it.k0 + i * kKeys + warp * 16;
    const uint32_t dst = copy_to + uint32_t(i % kStages) * (2 * kTile);
    if (whole) {
      int valid = min(it.k1 - j0, 16);
      if (unsigned(page) >= unsigned(a.num_pages)) {
        if (valid > 0) atomicOr(&g_prefix_flags, kFlagBadIndex);
        valid = 0;
      }
      const int slot = (a.page_shift >= 0 ? j0 & (a.page_size - 1) : j0 % a.page_size) + copy_row;
      const char* ks = k_head + int64_t(page) * a.k_ps + int64_t(slot) * a.k_ss;
      const char* vs = v_head + int64_t(page) * a.v_ps + int64_t(slot) * a.v_ss;
      if (valid == 16 && a.dim == DP) {
#pragma unroll
        for (int x = 0; x < 16 / RPI; ++x) {
          cp_async16(dst + uint32_t(x * RPI) * kPitch<DP>, ks, true);
          cp_async16(dst + uint32_t(x * RPI) * kPitch<DP> + kTile, vs, true);
          ks += RPI * a.k_ss;
          vs += RPI * a.v_ss;
        }
      } else {
#pragma unroll 2
        for (int x = 0; x < 16 / RPI; ++x) {
          const bool there = x * RPI + copy_row < valid && column;
          cp_async16(dst + uint32_t(x * RPI) * kPitch<DP>, there ? ks : a.q, there);
          cp_async16(dst + uint32_t(x * RPI) * kPitch<DP> + kTile, there ? vs : a.q, there);
          ks += RPI * a.k_ss;
          vs += RPI * a.v_ss;
        }
      }
      return;
    }
    const int j = j0 + (lane & 15);
    KeyOffset off{0, 0};
    if (!(j < it.k1 && key_offset(a, it, j, page, &g_prefix_flags, &off))) off.k = off.v = -1;
#pragma unroll 2
    for (int x = 0; x < 16 / RPI; ++x) {
      const int64_t ko = __shfl_sync(0xffffffffu, off.k, x * RPI + copy_row);
      const int64_t vo = __shfl_sync(0xffffffffu, off.v, x * RPI + copy_row);
      const bool there = ko >= 0 && column;
      cp_async16(dst + uint32_t(x * RPI) * kPitch<DP>, there ? a.k + ko + copy_chunk * 16 : a.q, there);
      cp_async16(dst + uint32_t(x * RPI) * kPitch<DP> + kTile, there ? a.v + vo + copy_chunk * 16 : a.q, there);
    }
  };

  // R = 16: a warp reads only what it brought, so that both stages are under
  // way from the start and no warp waits for another
  constexpr int kAhead = R == 64 ? kStages - 1 : kStages;
  int page = fetch_page(0), next_page = fetch_page(1);
#pragma unroll 1
  for (int i = 0; i < kAhead; ++i) {
    if (i < ntiles) copy_tile(i, page);
    cp_async_commit();
    page = next_page;
    if (i + 1 < kAhead) next_page = fetch_page(i + 2);
  }

  // the item's rows of Q as A fragments
  const int rbase = R == 64 ? warp * 16 : 0;
  const int ra = rbase + (lane >> 2), rb = ra + 8;  // this thread's two rows of the tile
  const bool two = R == 64 || it.rows > 8;          // there is a second one
  uint32_t qf[DP / 16][4];
  {
    const char* qp[2];
    bool there[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int rl = x ? rb : ra;
      there[x] = rl < it.rows;
      qp[x] = a.q;
      if (x && !two) break;
      const int r = it.r0 + (there[x] ? rl : 0);
      qp[x] = a.q + int64_t(it.t0 + r / a.group) * a.q_ts + int64_t(it.head * a.group + r % a.group) * a.q_hs;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int s = 0; s < DP / 16; ++s) qf[s][x] = qf[s][x + 2] = 0u;
      if (x && !two) break;
#pragma unroll
      for (int s = 0; s < DP / 16; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int d = s * 16 + h * 8 + (lane & 3) * 2;
          if (there[x] && d < a.dim) qf[s][x + 2 * h] = *reinterpret_cast<const uint32_t*>(qp[x] + d * 2);
        }
    }
  }
  // keys (within the segment) that the two rows see
  const int lima = ra < it.rows ? min(visible_keys<T>(it, (it.r0 + ra) / a.group), it.k1) : 0;
  const int limb = rb < it.rows ? min(visible_keys<T>(it, (it.r0 + rb) / a.group), it.k1) : 0;
  // up to here no row of the tile is masked
  const int free_to = min(unmasked_keys<T>(it, it.r0 / a.group), it.k1);

  float o[DP / 8][4];
#pragma unroll
  for (int i = 0; i < DP / 8; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x) o[i][x] = 0.0f;
  float ma = -INFINITY, mb = -INFINITY, la = 0.0f, lb = 0.0f;

  auto copy_next = [&](int i) {
    if (i + kAhead < ntiles) {
      copy_tile(i + kAhead, page);
      page = fetch_page(i + kAhead + 1);
    }
    cp_async_commit();
  };
  const int kw = R == 64 ? 0 : warp * KW;  // first key of a stage for this warp
  const uint32_t klane = sbase + uint32_t(kw + (lane & 7) + ((lane >> 4) << 3)) * kPitch<DP> + ((lane & 8) << 1);
  const uint32_t vlane = sbase + kTile + uint32_t(kw + (lane & 15)) * kPitch<DP> + (lane & 16);
  bool first = true;
  for (int i = 0; i < ntiles; ++i) {
    cp_async_wait<kAhead - 1>();
    if constexpr (R == 64) {
      __syncthreads();  // tile i landed for every warp; everyone is done with tile i - 1's stage
      copy_next(i);
    } else {
      __syncwarp();
    }
    const uint32_t stage = uint32_t(i % kStages) * (2 * kTile);
    if (it.k0 + i * kKeys + kw < it.k1) {  // some of this warp's keys are there
      float s[NB][4];
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[n][x] = 0.0f;
#pragma unroll
      for (int st = 0; st < DP / 16; ++st)
#pragma unroll
        for (int n = 0; n < NB / 2; ++n) {
          uint32_t b[4];
          ldsm4(klane + stage + uint32_t(n * 16) * kPitch<DP> + uint32_t(st * 32), b);
          mma16816<H>(s[2 * n], qf[st], b[0], b[1]);
          mma16816<H>(s[2 * n + 1], qf[st], b[2], b[3]);
        }

      const int j0 = it.k0 + i * kKeys + kw + (lane & 3) * 2;
      if (it.k0 + (i + 1) * kKeys > free_to) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (j0 + n * 8 + (x & 1) >= (x < 2 ? lima : limb)) s[n][x] = -INFINITY;
        if constexpr (T) {
          if (it.own) {  // at most 64 keys of a warp: one window per row
            const int first_key = it.k0 + i * kKeys + kw;
            const uint64_t wa = lima > 0 ? tree_window(a, it, it.t0 + (it.r0 + ra) / a.group, first_key) : 0ull;
            const uint64_t wb = limb > 0 ? tree_window(a, it, it.t0 + (it.r0 + rb) / a.group, first_key) : 0ull;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (!((x < 2 ? wa : wb) >> (n * 8 + (lane & 3) * 2 + (x & 1)) & 1ull)) s[n][x] = -INFINITY;
          }
        }
      }
      float xa = -INFINITY, xb = -INFINITY;
#pragma unroll
      for (int n = 0; n < NB; ++n) xa = fmaxf(xa, fmaxf(s[n][0], s[n][1]));
      if (two) {
#pragma unroll
        for (int n = 0; n < NB; ++n) xb = fmaxf(xb, fmaxf(s[n][2], s[n][3]));
      }
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, d));
        if (two) xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, d));
      }
      xa *= a.scale_log2;
      xb *= a.scale_log2;
      // m is the maximum at the time of the last rescale; l and o share it
      if (first) {
        ma = xa;
        mb = xb;
        first = false;
      } else if (__any_sync(0xffffffffu, xa > ma + kGrowth || xb > mb + kGrowth)) {
        const float na = fmaxf(ma, xa), nb = fmaxf(mb, xb);
        const float fa = na == -INFINITY ? 1.0f : ex2(ma - na), fb = nb == -INFINITY ? 1.0f : ex2(mb - nb);
        ma = na;
        mb = nb;
        la *= fa;
        lb *= fb;
#pragma unroll
        for (int d = 0; d < DP / 8; ++d) {
          o[d][0] *= fa;
          o[d][1] *= fa;
          o[d][2] *= fb;
          o[d][3] *= fb;
        }
      }
      const float ba = ma == -INFINITY ? 0.0f : ma - kLift<H>, bb = mb == -INFINITY ? 0.0f : mb - kLift<H>;
      uint32_t pf[NB][2];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const float p0 = ex2(fmaf(s[n][0], a.scale_log2, -ba)), p1 = ex2(fmaf(s[n][1], a.scale_log2, -ba));
        la += p0 + p1;
        pf[n][0] = H::down2(p0, p1);
        pf[n][1] = 0u;
        if (two) {
          const float p2 = ex2(fmaf(s[n][2], a.scale_log2, -bb)), p3 = ex2(fmaf(s[n][3], a.scale_log2, -bb));
          lb += p2 + p3;
          pf[n][1] = H::down2(p2, p3);
        }
      }
#pragma unroll
      for (int n = 0; n < NB / 2; ++n) {
        const uint32_t pa[4] = {pf[2 * n][0], pf[2 * n][1], pf[2 * n + 1][0], pf[2 * n + 1][1]};
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
          uint32_t b[4];
          ldsm4t(vlane + stage + uint32_t(n * 16) * kPitch<DP> + uint32_t(d * 32), b);
          mma16816<H>(o[2 * d], pa, b[0], b[1]);
          mma16816<H>(o[2 * d + 1], pa, b[2], b[3]);
        }
      }
    }
    if constexpr (R != 64) {
      __syncwarp();  // every lane is done with the stage
      copy_next(i);
    }
  }
  ma -= kLift<H>;  // from here what l and o are relative to
  mb -= kLift<H>;
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    la += __shfl_xor_sync(0xffffffffu, la, d);
    lb += __shfl_xor_sync(0xffffffffu, lb, d);
  }
  cp_async_wait<0>();

  if constexpr (R != 64) {
    // join the four warps' key shares: maxima and sums first, then the
    // outputs scaled to the common maximum, added in warp order
    __syncthreads();  // the stages are free
    float2* sml = reinterpret_cast<float2*>(smem);             // [warp][16]
    float* so = reinterpret_cast<float*>(smem + 512);          // [warp][16][DP + 4]
    constexpr int kStep = DP + 4;
    if ((lane & 3) == 0) {
      sml[warp * 16 + ra] = make_float2(ma, la);
      sml[warp * 16 + rb] = make_float2(mb, lb);
    }
    __syncthreads();
    float ta = -INFINITY, tb = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      ta = fmaxf(ta, sml[w * 16 + ra].x);
      tb = fmaxf(tb, sml[w * 16 + rb].x);
    }
    const float fa = ma == -INFINITY ? 0.0f : ex2(ma - ta), fb = mb == -INFINITY ? 0.0f : ex2(mb - tb);
#pragma unroll
    for (int d = 0; d < DP / 8; ++d) {
      const int col = d * 8 + (lane & 3) * 2;
      if (ra < it.rows)
        *reinterpret_cast<float2*>(so + (warp * 16 + ra) * kStep + col) = make_float2(o[d][0] * fa, o[d][1] * fa);
      if (rb < it.rows)
        *reinterpret_cast<float2*>(so + (warp * 16 + rb) * kStep + col) = make_float2(o[d][2] * fb, o[d][3] * fb);
    }
    __syncthreads();
    // four lanes of a chunk of 4 elements each: thread -> (row, 4 columns)
    for (int e = threadIdx.x; e < it.rows * (DP / 4); e += kThreads) {
      const int r = e / (DP / 4), col = (e % (DP / 4)) * 4;
      if (col >= a.dim) continue;
      float m = -INFINITY, l = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sml[w * 16 + r].x);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 x = sml[w * 16 + r];
        l += x.x == -INFINITY ? x.y : x.y * ex2(x.x - m);  // x.y is 0, or NaN
        const float4 y = *reinterpret_cast<const float4*>(so + (w * 16 + r) * kStep + col);
        v.x += y.x;
        v.y += y.y;
        v.z += y.z;
        v.w += y.w;
      }
      const RowOut ro = row_out(a, it, it.r0 + r);
      if (!a.direct) {
        *reinterpret_cast<float4*>(ro.part + col) = v;
        if (col == 0) *ro.ml = make_float2(m, l);
      } else {
        if (!part_holds(make_float2(m, l))) v = make_float4(0.f, 0.f, 0.f, 0.f);
        write_row<H>(ro.out, ro.lse, col, m, l, v);
      }
    }
  } else {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = x ? rb : ra;
      if (r >= it.rows) continue;
      const float m = x ? mb : ma, l = x ? lb : la;
      const RowOut ro = row_out(a, it, it.r0 + r);
      if (!a.direct) {
#pragma unroll
        for (int d = 0; d < DP / 8; ++d) {
          const int col = d * 8 + (lane & 3) * 2;
          if (col < a.dim) *reinterpret_cast<float2*>(ro.part + col) = make_float2(o[d][2 * x], o[d][2 * x + 1]);
        }
        if ((lane & 3) == 0) *ro.ml = make_float2(m, l);
      } else {
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
        for (int d = 0; d < DP / 8; ++d) {
          const int col = d * 8 + (lane & 3) * 2;
          if (col < a.dim)
            *reinterpret_cast<uint32_t*>(ro.out + col * 2) =
                part_holds(make_float2(m, l)) ? H::down2(o[d][2 * x] * inv, o[d][2 * x + 1] * inv) : 0u;
        }
        if ((lane & 3) == 0 && ro.lse) *ro.lse = l > 0.0f || l != l ? fmaf(m, kLn2, logf(l)) : -INFINITY;
      }
    }
  }
}

// `beside`: the launch before this one is other items of the same call, which
// this one does not depend on. Its CTAs all waited for the grids before it
// ahead of letting this one start, so there is nothing to wait for here; but
// what follows (the join) only waits for this launch, so its last CTA ends
// after the other launch did.
template <typename H, int DP, int R, int W, bool T>
__global__ void __launch_bounds__(Shape<R, W>::kThreads, R == 64 ? 2 : (DP == 64 ? 20 : 12) / W)
    prefix_mma_kernel(const __grid_constant__ PrefixArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  if (!a.beside) pdl_wait_prior_grid();
  pdl_allow_dependents();
  const PrefixItem it = prefix_item<T>(a, unsigned(a.first) + blockIdx.x, &g_prefix_flags);
  if (it.rows > 0) attend<H, DP, R, W, T>(a, it, smem);
  if (a.fused) unheld_rows<H>(a, W, &g_prefix_flags);
  if (a.beside && blockIdx.x + 1 == gridDim.x) pdl_wait_prior_grid();
}

// Joins a row's partial results: 1 to 8 warps per row, four elements per lane,
// kBatch ranges per warp and round; the launch takes as many warps as make one
// round (up to 128 ranges). The partial outputs are asked for together with the
// maxima and sums, not after them (those of ranges that hold nothing are read and
// dropped): one latency, which is most of this kernel's time. The order of
// the sums depends on the plan alone.
constexpr int kJoinWarps = 8;
template <typename H, int kBatch>
__device__ __forceinline__ void join_rows(const PrefixArgs& a, int per_row) {
  static_assert(kBatch <= 32, "a lane per range of a round");
  __shared__ float4 sv[kJoinWarps][32];
  __shared__ float sl[kJoinWarps];
  pdl_allow_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * (kJoinWarps / per_row) + warp / per_row;
  const int share = warp % per_row;
  const int64_t rows = int64_t(a.tokens) * a.q_heads;
  const bool there = row < rows;
  const int t = there ? int(row / a.q_heads) : 0;
  const bool mine = lane * 4 < a.dim;
  pdl_wait_prior_grid();
  float l = 0.0f, m = -INFINITY;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (there) {
    const float2* ml = a.ml + row * a.splits;
    const float* src = a.part + row * a.dim + lane * 4;
    const int64_t step = rows * a.dim;
    int n = a.splits;
    float4 y[kBatch];
    auto load = [&](int s0) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        y[u] = mine && s0 + u < n ? *reinterpret_cast<const float4*>(src + (s0 + u) * step)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(share * kBatch);
    // this lane's range of the first round, and everybody's maxima
    float2 x = share * kBatch + lane < n ? ml[share * kBatch + lane] : make_float2(-INFINITY, 0.0f);
    float all[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) all[i] = 32 * i + lane < n ? ml[32 * i + lane].x : -INFINITY;
    if (a.cu_q && a.suffix_splits > 0 && (t < a.cu_q[0] || t >= a.cu_q[a.batch])) n = a.prefix_splits;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (32 * i + lane < n) m = fmaxf(m, all[i]);
    for (int s = 128 + lane; s < n; s += 32) m = fmaxf(m, ml[s].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    for (int s0 = share * kBatch; s0 < n; s0 += per_row * kBatch) {
      if (s0 > share * kBatch) {
        load(s0);
        x = s0 + lane < n ? ml[s0 + lane] : make_float2(-INFINITY, 0.0f);
      }
      // the range's weight; 0: it holds nothing, and its partial output is not to be looked at
      const bool holds = s0 + lane < n && lane < kBatch && !(x.x == -INFINITY && x.y == 0.0f);
      const float w = !holds ? 0.0f : x.x == -INFINITY ? 1.0f : ex2(x.x - m);
      const unsigned which = __ballot_sync(0xffffffffu, holds);
      const float part_l = holds ? x.y * w : 0.0f;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const float wu = __shfl_sync(0xffffffffu, w, u);
        l += __shfl_sync(0xffffffffu, part_l, u);
        if (which >> u & 1u) {
          v.x = fmaf(y[u].x, wu, v.x);
          v.y = fmaf(y[u].y, wu, v.y);
          v.z = fmaf(y[u].z, wu, v.z);
          v.w = fmaf(y[u].w, wu, v.w);
        }
      }
    }
  }
  if (per_row > 1) {
    sv[warp][lane] = v;
    if (lane == 0) sl[warp] = l;
    __syncthreads();
    if (share != 0) return;
    for (int s = 1; s < per_row; ++s) {
      const float4 y = sv[warp + s][lane];
      v.x += y.x;
      v.y += y.y;
      v.z += y.z;
      v.w += y.w;
      l += sl[warp + s];
    }
  }
  if (!there) return;
  const bool any = l > 0.0f || l != l;
  const float inv = any ? 1.0f / l : 0.0f;
  if (mine) {
    char* out = a.out + int64_t(t) * a.out_ts + int64_t(row - int64_t(t) * a.q_heads) * a.out_hs;
    *reinterpret_cast<uint2*>(out + lane * 8) =
        make_uint2(H::down2(v.x * inv, v.y * inv), H::down2(v.z * inv, v.w * inv));
  }
  if (lane == 0 && a.lse) a.lse[row] = any ? fmaf(m, kLn2, logf(l)) : -INFINITY;
}

// The same for few ranges and many rows: four rows per warp, all their loads
// in flight together (37900 rows of two ranges: the call 137 -> 130 us).
constexpr int kFewRows = 4;
template <typename H, int kRanges>
__device__ __forceinline__ void join_rows_few(const PrefixArgs& a) {
  pdl_allow_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t rows = int64_t(a.tokens) * a.q_heads;
  const int64_t first = (int64_t(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5)) * kFewRows;
  const bool mine = lane * 4 < a.dim;
  pdl_wait_prior_grid();
  if (first >= rows) return;
  float4 y[kFewRows][kRanges];
  float2 x[kFewRows][kRanges];
#pragma unroll
  for (int k = 0; k < kFewRows; ++k) {
    const int64_t row = first + k < rows ? first + k : rows - 1;
#pragma unroll
    for (int s = 0; s < kRanges; ++s) {
      x[k][s] = s < a.splits ? a.ml[row * a.splits + s] : make_float2(-INFINITY, 0.0f);
      y[k][s] = mine && s < a.splits
                    ? *reinterpret_cast<const float4*>(a.part + (s * rows + row) * a.dim + lane * 4)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  int held[2] = {0, a.tokens};  // the tokens that some sequence holds
  if (a.cu_q && a.suffix_splits > 0) {
    held[0] = a.cu_q[0];
    held[1] = a.cu_q[a.batch];
  }
#pragma unroll
  for (int k = 0; k < kFewRows; ++k) {
    const int64_t row = first + k;
    if (row >= rows) break;
    const int t = int(row / a.q_heads);
    const int n = t >= held[0] && t < held[1] ? a.splits : a.prefix_splits;
    float m = -INFINITY, l = 0.0f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < kRanges; ++s)
      if (s < n) m = fmaxf(m, x[k][s].x);
#pragma unroll
    for (int s = 0; s < kRanges; ++s) {
      if (s >= n || (x[k][s].x == -INFINITY && x[k][s].y == 0.0f)) continue;
      const float w = x[k][s].x == -INFINITY ? 1.0f : ex2(x[k][s].x - m);
      l = fmaf(x[k][s].y, w, l);
      v.x = fmaf(y[k][s].x, w, v.x);
      v.y = fmaf(y[k][s].y, w, v.y);
      v.z = fmaf(y[k][s].z, w, v.z);
      v.w = fmaf(y[k][s].w, w, v.w);
    }
    const bool any = l > 0.0f || l != l;
    const float inv = any ? 1.0f / l : 0.0f;
    if (mine) {
      char* out = a.out + int64_t(t) * a.out_ts + int64_t(row - int64_t(t) * a.q_heads) * a.out_hs;
      *reinterpret_cast<uint2*>(out + lane * 8) =
          make_uint2(H::down2(v.x * inv, v.y * inv), H::down2(v.z * inv, v.w * inv));
    }
    if (lane == 0 && a.lse) a.lse[row] = any ? fmaf(m, kLn2, logf(l)) : -INFINITY;
  }
}

// The joins, and the check of cu_q that the items leave over.
template <typename H, int kBatch, bool kCheck>
__global__ void __launch_bounds__(32 * kJoinWarps)
    prefix_join_kernel(const __grid_constant__ PrefixArgs a, int per_row) {
  join_rows<H, kBatch>(a, per_row);
  if (kCheck) check_cu_q(a, kJoinWarps, &g_prefix_flags);
}
template <typename H, int kRanges, bool kCheck>
__global__ void __launch_bounds__(32 * kJoinWarps) prefix_join_few_kernel(const __grid_constant__ PrefixArgs a) {
  join_rows_few<H, kRanges>(a);
  if (kCheck) check_cu_q(a, kJoinWarps, &g_prefix_flags);
}

// A call without a single key.
template <typename H>
__global__ void __launch_bounds__(128) prefix_empty_kernel(const __grid_constant__ PrefixArgs a) {
  pdl_allow_dependents();
  pdl_wait_prior_grid();
  const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= int64_t(a.tokens) * a.q_heads) return;
  const int64_t t = row / a.q_heads;
  char* out = a.out + t * a.out_ts + (row - t * a.q_heads) * a.out_hs;
  if (lane * 4 < a.dim) *reinterpret_cast<uint2*>(out + lane * 8) = make_uint2(0u, 0u);
  if (lane == 0 && a.lse) a.lse[row] = -INFINITY;
}

template <typename H, int DP, int R, int W, bool T>
cudaError_t launch_mma(const PrefixArgs& p, unsigned items, cudaStream_t stream) {
  auto kern = prefix_mma_kernel<H, DP, R, W, T>;
  constexpr int smem = kStages * 2 * Shape<R, W>::kKeys * int(kPitch<DP>);
  static PerDeviceCache attr_set;
  const cudaError_t e = set_max_dynamic_smem_once(kern, smem, attr_set);
  if (e != cudaSuccess) return e;
  return launch_k(kern, dim3(items), dim3(Shape<R, W>::kThreads), smem, stream, p);
}

template <typename H, int DP, bool T>
cudaError_t launch_rows(const PrefixArgs& p, int rows, unsigned items, cudaStream_t stream) {
  if (rows == 64) return launch_mma<H, DP, 64, 4, T>(p, items, stream);
  return items <= kFewItems ? launch_mma<H, DP, 16, 4, T>(p, items, stream)
                            : launch_mma<H, DP, 16, 2, T>(p, items, stream);
}
template <typename H, bool T>
cudaError_t launch_rows(const PrefixArgs& p, int rows, unsigned items, cudaStream_t stream) {
  return p.dim <= 64 ? launch_rows<H, 64, T>(p, rows, items, stream) : launch_rows<H, 128, T>(p, rows, items, stream);
}

template <typename H, bool kCheck>
cudaError_t launch_join(const PrefixArgs& p, cudaStream_t stream) {
  const int64_t rows = int64_t(p.tokens) * p.q_heads;
  const int64_t few = int64_t(kJoinWarps) * kFewRows;
  if (p.splits <= 4 && rows >= few * kSms)
    return launch_k(p.splits <= 2 ? prefix_join_few_kernel<H, 2, kCheck> : prefix_join_few_kernel<H, 4, kCheck>,
                    dim3(unsigned((rows + few - 1) / few)), dim3(32 * kJoinWarps), 0, stream, p);
  int per_row = 1;
  while (per_row < kJoinWarps && per_row * 8 < p.splits) per_row *= 2;
  const int64_t blocks = (rows * per_row + kJoinWarps - 1) / kJoinWarps;
  return launch_k(p.splits <= 4    ? prefix_join_kernel<H, 4, kCheck>
                  : p.splits <= 64 ? prefix_join_kernel<H, 8, kCheck>
                                   : prefix_join_kernel<H, 16, kCheck>,
                  dim3(unsigned(blocks)), dim3(32 * kJoinWarps), 0, stream, p, per_row);
}

template <typename H>
cudaError_t launch_typed(const PrefixArgs& p, cudaStream_t stream) {
  const int64_t rows = int64_t(p.tokens) * p.q_heads;
  if (p.splits == 0 && !p.fused)
    return launch_k(prefix_empty_kernel<H>, dim3(unsigned((rows + 3) / 4)), dim3(128), 0, stream, p);
  const int64_t prefix_items = int64_t(p.prefix_tiles) * p.prefix_splits * p.k_heads;
  const int64_t suffix_items = int64_t(p.suffix_tiles) * p.suffix_splits * p.k_heads;
  if (prefix_items + suffix_items > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  // Prefix items, then suffix items; one launch where both take the same kernel.
  const int64_t counts[2] = {prefix_items, suffix_items};
  const int tile_rows[2] = {p.prefix_rows, p.suffix_rows};
  int64_t first = 0;
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
    int64_t items = counts[i];
    const int tile = tile_rows[i];
    if (i == 0 && tile == tile_rows[1] && !p.fused) items += counts[1];
    if (items == 0 || first == prefix_items + suffix_items) continue;
    PrefixArgs q = p;
    q.first = int(first);
    q.beside = first > 0;
    q.fused = p.fused && i == 1;
    q.direct = p.direct || q.fused;
    const bool tree = p.tree && first + items > prefix_items;  // own keys are among them
    e = tile == 256 ? launch_prefix_tc(q, H::kDtype, tree, unsigned(items), stream)
        : tree      ? launch_rows<H, true>(q, tile, unsigned(items), stream)
                    : launch_rows<H, false>(q, tile, unsigned(items), stream);
    first += items;
  }
  if (e != cudaSuccess || p.direct || p.fused) return e;
  const bool check = p.cu_q && p.suffix_splits > 0 && p.batch > 32;  // (its mere presence costs 0.3 us)
  return check ? launch_join<H, true>(p, stream) : launch_join<H, false>(p, stream);
}

}  // namespace

namespace {

constexpr int64_t kStreamBytes = 32 << 20;  // a quarter of L2
constexpr int kMaxRanges = 152;  // per row, of the shared and of the own keys each (more where ranges reach kMostKeys)

// Keys per range of the mma kernel, in units of 64: about eight items per SM
// where there is that much, else one for each CTA that fits on the SMs (128
// sequences x 2000 keys of one head: 35.3 -> 31.9 us); at most kMaxRanges ranges.
int64_t mma_range(int64_t tiles, int64_t units, int dim) {
  const int64_t total = tiles * units, resident = kSms * (dim <= 64 ? 10 : 6);
  int64_t per = total / (kSms * 8);
  if (per < 6) per = (total + resident - 1) / resident;
  per = per < 1 ? 1 : per;
  return units > per * kMaxRanges ? (units + kMaxRanges - 1) / kMaxRanges : per;
}

// Keys per range of the tcgen05 kernel (one CTA per SM), in half tiles but
// whole tiles of them: the number of ranges that ends soonest, counting a wave
// of CTAs as its key tiles plus about three for its start and end, and the
// partial results of a range (written and read in binary32, about 8 TB/s) in
// the same unit of about a microsecond. Candidates: what fills one to six
// waves, and three, two and one quarters of that.
int64_t tc_range(int64_t row_tiles, int64_t key_tiles, int64_t rows, int sms) {
  int32_t best = int32_t(key_tiles);
  const int32_t keys = best, tiles = row_tiles < (1 << 30) ? int32_t(row_tiles) : 1 << 30;
  double least = double((row_tiles + sms - 1) / sms) * double(key_tiles + 3);  // one range
  for (int32_t w = 1; w <= 6; ++w) {
    int32_t most = w * sms / tiles;
    most = most < kMaxRanges ? most : kMaxRanges;
    most = most < keys ? most : keys;
    for (int32_t q = 4; q >= 1; --q) {
      const int32_t s = most * q / 4;
      if (s < 2) break;
      const int32_t per = (keys + s - 1) / s, used = (keys + per - 1) / per;
      const int32_t waves = (tiles * used + sms - 1) / sms;  // at most 6 waves of CTAs
      const double cost = double(waves) * double(per + 3) + double(used) * double(rows) * 1e-4;
      if (cost < least) {
        least = cost;
        best = per;
      }
    }
  }
  return 2 * int64_t(best);
}

// The own keys run on another kernel beside the shared ones. Where they are the
// longer part (bound by their bytes, at about 6 TB/s; sequences hold some 80% of
// the longest on average), the shared keys are cut into fewer ranges, which
// cost less start and partial results and leave the other SMs to the own keys:
// the number that lets both end soonest. A key tile takes about 1.7 us beside
// own keys (2.0 with two tiles of rows; 0.8 of that at 64 elements), a range
// three more. 64 sequences x 32 heads over 2048 shared and 187 own keys take 45
// us, 53 with ranges for every SM; 128 x 32 heads over 8, 4000 and 300: 44 and 55.
int64_t beside_range(const nf4_prefix_attention_args& a, const PrefixArgs& p, int64_t tiles, int64_t key_tiles,
                     int64_t rows, int64_t per) {
  const double own = double(a.batch) * double(p.suffix_max) * double(p.k_heads) * double(p.dim) * 4.0 * 0.8 / 6e6;
  const double tile = (rows <= 128 ? 1.7 : 2.0) * (p.dim <= 64 ? 0.8 : 1.0);
  if (own < (double(per) * 0.5 + 3.0) * 1.2) return per;
  double least = 0.0;
  for (int64_t s = 1; s * tiles <= kSms && s <= key_tiles; ++s) {
    const int64_t each = (key_tiles + s - 1) / s, ctas = tiles * ((key_tiles + each - 1) / each);
    const double shared = double(each + 3) * tile;
    const double alone = shared * double(kSms - ctas);  // of the SMs left to the own keys
    const double cost = (own * kSms <= alone ? shared : own + shared - alone / kSms) +
                        double(s) * double(rows) * double(p.k_heads) * 1e-4;
    if (least == 0.0 || cost < least) {
      least = cost;
      per = 2 * each;
    }
  }
  return per;
}

// Where the shared keys would take every SM once, and the own keys are little
// work: the SMs to leave to them, so that they end meanwhile (a CTA of theirs
// takes about 5 us, three or six run on an SM; a key tile about 1.5 us). 0: none.
int sms_for_own(const PrefixArgs& p, int64_t own_items, int64_t tiles, int64_t per, int64_t units) {
  const int64_t ctas = tiles * ((units + per - 1) / per);
  if (ctas > kSms) return 0;
  const double own = double(own_items) * (own_items <= kFewItems ? 5.0 / 3.0 : 5.0 / 6.0);
  const double keep = own / ((double(per) * 0.5 + 3.0) * 1.5) + 1.0;
  return keep < kSms / 8 && ctas > kSms - int64_t(keep) ? int(keep) : 0;
}

// Trees (many short runs of rows, each over keys of its own): which kernel, and how
// long the ranges. A model of three plans, in microseconds, of which the least is
// taken; "units" are 64 keys of a tile of 64 rows, "tiles" whole key tiles of 256.
//   * everything on 64-row tiles in one launch: 7 + 2.4 per unit and SM's two CTAs (3.4 where some are shared), or, with
//     more items than those, 2.5 and 3.9 for each of them; a fifth more for many ranges.
//     2 trees of 8 over 300 + 60 keys (12 heads over 2): 6.7 us, 9.4 on two kernels;
//   * everything on the tcgen05 kernel in one launch: 6.5 of start and end per item and 1 per
//     tile (1.75 with more than 128 rows; 0.8 of that at 64 elements), in the ranges that end
//     soonest, or the bytes at 6.3 TB/s. One tree of 25 over 50000 keys of 32 heads: 124 us,
//     214 on 16-row tiles; 37 trees of up to 13 over 777 + 500 keys in pages of 24: 18, 21 on
//     64-row tiles;
//   * up to 16 rows of a sequence: own keys on 16-row tiles, at about 5.5 TB/s (up to
//     32, at 2.7 to 3.8, where two tiles read the same keys), and shared ones on the tcgen05
//     kernel beside them: 8 sequences x 32 heads x 16 nodes over 500 + 300 keys 22.3 us, 24.4
//     on 64-row tiles. (64 sequences x 8 heads x 24 rows over 2000 keys: 107 us on 16-row
//     tiles, 89 on the tcgen05 kernel, which is taken.)
// Over 192 shapes drawn at random the choice of the kernel costs 1% against the best
// of them; with its ranges the plan's time is 2% below the best of the kernels with 1, 2, 4,
// 8, 16, 48 and 128 ranges tried for each, and at worst 1.45 times it: 8 trees of nearly
// equal lengths of 23162 keys, 65 us, 45 in 4 ranges, where lengths are taken for uneven.
// Sequences hold some 80% of the longest one's keys on average.
struct TreePlan {
  int prefix_rows, suffix_rows;
  int64_t per;  // keys of a range, in half key tiles (tcgen05) or units (64 rows); 0: as for other calls
};
TreePlan plan_tree(const nf4_prefix_attention_args& a, int64_t suffix_max, int64_t tile_keys) {
  const double kFull = 0.8, kItem = 6.5, kBytes = 6.3e6;
  const double heads = double(a.k_heads);
  const int64_t group = a.q_heads / a.k_heads, rows = a.tokens * group;
  const int64_t each = a.batch > 0 ? (rows + a.batch - 1) / a.batch : 0;  // of a sequence
  auto tiles = [](int64_t n, int64_t of) { return (n + of - 1) / of; };
  const double own_bytes = double(a.batch * suffix_max) * heads * double(a.head_dim) * 4.0 * kFull;
  const double bytes = own_bytes + double(a.prefix_len) * heads * double(a.head_dim) * 4.0;

  // 256 rows. The ranges that end soonest: shared items, all alike, in rounds (16 sequences and heads over 47458 keys
  // took 77 us in 9 ranges, one round, 111 in 10), then own ones on the SMs that the last round leaves and behind it.
  // Those are counted too, for a few items too many are a round more (6 sequences x 6 heads of 96 over 28842 keys: 4
  // ranges, 144 items, 95 us, 5 ranges 147): a third as if sequences were all as long as the longest, the rest with
  // lengths spread evenly from 60% of it up, where a range behind a sequence's end costs nothing (37 sequences over 500
  // keys in ranges of 480: 17.8 us, in one range 20.8).
  const double own_items = double(a.batch * tiles(each, 256)) * heads, shared_items = double(tiles(rows, 256)) * heads;
  const int64_t own_tiles = tiles(suffix_max, tile_keys), shared_tiles = tiles(a.prefix_len, tile_keys);
  const double narrow = a.head_dim <= 64 ? 0.8 : 1.0;
  const double own_tile = (each > 128 ? 1.75 : 1.0) * narrow, shared_tile = (rows > 128 ? 1.75 : 1.0) * narrow;
  const double own_work = own_items * double(own_tiles) * kFull * own_tile;
  const int64_t longest = own_tiles > shared_tiles ? own_tiles : shared_tiles;
  double best = 0.0;
  int64_t best_per = 0;
  for (int64_t parts = 1; parts <= kMaxRanges && parts <= longest; parts += parts / 16 + 1) {
    const int64_t per = tiles(longest, parts);
    const int64_t s = tiles(shared_tiles, per), o = tiles(own_tiles, per);
    // ranges of a sequence that hold keys, on average: `all` that every sequence reaches, and of the others the part
    // (1 - start / longest) / 0.4 of sequences; one sequence is the longest
    const double spread_of = 2.0 * (1.0 - kFull) * double(own_tiles);
    const int64_t reach = int64_t((double(own_tiles) - spread_of) / double(per)) + 1, all = o < reach ? o : reach;
    const double others =
        o > all ? double(o - all) * (double(own_tiles) - 0.5 * double(per) * double(all + o - 1)) / spread_of : 0.0;
    const double uneven = a.batch > 0 ? (double(o) + (double(all) + others) * double(a.batch - 1)) / double(a.batch) : 0.0;
    const double shared_all = shared_items * double(s);
    const double item = double(per < shared_tiles ? per : shared_tiles) * shared_tile + kItem;
    const double own_item = double(per < own_tiles ? per : own_tiles) * own_tile + kItem;
    const double whole = double(int64_t(shared_all) / kSms), rest = shared_all - whole * kSms;
    const double spare = kSms - rest, last = rest > 0.0 ? item : 0.0;
    const double beside = spare * double(int64_t(last / own_item));
    auto end = [&](double ranges, double work) {  // behind the whole rounds
      const double count = own_items * ranges;
      if (count > 0.0 && count <= spare) return last > own_item ? last : own_item;  // all at once
      if (count <= beside) return last;
      const double more = work + kItem * count - spare * last;
      const double rounds = double((int64_t(count - beside) + kSms - 1) / kSms) * own_item;
      const double spread = (more > 0.0 ? more / kSms : 0.0) + 0.5 * own_item;
      return last + (rounds < spread ? rounds : spread);
    };
    double time = whole * item + end(double(o), own_work / kFull) / 3.0 + end(uneven, own_work) * 2.0 / 3.0;
    if (time < bytes / kBytes + kItem) time = bytes / kBytes + kItem;
    // partial results and their join
    const double cost = time + double(s + o) * double(rows) * heads * 1.5e-4 + (s + o > 1 ? 2.0 : 0.0);
    if (parts == 1 || cost < best) {
      best = cost;
      best_per = 2 * per;
    }
  }
  const double est256 = 0.95 * (2.0 + best);

  // 64 rows
  const int64_t own_units = tiles(suffix_max, kUnit), shared_units = tiles(a.prefix_len, kUnit);
  const double own64 = double(a.batch * tiles(each, 64)) * heads, shared64 = double(tiles(rows, 64)) * heads;
  const double work64 = (own64 * double(own_units) * kFull + shared64 * double(shared_units)) / (2.0 * kSms);
  const double items64 = (own64 + (shared_units > 0 ? shared64 : 0.0)) / (2.0 * kSms);
  const double few64 = 7.0 + (shared_units > 0 ? 3.4 : 2.4) * work64, many64 = 3.5 + 2.5 * work64 + 3.9 * items64;
  const double est64 = (items64 > 1.0 && many64 > few64 ? many64 : few64) *
                       (own_units > 32 || shared_units > 32 ? 1.2 : 1.0);
  if (each <= 32) {
    double est16 = 8.0 + own_bytes / (each <= 16 ? 5.5e6 : 2.7e6);
    if (a.prefix_len > 0)
      est16 += 5.0 + 1.5 * shared_items * (double(shared_tiles) * (rows > 128 ? 1.75 : 1.0) + kItem) / kSms;
    if (est16 < est64 && est16 < est256)
      return {rows > 16 || a.prefix_len > 1024 ? 256 : 16, 16, 0};
  }
  if (est64 >= est256) return {256, 256, best_per};
  // as many items as there are places, of one unit or more; longer ones in about four rounds
  const int64_t units = int64_t(own64 * double(own_units) + shared64 * double(shared_units));
  const int64_t whole = tiles(units, 2 * kSms), four = units / (4 * kSms);
  // one range where that is one unit more at most: it saves the join (12 trees of 47 over up to 128 keys, 16 heads over
  // 4: 9.7 us in two ranges, 6.0 in one)
  const bool one = shared_units == 0 && whole <= 6 && own_units <= whole + 1;
  return {64, 64, one ? whole + 1 : whole <= 6 ? whole : four < 6 ? 6 : four};
}

}  // namespace

// Rows per tile, and the ranges of keys. Everything follows from the sizes
// that the host knows (never from lengths on the device).
void plan_prefix_attention(const nf4_prefix_attention_args& a, bool tree, PrefixArgs* p, size_t* bytes) {
  p->batch = int(a.batch);
  p->tokens = int(a.tokens);
  p->q_heads = int(a.q_heads);
  p->k_heads = int(a.k_heads);
  p->group = int(a.q_heads / a.k_heads);
  p->dim = int(a.head_dim);
  p->prefix_len = int(a.prefix_len);
  p->suffix_max = a.batch > 0 ? int(a.suffix_pages_width * a.page_size) : 0;
  const int64_t rows = a.tokens * p->group;  // of a key/value head
  // The shared keys go to the tcgen05 kernel however few the rows: it streams
  // them faster (one token, 12 heads over 2, 100000 keys: 26.7 us against 36 us)
  // and no slower when they are few; only where they are few and so are the
  // rows, the call is one launch fewer with everything on the other kernel.
  p->prefix_rows = rows > 16 || p->prefix_len > 1024 ? 256 : 16;
  p->suffix_rows = rows > 64 * a.batch ? 256 : rows > 32 * a.batch ? 64 : 16;
  TreePlan plan = {};
  if (tree) {
    plan = plan_tree(a, p->suffix_max, prefix_tile_keys(a.page_size));
    p->prefix_rows = plan.prefix_rows;
    p->suffix_rows = plan.suffix_rows;
  }
  p->prefix_tiles = int((rows + p->prefix_rows - 1) / p->prefix_rows);
  // the two ways of first_tile()
  const int64_t whole = rows / p->suffix_rows + a.batch;
  p->tile_per_row = rows <= whole;
  p->suffix_tiles = int(p->tile_per_row ? rows : whole);
  // as many as there are when the tokens are spread evenly (the ranges are made for these)
  const int64_t likely = a.batch > 0 ? a.batch * ((rows / a.batch + p->suffix_rows - 1) / p->suffix_rows) : 0;
  // units of both, of which the tcgen05 kernel's ranges have an even number: whole tiles
  const int64_t half = prefix_tile_keys(a.page_size) / 2;
  const int64_t pu = p->prefix_rows == 256 ? half : kUnit, su = p->suffix_rows == 256 ? half : kUnit;
  const int64_t pk = (int64_t(p->prefix_len) + pu - 1) / pu, sk = (int64_t(p->suffix_max) + su - 1) / su;
  // (whole tiles: units are 56, 60 or 64 keys)
  auto bounded = [&](int64_t per, int64_t unit) {
    const int64_t most = kMostKeys / (2 * unit) * 2;
    return per < most ? per : most;
  };
  // a tree's ranges, whole ones of these units
  auto planned = [&](int64_t units, int64_t unit, int tile_rows) {
    const int64_t least = (units + kMaxRanges - 1) / kMaxRanges, even = tile_rows == 256 ? 2 : 1;
    const int64_t per = plan.per > least ? plan.per : least;
    return bounded((per + even - 1) / even * even, unit);
  };
  if (sk > 0) {
    const int64_t per =
        plan.per > 0 ? planned(sk, su, p->suffix_rows) :
        bounded(p->suffix_rows == 256 ? tc_range(likely * p->k_heads, (sk + 1) / 2, rows * p->k_heads, kSms)
                                      : mma_range(likely * p->k_heads, sk, p->dim),
                su);
    p->suffix_chunk = int(per * su);
    p->suffix_splits = int((sk + per - 1) / per);
  }
  if (pk > 0) {
    const int64_t tiles = int64_t(p->prefix_tiles) * p->k_heads;
    int64_t per;
    if (plan.per > 0) {
      per = planned(pk, pu, p->prefix_rows);  // (no fused items: trees bring few rows)
    } else if (p->prefix_rows != 256) {
      per = mma_range(tiles, pk, p->dim);  // (at most 1024 keys)
    } else {
      const int64_t longest = (pk + 1) / 2;
      per = bounded(tc_range(tiles, longest, rows * p->k_heads, kSms), pu);
      // One range of each and many rows: the items of own keys join the shared
      // part themselves, in place of a launch that reads both parts again (8 prompts
      // of 257 to 512 tokens over 8190 + 700 keys 131 -> 125 us, 4 of 300 over 1000 +
      // 400 with 32 heads over 8 41.4 -> 35.2; 20 of 50 33.1 and 33.5). Not with the
      // few-row kernel, whose items would hold their SMs waiting for the shared part:
      // 64 sequences x 32 heads over 2048 + 190 took 56 us instead of 49; nor with two
      // ranges and more to read back: 16 prompts of 100 35 instead of 29.
      p->fused = !tree && p->suffix_splits == 1 && p->suffix_rows == 256 && pk <= per;
      if (!p->fused && p->suffix_rows != 256 && sk > 0) {
        per = beside_range(a, *p, tiles, longest, rows, per);
        const int keep = sms_for_own(*p, likely * p->k_heads * p->suffix_splits, tiles, per, pk);
        if (keep > 0) per = tc_range(tiles, longest, rows * p->k_heads, kSms - keep);
        per = bounded(per, pu);
      }
    }
    p->prefix_chunk = int(per * pu);
    p->prefix_splits = int((pk + per - 1) / per);
  }
  // A long stream of shared keys that one tile of rows reads leaves L2 first, and
  // leaves partial results, page tables and code there: 12 heads of 16 tokens over
  // 131071 keys 35.4 -> 32.0 us. A short one stays, for whoever reads it next: 32
  // sequences over 8192 keys 13.7 us, 14.1 where it leaves first.
  p->stream = p->prefix_tiles == 1 && p->prefix_len * a.k_heads * a.head_dim * 4 > kStreamBytes;
  if (pk == 0) p->fused = p->suffix_splits == 1;  // own keys in one range are all there is
  if (rows == 0) p->prefix_splits = p->suffix_splits = p->fused = 0;
  p->splits = p->prefix_splits + (p->fused ? 0 : p->suffix_splits);
  const int64_t all = a.tokens * a.q_heads;
  p->direct = p->prefix_splits == 1 && p->suffix_splits == 0;
  *bytes = p->splits > 0 && !p->direct ? size_t(all) * size_t(p->splits) * (size_t(a.head_dim) * 4 + 8) : 0;
}

size_t prefix_attention_workspace_bytes(const nf4_prefix_attention_args& a, bool tree) {
  PrefixArgs p = {};
  size_t bytes = 0;
  plan_prefix_attention(a, tree, &p, &bytes);
  return bytes;
}

cudaError_t launch_prefix_attention(const nf4_prefix_attention_args& a, const nf4_tree_attention_args* tree,
                                    void* workspace, size_t workspace_bytes, bool* enough, cudaStream_t stream) {
  PrefixArgs p = {};
  size_t bytes = 0;
  plan_prefix_attention(a, tree != nullptr, &p, &bytes);
  *enough =
      bytes == 0 || (workspace && workspace_bytes >= bytes && (reinterpret_cast<uintptr_t>(workspace) & 15u) == 0);
  if (!*enough) return cudaSuccess;
  p.q = static_cast<const char*>(a.q);
  p.out = static_cast<char*>(a.out);
  p.k = static_cast<const char*>(a.k_cache);
  p.v = static_cast<const char*>(a.v_cache);
  p.q_ts = a.q_token_stride * 2;
  p.q_hs = a.q_head_stride * 2;
  p.out_ts = a.out_token_stride * 2;
  p.out_hs = a.out_head_stride * 2;
  p.k_ps = a.k_page_stride * 2;
  p.k_ss = a.k_slot_stride * 2;
  p.k_hs = a.k_head_stride * 2;
  p.v_ps = a.v_page_stride * 2;
  p.v_ss = a.v_slot_stride * 2;
  p.v_hs = a.v_head_stride * 2;
  p.lse = a.lse;
  p.prefix_pages = a.prefix_pages;
  p.suffix_pages = a.suffix_pages;
  p.suffix_lens = a.suffix_lens;
  p.cu_q = a.cu_q;
  if (tree) {
    p.tree = tree->tree_mask;
    p.tree_stride = tree->tree_mask_stride;
    p.tree_words = int(tree->tree_words);
  }
  p.suffix_pages_stride = a.suffix_pages_stride;
  p.page_size = int(a.page_size);
  p.page_shift = -1;
  for (int s = 0; s <= 16; ++s)
    if (p.page_size == 1 << s) p.page_shift = s;
  p.num_pages = int(a.num_pages);
  p.scale_log2 = float(a.scale * 1.4426950408889634);
  if (bytes > 0) {
    p.part = static_cast<float*>(workspace);
    p.ml = reinterpret_cast<float2*>(p.part + int64_t(p.splits) * a.tokens * a.q_heads * a.head_dim);
  }
  return a.dtype == NF4_BF16 ? launch_typed<Bf16>(p, stream) : launch_typed<Fp16>(p, stream);
}

cudaError_t prefix_flags(unsigned int** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_prefix_flags);
}

}  // namespace nf4
