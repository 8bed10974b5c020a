// nf4_rope.cu -- rotary position tables, the per-head norm and rotation of
// queries and keys, and the append of keys and values to a paged cache.
//
// A head row x becomes u = x * rsqrt(mean(x^2) + eps) * w (or u = x without a
// weight), then every pair (a, b) of its rotated part becomes
// (a cos - b sin, b cos + a sin). Every element is read once and written
// once, about seven operations each: bound by memory, and for a few tokens by
// the latency of one launch and three dependent loads (position, table row,
// result).
//
// Split: a row is cut into units of two 16-byte chunks that hold whole pairs
// (one of each half of the rotated part, in either layout, and one of each half
// of the rest), so that neighbouring lanes hold neighbouring chunks; with two
// neighbouring chunks per lane for the interleaved layout, half a sector to
// each instruction, the prompt below took 57 us. One lane per unit: a row's
// norm is a butterfly over the 2^k lanes that share it, both elements of a pair
// are in one lane's registers, and an output may be its input. A warp
// takes one token: the weights times the token's cosines and sines are formed
// once and serve all the heads that the warp walks over (two multiplications
// and additions per element, packed two to an instruction), and the next four
// rows are under way in shared memory, each lane reading back only what it
// brought. 8192 tokens x 64 heads of 128 in bf16 take 44.7 us (6.1 TB/s, 91% of
// measured copy bandwidth; interleaved 44.2), an append of 8000 x 96 heads 62.4
// us (95%).
#include <math.h>

#include <initializer_list>

#include "nf4_attn.cuh"

namespace nf4 {
namespace {

__device__ unsigned int g_rope_flags = 0;  // kFlagBadIndex

constexpr int kMaxFreqs = 256;

struct TableArgs {
  float2* cs;
  int64_t positions;
  int pairs;
  float magnitude;
  double freq[kMaxFreqs];
};

// One (cos, sin) per thread. The angle is reduced in binary64 (2 pi in two
// parts), its binary32 head goes through sincosf and the rest r enters to
// first order: cos(h + r) = cos h - r sin h, |r| < 2e-7.
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ TableArgs a) {
  pdl_allow_dependents();
  pdl_wait_prior_grid();
  const int64_t total = a.positions * a.pairs;
  for (int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x; e < total; e += int64_t(gridDim.x) * 256) {
    const int64_t p = e / a.pairs;
    const int i = int(e - p * a.pairs);
    const double angle = double(p) * a.freq[i];
    const double turns = rint(angle * 0.15915494309189533577);
    const double red = fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586477, angle));
    const float h = float(red);
    const float r = float(red - double(h));
    float s, c;
    sincosf(h, &s, &c);
    const float cc = fmaf(-r, s, c), ss = fmaf(r, c, s);
    a.cs[e] = make_float2(a.magnitude * cc, a.magnitude * ss);
  }
}

struct RowSet {
  const char* in;
  char* out;
  int64_t in_ts, in_hs, out_ts, out_hs;  // elements; of a cache only out_hs is used
  int heads;
};

struct RopeArgs {
  RowSet q, k, v;             // v.heads 0 without a cache
  const void* qw;
  const void* kw;
  const int64_t* positions;
  const float2* cs;
  const int64_t* slots;       // null: k goes to k.out by token
  int64_t max_positions;
  int64_t k_page_stride, k_slot_stride, v_page_stride, v_slot_stride;
  int64_t num_slots;
  int page_size;
  int dim, rot, interleaved;
  float eps, inv_dim;
  int tokens;
  int lane_bits;              // log2 of the lanes per row
  int gq, gk, gv;             // groups of 32 >> lane_bits rows
  int per_warp, parts;        // groups a warp walks over; warps per token
};

// Two chunks of P elements as P pairs (a_i, b_i) of binary32 and back: in the
// half layout a comes from the first chunk and b from the second, in the
// interleaved layout they alternate.
template <int kBytes>
struct ChunkOf;
template <>
struct ChunkOf<16> {
  using type = uint4;
  static __device__ __forceinline__ void get(const uint4& x, uint32_t* w) {
    w[0] = x.x;
    w[1] = x.y;
    w[2] = x.z;
    w[3] = x.w;
  }
  static __device__ __forceinline__ uint4 put(const uint32_t* w) { return make_uint4(w[0], w[1], w[2], w[3]); }
  static __device__ __forceinline__ void copy(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  }
};
template <>
struct ChunkOf<8> {
  using type = uint2;
  static __device__ __forceinline__ void get(const uint2& x, uint32_t* w) {
    w[0] = x.x;
    w[1] = x.y;
  }
  static __device__ __forceinline__ uint2 put(const uint32_t* w) { return make_uint2(w[0], w[1]); }
  static __device__ __forceinline__ void copy(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
  }
};

template <typename H, int kBytes>
struct Elem : ChunkOf<kBytes> {
  static constexpr int kSize = 2, kPer = kBytes / 2;
  using Chunk = typename ChunkOf<kBytes>::type;
  template <bool kInterleaved>
  static __device__ __forceinline__ void up(const Chunk& x0, const Chunk& x1, float (&a)[kPer], float (&b)[kPer]) {
    uint32_t w[kPer];
    Elem::get(x0, w);
    Elem::get(x1, w + kPer / 2);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float2 p = H::up2(w[i]);
      if (kInterleaved) {
        a[i] = p.x;
        b[i] = p.y;
      } else {
        float* to = i < kPer / 2 ? a + 2 * i : b + 2 * i - kPer;
        to[0] = p.x;
        to[1] = p.y;
      }
    }
  }
  template <bool kInterleaved>
  static __device__ __forceinline__ void down(const float (&a)[kPer], const float (&b)[kPer], Chunk& x0, Chunk& x1) {
    uint32_t w[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float* from = i < kPer / 2 ? a + 2 * i : b + 2 * i - kPer;
      w[i] = kInterleaved ? H::down2(a[i], b[i]) : H::down2(from[0], from[1]);
    }
    x0 = Elem::put(w);
    x1 = Elem::put(w + kPer / 2);
  }
  static __device__ __forceinline__ float load(const char* p) {
    return H::up2(*reinterpret_cast<const uint16_t*>(p)).x;
  }
  static __device__ __forceinline__ void store(char* p, float v) {
    *reinterpret_cast<uint16_t*>(p) = uint16_t(H::down2(v, v) & 0xffffu);
  }
};
template <>
struct Elem<float, 16> : ChunkOf<16> {
  static constexpr int kSize = 4, kPer = 4;
  using Chunk = uint4;
  template <bool kInterleaved>
  static __device__ __forceinline__ void up(const uint4& x0, const uint4& x1, float (&a)[4], float (&b)[4]) {
    const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = __uint_as_float(w[kInterleaved ? 2 * i : i]);
      b[i] = __uint_as_float(w[kInterleaved ? 2 * i + 1 : i + 4]);
    }
  }
  template <bool kInterleaved>
  static __device__ __forceinline__ void down(const float (&a)[4], const float (&b)[4], uint4& x0, uint4& x1) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[kInterleaved ? 2 * i : i] = __float_as_uint(a[i]);
      w[kInterleaved ? 2 * i + 1 : i + 4] = __float_as_uint(b[i]);
    }
    x0 = put(w);
    x1 = put(w + 4);
  }
  static __device__ __forceinline__ float load(const char* p) { return *reinterpret_cast<const float*>(p); }
  static __device__ __forceinline__ void store(char* p, float v) { *reinterpret_cast<float*>(p) = v; }
};

// Two binary32 operations in one instruction, each rounded to nearest even.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where a token's key and value go: the first byte of (slot, head 0) of each
// cache. False: nowhere (a negative slot, or one past the cache, which is
// reported).
__device__ __forceinline__ bool slot_base(const RopeArgs& a, int64_t slot, int size, char** k, char** v) {
  if (slot < 0) return false;
  if (slot >= a.num_slots) {
    atomicOr(&g_rope_flags, kFlagBadIndex);
    return false;
  }
  int64_t page, off;
  if (slot <= 0xffffffffll) {
    page = uint32_t(slot) / uint32_t(a.page_size);
    off = uint32_t(slot) % uint32_t(a.page_size);
  } else {
    page = slot / a.page_size;
    off = slot % a.page_size;
  }
  *k = a.k.out + (page * a.k_page_stride + off * a.k_slot_stride) * size;
  *v = a.v.out + (page * a.v_page_stride + off * a.v_slot_stride) * size;
  return true;
}

constexpr int kRopeThreads = 128;
// Blocks of four warps, five on an SM (96 registers; six where a chunk has four
// elements and 80 do), four rows under way per warp through shared memory. 8192
// tokens x 64 heads of 128 in bf16, us: rows under way in registers, the next one
// only, 51.6, four 60.3 (too few warps); through shared memory two 48.0, four
// 45.2, six 46.1 (and with six blocks 46.0, with eight, whose 64 registers spill,
// 51.4).
template <typename E>
constexpr int kRopeBlocks = E::kPer == 8 ? 5 : 6;
constexpr int kInFlight = 4;
constexpr int kPerWarp = 8;  // row groups that one warp walks over at least, where there are many tokens (4: 54 us)

template <typename E, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks<E>) rope_rows_kernel(const __grid_constant__ RopeArgs a) {
  using Chunk = typename E::Chunk;
  constexpr int P = E::kPer;  // elements per chunk = pairs per unit
  constexpr int kBytes = sizeof(Chunk);
  pdl_allow_dependents();
  const int64_t w = int64_t(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int t = int(w / a.parts);
  const int part = int(w - int64_t(t) * a.parts);
  pdl_wait_prior_grid();
  if (t >= a.tokens) return;
  const int unit = lane & ((1 << a.lane_bits) - 1);
  const int sub = lane >> a.lane_bits;
  const int rows = 32 >> a.lane_bits;
  const int rot_units = a.rot / (2 * P);
  const bool active = unit < a.dim / (2 * P);
  const bool turned = unit < rot_units;
  // byte offset of the unit's first chunk, and from there to the second (a lane
  // past the row's end takes the row's first chunk, and stores nothing)
  const int c0 = !active ? 0 : kBytes * (turned ? unit : unit + rot_units);
  const int c1 = kBytes * (turned ? rot_units : a.dim / (2 * P) - rot_units);
  // this warp's row groups: q's, then k's, then v's
  const int g = part * a.per_warp;
  const int g_end = min(g + a.per_warp, a.gq + a.gk + a.gv);

  // The groups of one kind (0 q, 1 k, 2 v) that this warp has: [from, to) of
  // the kind's own. Lanes without a row of their own read the last head's.
  struct Part {
    const char* src;   // this lane's first chunk of head 0
    int from, to;
    int last;          // the last head
    int head_step;     // bytes
  };
  auto part_of = [&](int kind) {
    const RowSet& r = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const int first = kind == 0 ? 0 : kind == 1 ? a.gq : a.gq + a.gk;
    const int n = kind == 0 ? a.gq : kind == 1 ? a.gk : a.gv;
    return Part{r.in + int64_t(t) * r.in_ts * E::kSize + c0, max(g - first, 0),
                min(g_end - first, n), r.heads - 1, int(r.in_hs) * E::kSize};
  };
  // Rows under way, in shared memory; every lane reads back only what it brought.
  __shared__ __align__(16) Chunk ring[kRopeThreads / 32][kInFlight][2][32];
  auto& mine = ring[threadIdx.x >> 5];
  auto load = [&](const Part& s, int gi) {
    if (gi < s.to) {
      const char* p = s.src + min(gi * rows + sub, s.last) * s.head_step;
      const int slot = (gi - s.from) % kInFlight;
      E::copy(smem_u32(&mine[slot][0][lane]), p);
      E::copy(smem_u32(&mine[slot][1][lane]), p + c1);
    }
    copy_commit();
  };
  // the first rows are on their way before the position and its table row are asked for
  const int kind0 = g < a.gq ? 0 : g < a.gq + a.gk ? 1 : 2;
  {
    const Part s = part_of(kind0);
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) load(s, s.from + u);
  }

  const int64_t slot = a.slots ? a.slots[t] : 0;
  const int64_t pos = a.rot > 0 ? a.positions[t] : 0;
  const bool good = a.rot == 0 || (pos >= 0 && pos < a.max_positions);
  if (!good && lane == 0) atomicOr(&g_rope_flags, kFlagBadIndex);
  char *kdst = nullptr, *vdst = nullptr;
  bool stored = true;
  if (a.slots) stored = slot_base(a, slot, E::kSize, &kdst, &vdst);

  // One kind of rows at a time: `kind` is the same for the whole warp.
  for (int kind = kind0; kind < 3; ++kind) {
    const Part s = part_of(kind);
    if (s.from >= s.to || (kind > 0 && !stored)) continue;
    if (kind != kind0) {
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) load(s, s.from + u);
    }
    char* dst = kind == 0   ? a.q.out + int64_t(t) * a.q.out_ts * E::kSize
                : !a.slots  ? a.k.out + int64_t(t) * a.k.out_ts * E::kSize
                : kind == 1 ? kdst
                            : vdst;
    dst += c0;
    const int out_step = int(kind == 0 ? a.q.out_hs : kind == 1 ? a.k.out_hs : a.v.out_hs) * E::kSize;

    // weight times cosine and sine: a' = a (wa c) - b (wb s), b' = b (wb c) + a (wa s)
    const char* wt = reinterpret_cast<const char*>(kind == 0 ? a.qw : kind == 1 ? a.kw : nullptr);
    uint64_t ac[P / 2], bs[P / 2], bc[P / 2], as[P / 2];
    if (kind < 2) {
      float wa[P], wb[P];
      if (wt) {
        E::template up<kInterleaved>(*reinterpret_cast<const Chunk*>(wt + c0),
                                     *reinterpret_cast<const Chunk*>(wt + c0 + c1), wa, wb);
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) wa[i] = wb[i] = 1.0f;
      }
      // a position out of the table: NaN in every element, turned or not
      // (interleaved, half of the unit's pairs are in each chunk)
      const float4* src = reinterpret_cast<const float4*>(a.cs + (good ? pos : 0) * (a.rot / 2)) +
                          unit * (kInterleaved ? P / 4 : P / 2);
      const int far = kInterleaved ? rot_units * (P / 4) - P / 4 : 0;
      const float none = good ? 1.0f : __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int i = 0; i < P / 2; ++i) {
        float4 f = make_float4(none, 0.0f, none, 0.0f);
        if (turned && good) f = src[i < P / 4 ? i : i + far];
        const uint64_t c = pack2(f.x, f.z);
        ac[i] = mul2(pack2(wa[2 * i], wa[2 * i + 1]), c);
        bc[i] = mul2(pack2(wb[2 * i], wb[2 * i + 1]), c);
        as[i] = mul2(pack2(wa[2 * i], wa[2 * i + 1]), pack2(f.y, f.w));
        bs[i] = mul2(pack2(wb[2 * i], wb[2 * i + 1]), pack2(-f.y, -f.w));
      }
    }

    for (int gi = s.from; gi < s.to; ++gi) {
      copy_wait<kInFlight - 1>();
      const int slot = (gi - s.from) % kInFlight;
      Chunk y0 = mine[slot][0][lane], y1 = mine[slot][1][lane];
      if (kind < 2) {
        float fa[P], fb[P];
        E::template up<kInterleaved>(y0, y1, fa, fb);
        uint64_t pa[P / 2], pb[P / 2];
#pragma unroll
        for (int i = 0; i < P / 2; ++i) {
          pa[i] = pack2(fa[2 * i], fa[2 * i + 1]);
          pb[i] = pack2(fb[2 * i], fb[2 * i + 1]);
        }
        float inv = 1.0f;
        if (wt) {
          uint64_t sq = mul2(pa[0], pa[0]);
#pragma unroll
          for (int i = 1; i < P / 2; ++i) sq = fma2(pa[i], pa[i], sq);
#pragma unroll
          for (int i = 0; i < P / 2; ++i) sq = fma2(pb[i], pb[i], sq);
          const float2 two = unpack2(sq);
          float ss = active ? two.x + two.y : 0.0f;
          for (int m = 1 << a.lane_bits >> 1; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
          inv = rsqrtf(fmaf(ss, a.inv_dim, a.eps));
        }
        const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
        for (int i = 0; i < P / 2; ++i) {
          uint64_t ya = mul2(pa[i], ac[i]), yb = mul2(pb[i], bc[i]);
          if (turned) {
            ya = fma2(pb[i], bs[i], ya);
            yb = fma2(pa[i], as[i], yb);
          }
          if (wt) {
            ya = mul2(ya, inv2);
            yb = mul2(yb, inv2);
          }
          const float2 u2 = unpack2(ya), v2 = unpack2(yb);
          fa[2 * i] = u2.x;
          fa[2 * i + 1] = u2.y;
          fb[2 * i] = v2.x;
          fb[2 * i + 1] = v2.y;
        }
        E::template down<kInterleaved>(fa, fb, y0, y1);
      }
      const int h = gi * rows + sub;
      if (active && h <= s.last) {
        char* p = dst + h * out_step;
        *reinterpret_cast<Chunk*>(p) = y0;
        *reinterpret_cast<Chunk*>(p + c1) = y1;
      }
      load(s, gi + kInFlight);
    }
    copy_wait<0>();
  }
  copy_wait<0>();  // rows that go nowhere were asked for too: the block's shared memory is not given back under them
}

// Any head size, alignment and rotated part: one warp per row, a lane per
// pair, then the rest of the row.
template <typename E>
__global__ void __launch_bounds__(kRopeThreads) rope_rows_any_kernel(const __grid_constant__ RopeArgs a) {
  pdl_allow_dependents();
  const int heads = a.q.heads + a.k.heads + a.v.heads;
  const int64_t w = int64_t(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int t = int(w / heads);
  pdl_wait_prior_grid();
  if (t >= a.tokens) return;
  int h = int(w - int64_t(t) * heads);
  const int kind = h < a.q.heads ? 0 : h < a.q.heads + a.k.heads ? 1 : 2;
  h -= kind == 0 ? 0 : kind == 1 ? a.q.heads : a.q.heads + a.k.heads;
  const RowSet& r = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
  const char* in = r.in + (int64_t(t) * r.in_ts + int64_t(h) * r.in_hs) * E::kSize;
  char* out;
  if (kind > 0 && a.slots) {
    char *kd = nullptr, *vd = nullptr;
    if (!slot_base(a, a.slots[t], E::kSize, &kd, &vd)) return;
    out = (kind == 1 ? kd : vd) + int64_t(h) * r.out_hs * E::kSize;
  } else {
    out = r.out + (int64_t(t) * r.out_ts + int64_t(h) * r.out_hs) * E::kSize;
  }
  if (kind == 2) {
    for (int i = lane; i < a.dim; i += 32) E::store(out + i * E::kSize, E::load(in + i * E::kSize));
    return;
  }
  const char* wt = reinterpret_cast<const char*>(kind == 0 ? a.qw : a.kw);
  float inv = 1.0f;
  if (wt) {
    float ss = 0.0f;
    for (int i = lane; i < a.dim; i += 32) {
      const float f = E::load(in + i * E::kSize);
      ss = fmaf(f, f, ss);
    }
    for (int m = 16; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    inv = rsqrtf(fmaf(ss, a.inv_dim, a.eps));
  }
  auto value = [&](int i) {
    float f = E::load(in + i * E::kSize);
    if (wt) f = f * inv * E::load(wt + i * E::kSize);
    return f;
  };
  bool good = true;
  const float2* cs = nullptr;
  if (a.rot > 0) {
    const int64_t pos = a.positions[t];
    good = pos >= 0 && pos < a.max_positions;
    if (!good && lane == 0) atomicOr(&g_rope_flags, kFlagBadIndex);
    cs = a.cs + (good ? pos : 0) * (a.rot / 2);
  }
  const float nan = __uint_as_float(0x7fc00000u);
  for (int i = lane; i < a.rot / 2; i += 32) {
    const int i0 = a.interleaved ? 2 * i : i, i1 = a.interleaved ? 2 * i + 1 : i + a.rot / 2;
    const float p = value(i0), b = value(i1);
    const float2 f = good ? cs[i] : make_float2(nan, nan);
    E::store(out + i0 * E::kSize, p * f.x - b * f.y);
    E::store(out + i1 * E::kSize, b * f.x + p * f.y);
  }
  for (int i = a.rot + lane; i < a.dim; i += 32) E::store(out + i * E::kSize, good ? value(i) : nan);
}

// Whether chunks of E hold every row: whole units, and all rows, weights and
// strides on a chunk's boundary.
template <typename E>
bool in_chunks(const RopeArgs& a) {
  constexpr int P = E::kPer;
  auto aligned = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % sizeof(typename E::Chunk) == 0; };
  // offsets of heads are of 32 bits (64 took up to 3% longer: instructions count here)
  auto near = [](int64_t heads, int64_t step) {
    const int64_t most = ((int64_t(1) << 31) - 1) / (E::kSize * heads);
    return -most <= step && step <= most;
  };
  auto fits = [&](const RowSet& r) {
    return r.heads == 0 ||
           (near(r.heads, r.in_hs) && near(r.heads, r.out_hs) && aligned(r.in) && aligned(r.out) &&
            r.in_ts % P == 0 && r.in_hs % P == 0 && r.out_ts % P == 0 && r.out_hs % P == 0);
  };
  return a.dim % (2 * P) == 0 && a.rot % (2 * P) == 0 && a.dim / (2 * P) <= 32 && fits(a.q) && fits(a.k) &&
         fits(a.v) && aligned(a.qw) && aligned(a.kw) && reinterpret_cast<uintptr_t>(a.cs) % 16 == 0 &&
         a.k_page_stride % P == 0 && a.k_slot_stride % P == 0 && a.v_page_stride % P == 0 &&
         a.v_slot_stride % P == 0;
}

template <typename E>
cudaError_t launch_chunks(RopeArgs& a, cudaStream_t stream) {
  const int P = E::kPer;
  const int per_block = kRopeThreads / 32;
  a.lane_bits = 0;
  while ((1 << a.lane_bits) < a.dim / (2 * P)) ++a.lane_bits;
  const int rows = 32 >> a.lane_bits;
  a.gq = (a.q.heads + rows - 1) / rows;
  a.gk = (a.k.heads + rows - 1) / rows;
  a.gv = (a.v.heads + rows - 1) / rows;
  // Warps per token. Few tokens: as many as the SMs hold at a time, one per
  // group at most (64 heads of 128 in bf16, us: 400 tokens 4.9, twice as many 6.1,
  // half as many 6.6; 1000 tokens 7.2, 8.8 and 8.0), and two rather than one
  // that would leave a third of the places empty (1700 tokens x 40 heads 9.1, one
  // 10.1). Many: one for every 8 to 15 groups, since a warp's table row and
  // weights serve all of them (8192 tokens x 40 heads, ten groups: 30.6, two
  // warps of five 35.8).
  const int groups = a.gq + a.gk + a.gv;
  const int64_t resident = 152 * kRopeBlocks<E> * (kRopeThreads / 32);
  const int64_t least = groups < 2 * kPerWarp ? 1 : groups / kPerWarp;
  const int64_t fit = 10 * int64_t(a.tokens) < 7 * resident && a.tokens * 2 > resident ? 2 : resident / a.tokens;
  a.parts = int(fit < least ? least : fit < groups ? fit : groups);
  a.per_warp = (groups + a.parts - 1) / a.parts;
  const int64_t blocks = (int64_t(a.tokens) * a.parts + per_block - 1) / per_block;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return launch_k(a.interleaved ? rope_rows_kernel<E, true> : rope_rows_kernel<E, false>, dim3(unsigned(blocks)),
                  dim3(kRopeThreads), 0, stream, a);
}

template <typename E>
cudaError_t launch_any(RopeArgs& a, cudaStream_t stream) {
  const int per_block = kRopeThreads / 32;
  const int64_t warps = int64_t(a.tokens) * (a.q.heads + a.k.heads + a.v.heads);
  const int64_t blocks = (warps + per_block - 1) / per_block;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return launch_k(rope_rows_any_kernel<E>, dim3(unsigned(blocks)), dim3(kRopeThreads), 0, stream, a);
}

// 16-byte chunks; 8-byte chunks where 16-byte ones do not hold whole units (a
// rotated part of 40 elements, say: 8000 tokens x 12 heads of 80 in bf16 take
// 15.2 us, element by element 30.3), which binary32 leaves to its four-element
// chunks of 16 bytes; elements otherwise.
template <typename H>
cudaError_t launch_half(RopeArgs& a, cudaStream_t stream) {
  if (in_chunks<Elem<H, 16>>(a)) return launch_chunks<Elem<H, 16>>(a, stream);
  if (in_chunks<Elem<H, 8>>(a)) return launch_chunks<Elem<H, 8>>(a, stream);
  return launch_any<Elem<H, 16>>(a, stream);
}
cudaError_t launch_float(RopeArgs& a, cudaStream_t stream) {
  if (in_chunks<Elem<float, 16>>(a)) return launch_chunks<Elem<float, 16>>(a, stream);
  return launch_any<Elem<float, 16>>(a, stream);
}

}  // namespace

cudaError_t rope_flags(unsigned int** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_rope_flags);
}

cudaError_t launch_rope_table(const nf4_rope_table_args& a, cudaStream_t stream) {
  TableArgs t;
  t.cs = reinterpret_cast<float2*>(a.cos_sin);
  t.positions = a.positions;
  t.pairs = int(a.rot_dim / 2);
  t.magnitude = float(a.magnitude);
  const double two_pi = 6.283185307179586477;
  auto corner = [&](double turns) {
    return double(a.rot_dim) * log(a.original_positions / (two_pi * turns)) / (2.0 * log(a.base));
  };
  double lo = 0.0, hi = 0.0;
  if (a.scaling == NF4_ROPE_RAMP) {
    lo = fmax(floor(corner(a.high)), 0.0);
    hi = fmin(ceil(corner(a.low)), double(a.rot_dim - 1));
  }
  for (int i = 0; i < t.pairs; ++i) {
    const double f = pow(a.base, -2.0 * i / double(a.rot_dim));
    double g = f;
    if (a.scaling == NF4_ROPE_LINEAR) {
      g = f / a.factor;
    } else if (a.scaling == NF4_ROPE_BANDS) {
      const double r = a.original_positions * f / two_pi;
      const double s = fmin(fmax((r - a.low) / (a.high - a.low), 0.0), 1.0);
      g = (1.0 - s) * f / a.factor + s * f;
    } else if (a.scaling == NF4_ROPE_RAMP) {
      const double s = fmin(fmax((i - lo) / fmax(hi - lo, 1e-3), 0.0), 1.0);
      g = (1.0 - s) * f + s * f / a.factor;
    }
    t.freq[i] = g;
  }
  const int64_t blocks = (a.positions * t.pairs + 255) / 256;
  const int64_t most = 152 * 32;
  return launch_k(rope_table_kernel, dim3(unsigned(blocks < most ? blocks : most)), dim3(256), 0, stream, t);
}

cudaError_t launch_qk_rope(const nf4_qk_norm_rope_args& q, const nf4_kv_append_args* c,
                           cudaStream_t stream) {
  RopeArgs a = {};
  a.q = RowSet{static_cast<const char*>(q.q), static_cast<char*>(q.q_out), q.q_token_stride, q.q_head_stride,
               q.q_out_token_stride, q.q_out_head_stride, int(q.q_heads)};
  a.k = RowSet{static_cast<const char*>(q.k), static_cast<char*>(q.k_out), q.k_token_stride, q.k_head_stride,
               q.k_out_token_stride, q.k_out_head_stride, int(q.k_heads)};
  a.page_size = 1;
  if (c) {
    a.k.out = static_cast<char*>(c->k_cache);
    a.k.out_ts = 0;
    a.k.out_hs = c->k_head_stride;
    a.v = RowSet{static_cast<const char*>(c->v), static_cast<char*>(c->v_cache), c->v_token_stride,
                 c->v_head_stride, 0, c->v_cache_head_stride, int(q.k_heads)};
    a.slots = c->slots;
    a.k_page_stride = c->k_page_stride;
    a.k_slot_stride = c->k_slot_stride;
    a.v_page_stride = c->v_page_stride;
    a.v_slot_stride = c->v_slot_stride;
    a.page_size = int(c->page_size);
    a.num_slots = c->num_pages * c->page_size;
  }
  // the stride of a dimension of one is never used
  for (RowSet* r : {&a.q, &a.k, &a.v}) {
    if (q.tokens == 1) r->in_ts = r->out_ts = 0;
    if (r->heads == 1) r->in_hs = r->out_hs = 0;
  }
  if (c && c->num_pages == 1) a.k_page_stride = a.v_page_stride = 0;
  if (c && c->page_size == 1) a.k_slot_stride = a.v_slot_stride = 0;
  a.qw = q.q_heads > 0 ? q.q_weight : nullptr;
  a.kw = q.k_heads > 0 ? q.k_weight : nullptr;
  a.positions = q.positions;
  a.cs = q.rot_dim > 0 ? reinterpret_cast<const float2*>(q.cos_sin) : nullptr;
  a.max_positions = q.max_positions;
  a.dim = int(q.head_dim);
  a.rot = int(q.rot_dim);
  a.interleaved = q.interleaved != 0;
  a.eps = float(q.eps);
  a.inv_dim = 1.0f / float(q.head_dim);
  a.tokens = int(q.tokens);
  switch (q.dtype) {
    case NF4_BF16: return launch_half<Bf16>(a, stream);
    case NF4_FP16: return launch_half<Fp16>(a, stream);
    default: return launch_float(a, stream);
  }
}

}  // namespace nf4
