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
// (the chunks at i and i + rot_dim / 2 of the half layout, two neighbouring
// chunks otherwise), one lane per unit, so that a row's norm is a butterfly
// over the 2^k lanes that share it and both elements of a pair are in one
// lane's registers: no shared memory, and an output may be its input. A warp
// takes one token: its table row and weights are loaded into registers once
// and serve all the heads that the warp walks over, four row groups in flight
// at a time.
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

template <typename T>
struct Elem;  // a 16-byte chunk as binary32 values and back
template <typename H>
struct Elem16 {
  static constexpr int kSize = 2, kPer = 8;
  static __device__ __forceinline__ void up(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = H::up2(w[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
  static __device__ __forceinline__ uint4 down(const float* f) {
    return make_uint4(H::down2(f[0], f[1]), H::down2(f[2], f[3]), H::down2(f[4], f[5]), H::down2(f[6], f[7]));
  }
  static __device__ __forceinline__ float load(const char* p) {
    return H::up2(*reinterpret_cast<const uint16_t*>(p)).x;
  }
  static __device__ __forceinline__ void store(char* p, float v) {
    *reinterpret_cast<uint16_t*>(p) = uint16_t(H::down2(v, v) & 0xffffu);
  }
};
template <>
struct Elem<Bf16> : Elem16<Bf16> {};
template <>
struct Elem<Fp16> : Elem16<Fp16> {};
template <>
struct Elem<float> {
  static constexpr int kSize = 4, kPer = 4;
  static __device__ __forceinline__ void up(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 down(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float load(const char* p) { return *reinterpret_cast<const float*>(p); }
  static __device__ __forceinline__ void store(char* p, float v) { *reinterpret_cast<float*>(p) = v; }
};

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

constexpr int kRopeThreads = 256;
constexpr int kInFlight = 4;  // row groups whose loads are issued together

template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_rows_kernel(const __grid_constant__ RopeArgs a) {
  using E = Elem<T>;
  constexpr int P = E::kPer;  // elements per chunk = pairs per unit
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
  int c0, c1;  // the unit's chunks
  if (turned && !a.interleaved) {
    c0 = unit;
    c1 = unit + rot_units;
  } else {
    c0 = 2 * unit;
    c1 = c0 + 1;
  }
  const int g0 = part * a.per_warp;
  const int g1 = min(g0 + a.per_warp, a.gq + a.gk + a.gv);

  // the row of group g that this lane works on: 0 q, 1 k, 2 v, and its head (-1: none)
  auto row_of = [&](int g, int* head) {
    const int kind = g < a.gq ? 0 : g < a.gq + a.gk ? 1 : 2;
    const int h = (g - (kind == 0 ? 0 : kind == 1 ? a.gq : a.gq + a.gk)) * rows + sub;
    const int n = kind == 0 ? a.q.heads : kind == 1 ? a.k.heads : a.v.heads;
    *head = (g < g1 && active && h < n) ? h : -1;
    return kind;
  };
  auto load = [&](int g, uint4& x0, uint4& x1) {
    int h;
    const int kind = row_of(g, &h);
    x0 = x1 = make_uint4(0u, 0u, 0u, 0u);
    if (h < 0) return;
    const RowSet& r = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const char* p = r.in + (int64_t(t) * r.in_ts + int64_t(h) * r.in_hs) * E::kSize;
    x0 = *reinterpret_cast<const uint4*>(p + c0 * 16);
    x1 = *reinterpret_cast<const uint4*>(p + c1 * 16);
  };

  uint4 x[kInFlight][2];
#pragma unroll
  for (int u = 0; u < kInFlight; ++u) load(g0 + u, x[u][0], x[u][1]);
  // the token's table row and place in the cache, and the weights
  float cosv[P], sinv[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    cosv[i] = 1.0f;
    sinv[i] = 0.0f;
  }
  if (a.rot > 0) {
    const int64_t pos = a.positions[t];
    const bool good = pos >= 0 && pos < a.max_positions;
    if (!good && lane == 0) atomicOr(&g_rope_flags, kFlagBadIndex);
    if (!good) {  // NaN in every element of the token's rows, turned or not
#pragma unroll
      for (int i = 0; i < P; ++i) cosv[i] = sinv[i] = __uint_as_float(0x7fc00000u);
    } else if (turned) {
      const float4* src = reinterpret_cast<const float4*>(a.cs + pos * (a.rot / 2) + unit * P);
#pragma unroll
      for (int i = 0; i < P / 2; ++i) {
        const float4 f = __ldg(src + i);
        cosv[2 * i] = f.x;
        sinv[2 * i] = f.y;
        cosv[2 * i + 1] = f.z;
        sinv[2 * i + 1] = f.w;
      }
    }
  }
  char *kdst = nullptr, *vdst = nullptr;
  bool stored = true;
  if (a.slots) stored = slot_base(a, a.slots[t], E::kSize, &kdst, &vdst);
  uint4 wq[2], wk[2];
  wq[0] = wq[1] = wk[0] = wk[1] = make_uint4(0u, 0u, 0u, 0u);
  if (active) {
    if (a.qw) {
      wq[0] = __ldg(reinterpret_cast<const uint4*>(a.qw) + c0);
      wq[1] = __ldg(reinterpret_cast<const uint4*>(a.qw) + c1);
    }
    if (a.kw) {
      wk[0] = __ldg(reinterpret_cast<const uint4*>(a.kw) + c0);
      wk[1] = __ldg(reinterpret_cast<const uint4*>(a.kw) + c1);
    }
  }

  for (int g = g0; g < g1; g += kInFlight) {
    if (g > g0) {
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) load(g + u, x[u][0], x[u][1]);
    }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      int h;
      const int kind = row_of(g + u, &h);
      uint4 y0 = x[u][0], y1 = x[u][1];
      if (kind < 2) {
        float f0[P], f1[P];
        E::up(y0, f0);
        E::up(y1, f1);
        if (kind == 0 ? a.qw != nullptr : a.kw != nullptr) {  // the same for the whole warp
          float ss = 0.0f;
#pragma unroll
          for (int i = 0; i < P; ++i) ss = fmaf(f0[i], f0[i], fmaf(f1[i], f1[i], ss));
          for (int m = 1 << a.lane_bits >> 1; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
          const float inv = rsqrtf(fmaf(ss, a.inv_dim, a.eps));
          float w0[P], w1[P];
          E::up(kind == 0 ? wq[0] : wk[0], w0);
          E::up(kind == 0 ? wq[1] : wk[1], w1);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            f0[i] = f0[i] * inv * w0[i];
            f1[i] = f1[i] * inv * w1[i];
          }
        }
        if (turned && a.interleaved) {
          // pairs (f0[0], f0[1]), ... then (f1[0], f1[1]), ...
#pragma unroll
          for (int i = 0; i < P / 2; ++i) {
            const float p = f0[2 * i], r = f0[2 * i + 1];
            f0[2 * i] = p * cosv[i] - r * sinv[i];
            f0[2 * i + 1] = r * cosv[i] + p * sinv[i];
            const float p1 = f1[2 * i], r1 = f1[2 * i + 1];
            f1[2 * i] = p1 * cosv[P / 2 + i] - r1 * sinv[P / 2 + i];
            f1[2 * i + 1] = r1 * cosv[P / 2 + i] + p1 * sinv[P / 2 + i];
          }
        } else {
          // the pairs (f0[i], f1[i]); for a unit that is not turned (1, 0), or NaN
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const float p = f0[i], r = f1[i];
            f0[i] = p * cosv[i];
            f1[i] = r * cosv[i];
            if (turned) {
              f0[i] -= r * sinv[i];
              f1[i] += p * sinv[i];
            }
          }
        }
        y0 = E::down(f0);
        y1 = E::down(f1);
      }
      if (h >= 0) {
        char* p;
        if (kind == 0)
          p = a.q.out + (int64_t(t) * a.q.out_ts + int64_t(h) * a.q.out_hs) * E::kSize;
        else if (!a.slots)
          p = a.k.out + (int64_t(t) * a.k.out_ts + int64_t(h) * a.k.out_hs) * E::kSize;
        else
          p = kind == 1 ? kdst + int64_t(h) * a.k.out_hs * E::kSize : vdst + int64_t(h) * a.v.out_hs * E::kSize;
        if (kind == 0 || stored) {
          *reinterpret_cast<uint4*>(p + c0 * 16) = y0;
          *reinterpret_cast<uint4*>(p + c1 * 16) = y1;
        }
      }
    }
  }
}

// Any head size, alignment and rotated part: one warp per row, a lane per
// pair, then the rest of the row.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_rows_any_kernel(const __grid_constant__ RopeArgs a) {
  using E = Elem<T>;
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
    const float2 f = good ? __ldg(cs + i) : make_float2(nan, nan);
    E::store(out + i0 * E::kSize, p * f.x - b * f.y);
    E::store(out + i1 * E::kSize, b * f.x + p * f.y);
  }
  for (int i = a.rot + lane; i < a.dim; i += 32) E::store(out + i * E::kSize, good ? value(i) : nan);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T>
cudaError_t launch_rows(RopeArgs& a, cudaStream_t stream) {
  using E = Elem<T>;
  const int P = E::kPer;
  auto fits = [&](const RowSet& r) {
    return r.heads == 0 || (aligned16(r.in) && aligned16(r.out) && r.in_ts % P == 0 && r.in_hs % P == 0 &&
                            r.out_ts % P == 0 && r.out_hs % P == 0);
  };
  const bool wide = a.dim % (2 * P) == 0 && a.rot % (2 * P) == 0 && a.dim / (2 * P) <= 32 && fits(a.q) &&
                    fits(a.k) && fits(a.v) && aligned16(a.qw) && aligned16(a.kw) && aligned16(a.cs) &&
                    a.k_page_stride % P == 0 && a.k_slot_stride % P == 0 && a.v_page_stride % P == 0 &&
                    a.v_slot_stride % P == 0;
  const int per_block = kRopeThreads / 32;
  if (!wide) {
    const int64_t warps = int64_t(a.tokens) * (a.q.heads + a.k.heads + a.v.heads);
    const int64_t blocks = (warps + per_block - 1) / per_block;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    return launch_k(rope_rows_any_kernel<T>, dim3(unsigned(blocks)), dim3(kRopeThreads), 0, stream, a);
  }
  a.lane_bits = 0;
  while ((1 << a.lane_bits) < a.dim / (2 * P)) ++a.lane_bits;
  const int rows = 32 >> a.lane_bits;
  a.gq = (a.q.heads + rows - 1) / rows;
  a.gk = (a.k.heads + rows - 1) / rows;
  a.gv = (a.v.heads + rows - 1) / rows;
  // Groups per warp: one while that does not fill the SMs (64 warps each),
  // more when there is plenty, so that a warp's table row and weights serve
  // several groups.
  const int groups = a.gq + a.gk + a.gv;
  int64_t per = int64_t(a.tokens) * groups / (152 * 64);
  per = per < 1 ? 1 : per > 16 ? 16 : per;
  a.parts = int((groups + per - 1) / per);
  a.per_warp = (groups + a.parts - 1) / a.parts;
  const int64_t blocks = (int64_t(a.tokens) * a.parts + per_block - 1) / per_block;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return launch_k(rope_rows_kernel<T>, dim3(unsigned(blocks)), dim3(kRopeThreads), 0, stream, a);
}

}  // namespace

cudaError_t read_and_clear_rope_flags(unsigned int* flags) {
  const unsigned int zero = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(flags, g_rope_flags, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_rope_flags, &zero, sizeof(unsigned int));
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
    case NF4_BF16: return launch_rows<Bf16>(a, stream);
    case NF4_FP16: return launch_rows<Fp16>(a, stream);
    default: return launch_rows<float>(a, stream);
  }
}

}  // namespace nf4
