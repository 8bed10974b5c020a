// nf4_attn.cuh -- definitions shared by the attention-side translation units
// (the entry points of include/nf4_attention.h).
#pragma once

#include "nf4_attention.h"
#include "nf4_internal.cuh"

namespace nf4 {

// Device error flags of the attention side, one word per translation unit and
// device (their addresses on the current one), read and cleared together with the
// tensor-core GEMV's.
constexpr unsigned kFlagWaitRanOut = 1u;  // a bounded wait ran out
constexpr unsigned kFlagBadIndex = 2u;    // a position, slot, page, length or cu_q entry out of range
cudaError_t rope_flags(unsigned int** word);
cudaError_t prefix_flags(unsigned int** word);
cudaError_t prefix_tc_flags(unsigned int** word);

nf4_status status_of(cudaError_t e);

cudaError_t launch_rope_table(const nf4_rope_table_args& a, cudaStream_t stream);
// The norm and rotation of q and k rows; with `cache`, keys and values go to
// its slots.
cudaError_t launch_qk_rope(const nf4_qk_norm_rope_args& a, const nf4_kv_append_args* cache,
                           cudaStream_t stream);
size_t prefix_attention_workspace_bytes(const nf4_prefix_attention_args& a);
// *enough is false, and nothing was launched, where the workspace does not do.
cudaError_t launch_prefix_attention(const nf4_prefix_attention_args& a, void* workspace, size_t workspace_bytes,
                                    bool* enough, cudaStream_t stream);

// 16-bit element types: conversions to and from binary32.
struct Bf16 {
  static constexpr nf4_dtype kDtype = NF4_BF16;
  static __device__ __forceinline__ float2 up2(uint32_t v) {  // low element first, exact
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t down2(float lo, float hi) {  // nearest even
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
struct Fp16 {
  static constexpr nf4_dtype kDtype = NF4_FP16;
  static __device__ __forceinline__ float2 up2(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
  static __device__ __forceinline__ uint32_t down2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

}  // namespace nf4
