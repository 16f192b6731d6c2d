// Epilogue pieces shared by the dense GEMM kernels (a shared expert's gated
// projection, the linear projection, and the products of their backward passes).
#pragma once

#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {

// Shared-memory descriptor of an MN-major operand (its rows along K, 64
// consecutive M or N elements per 128-byte row) stored by TMA boxes of
// 64 elements x 64 K rows with the 128-byte swizzle: 8-row atoms of 1024 bytes
// follow one another along K (stride byte offset), the boxes of further 64
// elements lie 8192 bytes apart (leading byte offset). A step of 16 along K
// advances the start address by 2048 bytes.
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(8192 >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// idesc_bf16_f32 with the majorness of the operands (bits 15 and 16).
__host__ __device__ constexpr uint32_t idesc_bf16_f32_major(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16_f32(M, N) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
}

// The activation of kAct (kActNone: the identity), and act * u of a gated pair.
template <int kAct>
__device__ __forceinline__ float act_t(float z) {
  return kAct == kActNone ? z : gated_act_t<kAct>(z, 1.0f);
}

// act(z) and act'(z):
//   silu z p, p (1 + z (1 - p)) with p = 1 / (1 + e^-z)
//   gelu z q, q + z e^(-z^2/2) / sqrt(2 pi) with q = (1 + erf(z / sqrt 2)) / 2
//   relu max(z, 0), [z > 0]
// silu's p saturates to 0 and 1 without an overflow: e^-z = inf gives p = 0.
__device__ __forceinline__ void act_and_slope(int act, float z, float& f, float& d) {
  if (act == MOE_ACT_SILU) {
    const float p = 1.0f / (1.0f + __expf(-z));
    f = p == 0.0f ? 0.0f : z * p;
    d = p == 0.0f ? 0.0f : p * fmaf(z, 1.0f - p, 1.0f);
  } else if (act == MOE_ACT_GELU) {
    const float q = 0.5f * (1.0f + erff(z * 0.7071067811865476f));
    f = z * q;
    d = fmaf(z * 0.3989422804014327f, __expf(-0.5f * z * z), q);
  } else if (act == MOE_ACT_RELU) {
    f = fmaxf(z, 0.0f);
    d = z > 0.0f ? 1.0f : 0.0f;
  } else {
    f = z;
    d = 1.0f;
  }
}

}  // namespace moe
