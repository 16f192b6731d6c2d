// Epilogue pieces shared by the dense GEMM kernels (a shared expert's gated
// projection, the linear projection, and the products of their backward passes).
#pragma once

#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {

// One lane of the converged warp, the same one each time. The producer and the
// MMA issuer run their loops with the whole warp and let this lane issue:
// descriptors and coordinates stay in uniform registers that way. With a single
// lane in the loop, a K step of four MMAs cost its thread 0.28 us whatever
// their size; so issued it takes 0.20 (128 columns; 256 reach the MMAs' own 0.277).
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// mbar_wait_bounded by a whole warp, with one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                          uint64_t limit_ns) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort_flag, status, limit_ns));
}

// After a wait that gave up: the loads that the producer had issued when it stopped at
// (stage, phase) land in the ring, or a millisecond a stage passes.
__device__ __forceinline__ void drain_loads(uint64_t* full, int stages, int stage, uint32_t phase, int* status) {
  for (int i = 0; i < stages; ++i) {
    if (--stage < 0) {
      stage = stages - 1;
      phase ^= 1;
    }
    int never = 0;
    mbar_wait_bounded(&full[stage], phase, &never, status, 1000000ull);
  }
}

// The two halves of cluster_sync.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Asynchronous store into the shared memory of a CTA of the cluster, its four
// bytes counted on a barrier there.
__device__ __forceinline__ void st_async_u32(uint32_t cluster_dst, uint32_t v, uint32_t cluster_bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(cluster_dst),
               "r"(v), "r"(cluster_bar)
               : "memory");
}

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

// 2^x and 1/x by the hardware's approximations (2^-22 and one ulp, relative;
// subnormal results are zero): one instruction each, where the epilogues' tail
// and the gradients' elementwise pass would be paced by the range handling
// of expf and a division.
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// Two fp32 values in one register pair: the packed multiply-add takes one issue slot for
// both, and the epilogues' tail and the gradients' elementwise pass are paced by issue.
struct Pair {
  unsigned long long v;
};
__device__ __forceinline__ Pair pair(float a, float b) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ Pair pair(float a) { return pair(a, a); }
__device__ __forceinline__ void split(Pair p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// The standard normal distribution function at two z, and e = exp(-z^2 / 2):
// Phi(-|z|) = e/2 erfcx(|z| / sqrt 2), with erfcx(x) = e^(x^2) erfc(x) as a
// polynomial of degree 7 without constant term in t = 1 / (1 + 0.375 x), the
// form of Abramowitz and Stegun 7.1.26, fitted here by weighted least squares to
// a relative error of 7e-7 on [0, 11] (its coefficients halved below). The negative
// side keeps its relative accuracy (4e-6 at z = -12), which 1 + erf(z / sqrt 2) loses
// from -4 on.
__device__ __forceinline__ Pair normal_cdf(Pair z, Pair& e) {
  float z0, z1, t0, t1;
  split(z, z0, z1);
  split(fma2(pair(0.375f * 0.7071067811865476f), pair(fabsf(z0), fabsf(z1)), pair(1.0f)), t0, t1);
  const Pair t = pair(rcp_approx(t0), rcp_approx(t1));
  Pair q = pair(0.5f * -0.13459716737270355f);
  q = fma2(q, t, pair(0.5f * 0.386208713054657f));
  q = fma2(q, t, pair(0.5f * -0.12719842791557312f));
  q = fma2(q, t, pair(0.5f * 0.2813640832901001f));
  q = fma2(q, t, pair(0.5f * 0.16730797290802002f));
  q = fma2(q, t, pair(0.5f * 0.2155657857656479f));
  q = fma2(q, t, pair(0.5f * 0.2113487720489502f));
  split(mul2(mul2(z, z), pair(-0.5f * kLog2e)), t0, t1);
  e = pair(exp2_approx(t0), exp2_approx(t1));
  split(mul2(mul2(q, t), e), t0, t1);  // the tail
  return pair(z0 >= 0.0f ? 1.0f - t0 : t0, z1 >= 0.0f ? 1.0f - t1 : t1);  // a NaN stays one
}

// Two values through the activation kAct (kActNone: the identity).
template <int kAct>
__device__ __forceinline__ void act2(float& a, float& b) {
  if (kAct == MOE_ACT_GELU) {
    Pair e;
    const Pair z = pair(a, b);
    split(mul2(z, normal_cdf(z, e)), a, b);
  } else if (kAct == MOE_ACT_RELU) {
    a = a > 0.0f || a != a ? a : 0.0f;
    b = b > 0.0f || b != b ? b : 0.0f;
  } else if (kAct == MOE_ACT_SILU) {
    a *= rcp_approx(1.0f + exp2_approx(a * -kLog2e));
    b *= rcp_approx(1.0f + exp2_approx(b * -kLog2e));
  }
}

// f = act(z) and d = act'(z) of two values:
//   silu z p, p (1 + z (1 - p)) with p = 1 / (1 + e^-z)
//   gelu z Phi(z), Phi(z) + z e^(-z^2/2) / sqrt(2 pi)
//   relu max(z, 0), [z > 0]
// silu's p goes to 0 without an overflow: e^-z = inf gives p = 0.
template <int kAct>
__device__ __forceinline__ void act_and_slope(float z, float& f, float& d) {
  if (kAct == MOE_ACT_SILU) {
    const float p = rcp_approx(1.0f + exp2_approx(z * -kLog2e));
    f = z * p;
    d = p * fmaf(z, 1.0f - p, 1.0f);
  } else if (kAct == MOE_ACT_RELU) {
    f = z > 0.0f || z != z ? z : 0.0f;
    d = z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  } else {
    f = z;
    d = 1.0f;
  }
}
template <int kAct>
__device__ __forceinline__ void act_and_slope2(const float (&z)[2], float (&f)[2], float (&d)[2]) {
  if (kAct == MOE_ACT_GELU) {
    Pair e;
    const Pair zz = pair(z[0], z[1]), q = normal_cdf(zz, e);
    split(mul2(zz, q), f[0], f[1]);
    split(fma2(mul2(zz, pair(0.3989422804014327f)), e, q), d[0], d[1]);
  } else {
    act_and_slope<kAct>(z[0], f[0], d[0]);
    act_and_slope<kAct>(z[1], f[1], d[1]);
  }
}

// Runs f with the activation as a compile-time constant; a gate always has one (kNone false).
template <int kAct>
struct ActTag {
  static constexpr int value = kAct;
};
template <bool kNone, typename F>
__host__ __device__ __forceinline__ auto with_act(int act, F&& f) {
  switch (act) {
    case MOE_ACT_SILU:
      return f(ActTag<MOE_ACT_SILU>{});
    case MOE_ACT_GELU:
      return f(ActTag<MOE_ACT_GELU>{});
    default:
      if constexpr (kNone) {
        if (act == kActNone) return f(ActTag<kActNone>{});
      }
      return f(ActTag<MOE_ACT_RELU>{});
  }
}

}  // namespace moe
