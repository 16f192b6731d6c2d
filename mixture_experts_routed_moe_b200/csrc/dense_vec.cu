// The dense products of a few tokens with the weights streamed through registers.
//
//   linear:  out[t, n] = bf16(act(<W[n], x[t]> + bias[n]) + residual[t, n])
//   gated:   out[t, n] = bf16(act(<W[n], x[t]>) * <W[N+n], x[t]>)
//
// Up to 24 tokens a weight is read for 48 operations at most: HBM's rate and what a
// call waits before and after its stream bound it, not the tensor cores. So a weight
// goes from global memory straight into the register of a warp-wide MMA (16 weight
// rows x 8 tokens x 16 of K), with no tensor map, shared memory, tensor memory or
// cluster on the way. The sum over K takes any order as long as both operands follow
// it: a lane's 32 contiguous bytes of a row are the K positions of its fragments in
// four MMAs, and the four lanes of a row take a 128-byte line in one load. A unit is
// 16 weight rows (gated: 8 gate rows and their 8 up rows, so that one lane holds
// both factors of an output); the warps of a block share its K range, and their
// partials are added in order in shared memory: no atomics, the same bits every run.
//
// On B200 in a CUDA graph, this form against the one with K split over a cluster of
// tcgen05 CTAs (its fixed path is 1 us longer): gated 2048 -> 1408 4.0 us against 5.4
// for 1 token, 4.1 against 5.6 for 8, 4.7 against 5.8 for 16; linear 2048 -> 7168 6.7
// against 8.4, 7.5 against 9.3, 8.1 against 9.4; gated 7168 -> 2048 10.8 against 12.6,
// 11.1 against 13.0, 11.8 against 13.3; gated 4096 -> 14336 34.6 (6.8 TB/s) against
// 39.4 for one token, 42.2 against 39.1 for 16, where the tokens' way through L1 is
// full. One token on fp32 multiply-adds instead took 4.5, 7.4, 11.6 and 37.3 us; loads
// of 16 bytes (half lines) 4.4, 7.7, 11.9 and 36.8.
#include <algorithm>

#include "dense_core.cuh"

namespace moe {
namespace {

constexpr int kMaxWarps = 16;
constexpr int kStep = 64;  // K of a warp's load: 4 lanes of a row, 16 bf16 each

struct VecParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* w;
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
  __nv_bfloat16* out;
  void* save;  // linear: bf16 z [T, N]; gated: fp32 [T, 2N]; or null
  int T, N, K, act;
};

// sixteen values of a row; those at K and beyond (`left` of them are below K, a
// multiple of 8) read as zero
struct Frag {
  uint32_t r[8];
};
template <bool kWide, bool kStream>
__device__ __forceinline__ Frag load(const __nv_bfloat16* p, int left) {
  Frag v;
  if constexpr (kWide) {  // one load of 32 bytes, whole or not at all
#pragma unroll
    for (int i = 0; i < 8; ++i) v.r[i] = 0u;
    if constexpr (kStream)
      asm volatile(
          "{ .reg .pred p; setp.gt.s32 p, %9, 0;\n\t"
          "@p ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8]; }"
          : "+r"(v.r[0]), "+r"(v.r[1]), "+r"(v.r[2]), "+r"(v.r[3]), "+r"(v.r[4]), "+r"(v.r[5]), "+r"(v.r[6]),
            "+r"(v.r[7])
          : "l"(p), "r"(left));
    else
      asm volatile(
          "{ .reg .pred p; setp.gt.s32 p, %9, 0;\n\t"
          "@p ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8]; }"
          : "+r"(v.r[0]), "+r"(v.r[1]), "+r"(v.r[2]), "+r"(v.r[3]), "+r"(v.r[4]), "+r"(v.r[5]), "+r"(v.r[6]),
            "+r"(v.r[7])
          : "l"(p), "r"(left));
  } else {
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const uint4* q = reinterpret_cast<const uint4*>(p);
    const uint4 l = left > 0 ? (kStream ? ld_stream_u4(q) : __ldg(q)) : zero;
    const uint4 h = left > 8 ? (kStream ? ld_stream_u4(q + 1) : __ldg(q + 1)) : zero;
    v = Frag{{l.x, l.y, l.z, l.w, h.x, h.y, h.z, h.w}};
  }
  return v;
}

// d += A B for 16 rows x 8 tokens x 16 of K: lane (g, c) = (lane / 4, lane % 4) gives
// rows g and g + 8 of A and token g of B, and holds tokens 2c and 2c + 1 of those rows
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// kGroups: groups of 8 tokens; kWide: rows start at multiples of 32 bytes
template <bool kGated, int kGroups, bool kWide>
__global__ void __launch_bounds__(32 * kMaxWarps, 1) dense_vec_kernel(const VecParams p) {
  pdl_wait();  // the previous kernel on the stream has completed; its writes are visible
  pdl_trigger();
  // 64 to 128 bytes of each row in flight a lane. (The bounds above say one block an SM, or
  // the compiler aims at 64 registers and takes the loads one by one: 4.9 us for 4.1.)
  constexpr int kBatch = kGroups == 1 ? 4 : 2;
  __shared__ float4 s_part[kMaxWarps][kGroups][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int n0 = blockIdx.x * (kGated ? 8 : 16);
  const bool two = kGated || n0 + 8 < p.N;  // N is a multiple of 8: a linear unit has one or two halves
  const int steps = (p.K + kStep - 1) / kStep;
  const int s0 = warp * steps / warps, s1 = (warp + 1) * steps / warps;
  const __nv_bfloat16* w0 = p.w + static_cast<size_t>(n0 + g) * p.K + c * 16;
  const __nv_bfloat16* w1 = p.w + static_cast<size_t>((kGated ? p.N : 8) + n0 + g) * p.K + c * 16;
  const __nv_bfloat16* x[kGroups];
  bool on[kGroups];
#pragma unroll
  for (int t = 0; t < kGroups; ++t) {
    on[t] = 8 * t + g < p.T;
    x[t] = p.x + static_cast<size_t>(on[t] ? 8 * t + g : 0) * p.K + c * 16;
  }
  float acc[kGroups][4] = {};
  for (int s = s0; s < s1; s += kBatch) {
    Frag a[kBatch], b[kBatch], v[kBatch][kGroups];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int k = (s + j) * kStep;
      const int left = s + j < s1 ? p.K - k - c * 16 : 0;
      a[j] = load<kWide, true>(w0 + k, left);
      b[j] = load<kWide, true>(w1 + k, two ? left : 0);
#pragma unroll
      for (int t = 0; t < kGroups; ++t) v[j][t] = load<kWide, false>(x[t] + k, on[t] ? left : 0);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
#pragma unroll
      for (int t = 0; t < kGroups; ++t)
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          mma(acc[t], a[j].r[i], b[j].r[i], a[j].r[i + 1], b[j].r[i + 1], v[j][t].r[i], v[j][t].r[i + 1]);
  }
#pragma unroll
  for (int t = 0; t < kGroups; ++t) s_part[warp][t][lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
  __syncthreads();
  if (warp >= kGroups) return;  // (a block has four warps or more)
  float z[4] = {};
  for (int q = 0; q < warps; ++q) {
    const float4 v = s_part[q][warp][lane];
    z[0] += v.x;
    z[1] += v.y;
    z[2] += v.z;
    z[3] += v.w;
  }
  // z: tokens 2c and 2c + 1 of row g, then of row g + 8
  const int t0 = 8 * warp + 2 * c;
  const int n = n0 + g;
  if constexpr (kGated) {
    if (p.save != nullptr) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (t0 + i >= p.T) continue;
        float* gu = static_cast<float*>(p.save) + static_cast<size_t>(t0 + i) * 2 * p.N + n;
        gu[0] = z[i];
        gu[p.N] = z[2 + i];
      }
    }
    with_act<false>(p.act, [&](auto tag) { act2<decltype(tag)::value>(z[0], z[1]); });
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (t0 + i < p.T) p.out[static_cast<size_t>(t0 + i) * p.N + n] = __float2bfloat16_rn(z[i] * z[2 + i]);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && !two) break;
      const int m = n + 8 * h;
      const size_t o = static_cast<size_t>(t0) * p.N + m;
      float y[2] = {z[2 * h], z[2 * h + 1]};
      if (p.bias != nullptr) {
        const float b = __bfloat162float(p.bias[m]);
        y[0] += b;
        y[1] += b;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (p.save != nullptr && t0 + i < p.T)
          static_cast<__nv_bfloat16*>(p.save)[o + i * static_cast<size_t>(p.N)] = __float2bfloat16_rn(y[i]);
      with_act<true>(p.act, [&](auto tag) { act2<decltype(tag)::value>(y[0], y[1]); });
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (t0 + i >= p.T) continue;
        const size_t at = o + i * static_cast<size_t>(p.N);
        // (not one FMA with the activation's last product: the bits are those of a call with save)
        if (p.residual != nullptr) y[i] = __fadd_rn(y[i], __bfloat162float(p.residual[at]));
        p.out[at] = __float2bfloat16_rn(y[i]);
      }
    }
  }
}

template <bool kGated, int kGroups>
cudaError_t launch_groups(const VecParams& p, bool wide, int units, int warps, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(units)), block(static_cast<unsigned>(32 * warps));
  return wide ? launch_pdl(dense_vec_kernel<kGated, kGroups, true>, grid, block, 0, st, p)
              : launch_pdl(dense_vec_kernel<kGated, kGroups, false>, grid, block, 0, st, p);
}

template <bool kGated>
cudaError_t launch_tokens(const VecParams& p, bool wide, int units, int warps, cudaStream_t st) {
  if (p.T <= 8) return launch_groups<kGated, 1>(p, wide, units, warps, st);
  if (p.T <= 16) return launch_groups<kGated, 2>(p, wide, units, warps, st);
  return launch_groups<kGated, 3>(p, wide, units, warps, st);
}

int units_of(const DenseGemm& g) { return g.order == kGatedNT ? g.N / 8 : (g.N + 15) / 16; }

}  // namespace

// Where this form is the faster one. More tokens take their loads through L1 once a unit,
// so that fewer units, or fewer bytes a unit, stay ahead: for 8 tokens gated 4096 -> 14336
// 35.7 us against 38.8, but linear 4096 -> 16384 26.1 against 24.0; for 16 linear 2048 ->
// 7168 8.2 against 9.3 and 5120 -> 5120 13.9 against 12.8; for 24 gated 2048 -> 1408 5.1
// against 6.3, but linear 2048 -> 7168 9.5 against 9.3 and for 20 gated 7168 -> 2048 13.6
// against 13.3; for 32 one of five sizes is ahead.
bool dense_vec_supported(const DenseGemm& g, int num_sms) {
  if (g.order != kGatedNT && g.order != kLinearNT) return false;
  const int units = units_of(g);
  if (g.M <= 1) return true;
  if (g.M <= 8) return g.order == kGatedNT || units <= 4 * num_sms;
  if (g.M <= 16) return units <= 2 * num_sms || (units <= 4 * num_sms && g.K <= 4096);
  return g.M <= 24 && units <= 2 * num_sms && g.K <= 4096;
}

cudaError_t launch_dense_vec(const DenseGemm& g, int num_sms, cudaStream_t st) {
  const bool gated = g.order == kGatedNT;
  VecParams p{};
  p.x = static_cast<const __nv_bfloat16*>(g.a);
  p.w = static_cast<const __nv_bfloat16*>(g.b);
  p.bias = static_cast<const __nv_bfloat16*>(g.bias);
  p.residual = static_cast<const __nv_bfloat16*>(g.residual);
  p.out = static_cast<__nv_bfloat16*>(g.out);
  p.save = g.save;
  p.T = g.M;
  p.N = g.N;
  p.K = g.K;
  p.act = g.act;
  const bool wide = g.K % 16 == 0 && reinterpret_cast<uintptr_t>(g.a) % 32 == 0 &&
                    reinterpret_cast<uintptr_t>(g.b) % 32 == 0;
  const int units = units_of(g);
  // Sixteen warps fill an SM's registers. One round of blocks with as many warps as fit:
  // linear 2048 -> 7168 (448 units) 6.8, 7.8 and 12.0 us with 4, 8 and 16 warps a block,
  // gated 7168 -> 2048 (256) 12.6, 11.1 and 13.0, linear 7168 -> 128 (8) 5.2, 4.4 and 4.1.
  // With more units two blocks of an SM cover one another's ends where K is long (gated 4096
  // -> 14336 37.9 against 34.6 us), four where it is short (gated 1024 -> 8192 7.1, 9.7).
  int warps = 4;
  if (units <= 2 * num_sms ? g.K >= 1024 : units > 4 * num_sms && g.K >= 4096) warps = 8;
  if (units <= num_sms && g.K >= 4096) warps = 16;
  return gated ? launch_tokens<true>(p, wide, units, warps, st) : launch_tokens<false>(p, wide, units, warps, st);
}

}  // namespace moe
