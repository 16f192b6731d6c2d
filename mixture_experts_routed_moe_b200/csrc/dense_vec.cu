// The dense products of a single token: matrix-vector products on the CUDA cores.
//
//   linear:  out[n] = bf16(act(<W[n], x> + bias[n]) + residual[n])
//   gated:   out[n] = bf16(act(<W[n], x>) * <W[N+n], x>)
//
// One token is bound by the launch, the first byte's way from HBM and then the
// weights' stream, not by arithmetic, and needs no tensor map, tensor memory or
// cluster. A unit is two weight rows (gated: the gate and the up row of one output;
// linear: two outputs); `split` neighbouring warps of a block share a unit, each
// with its range of K in batches of 16-byte loads, and their fp32 sums are added
// in order. Enough warps are in flight to cover HBM's latency: many short rows
// take a warp each, few long ones several.
//
// On B200 in a CUDA graph, against the few-token form on the tensor cores: gated
// 2048 -> 1408 4.5 us against 5.4, linear 2048 -> 7168 7.4 against 8.4, gated 4096 ->
// 14336 37.3 (6.3 TB/s) against 39.5; from two tokens on that form wins (here the tokens
// would be read from L1 once a weight row).
#include <algorithm>

#include "dense_core.cuh"

namespace moe {
namespace {

constexpr int kMaxSplit = 8;  // warps of a unit at most
constexpr int kBatch = 4;  // 16-byte loads of a row in flight a lane

struct VecParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* w;
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
  __nv_bfloat16* out;
  void* save;  // linear: bf16 z [N]; gated: fp32 [2N]; or null
  int N, K, act;
  int split;  // warps of a unit: 1, 2, 4 or 8
};

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float acc) {
  const uint32_t p[4] = {a.x, a.y, a.z, a.w}, q[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = fmaf(bf16_lo(p[i]), bf16_lo(q[i]), acc);
    acc = fmaf(bf16_hi(p[i]), bf16_hi(q[i]), acc);
  }
  return acc;
}

template <bool kGated>
__global__ void __launch_bounds__(32 * kMaxSplit, 4) dense_vec_kernel(const VecParams p) {
  pdl_wait();  // the previous kernel on the stream has completed; its writes are visible
  pdl_trigger();
  __shared__ float2 s_sum[kMaxSplit];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int unit = (blockIdx.x * (blockDim.x >> 5) + warp) / p.split, part = warp % p.split;
  const int n = kGated ? unit : 2 * unit;  // (N is even: both rows of a linear unit exist)
  const int vecs = p.K / 8;
  const int v0 = static_cast<int>(static_cast<long long>(part) * vecs / p.split);
  const int v1 = n < p.N ? static_cast<int>(static_cast<long long>(part + 1) * vecs / p.split) : v0;
  const uint4* w0 = reinterpret_cast<const uint4*>(p.w + static_cast<size_t>(n) * p.K);
  const uint4* w1 = reinterpret_cast<const uint4*>(p.w + static_cast<size_t>(kGated ? p.N + n : n + 1) * p.K);
  const uint4* x = reinterpret_cast<const uint4*>(p.x);
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  float z0 = 0.f, z1 = 0.f;
  for (int i0 = v0 + lane; i0 < v1; i0 += 32 * kBatch) {
    uint4 a[kBatch], b[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + 32 * j;
      a[j] = i < v1 ? ld_stream_u4(w0 + i) : zero;
      b[j] = i < v1 ? ld_stream_u4(w1 + i) : zero;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + 32 * j;
      if (i >= v1) continue;
      const uint4 v = __ldg(x + i);
      z0 = dot8(a[j], v, z0);
      z1 = dot8(b[j], v, z1);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    z0 += __shfl_xor_sync(0xffffffffu, z0, o);
    z1 += __shfl_xor_sync(0xffffffffu, z1, o);
  }
  if (p.split > 1) {
    if (lane == 0) s_sum[warp] = make_float2(z0, z1);
    __syncthreads();
    if (part != 0) return;
    for (int q = 1; q < p.split; ++q) {
      z0 += s_sum[warp + q].x;
      z1 += s_sum[warp + q].y;
    }
  }
  if (lane != 0 || n >= p.N) return;
  if (kGated) {
    if (p.save != nullptr) {
      float* s = static_cast<float*>(p.save) + n;
      s[0] = z0;
      s[p.N] = z1;
    }
    p.out[n] = __float2bfloat16_rn(
        with_act(p.act, [&](auto tag) { return act_t<decltype(tag)::value>(z0) * z1; }));
  } else {
    if (p.bias != nullptr) {
      const uint32_t b = __ldg(reinterpret_cast<const uint32_t*>(p.bias + n));
      z0 += bf16_lo(b);
      z1 += bf16_hi(b);
    }
    if (p.save != nullptr)
      *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.save) + n) = pack_bf16x2(z0, z1);
    with_act(p.act, [&](auto tag) {
      z0 = act_t<decltype(tag)::value>(z0);
      z1 = act_t<decltype(tag)::value>(z1);
    });
    if (p.residual != nullptr) {
      const uint32_t r = *reinterpret_cast<const uint32_t*>(p.residual + n);
      z0 += bf16_lo(r);
      z1 += bf16_hi(r);
    }
    *reinterpret_cast<uint32_t*>(p.out + n) = pack_bf16x2(z0, z1);
  }
}

}  // namespace

// Weights of 100 MB and more with rows beyond 4096 stay with the few-token form: gated
// 16384 -> 8192 takes 83.7 us here and 81.8 there, 32768 -> 8192 180 and 155 (below that
// size this form wins throughout, 1.1 to 2 times; 4096 -> 14336 with 235 MB as well).
bool dense_vec_supported(const DenseGemm& g) {
  if (g.M != 1 || (g.order != kGatedNT && g.order != kLinearNT)) return false;
  return g.K <= 4096 || 2ll * g.K * g.N * (g.order == kGatedNT ? 2 : 1) < 100000000ll;
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
  p.N = g.N;
  p.K = g.K;
  p.act = g.act;
  // As many warps as fit on the SMs at once (32 each), each with two loads of a row a lane or
  // more. Blocks of four warps end sooner than blocks of eight (gated 2048 -> 1408 4.48 us
  // against 4.60); eight warps of a unit pay from K 4096 (16384 -> 8: 5.1 us to 3.6).
  const long long units = gated ? g.N : g.N / 2;
  p.split = 1;
  while (p.split < kMaxSplit && 2 * units * p.split <= 32ll * num_sms && g.K >= 1024 * p.split) p.split *= 2;
  const int warps = std::max(4, p.split);
  const long long per = warps / p.split;
  const dim3 grid(static_cast<unsigned>((units + per - 1) / per)), block(32 * warps);
  return gated ? launch_pdl(dense_vec_kernel<true>, grid, block, 0, st, p)
               : launch_pdl(dense_vec_kernel<false>, grid, block, 0, st, p);
}

}  // namespace moe
