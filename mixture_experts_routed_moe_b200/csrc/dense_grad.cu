// Elementwise halves of the dense operators' backward passes: the gradients
// at the pre-activations, from the pre-activations the forward kept (g and u in
// fp32, z in bf16: what that costs the slope stands at dense_gemm.cu's head).
//
//   gated:  dg = dh u act'(g),  du = dh act(g)        -> bf16 [T, 2I]
//   linear: dz = dy act'(z)                           -> bf16 [T, N]
//           db = sum_t dz                             (from the fp32 dz)
//
// HBM-bound: 16-byte loads and stores, each element once; gelu's slope is paced by issue
// as much, so that it works on packed pairs (4096 x 14336 gated 7 us less, now 115 = 7.2 TB/s
// with the last writes still in L2, silu 117; dz and db 69.4 -> 62.8, there with the
// 16-byte loads, silu 57.8). dg, du and dz are
// rounded to bf16 because they are the tensor cores' operands of the products
// that follow; the column sums are fp32 in a fixed order.
#include <algorithm>

#include "dense_core.cuh"

namespace moe {
namespace {

constexpr int kGradCols = 256;  // columns of a block of linear_grad_kernel

template <int kAct>
__global__ void __launch_bounds__(256) gated_grad_kernel(const float* __restrict__ gu,
                                                         const __nv_bfloat16* __restrict__ dh,
                                                         __nv_bfloat16* __restrict__ dgu, long long T, int I) {
  pdl_wait();  // the previous kernel on the stream has completed; its writes are visible
  pdl_trigger();
  const int nv = I / 8;
  const long long n = T * nv;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += stride) {
    const long long t = i / nv;
    const int c = static_cast<int>(i - t * nv) * 8;
    const float4* gp = reinterpret_cast<const float4*>(gu + 2 * t * I + c);
    const float4* up = reinterpret_cast<const float4*>(gu + 2 * t * I + I + c);
    const float4 g0 = gp[0], g1 = gp[1], u0 = up[0], u1 = up[1];
    const uint4 d = *reinterpret_cast<const uint4*>(dh + t * I + c);
    const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
    const float u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
    const uint32_t dw[4] = {d.x, d.y, d.z, d.w};
    uint32_t og[4], ou[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float f[2], s[2];
      act_and_slope2<kAct>({g[2 * q], g[2 * q + 1]}, f, s);
      const float a = bf16_lo(dw[q]), b = bf16_hi(dw[q]);
      og[q] = pack_bf16x2(a * u[2 * q] * s[0], b * u[2 * q + 1] * s[1]);
      ou[q] = pack_bf16x2(a * f[0], b * f[1]);
    }
    *reinterpret_cast<uint4*>(dgu + 2 * t * I + c) = make_uint4(og[0], og[1], og[2], og[3]);
    *reinterpret_cast<uint4*>(dgu + 2 * t * I + I + c) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
  }
}

// Block (x, y): 256 columns (8 a lane of a warp), rows y, y + 8, ... by its
// eight warps within the row range of blockIdx.y, two rows' loads in flight; dz
// written, the fp32 column sums of the range added over the warps in order and
// left in partial[y].
template <int kAct>
__global__ void __launch_bounds__(256, 4)
    linear_grad_kernel(const __nv_bfloat16* __restrict__ z, const __nv_bfloat16* __restrict__ dy,
                       __nv_bfloat16* __restrict__ dz, float* __restrict__ partial, long long T, int N) {
  pdl_wait();
  pdl_trigger();
  constexpr int kRows = 2;
  __shared__ float s_sum[8][kGradCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * kGradCols + lane * 8;
  const long long t0 = blockIdx.y * T / gridDim.y, t1 = (blockIdx.y + 1) * T / gridDim.y;
  float sum[8] = {};
  if (c < N) {
    for (long long t = t0 + warp; t < t1; t += 8 * kRows) {
      uint4 d[kRows], zz[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const size_t at = static_cast<size_t>(t + 8 * k) * N + c;
        d[k] = t + 8 * k < t1 ? *reinterpret_cast<const uint4*>(dy + at) : make_uint4(0u, 0u, 0u, 0u);
        if (kAct != kActNone)
          zz[k] = t + 8 * k < t1 ? *reinterpret_cast<const uint4*>(z + at) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const uint32_t dw[4] = {d[k].x, d[k].y, d[k].z, d[k].w};
        const uint32_t zw[4] = {zz[k].x, zz[k].y, zz[k].z, zz[k].w};
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v0 = bf16_lo(dw[q]), v1 = bf16_hi(dw[q]);
          if (kAct != kActNone) {
            float f[2], s[2];
            act_and_slope2<kAct>({bf16_lo(zw[q]), bf16_hi(zw[q])}, f, s);
            v0 *= s[0];
            v1 *= s[1];
            o[q] = pack_bf16x2(v0, v1);
          }
          sum[2 * q] += v0;
          sum[2 * q + 1] += v1;
        }
        if (kAct != kActNone && t + 8 * k < t1)
          *reinterpret_cast<uint4*>(dz + static_cast<size_t>(t + 8 * k) * N + c) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  if (partial == nullptr) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) s_sum[warp][lane * 8 + q] = sum[q];
  __syncthreads();
  const int col = blockIdx.x * kGradCols + threadIdx.x;
  if (threadIdx.x < kGradCols && col < N) {
    float t = s_sum[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < 8; ++w) t += s_sum[w][threadIdx.x];
    partial[static_cast<size_t>(blockIdx.y) * N + col] = t;
  }
}

}  // namespace

cudaError_t launch_gated_grad(const float* gu, const void* dh, void* dgu, int T, int I, int act, int num_sms,
                              cudaStream_t st) {
  const long long n = static_cast<long long>(T) * (I / 8);
  // a thread a vector (4096 x 14336: 117 us; one wave of blocks that walk 126)
  const long long blocks = std::min<long long>((n + 255) / 256, static_cast<long long>(num_sms) * 256);
  return with_act<false>(act, [&](auto tag) {
    return launch_pdl(gated_grad_kernel<decltype(tag)::value>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st,
                      gu, static_cast<const __nv_bfloat16*>(dh), static_cast<__nv_bfloat16*>(dgu),
                      static_cast<long long>(T), I);
  });
}

int linear_grad_rows(int T, int N) {
  // row ranges: one wave of four blocks an SM of a B200, at least 16 rows each (two a warp)
  const int cols = (N + kGradCols - 1) / kGradCols;
  return std::max(1, std::min((T + 15) / 16, std::max(1, 592 / cols)));
}

cudaError_t launch_linear_grad(const void* z, const void* dy, void* dz, float* partial, void* db, int T, int N,
                               int act, cudaStream_t st) {
  const int rows = linear_grad_rows(T, N);
  const dim3 grid(static_cast<unsigned>((N + kGradCols - 1) / kGradCols), static_cast<unsigned>(rows));
  const cudaError_t err = with_act<true>(act, [&](auto tag) {
    return launch_pdl(linear_grad_kernel<decltype(tag)::value>, grid, dim3(256), 0, st,
                      static_cast<const __nv_bfloat16*>(z),
                      static_cast<const __nv_bfloat16*>(dy), static_cast<__nv_bfloat16*>(dz),
                      db != nullptr ? partial : static_cast<float*>(nullptr), static_cast<long long>(T), N);
  });
  if (err != cudaSuccess || db == nullptr) return err;
  return launch_column_sum(partial, rows, N, db, st);
}

}  // namespace moe
