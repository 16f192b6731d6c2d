// Root-mean-square norm with the residual's addition ahead of the router and
// the experts, its e4m3 form, and its backward pass.
//
//   s = bf16(x + residual)   (x itself without a residual: the residual stream)
//   r = (mean_i s_i^2 + eps)^(-1/2),   y_i = s_i r w_i
//   codes, scales: per 128 columns of the fp32 y, scale = amax / 448 (1 for an
//   all-zero group), code = e4m3(y / scale), as the FP8 experts' activations
//   dx_i = r (w_i dy_i - s_i r^2 mean_j(w_j dy_j s_j)) + dresidual_i
//   dw_i = sum_t dy_i s_i r
//
// Bound by HBM: every element is read once and written once, the row stays in
// registers between the sum of squares and the scaling. The sum of squares,
// r, the scaling and all gradient sums are fp32; s is rounded to bf16 because
// that is the value the residual stream keeps (and the backward pass reads),
// y, dx and dw are rounded once at the end, the codes straight from fp32.
// Every sum runs in a fixed order, so results are deterministic.
#include <algorithm>

#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

struct NormParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* residual;  // or null
  const __nv_bfloat16* weight;
  __nv_bfloat16* y;             // or null
  __nv_bfloat16* residual_out;  // or null
  uint8_t* codes;               // or null
  float* scales;
  float* rstd;  // or null
  int T, H;
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = bf16_lo(v.x);
  f[1] = bf16_hi(v.x);
  f[2] = bf16_lo(v.y);
  f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z);
  f[5] = bf16_hi(v.z);
  f[6] = bf16_lo(v.w);
  f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Sum over the `nthr` threads (a multiple of 32) that share a row, the same
// value in all of them; one warp needs no shared memory. The warp sums are
// added in warp order. `s_red` holds one float per warp and is free again
// after the row's next barrier.
__device__ __forceinline__ float row_sum(float v, int nthr, float* s_red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (nthr == 32) return v;
  const int warp = threadIdx.x >> 5, nw = nthr >> 5;
  if ((threadIdx.x & 31) == 0) s_red[warp] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  float t = lane < nw ? s_red[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

// One row per `tpr` threads: a warp with rows_per_block rows in a block, or the
// whole block. Thread i of the row holds the 16-byte vectors i, i + tpr, ...;
// the 16 vectors of a 128-column group lie in one half-warp.
template <int kVec>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormParams p, int tpr) {
  pdl_wait();  // the previous kernel on the stream has completed; its writes are visible
  pdl_trigger();
  __shared__ float s_red[32];
  const int rpb = blockDim.x / tpr;
  const long long t = static_cast<long long>(blockIdx.x) * rpb + threadIdx.x / tpr;
  if (t >= p.T) return;  // whole warps leave; a block-wide row always exists
  const int i0 = threadIdx.x % tpr;
  const int nvec = p.H / 8;
  const size_t base = static_cast<size_t>(t) * p.H;
  const uint4* x = reinterpret_cast<const uint4*>(p.x + base);
  const uint4* res = reinterpret_cast<const uint4*>(p.residual + base);
  const uint4* wv = reinterpret_cast<const uint4*>(p.weight);

  uint4 s[kVec], w[kVec];
  uint4 rv[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int i = i0 + j * tpr;
    s[j] = i < nvec ? x[i] : make_uint4(0u, 0u, 0u, 0u);
  }
  if (p.residual != nullptr) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int i = i0 + j * tpr;
      rv[j] = i < nvec ? res[i] : make_uint4(0u, 0u, 0u, 0u);
    }
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int i = i0 + j * tpr;
    w[j] = i < nvec ? __ldg(wv + i) : make_uint4(0u, 0u, 0u, 0u);
  }
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    float a[8];
    unpack8(s[j], a);
    if (p.residual != nullptr) {
      float b[8];
      unpack8(rv[j], b);
#pragma unroll
      for (int q = 0; q < 8; ++q) a[q] += b[q];
      s[j] = pack8(a);
      unpack8(s[j], a);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) sum = fmaf(a[q], a[q], sum);
  }
  if (p.residual_out != nullptr) {
    uint4* ro = reinterpret_cast<uint4*>(p.residual_out + base);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int i = i0 + j * tpr;
      if (i < nvec) ro[i] = s[j];
    }
  }
  sum = row_sum(sum, tpr, s_red);
  const float r = rsqrtf(sum / static_cast<float>(p.H) + p.eps);
  if (p.rstd != nullptr && i0 == 0) p.rstd[t] = r;
  const unsigned hmask = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int i = i0 + j * tpr;
    if (i >= nvec) continue;  // H % 128 == 0 with codes: whole half-warps skip
    float a[8], g[8];
    unpack8(s[j], a);
    unpack8(w[j], g);
#pragma unroll
    for (int q = 0; q < 8; ++q) a[q] = a[q] * r * g[q];
    if (p.y != nullptr) reinterpret_cast<uint4*>(p.y + base)[i] = pack8(a);
    if (p.codes != nullptr) {
      float amax = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) amax = fmaxf(amax, fabsf(a[q]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(hmask, amax, o));
      const float sc = amax > 0.f ? __fdiv_rn(amax, 448.0f) : 1.0f;
      const GroupDivisor dv = make_group_divisor(sc);
      uint32_t c[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(
            make_float2(group_div(dv, a[4 * q]), group_div(dv, a[4 * q + 1])), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(group_div(dv, a[4 * q + 2]), group_div(dv, a[4 * q + 3])), __NV_SATFINITE, __NV_E4M3);
        c[q] = lo | (hi << 16);
      }
      reinterpret_cast<uint2*>(p.codes + base)[i] = make_uint2(c[0], c[1]);
      if ((threadIdx.x & 15) == 0) p.scales[base / 128 + i / 16] = sc;
    }
  }
}

struct NormBwdParams {
  const __nv_bfloat16* dy;
  const __nv_bfloat16* s;
  const __nv_bfloat16* weight;
  const float* rstd;
  const __nv_bfloat16* dresidual;  // or null
  __nv_bfloat16* dx;
  float* partial;  // [gridDim.x, H]
  int T, H;
};

// Block b takes the rows b, b + grid, ...: dx of each row, and the block's sum
// of dy s r over its rows in registers, written once as a partial row that
// column_sum_kernel adds over the blocks.
template <int kVec>
__global__ void __launch_bounds__(1024) rms_norm_backward_kernel(const NormBwdParams p) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s_red[2][32];
  const int nvec = p.H / 8, tpr = blockDim.x;
  const uint4* wv = reinterpret_cast<const uint4*>(p.weight);
  uint4 w[kVec];
  float dw[kVec][8];
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int i = threadIdx.x + j * tpr;
    w[j] = i < nvec ? __ldg(wv + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int q = 0; q < 8; ++q) dw[j][q] = 0.f;
  }
  const float inv_h = 1.0f / static_cast<float>(p.H);
  int flip = 0;
  for (long long t = blockIdx.x; t < p.T; t += gridDim.x, flip ^= 1) {
    const size_t base = static_cast<size_t>(t) * p.H;
    const uint4* dyp = reinterpret_cast<const uint4*>(p.dy + base);
    const uint4* sp = reinterpret_cast<const uint4*>(p.s + base);
    const uint4* rp = reinterpret_cast<const uint4*>(p.dresidual + base);
    uint4 dy[kVec], s[kVec], dr[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int i = threadIdx.x + j * tpr;
      const bool in = i < nvec;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      dy[j] = in ? dyp[i] : zero;
      s[j] = in ? sp[i] : zero;
      dr[j] = in && p.dresidual != nullptr ? rp[i] : zero;
    }
    const float r = p.rstd[t];
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      float a[8], b[8], g[8];
      unpack8(dy[j], a);
      unpack8(s[j], b);
      unpack8(w[j], g);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float xh = b[q] * r;
        dw[j][q] = fmaf(a[q], xh, dw[j][q]);
        dot = fmaf(a[q] * g[q], xh, dot);
      }
    }
    // two buffers in turn: a warp may still read one row's sums while another
    // writes the next row's
    dot = row_sum(dot, tpr, s_red[flip]) * inv_h;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int i = threadIdx.x + j * tpr;
      if (i >= nvec) continue;
      float a[8], b[8], g[8], d[8];
      unpack8(dy[j], a);
      unpack8(s[j], b);
      unpack8(w[j], g);
      unpack8(dr[j], d);
#pragma unroll
      for (int q = 0; q < 8; ++q) d[q] = fmaf(r, a[q] * g[q] - b[q] * r * dot, d[q]);
      reinterpret_cast<uint4*>(p.dx + base)[i] = pack8(d);
    }
  }
  float* out = p.partial + static_cast<size_t>(blockIdx.x) * p.H;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int i = threadIdx.x + j * tpr;
    if (i >= nvec) continue;
    reinterpret_cast<float4*>(out)[2 * i] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
    reinterpret_cast<float4*>(out)[2 * i + 1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
  }
}

// out[c] = bf16(sum_r partial[r][c]), r ascending within each of eight row
// classes, the classes added in order. A block takes 32 columns.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* __restrict__ partial, int rows, int cols,
                                                         __nv_bfloat16* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s_sum[8][33];
  const int lane = threadIdx.x & 31, cls = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < cols)
    for (int r = cls; r < rows; r += 8) v += partial[static_cast<size_t>(r) * cols + c];
  s_sum[cls][lane] = v;
  __syncthreads();
  if (cls == 0 && c < cols) {
    float t = s_sum[0][lane];
#pragma unroll
    for (int q = 1; q < 8; ++q) t += s_sum[q][lane];
    out[c] = __float2bfloat16_rn(t);
  }
}

int round32(int v) { return (v + 31) / 32 * 32; }

}  // namespace

cudaError_t launch_column_sum(const float* partial, int rows, int cols, void* out, cudaStream_t st) {
  return launch_pdl(column_sum_kernel, dim3(static_cast<unsigned>((cols + 31) / 32)), dim3(256), 0, st, partial, rows,
                    cols, static_cast<__nv_bfloat16*>(out));
}

cudaError_t launch_rms_norm(const void* x, const void* residual, const void* weight, int T, int H, float eps, void* y,
                            void* residual_out, uint8_t* codes, float* scales, float* rstd, cudaStream_t st) {
  NormParams p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.residual = static_cast<const __nv_bfloat16*>(residual);
  p.weight = static_cast<const __nv_bfloat16*>(weight);
  p.y = static_cast<__nv_bfloat16*>(y);
  p.residual_out = static_cast<__nv_bfloat16*>(residual_out);
  p.codes = codes;
  p.scales = scales;
  p.rstd = rstd;
  p.T = T;
  p.H = H;
  p.eps = eps;
  const int nvec = H / 8;
  // a warp per row up to four vectors a lane, else a block per row with at
  // least eight warps' worth of vectors spread over it
  int vec, tpr, block;
  if (nvec <= 128) {
    vec = nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4;
    tpr = 32;
    block = 128;
  } else {
    vec = nvec <= 512 ? 1 : nvec <= 1024 ? 2 : nvec <= 4096 ? 4 : 8;
    tpr = block = round32((nvec + vec - 1) / vec);
  }
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(T) + block / tpr - 1) / (block / tpr)));
  switch (vec) {
    case 1:
      return launch_pdl(rms_norm_kernel<1>, grid, dim3(block), 0, st, p, tpr);
    case 2:
      return launch_pdl(rms_norm_kernel<2>, grid, dim3(block), 0, st, p, tpr);
    case 4:
      return launch_pdl(rms_norm_kernel<4>, grid, dim3(block), 0, st, p, tpr);
    default:
      return launch_pdl(rms_norm_kernel<8>, grid, dim3(block), 0, st, p, tpr);
  }
}

int rms_norm_backward_blocks(int T) { return std::min(T, kNormBackwardBlocks); }

cudaError_t launch_rms_norm_backward(const void* dy, const void* s, const void* weight, const float* rstd,
                                     const void* dresidual, int T, int H, void* dx, void* dw, float* partial,
                                     cudaStream_t st) {
  NormBwdParams p{};
  p.dy = static_cast<const __nv_bfloat16*>(dy);
  p.s = static_cast<const __nv_bfloat16*>(s);
  p.weight = static_cast<const __nv_bfloat16*>(weight);
  p.rstd = rstd;
  p.dresidual = static_cast<const __nv_bfloat16*>(dresidual);
  p.dx = static_cast<__nv_bfloat16*>(dx);
  p.partial = partial;
  p.T = T;
  p.H = H;
  const int nvec = H / 8;
  const int vec = nvec <= 256 ? 1 : nvec <= 1024 ? 2 : nvec <= 4096 ? 4 : 8;
  const dim3 grid(static_cast<unsigned>(rms_norm_backward_blocks(T)));
  const dim3 block(static_cast<unsigned>(round32((nvec + vec - 1) / vec)));
  cudaError_t err;
  switch (vec) {
    case 1:
      err = launch_pdl(rms_norm_backward_kernel<1>, grid, block, 0, st, p);
      break;
    case 2:
      err = launch_pdl(rms_norm_backward_kernel<2>, grid, block, 0, st, p);
      break;
    case 4:
      err = launch_pdl(rms_norm_backward_kernel<4>, grid, block, 0, st, p);
      break;
    default:
      err = launch_pdl(rms_norm_backward_kernel<8>, grid, block, 0, st, p);
  }
  if (err != cudaSuccess) return err;
  return launch_column_sum(partial, static_cast<int>(grid.x), H, dw, st);
}

}  // namespace moe
