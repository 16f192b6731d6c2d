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
// registers between the sum of squares and the scaling. (Beyond 16384 columns a thread
// holds eight vectors, more than its 64 registers take: 0.7 to 1.5 KB a thread are spilled,
// and 4096 x 32768 with a residual takes 591 us = 1.8 TB/s, its backward pass 559; 4096 x
// 16384 91 and 166 us.) The sum of squares,
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
  __nv_bfloat16* residual_out;  // s, or null
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

// Sum over the threads that share a row, the same value in all of them. One
// warp: a butterfly over the lanes' sums of v. A block (tpr threads, a multiple
// of 32; one barrier of the whole block): v[j] of a warp belongs to the 32
// consecutive vectors of chunk j * tpr / 32 + warp; the chunks' sums are added in
// an order of their own numbers, so that a row's sum does not depend on how
// many vectors a thread holds. s_red holds a float for each chunk of the
// block's rows; two such buffers in turn make one barrier a row enough.
template <int kVec>
struct RowSum {
  int nw, warp, lane, first;  // warps of a row, this one's number in it, the row's first slot

  __device__ __forceinline__ explicit RowSum(int tpr)
      : nw(tpr >> 5), lane(threadIdx.x & 31) {
    const int group = (threadIdx.x >> 5) / nw;
    warp = (threadIdx.x >> 5) - group * nw;
    first = group * nw * kVec;
  }
  static __device__ __forceinline__ float butterfly(float t) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t;
  }
  __device__ __forceinline__ float operator()(const float (&v)[kVec], float* s_red) const {
    if (nw == 1) {
      float t = v[0];
#pragma unroll
      for (int j = 1; j < kVec; ++j) t += v[j];
      return butterfly(t);
    }
    float* red = s_red + first;
    float c[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) c[j] = butterfly(v[j]);
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) red[j * nw + warp] = c[j];
    }
    __syncthreads();
    float t = lane < nw * kVec ? red[lane] : 0.f;
#pragma unroll
    for (int q = 1; q < kVec; ++q)
      if (lane + 32 * q < nw * kVec) t += red[lane + 32 * q];
    return butterfly(t);
  }
};

// Scales one thread's vectors of row t and writes y, the codes and the scales.
template <int kVec, bool kCodes, bool kLean>
__device__ __forceinline__ void norm_write(const NormParams& p, const uint4 (&s)[kVec], const uint4 (&w)[kVec], float r,
                                           size_t base, int i0, int tpr, int nvec) {
  const unsigned hmask = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int i = i0 + j * tpr;
    if (i >= nvec) continue;  // H % 128 == 0 with codes: whole half-warps skip
    float a[8], g[8];
    unpack8(s[j], a);
    unpack8(kLean ? __ldg(reinterpret_cast<const uint4*>(p.weight) + i) : w[j], g);
#pragma unroll
    for (int q = 0; q < 8; ++q) a[q] = a[q] * r * g[q];
    if (!kCodes || p.y != nullptr) reinterpret_cast<uint4*>(p.y + base)[i] = pack8(a);
    if (kCodes) {
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

// Where the residual stream s comes from, and whether it is written. kAlone: s is x, which
// the caller keeps (the test for a buffer alone cost these forms up to 7%: 8192 x 2048
// 13.3 us against 14.3); kCopied: s is x, written to a buffer of its own; kAdded: x +
// residual, written where it is wanted.
enum Stream { kAlone, kCopied, kAdded };

// s = x + residual rounded to bf16 (x where the row has none), and the sum of its squares.
template <bool kRes>
__device__ __forceinline__ uint4 add_residual(const uint4& x, const uint4& res, float& sum) {
  float a[8];
  unpack8(x, a);
  uint4 s = x;
  if (kRes) {
    float b[8];
    unpack8(res, b);
#pragma unroll
    for (int q = 0; q < 8; ++q) a[q] += b[q];
    s = pack8(a);
    unpack8(s, a);
  }
  sum = a[0] * a[0];
#pragma unroll
  for (int q = 1; q < 8; ++q) sum = fmaf(a[q], a[q], sum);
  return s;
}

// Blocks of kMaxThreads an SM that the registers are bounded for, and so the threads that
// the grid may count on. (With the bound left at one block, codes at 70 registers a thread
// let 1024-thread grids run in two rounds: 8192 x 2048 35.6 us against 25.7.) Without a
// residual a row has half the bytes, so that more rows have to be in flight (13.4 us with
// 1536 threads, 17.1 with 1024); 640 threads are rows of 4104 to 5120 columns, two an SM.
constexpr int norm_residency(int vec, int threads, bool res, bool lean) {
  if (lean) return threads <= 256 ? 4 : threads <= 320 ? 3 : 2;
  if (threads == 640) return 2;
  if (threads != 512 || vec > 2) return 1;
  return vec == 1 && !res ? 3 : 2;
}

// A row is held by `tpr` threads: one warp, with blockDim / 32 rows in a
// block, or the whole block. Thread i of the row holds the 16-byte vectors i,
// i + tpr, ...; the 16 vectors of a 128-column group lie in one half-warp. The
// grid is a few blocks an SM; each row group walks over its rows with the next
// row's loads in flight while it reduces and stores the current one.
//
// kLean: the weights are read again for every row, from L1, and beyond 6144 columns the
// next row's loads go out after the sum: registers for one more block an SM.
//
// Measured on B200 (CUDA graph, inputs from HBM): 8192 x 2048 with a residual
// 22.9 us = 5.86 TB/s, 0.89 of the measured copy bandwidth; 4096 x 8192 43.4 us =
// 6.18 TB/s; 4096 x 7168 with codes 43.7 us = 6.05 TB/s; one row 1.7 us. Bulk copies
// of rows through a ring in shared memory (3 to 6 stages) measured 24 to 30 us
// on the first, one block a row without the walk 26.
template <int kVec, int kMaxThreads, int kStream, bool kCodes, bool kLean>
__global__ void __launch_bounds__(kMaxThreads, norm_residency(kVec, kMaxThreads, kStream == kAdded, kLean))
    rms_norm_kernel(const NormParams p, int tpr) {
  pdl_wait();  // the previous kernel on the stream has completed; its writes are visible
  pdl_trigger();
  constexpr bool kRes = kStream == kAdded;
  __shared__ float s_red[2][32 * kVec];
  const int rpb = blockDim.x / tpr;
  const RowSum<kVec> row_sum(tpr);
  const int i0 = threadIdx.x % tpr;
  const int nvec = p.H / 8;
  constexpr bool kLate = kLean && kMaxThreads > 384;  // (before the sum at 6144 columns: 38.1 us, after it 38.6)
  const long long step = static_cast<long long>(gridDim.x) * rpb;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint4 w[kVec], xv[kVec], rv[kVec];
  auto load = [&](long long t) {
    const uint4* x = reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(t) * p.H);
    const uint4* r = reinterpret_cast<const uint4*>(p.residual + static_cast<size_t>(t) * p.H);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int i = i0 + j * tpr;
      xv[j] = i < nvec ? x[i] : zero;
      if (kRes) rv[j] = i < nvec ? r[i] : zero;
    }
  };
  long long t = static_cast<long long>(blockIdx.x) * rpb + threadIdx.x / tpr;
  if (t < p.T) load(t);
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int i = i0 + j * tpr;
    w[j] = i < nvec ? __ldg(reinterpret_cast<const uint4*>(p.weight) + i) : zero;
  }
  const float inv_h = 1.0f / static_cast<float>(p.H);
  int flip = 0;
  // a row group of a block-wide row leaves the loop together, a warp on its own
  for (; t < p.T; t += step, flip ^= 1) {
    const size_t base = static_cast<size_t>(t) * p.H;
    uint4 s[kVec];
    float sq[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      s[j] = add_residual<kRes>(xv[j], rv[j], sq[j]);
      const int i = i0 + j * tpr;
      if (kStream != kAlone && p.residual_out != nullptr && i < nvec)
        reinterpret_cast<uint4*>(p.residual_out + base)[i] = s[j];
    }
    if (!kLate && t + step < p.T) load(t + step);
    const float sum = row_sum(sq, s_red[flip]);
    const float r = rsqrtf(fmaf(sum, inv_h, p.eps));
    if (kLate && t + step < p.T) load(t + step);
    if (p.rstd != nullptr && i0 == 0) p.rstd[t] = r;
    norm_write<kVec, kCodes, kLean>(p, s, w, r, base, i0, tpr, nvec);
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

// A row is held by `tpr` threads, with blockDim / tpr rows in a block at a time;
// a row group takes every (grid x groups)-th row: dx of each, and the sum of dy s
// r over its rows in registers. The block adds its groups' sums in order and
// writes one partial row, which column_sum_kernel adds over the blocks. With
// kPrefetch the next row's loads are in flight during the reduction and the
// stores of the current one (4099 x 4096 with a residual's gradient: 26.7 us, the
// column sums included, = 5.03 TB/s); without (rows so wide that the sums of dw take the
// registers) the second pass over the row reads it again, from the caches.
template <int kVec, int kMaxThreads, bool kPrefetch>
__global__ void __launch_bounds__(kMaxThreads) rms_norm_backward_kernel(const NormBwdParams p, int tpr) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float s_dw[];  // [groups - 1][H]
  __shared__ float s_red[2][32 * kVec];
  const int nvec = p.H / 8, groups = blockDim.x / tpr;
  const int group = threadIdx.x / tpr, i0 = threadIdx.x - group * tpr;
  const RowSum<kVec> row_sum(tpr);
  const long long step = static_cast<long long>(gridDim.x) * groups;
  const uint4* wv = reinterpret_cast<const uint4*>(p.weight);
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  constexpr int kHeld = kPrefetch ? kVec : 1;
  uint4 ndy[kHeld], ns[kHeld], ndr[kHeld], w[kHeld];
  float nr = 0.f;
  auto vec_of = [&](const __nv_bfloat16* m, long long t, int i) {
    return t < p.T && i < nvec && m != nullptr
               ? reinterpret_cast<const uint4*>(m + static_cast<size_t>(t) * p.H)[i]
               : zero;
  };
  auto load = [&](long long t) {
    nr = t < p.T ? __ldg(p.rstd + t) : 0.f;
#pragma unroll
    for (int j = 0; j < (kPrefetch ? kVec : 0); ++j) {
      ndy[j] = vec_of(p.dy, t, i0 + j * tpr);
      ns[j] = vec_of(p.s, t, i0 + j * tpr);
      ndr[j] = vec_of(p.dresidual, t, i0 + j * tpr);
    }
  };
  long long t0 = static_cast<long long>(blockIdx.x) * groups;  // the block's first row of this step
  load(t0 + group);
  float dw[kVec][8];
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    if (kPrefetch) w[j] = i0 + j * tpr < nvec ? __ldg(wv + i0 + j * tpr) : zero;
#pragma unroll
    for (int q = 0; q < 8; ++q) dw[j][q] = 0.f;
  }
  const float inv_h = 1.0f / static_cast<float>(p.H);
  int flip = 0;
  while (t0 < p.T) {
    const long long t = t0 + group;
    uint4 dy[kHeld], s[kHeld], dr[kHeld];
#pragma unroll
    for (int j = 0; j < (kPrefetch ? kVec : 0); ++j) {
      dy[j] = ndy[j];
      s[j] = ns[j];
      dr[j] = ndr[j];
    }
    const float r = nr;
    t0 += step;
    if (t0 < p.T) load(t0 + group);
    float part[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int i = i0 + j * tpr;
      float a[8], b[8], g[8];
      part[j] = 0.f;
      unpack8(kPrefetch ? dy[kPrefetch ? j : 0] : vec_of(p.dy, t, i), a);
      unpack8(kPrefetch ? s[kPrefetch ? j : 0] : vec_of(p.s, t, i), b);
      unpack8(kPrefetch ? w[kPrefetch ? j : 0] : vec_of(p.weight, 0, i), g);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float xh = b[q] * r;
        dw[j][q] = fmaf(a[q], xh, dw[j][q]);
        part[j] = fmaf(a[q] * g[q], xh, part[j]);
      }
    }
    const float dot = row_sum(part, s_red[flip]) * inv_h;
    flip ^= 1;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int i = i0 + j * tpr;
      if (t >= p.T || i >= nvec) continue;
      float a[8], b[8], g[8], d[8];
      unpack8(kPrefetch ? dy[kPrefetch ? j : 0] : vec_of(p.dy, t, i), a);
      unpack8(kPrefetch ? s[kPrefetch ? j : 0] : vec_of(p.s, t, i), b);
      unpack8(kPrefetch ? w[kPrefetch ? j : 0] : vec_of(p.weight, 0, i), g);
      unpack8(kPrefetch ? dr[kPrefetch ? j : 0] : vec_of(p.dresidual, t, i), d);
#pragma unroll
      for (int q = 0; q < 8; ++q) d[q] = fmaf(r, a[q] * g[q] - b[q] * r * dot, d[q]);
      reinterpret_cast<uint4*>(p.dx + static_cast<size_t>(t) * p.H)[i] = pack8(d);
    }
  }
  if (groups > 1) {
    if (group > 0) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const int i = i0 + j * tpr;
        if (i >= nvec) continue;
#pragma unroll
        for (int q = 0; q < 8; ++q) s_dw[(group - 1) * p.H + 8 * i + q] = dw[j][q];
      }
    }
    __syncthreads();
    if (group > 0) return;
  }
  float* out = p.partial + static_cast<size_t>(blockIdx.x) * p.H;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int i = i0 + j * tpr;
    if (i >= nvec) continue;
    for (int g = 0; g < groups - 1; ++g)
#pragma unroll
      for (int q = 0; q < 8; ++q) dw[j][q] += s_dw[g * p.H + 8 * i + q];
    reinterpret_cast<float4*>(out)[2 * i] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
    reinterpret_cast<float4*>(out)[2 * i + 1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
  }
}

// out[c] = bf16(sum_r partial[r][c]), r ascending within each of 32 row
// classes, the classes added in order. A block takes 32 columns.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* __restrict__ partial, int rows, int cols,
                                                          __nv_bfloat16* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s_sum[32][33];
  const int lane = threadIdx.x & 31, cls = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int r = cls; r < rows; r += 32) v += partial[static_cast<size_t>(r) * cols + c];
  }
  s_sum[cls][lane] = v;
  __syncthreads();
  if (cls == 0 && c < cols) {
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 32; ++q) t += s_sum[q][lane];
    out[c] = __float2bfloat16_rn(t);
  }
}

int round32(int v) { return (v + 31) / 32 * 32; }

}  // namespace

cudaError_t launch_column_sum(const float* partial, int rows, int cols, void* out, cudaStream_t st) {
  return launch_pdl(column_sum_kernel, dim3(static_cast<unsigned>((cols + 31) / 32)), dim3(1024), 0, st, partial, rows,
                    cols, static_cast<__nv_bfloat16*>(out));
}

namespace {

template <int kVec, int kMaxThreads, bool kLean, int kStream, bool kCodes>
cudaError_t launch_norm_s(const NormParams& p, int block, int tpr, int num_sms, cudaStream_t st) {
  constexpr bool kRes = kStream == kAdded;
  const long long rpb = block / tpr;
  // as many blocks as are resident; four vectors with a residual run in two rounds, whose
  // first loads overlap the others' last rows (4096 x 8192 43.3 us against 46.0)
  const int fit = kVec == 4 && kRes && !kCodes ? 1024 : kMaxThreads * norm_residency(kVec, kMaxThreads, kRes, kLean);
  const int per_sm = std::max(1, fit / block);
  const long long blocks = std::min<long long>((p.T + rpb - 1) / rpb, static_cast<long long>(num_sms) * per_sm);
  return launch_pdl(rms_norm_kernel<kVec, kMaxThreads, kStream, kCodes, kLean>, dim3(static_cast<unsigned>(blocks)),
                    dim3(static_cast<unsigned>(block)), 0, st, p, tpr);
}

template <int kVec, int kMaxThreads, bool kLean, bool kRes, bool kCodes>
cudaError_t launch_norm_k(const NormParams& p, int block, int tpr, int num_sms, cudaStream_t st) {
  if constexpr (kRes) {
    return launch_norm_s<kVec, kMaxThreads, kLean, kAdded, kCodes>(p, block, tpr, num_sms, st);
  } else {
    return p.residual_out != nullptr
               ? launch_norm_s<kVec, kMaxThreads, kLean, kCopied, kCodes>(p, block, tpr, num_sms, st)
               : launch_norm_s<kVec, kMaxThreads, kLean, kAlone, kCodes>(p, block, tpr, num_sms, st);
  }
}

template <int kVec, int kMaxThreads>
cudaError_t launch_norm_t(const NormParams& p, int block, int tpr, int num_sms, cudaStream_t st) {
  if (p.residual != nullptr)
    return p.codes != nullptr ? launch_norm_k<kVec, kMaxThreads, false, true, true>(p, block, tpr, num_sms, st)
                              : launch_norm_k<kVec, kMaxThreads, false, true, false>(p, block, tpr, num_sms, st);
  return p.codes != nullptr ? launch_norm_k<kVec, kMaxThreads, false, false, true>(p, block, tpr, num_sms, st)
                            : launch_norm_k<kVec, kMaxThreads, false, false, false>(p, block, tpr, num_sms, st);
}

// The lean form with codes, one row a block.
template <int kMaxThreads>
cudaError_t launch_norm_lean(const NormParams& p, int threads, int num_sms, cudaStream_t st) {
  return p.residual != nullptr ? launch_norm_k<2, kMaxThreads, true, true, true>(p, threads, threads, num_sms, st)
                               : launch_norm_k<2, kMaxThreads, true, false, true>(p, threads, threads, num_sms, st);
}

}  // namespace

cudaError_t launch_rms_norm(const void* x, const void* residual, const void* weight, int T, int H, float eps, void* y,
                            void* residual_out, uint8_t* codes, float* scales, float* rstd, int num_sms,
                            cudaStream_t st) {
  NormParams p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.residual = static_cast<const __nv_bfloat16*>(residual);
  p.weight = static_cast<const __nv_bfloat16*>(weight);
  p.y = static_cast<__nv_bfloat16*>(y);
  // (without a residual the stream is x: only a buffer of its own has to be written)
  p.residual_out = residual == nullptr && residual_out == x ? nullptr : static_cast<__nv_bfloat16*>(residual_out);
  p.codes = codes;
  p.scales = scales;
  p.rstd = rstd;
  p.T = T;
  p.H = H;
  p.eps = eps;
  const int nvec = H / 8;
  // a warp per row up to four vectors a lane, else a block per row
  if (nvec <= 32) return launch_norm_t<1, 512>(p, 128, 32, num_sms, st);
  if (nvec <= 64) return launch_norm_t<2, 512>(p, 128, 32, num_sms, st);
  if (nvec <= 128) return launch_norm_t<4, 512>(p, 128, 32, num_sms, st);
  auto threads = [&](int vec) { return round32((nvec + vec - 1) / vec); };
  // Codes over many rows: two vectors a thread in the lean form, where half the threads a row
  // and few registers let two to four rows run on an SM and cover one another's waits
  // (4096 x 7168 47.2 -> 43.7 us, 8192 columns 52.1 -> 50.1; without residual 35.1 -> 31.7, 4096
  // columns 22.2 -> 18.5); with a residual up to 5120 columns one vector is as fast or
  // faster (8192 x 2048 25.7 us against 27.8, 4096 x 5120 31.9 against 33.9).
  if (codes != nullptr && T > 2 * num_sms) {
    const int one = threads(1), two = threads(2);
    if (nvec <= 640 && residual == nullptr)
      return nvec <= 512 ? launch_norm_k<2, 256, true, false, true>(p, two, two, num_sms, st)
                         : launch_norm_k<2, 320, true, false, true>(p, two, two, num_sms, st);
    if (nvec > 512 && nvec <= 640) return launch_norm_k<1, 640, false, true, true>(p, one, one, num_sms, st);
    if (nvec > 640 && nvec <= 768) return launch_norm_lean<384>(p, two, num_sms, st);
    if (nvec > 768 && nvec <= 896) return launch_norm_lean<448>(p, two, num_sms, st);
    if (nvec > 896 && nvec <= 1024) return launch_norm_lean<512>(p, two, num_sms, st);
  }
  if (nvec <= 512) return launch_norm_t<1, 512>(p, threads(1), threads(1), num_sms, st);
  // One vector a thread shortens a row's path, which counts where few rows run
  // (16 x 7168 with codes: 2.8 us against 3.7 with four); four keep more bytes
  // in flight (4096 x 7168 without codes: 37.6 us against 43).
  if (nvec <= 1024 && T <= 2 * num_sms)
    return launch_norm_t<1, 1024>(p, threads(1), threads(1), num_sms, st);
  if (nvec <= 2048) return launch_norm_t<4, 512>(p, threads(4), threads(4), num_sms, st);
  return launch_norm_t<8, 1024>(p, threads(8), threads(8), num_sms, st);
}

namespace {

// Threads that share a row of the backward pass, and rows of a block at a time: as many as
// fit into 256 threads, or one (blocks of 160 to 512 threads with one vector a thread).
int backward_vec(int nvec) { return nvec <= 512 ? 1 : nvec <= 1024 ? 2 : nvec <= 2048 ? 4 : 8; }
int backward_tpr(int nvec) { return round32((nvec + backward_vec(nvec) - 1) / backward_vec(nvec)); }
int backward_groups(int nvec) { return std::max(1, 256 / backward_tpr(nvec)); }

}  // namespace

// Partial rows of the weight gradient: the blocks that run at once, with one vector a
// thread as many as 1024 threads an SM allow and at most four (640 to 1024 threads, by the
// width; 8192 x 768 15.5 us, x 1280 21.9, x 2048 26.6), else one block (its registers fill the
// SM; two blocks an SM leave twice the partial rows: 4096 x 7168 46.6 us against 44.4).
int rms_norm_backward_blocks(int T, int H) {
  const int nvec = H / 8, groups = backward_groups(nvec), block = groups * backward_tpr(nvec);
  const int per_sm = backward_vec(nvec) == 1 ? std::max(1, std::min(4, 1024 / block)) : 1;
  return std::min((T + groups - 1) / groups, kNormBackwardSms * per_sm);
}

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
  const int nvec = H / 8, tpr = backward_tpr(nvec), groups = backward_groups(nvec);
  const dim3 grid(static_cast<unsigned>(rms_norm_backward_blocks(T, H)));
  const size_t smem = static_cast<size_t>(groups - 1) * H * sizeof(float);  // below 8 KB: H <= 1024 where groups > 1
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(static_cast<unsigned>(tpr * groups)), smem, st, p, tpr);
  };
  cudaError_t err;
  switch (backward_vec(nvec)) {
    case 1:
      err = go(rms_norm_backward_kernel<1, 512, true>);
      break;
    case 2:
      err = go(rms_norm_backward_kernel<2, 512, true>);
      break;
    case 4:
      err = go(rms_norm_backward_kernel<4, 512, false>);
      break;
    default:
      err = go(rms_norm_backward_kernel<8, 1024, false>);
  }
  if (err != cudaSuccess) return err;
  return launch_column_sum(partial, static_cast<int>(grid.x), H, dw, st);
}

}  // namespace moe
