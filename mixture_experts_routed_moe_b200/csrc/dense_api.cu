// C entry points of the dense operators (declared in include/moe_b200.h):
// host-side argument checks, workspace sizes and the launch sequences.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "moe_common.cuh"
#include "moe_internal.h"

using namespace moe;

namespace {

constexpr int32_t kMaxDim = 1 << 20;
constexpr int32_t kMaxNormH = 65536;
constexpr int32_t kMaxT = 1 << 30;  // row numbers of a last tile stay below 2^31

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool rows_ok(int32_t T) { return T >= 0 && T <= kMaxT; }
bool dim_ok(int32_t v) { return v >= 8 && v <= kMaxDim && v % 8 == 0; }
bool gate_ok(int32_t act) { return act == MOE_ACT_SILU || act == MOE_ACT_GELU || act == MOE_ACT_RELU; }
bool act_ok(int32_t act) { return act == MOE_ACT_NONE || gate_ok(act); }

struct Span {
  const void* p;
  size_t bytes;
};

// No two spans of `outs` meet, and none meets a span of `ins`; null spans and
// empty ones never do. same[i] may be the very buffer of outs[i].
bool overlap(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}
bool disjoint(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span* q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) return false;
    for (const Span& i : ins)
      if (overlap(*o, i)) return false;
  }
  return true;
}
// disjoint, or the same buffer
bool same_or_disjoint(const Span& out, const Span& in) { return out.p == in.p || !overlap(out, in); }

size_t bf16_bytes(int64_t rows, int64_t cols) { return static_cast<size_t>(rows) * static_cast<size_t>(cols) * 2; }
size_t f32_bytes(int64_t rows, int64_t cols) { return static_cast<size_t>(rows) * static_cast<size_t>(cols) * 4; }
size_t round256(size_t v) { return (v + 255) / 256 * 256; }

moe_status done(cudaError_t err) { return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

cudaError_t run(const DenseGemm& g, int sms, cudaStream_t st) {
  if (dense_vec_supported(g, sms)) return launch_dense_vec(g, sms, st);
  return dense_small_us(g, sms) < dense_gemm_us(g, sms) ? launch_dense_small(g, sms, st)
                                                        : launch_dense_gemm(g, sms, st);
}

// dx = d W (d [T, M], W [M, K]) and dw = d^T x; either may be null. Both
// products share one launch, unless few tokens make dx faster as a stream of the weights.
cudaError_t backward_products(const void* d, const void* x, const void* w, int T, int M, int K, void* dx, void* dw,
                              int sms, cudaStream_t st) {
  DenseGemm gx{}, gw{};
  gx.order = kLinearNN;
  gx.M = T;
  gx.N = K;
  gx.K = M;
  gx.a = d;
  gx.b = w;
  gx.out = dx;
  gw.order = kLinearTN;
  gw.M = M;
  gw.N = K;
  gw.K = T;
  gw.a = d;
  gw.b = x;
  gw.out = dw;
  if (dx != nullptr && dw != nullptr &&
      dense_small_us(gx, sms) + dense_gemm_us(gw, sms) >= dense_gemm_backward_us(gx, gw, sms))
    return launch_dense_gemm_backward(gx, gw, sms, st);
  if (dx != nullptr) {
    const cudaError_t err = run(gx, sms, st);
    if (err != cudaSuccess) return err;
  }
  return dw != nullptr ? launch_dense_gemm(gw, sms, st) : cudaSuccess;
}

}  // namespace

extern "C" {

moe_status moe_rms_norm(const void* x, const void* residual, const void* weight, int32_t T, int32_t H, float eps,
                        void* y, void* residual_out, uint8_t* codes, float* scales, float* rstd, void* stream) {
  if (!rows_ok(T) || !dim_ok(H) || H > kMaxNormH || !std::isfinite(eps) || !(eps > 0.0f)) return MOE_ERR_INVALID_ARG;
  if ((codes == nullptr) != (scales == nullptr) || (codes != nullptr && H % 128 != 0)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (x == nullptr || weight == nullptr || (y == nullptr && codes == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(y, 16) ||
      !aligned(residual_out, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(rstd, 4))
    return MOE_ERR_INVALID_ARG;
  const size_t n = bf16_bytes(T, H);
  const Span sx{x, n}, sr{residual, n}, sw{weight, bf16_bytes(1, H)}, sy{y, n}, so{residual_out, n};
  const Span sc{codes, n / 2}, ss{scales, f32_bytes(T, H / 128)}, st{rstd, f32_bytes(T, 1)};
  if (!disjoint({sy, so, sc, ss, st}, {sw}) || !disjoint({sc, ss, st}, {sx, sr})) return MOE_ERR_INVALID_ARG;
  for (const Span& o : {sy, so})
    for (const Span& i : {sx, sr})
      if (!same_or_disjoint(o, i)) return MOE_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  return done(launch_rms_norm(x, residual, weight, T, H, eps, y, residual_out, codes, scales, rstd, sms,
                              static_cast<cudaStream_t>(stream)));
}

size_t moe_rms_norm_backward_workspace_size(int32_t T, int32_t H) {
  if (!rows_ok(T) || !dim_ok(H) || H > kMaxNormH) return 0;
  return round256(f32_bytes(std::max(1, rms_norm_backward_blocks(T, H)), H));
}

moe_status moe_rms_norm_backward(const void* dy, const void* s, const void* weight, const float* rstd,
                                 const void* dresidual, int32_t T, int32_t H, void* dx, void* dw, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const size_t need = moe_rms_norm_backward_workspace_size(T, H);
  if (need == 0 || dw == nullptr || !aligned(dw, 16)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) return done(cudaMemsetAsync(dw, 0, bf16_bytes(1, H), st));
  if (dy == nullptr || s == nullptr || weight == nullptr || rstd == nullptr || dx == nullptr || workspace == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(s, 16) || !aligned(weight, 16) || !aligned(rstd, 4) || !aligned(dresidual, 16) ||
      !aligned(dx, 16) || !aligned(workspace, 256))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  const size_t n = bf16_bytes(T, H), row = bf16_bytes(1, H);
  const Span sdy{dy, n}, ss{s, n}, sw{weight, row}, sr{rstd, f32_bytes(T, 1)}, sd{dresidual, n};
  const Span sx{dx, n}, sdw{dw, row}, sws{workspace, need};
  if (!disjoint({sx, sdw, sws}, {ss, sw, sr}) || !disjoint({sdw, sws}, {sdy, sd}) || !same_or_disjoint(sx, sdy) ||
      !same_or_disjoint(sx, sd))
    return MOE_ERR_INVALID_ARG;
  return done(launch_rms_norm_backward(dy, s, weight, rstd, dresidual, T, H, dx, dw, static_cast<float*>(workspace),
                                       st));
}

moe_status moe_gated_ffn(const void* x, const void* w_gate_up, int32_t T, int32_t H, int32_t I, int32_t act, void* h,
                         float* gu, void* stream) {
  if (!rows_ok(T) || !dim_ok(H) || !dim_ok(I) || !gate_ok(act)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (x == nullptr || w_gate_up == nullptr || h == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w_gate_up, 16) || !aligned(h, 16) || !aligned(gu, 16)) return MOE_ERR_INVALID_ARG;
  if (!disjoint({{h, bf16_bytes(T, I)}, {gu, f32_bytes(T, 2ll * I)}},
                {{x, bf16_bytes(T, H)}, {w_gate_up, bf16_bytes(2ll * I, H)}}))
    return MOE_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  DenseGemm g{};
  g.order = kGatedNT;
  g.M = T;
  g.N = I;
  g.K = H;
  g.a = x;
  g.b = w_gate_up;
  g.out = h;
  g.act = act;
  g.save = gu;
  return done(run(g, sms, static_cast<cudaStream_t>(stream)));
}

size_t moe_gated_ffn_backward_workspace_size(int32_t T, int32_t I) {
  if (!rows_ok(T) || !dim_ok(I)) return 0;
  return round256(std::max<size_t>(256, bf16_bytes(T, 2ll * I)));
}

moe_status moe_gated_ffn_backward(const void* dh, const void* x, const void* w_gate_up, const float* gu, int32_t T,
                                  int32_t H, int32_t I, int32_t act, void* dx, void* dw, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  const size_t need = moe_gated_ffn_backward_workspace_size(T, I);
  if (need == 0 || !dim_ok(H) || !gate_ok(act) || !aligned(dx, 16) || !aligned(dw, 16)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) return dw == nullptr ? MOE_OK : done(cudaMemsetAsync(dw, 0, bf16_bytes(2ll * I, H), st));
  if (dx == nullptr && dw == nullptr) return MOE_OK;
  if (dh == nullptr || x == nullptr || w_gate_up == nullptr || gu == nullptr || workspace == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (!aligned(dh, 16) || !aligned(x, 16) || !aligned(w_gate_up, 16) || !aligned(gu, 16) || !aligned(workspace, 256))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  if (!disjoint({{dx, bf16_bytes(T, H)}, {dw, bf16_bytes(2ll * I, H)}, {workspace, need}},
                {{dh, bf16_bytes(T, I)}, {x, bf16_bytes(T, H)}, {w_gate_up, bf16_bytes(2ll * I, H)},
                 {gu, f32_bytes(T, 2ll * I)}}))
    return MOE_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  cudaError_t err = launch_gated_grad(gu, dh, workspace, T, I, act, sms, st);
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  return done(backward_products(workspace, x, w_gate_up, T, 2 * I, H, dx, dw, sms, st));
}

moe_status moe_linear(const void* x, const void* w, const void* bias, const void* residual, int32_t T, int32_t K,
                      int32_t N, int32_t act, void* y, void* z, void* stream) {
  if (!rows_ok(T) || !dim_ok(K) || !dim_ok(N) || !act_ok(act)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (x == nullptr || w == nullptr || y == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 16) || !aligned(residual, 16) || !aligned(y, 16) ||
      !aligned(z, 16))
    return MOE_ERR_INVALID_ARG;
  const Span sy{y, bf16_bytes(T, N)}, sz{z, bf16_bytes(T, N)}, sr{residual, bf16_bytes(T, N)};
  if (!disjoint({sy, sz}, {{x, bf16_bytes(T, K)}, {w, bf16_bytes(N, K)}, {bias, bf16_bytes(1, N)}}) ||
      !disjoint({sz}, {sr}) || !same_or_disjoint(sy, sr))
    return MOE_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  DenseGemm g{};
  g.order = kLinearNT;
  g.M = T;
  g.N = N;
  g.K = K;
  g.a = x;
  g.b = w;
  g.out = y;
  g.act = act;
  g.bias = bias;
  g.residual = residual;
  g.save = z;
  return done(run(g, sms, static_cast<cudaStream_t>(stream)));
}

size_t moe_linear_backward_workspace_size(int32_t T, int32_t N, int32_t act, int32_t has_db) {
  if (!rows_ok(T) || !dim_ok(N) || !act_ok(act)) return 0;
  return 256 + (act != MOE_ACT_NONE ? round256(bf16_bytes(T, N)) : 0) +
         (has_db ? round256(f32_bytes(linear_grad_rows(T, N), N)) : 0);
}

moe_status moe_linear_backward(const void* dy, const void* x, const void* w, const void* z, int32_t T, int32_t K,
                               int32_t N, int32_t act, void* dx, void* dw, void* db, void* workspace,
                               size_t workspace_bytes, void* stream) {
  const size_t need = moe_linear_backward_workspace_size(T, N, act, db != nullptr);
  if (need == 0 || !dim_ok(K) || !aligned(dx, 16) || !aligned(dw, 16) || !aligned(db, 16)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    cudaError_t err = cudaSuccess;
    if (dw != nullptr) err = cudaMemsetAsync(dw, 0, bf16_bytes(N, K), st);
    if (err == cudaSuccess && db != nullptr) err = cudaMemsetAsync(db, 0, bf16_bytes(1, N), st);
    return done(err);
  }
  if (dx == nullptr && dw == nullptr && db == nullptr) return MOE_OK;
  if (dy == nullptr || x == nullptr || w == nullptr || workspace == nullptr || (act != MOE_ACT_NONE && z == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(z, 16) || !aligned(workspace, 256))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  if (!disjoint({{dx, bf16_bytes(T, K)}, {dw, bf16_bytes(N, K)}, {db, bf16_bytes(1, N)}, {workspace, need}},
                {{dy, bf16_bytes(T, N)}, {x, bf16_bytes(T, K)}, {w, bf16_bytes(N, K)},
                 {act != MOE_ACT_NONE ? z : nullptr, bf16_bytes(T, N)}}))
    return MOE_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const void* d = dy;
  void* dz = nullptr;
  if (act != MOE_ACT_NONE) {
    dz = ws;
    d = dz;
    ws += round256(bf16_bytes(T, N));
  }
  if (act != MOE_ACT_NONE || db != nullptr) {
    const cudaError_t err = launch_linear_grad(z, dy, dz, reinterpret_cast<float*>(ws), db, T, N, act, st);
    if (err != cudaSuccess) return MOE_ERR_CUDA;
  }
  return done(backward_products(d, x, w, T, N, K, dx, dw, sms, st));
}

}  // extern "C"
