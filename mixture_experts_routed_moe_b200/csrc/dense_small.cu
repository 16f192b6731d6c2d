// The dense GEMMs for few tokens: the weight rows are the MMA's M, the tokens
// its N, and K is split over a cluster, so that a decode batch streams the
// weights at HBM rate from every SM instead of filling a few token tiles.
//
//   linear:  out[t, n] = bf16(act(sum_k W[n,k] X[t,k] + bias[n]) + residual[t, n])
//   gated:   out[t, n] = bf16(act(sum_k W[n,k] X[t,k]) * sum_k W[N+n,k] X[t,k])
//
// for batches of up to a few hundred tokens (the smallest go through registers instead,
// but for dx and the largest weights), in even token tiles of at most 128, with W read
// K-major, or MN-major (linear only: dx = dz W of the backward pass, where W^T's rows
// are the outputs). A unit is up to 128 weight rows
// (gated: as many gate rows as up rows); a cluster of C CTAs owns a unit, CTA r
// taking the r-th of C ranges of K through a TMA ring into one TMEM
// accumulator of 128 x n_pad. The CTAs share out the unit's outputs, each adding
// the C partials of its part in rank order (one fixed order: deterministic, no
// atomics) and applying the epilogue in fp32. A partial goes straight from TMEM
// by asynchronous stores into the shared memory of the CTA that adds it, a
// region of its own beside the ring, counted on a barrier there: nobody waits for a
// remote load, for another CTA's ring or for a barrier of the cluster (from the
// last MMA to the end, 16 x 2048 -> 7168: 3.1 us with partials read through
// distributed shared memory between two cluster barriers, 1.9 so).
//
// Warps: 0 TMA producer, 1 MMA issuer; then all send and add. Every wait
// is bounded; a cluster with a wait that gave up writes NaN, and none of its CTAs that
// gave up ends before the others have stopped sending.
#include <algorithm>
#include <limits>
#include <type_traits>

#include "dense_core.cuh"

namespace moe {
namespace {

constexpr int kBK = 64;
constexpr int kThreads = 256;
constexpr int kManyThreads = 512;  // for large partials: see threads_of
constexpr int kA = kTileM * kBK * 2;  // 16 KB of weights a stage
constexpr int kMaxStages = 12;
constexpr int kTileTokens = 128;  // most tokens of a token tile
constexpr int kHalfTokens = 64;   // most tokens of a tile whose CTA takes half an SM

struct SmallParams {
  int T, N, num_kb;
  int tile_t, tiles; // tokens of a token tile, token tiles
  int n_pad;         // tile_t rounded up to a multiple of 16 (MMA N)
  uint32_t n_alloc;  // TMEM columns (power of two >= 32)
  int stages;        // of the ring, kA + n_pad * 128 bytes each
  int rows;          // outputs of a unit, a multiple of 8
  int act, stall;    // stall (failure tests): the last CTA of a cluster issues no loads
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
  __nv_bfloat16* out;
  void* save;  // linear: bf16 z [T, N]; gated: fp32 [T, 2N]; or null
  unsigned long long timeout_ns;
};

// Shared memory of a CTA, the ring and the partials' region: half an SM's (two
// CTAs of it, or one and the next kernel's, which starts early), or all of it for
// wide token tiles.
constexpr int kSlack = 1024, kBarrierBytes = 512;
__host__ __device__ constexpr int smem_bytes(int tile_t) { return tile_t <= kHalfTokens ? 114688 : 229376; }
__host__ __device__ constexpr int room(int tile_t) { return smem_bytes(tile_t) - kSlack - kBarrierBytes; }
__host__ __device__ constexpr int region_bytes(int tile_t) { return tile_t * kTileM * 4; }
int ring_stages(int tile_t, int n_pad) {
  return std::min(kMaxStages, (room(tile_t) - region_bytes(tile_t)) / (kA + n_pad * kBK * 2));
}

// Four consecutive outputs of one token, from their sums: bias, activation,
// residual, the one rounding. `res` and `bias` are the four values' inputs.
template <bool kGated>
__device__ __forceinline__ void write_outputs(const SmallParams& p, float4 z, float4 u, uint2 bias, uint2 res, int t,
                                              int n) {
  const size_t at = static_cast<size_t>(t) * p.N + n;
  float v[4];
  if (!kGated && p.bias != nullptr) {
    z.x += bf16_lo(bias.x);
    z.y += bf16_hi(bias.x);
    z.z += bf16_lo(bias.y);
    z.w += bf16_hi(bias.y);
  }
  if (p.save != nullptr) {
    if (kGated) {
      float* s = static_cast<float*>(p.save) + 2 * static_cast<size_t>(t) * p.N + n;
      *reinterpret_cast<float4*>(s) = z;
      *reinterpret_cast<float4*>(s + p.N) = u;
    } else {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.save) + at) =
          make_uint2(pack_bf16x2(z.x, z.y), pack_bf16x2(z.z, z.w));
    }
  }
  with_act<!kGated>(p.act, [&](auto tag) {
    constexpr int kAct = decltype(tag)::value;
    act2<kAct>(z.x, z.y);
    act2<kAct>(z.z, z.w);
  });
  v[0] = z.x;
  v[1] = z.y;
  v[2] = z.z;
  v[3] = z.w;
  if (kGated) {
    v[0] *= u.x;
    v[1] *= u.y;
    v[2] *= u.z;
    v[3] *= u.w;
  } else if (p.residual != nullptr) {
    v[0] += bf16_lo(res.x);
    v[1] += bf16_hi(res.x);
    v[2] += bf16_lo(res.y);
    v[3] += bf16_hi(res.y);
  }
  *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// The bias and the residual of four outputs.
__device__ __forceinline__ void load_addends(const SmallParams& p, int t, int n, uint2& bias, uint2& res) {
  bias = res = make_uint2(0u, 0u);
  if (n >= p.N) return;
  if (p.bias != nullptr) bias = __ldg(reinterpret_cast<const uint2*>(p.bias + n));
  if (p.residual != nullptr) res = *reinterpret_cast<const uint2*>(p.residual + static_cast<size_t>(t) * p.N + n);
}

// s_part holds [C][nt][len], the partials of this CTA's rows / C outputs (gated:
// the gate sums, then the up sums). The addends are loaded kAhead steps ahead,
// the first ones while the partials travel.
constexpr int kAhead = 2;
template <bool kGated, int kC>
__device__ __forceinline__ void finish(const SmallParams& p, const float* s_part, int n0, int t0, int nt, int rank,
                                       bool aborted, uint2 (&bias)[kAhead], uint2 (&res)[kAhead]) {
  const int own = p.rows / kC, len = kGated ? 2 * own : own, per = own / 4;
  auto step = [&](int i, uint2 bi, uint2 re) {
    const int t = i / per, r = (i - t * per) * 4;
    const int n = n0 + rank * own + r;
    if (n >= p.N) return;
    float4 g[kC], u[kC];
#pragma unroll
    for (int q = 0; q < kC; ++q) {
      const float* s = s_part + (q * nt + t) * len + r;
      g[q] = *reinterpret_cast<const float4*>(s);
      if (kGated) u[q] = *reinterpret_cast<const float4*>(s + own);
    }
#pragma unroll
    for (int q = 1; q < kC; ++q) {
      g[0].x += g[q].x;
      g[0].y += g[q].y;
      g[0].z += g[q].z;
      g[0].w += g[q].w;
      if (kGated) {
        u[0].x += u[q].x;
        u[0].y += u[q].y;
        u[0].z += u[q].z;
        u[0].w += u[q].w;
      }
    }
    if (aborted) {  // sums that never came: NaN in what is kept, and so in the output
      const float nan = __int_as_float(0x7FC00000);
      g[0] = u[0] = make_float4(nan, nan, nan, nan);
    }
    write_outputs<kGated>(p, g[0], u[0], bi, re, t0 + t, n);
  };
  for (int i = threadIdx.x; i < nt * per; i += blockDim.x) {
    const uint2 bi = bias[0], re = res[0];
#pragma unroll
    for (int k = 1; k < kAhead; ++k) {
      bias[k - 1] = bias[k];
      res[k - 1] = res[k];
    }
    if (!kGated) {
      const int j = i + kAhead * static_cast<int>(blockDim.x), t = j / per;
      if (t < nt) load_addends(p, t0 + t, n0 + rank * own + (j - t * per) * 4, bias[kAhead - 1], res[kAhead - 1]);
    }
    step(i, bi, re);
  }
}

template <bool kAmn, bool kGated>
__global__ void __launch_bounds__(kManyThreads)
    dense_small_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                       const SmallParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int kB = p.n_pad * kBK * 2;
  const int kStages = p.stages;
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * kA;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + room(p.tile_t));
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* arrived = tfull + 1;  // the partials of this CTA's outputs
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(arrived + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_status = reinterpret_cast<int*>(s_tmem + 2);
  float* s_part = reinterpret_cast<float*>(sB + kStages * kB);  // [C][nt][len], by source

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int csize = static_cast<int>(cluster_nctarank());
  const int rank = static_cast<int>(cluster_ctarank());
  // consecutive clusters take the token tiles of one unit: its weights meet in L2
  const int unit = blockIdx.x / csize / p.tiles;
  const int n0 = unit * p.rows;
  const int t0 = (blockIdx.x / csize - unit * p.tiles) * p.tile_t;
  const int nt = min(p.tile_t, p.T - t0);
  const int kb0 = rank * p.num_kb / csize, kb1 = (rank + 1) * p.num_kb / csize;
  // outputs that each CTA adds up, and their values a token
  const int own = p.rows / csize, len = kGated ? 2 * own : own;
  // bytes a stage receives (an MN-major unit always has 128 rows)
  const uint32_t stage_bytes = static_cast<uint32_t>((kGated ? 2 : 1) * (kAmn ? 128 : p.rows) * 128 + kB);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(arrived, 1);
    *s_abort = 0;
    *s_status = 0;
    fence_mbarrier_init();
    mbar_arrive_expect_tx(arrived, static_cast<uint32_t>(nt * (kGated ? 2 : 1) * p.rows * 4));
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, p.n_alloc);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  cluster_arrive();  // this CTA's barriers exist: its peers may copy into it after their wait
  pdl_wait();  // the previous kernel on the stream has completed; its writes are visible
  pdl_trigger();

  int next = 0;  // where the producer stops: the ring's next stage, its phase
  uint32_t next_ph = 0;
  if (warp == 0) {
    if (!p.stall || rank + 1 < csize) {
      const bool one = elect_one();
      int stage = 0;
      uint32_t ph = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait(&empty[stage], ph ^ 1, s_abort, s_status, p.timeout_ns)) break;
        if (one) {
          mbar_arrive_expect_tx(&full[stage], stage_bytes);
          uint8_t* a = sA + stage * kA;
          const int k0 = kb * kBK;
          if (kAmn) {
            tma_load_2d(a, &tmW, &full[stage], n0, k0);
            tma_load_2d(a + 8192, &tmW, &full[stage], n0 + 64, k0);
          } else if (kGated) {
            tma_load_2d(a, &tmW, &full[stage], k0, n0);
            tma_load_2d(a + p.rows * 128, &tmW, &full[stage], k0, p.N + n0);
          } else {
            tma_load_2d(a, &tmW, &full[stage], k0, n0);
          }
          tma_load_2d(sB + stage * kB, &tmX, &full[stage], k0, t0);
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          ph ^= 1;
        }
      }
      next = stage;
      next_ph = ph;
    }
  } else if (warp == 1) {
    const bool one = elect_one();
    const uint32_t idesc = idesc_bf16_f32_major(kTileM, p.n_pad, kAmn, false);
    int stage = 0;
    uint32_t ph = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!warp_wait(&full[stage], ph, s_abort, s_status, p.timeout_ns)) break;
      tc_fence_after();
      if (one) {
        const uint32_t a0 = smem_u32(sA + stage * kA);
        const uint32_t b0 = smem_u32(sB + stage * kB);
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k)
          umma_bf16(tmem_base, kAmn ? sdesc_mnmajor_sw128(a0 + k * 2048) : sdesc_kmajor_sw128(a0 + k * 32),
                    sdesc_kmajor_sw128(b0 + k * 32), idesc, (kb > kb0 || k != 0) ? 1u : 0u);
        umma_commit(&empty[stage]);
      }
      __syncwarp();
      if (++stage == kStages) {
        stage = 0;
        ph ^= 1;
      }
    }
    if (one) umma_commit(tfull);
    __syncwarp();
  }
  // All warps send the partial: two or four per TMEM lane quadrant, taking the blocks
  // of 16 tokens in turn (the producer's and the issuer's last).
  __syncwarp();
  {
    const int warps = blockDim.x / 32, quad = warp & 3, first = 16 * ((warp + warps - 2) % warps / 4);
    const int r = quad * 32 + lane;
    const bool busy = first < p.n_pad;
    const bool got = busy && mbar_wait_bounded(tfull, 0, s_abort, s_status, p.timeout_ns) && *s_abort == 0;
    const bool ok = __all_sync(0xffffffffu, got);
    cluster_wait();  // every CTA of the cluster runs, with its barriers
    if (ok) {
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
      const int up = kGated && r >= p.rows ? 1 : 0, ru = r - up * p.rows;
      const bool store = ru < p.rows;  // rows past the unit go nowhere
      const int owner = store ? ru / own : 0;
      const uint32_t dst = cluster_map(smem_u32(s_part + rank * nt * len + up * own + (ru - owner * own)),
                                       static_cast<uint32_t>(owner));
      const uint32_t bar = cluster_map(smem_u32(arrived), static_cast<uint32_t>(owner));
      for (int c = first; c < p.n_pad; c += 4 * warps) {
        uint32_t v[16];
        tmem_ld16(tb + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (store && c + i < nt) st_async_u32(dst + static_cast<uint32_t>((c + i) * len * 4), v[i], bar);
      }
    }
  }
  uint2 bias[kAhead], res[kAhead];
  if (!kGated) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = threadIdx.x + k * static_cast<int>(blockDim.x), per = own / 4, t = i / per;
      bias[k] = res[k] = make_uint2(0u, 0u);
      if (t < nt) load_addends(p, t0 + t, n0 + rank * own + (i - t * per) * 4, bias[k], res[k]);
    }
  }
  // without regard to this CTA's own abort flag: copies of other CTAs may still be on their way here
  int never = 0;
  const bool aborted = !mbar_wait_bounded(arrived, 0, &never, s_status, p.timeout_ns);
  tc_fence_before();
  auto end = [&](auto c) {
    finish<kGated, decltype(c)::value>(p, s_part, n0, t0, nt, rank, aborted, bias, res);
  };
  switch (csize) {
    case 1:
      end(std::integral_constant<int, 1>{});
      break;
    case 2:
      end(std::integral_constant<int, 2>{});
      break;
    case 4:
      end(std::integral_constant<int, 4>{});
      break;
    default:
      end(std::integral_constant<int, 8>{});
  }
  if (__syncthreads_or(aborted)) {
    // A wait gave up (never in normal operation), here or in a role whose part of this CTA's
    // partial then went to nobody, after the loads and MMAs that it waited for or stopped
    // were issued: they end before the shared and the tensor memory are given back.
    never = 0;
    if (threadIdx.x == 0) drain_loads(full, kStages, next, next_ph, s_status);
    if (threadIdx.x == 32) mbar_wait_bounded(tfull, 0, &never, s_status, 1000000ull);
    __syncthreads();
    // Slower peers may still send partials into this CTA. It stays until every peer has come
    // here too or has ended (threads that have do not count in the barrier, so that the
    // others pass by it), and then for what was sent last to land.
    cluster_arrive();
    cluster_wait();
    if (threadIdx.x == 0) mbar_wait_bounded(arrived, 0, &never, s_status, 1000000ull);
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, p.n_alloc);
  }
}

// Token tiles, rows of a unit, CTAs of a cluster, threads of a CTA.
struct Plan {
  int tile_t, tiles, rows, csize, ctas, threads;
  double us;  // estimated time; infinite where the CTAs would not be resident together
};

// Sixteen warps where a CTA sends and adds a large partial (linear with a residual 2048 ->
// 7168 for 96 tokens 13.4 us with eight, 11.5 with sixteen, 4096 -> 4096 for 256 20.4 and
// 17.9); with small ones and with the gated epilogue they cost up to 8%.
int threads_of(const DenseGemm& g, int tile_t, int rows, int csize) {
  return g.order != kGatedNT && tile_t * rows / csize >= 6000 ? kManyThreads : kThreads;
}

// The estimate, in us, fitted to sweeps on B200 (weights of 2048 x 1408 to 7168 x
// 2048, 1 to 512 tokens, every shape): 2.1 for the launch, the first loads and
// the end; a K step of a CTA at no less than 0.22, the ring's bytes in flight over
// 0.94, and 266 KB/us (172 for two CTAs of an SM); the partials and the outputs;
// a third of the weights' time from HBM, and some more where SMs with two CTAs
// run next to SMs with one. Over the sweep it is off by 9% and the shapes it
// picks are 1% from the best; the tile kernel's estimate is compared with it.
Plan plan_small(const DenseGemm& g, int num_sms) {
  const int num_kb = (g.K + kBK - 1) / kBK;
  const bool gated = g.order == kGatedNT;
  const double weights = 2.0 * g.N * g.K * (gated ? 2 : 1) / 6.0e6;
  Plan best{};
  best.us = std::numeric_limits<double>::infinity();
  for (int cap = 16; cap <= kTileTokens; cap *= 2) {
    const long long tiles = (g.M + cap - 1ll) / cap;
    const int tile_t = static_cast<int>((g.M + tiles - 1) / tiles);
    const int n_pad = (tile_t + 15) / 16 * 16;
    for (int c = 1; c <= 8; c *= 2) {
      if (c > 1 && 2 * c > num_kb) break;
      for (int rows = gated ? 64 : 128; rows >= 64; rows -= 64) {
        if (g.order == kLinearNN && rows != 128) continue;  // an MN-major unit is one box pair
        const long long ctas = ((g.N + rows - 1ll) / rows) * tiles * c;
        // clusters that fit, at two CTAs an SM or one
        if (tile_t <= kHalfTokens ? ctas > num_sms * (c == 8 ? 1.78 : c == 4 ? 1.91 : 2.0)
                                  : ctas > num_sms * (c == 8 ? 0.81 : c == 4 ? 0.89 : 1.0))
          continue;
        const double share = ctas > num_sms ? 2 : 1;
        const double bytes = (gated ? 2 : 1) * rows * 128 + n_pad * 128;
        const double step = std::max({0.22, 0.94 / ring_stages(tile_t, n_pad), bytes / (share > 1 ? 86e3 : 266e3)});
        const int threads = threads_of(g, tile_t, rows, c);
        const double us = 2.1 + (num_kb + c - 1) / c * step + 0.13 * c + 0.022 * tile_t +
                          (threads == kThreads ? 0.47 : 0.17) * tile_t * rows / c / 1024 + 0.36 * weights +
                          (share > 1 ? 1.1 + 0.16 * weights : 0.0);
        if (us < best.us) best = Plan{tile_t, static_cast<int>(tiles), rows, c, static_cast<int>(ctas), threads, us};
      }
    }
  }
  return best;
}

template <bool kAmn, bool kGated>
cudaError_t launch_t(const DenseGemm& g, int num_sms, cudaStream_t st) {
  // here the weights are g.b (rows = outputs) and the tokens g.a
  SmallParams p{};
  p.T = g.M;
  p.N = g.N;
  p.num_kb = (g.K + kBK - 1) / kBK;
  const Plan plan = plan_small(g, num_sms);
  p.tile_t = plan.tile_t;
  p.tiles = plan.tiles;
  p.rows = plan.rows;
  const int csize = plan.csize;
  p.n_pad = (p.tile_t + 15) / 16 * 16;
  p.n_alloc = 32;
  while (p.n_alloc < static_cast<uint32_t>(p.n_pad)) p.n_alloc <<= 1;
  p.stages = ring_stages(p.tile_t, p.n_pad);
  p.act = g.act;
  p.stall = stall_gate_up_loads();
  p.bias = static_cast<const __nv_bfloat16*>(g.bias);
  p.residual = static_cast<const __nv_bfloat16*>(g.residual);
  p.out = static_cast<__nv_bfloat16*>(g.out);
  p.save = g.save;
  p.timeout_ns = wait_limit_ns();

  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap tmW, tmX;
  const bool ok =
      (kAmn ? encode_tensor_map_2d(&tmW, bf16, 2, g.b, g.N, g.K, 64, kBK)
            : encode_tensor_map_2d(&tmW, bf16, 2, g.b, g.K, kGated ? 2 * static_cast<uint64_t>(g.N) : g.N, kBK,
                                   p.rows)) &&
      encode_tensor_map_2d(&tmX, bf16, 2, g.a, g.K, g.M, kBK, p.n_pad);
  if (!ok) return cudaErrorInvalidValue;

  auto kernel = dense_small_kernel<kAmn, kGated>;
  static unsigned long long done = 0;
  cudaError_t err = ensure_max_smem(reinterpret_cast<const void*>(kernel), &done);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(plan.ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(plan.threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem_bytes(p.tile_t));
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(csize);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, p);
}

}  // namespace

double dense_small_us(const DenseGemm& g, int num_sms) {
  return g.order == kLinearTN ? std::numeric_limits<double>::infinity() : plan_small(g, num_sms).us;
}

cudaError_t launch_dense_small(const DenseGemm& g, int num_sms, cudaStream_t st) {
  if (g.order == kGatedNT) return launch_t<false, true>(g, num_sms, st);
  if (g.order == kLinearNT) return launch_t<false, false>(g, num_sms, st);
  return launch_t<true, false>(g, num_sms, st);
}

}  // namespace moe
