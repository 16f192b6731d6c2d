// Dense GEMM on CTA pairs or single CTAs: tcgen05 tiles of one matrix for the
// whole batch (no routing), with the epilogues a shared expert needs.
//
//   linear:  out[m, n] = bf16(act(sum_k A[m,k] B[n,k] + bias[n]) + residual[m, n])
//   gated:   out[m, n] = bf16(act(sum_k A[m,k] B[n,k]) * sum_k A[m,k] B[N+n,k])
// optionally keeping the pre-activations for the backward pass: the gated g and u
// in fp32 (they multiply the gradients), the linear z in bf16, for half the bytes (1 to 2
// us of 2050 x 2048 -> 4104): only act'(z) is taken of it, which is then off by up to
// |z act''(z)| 2^-8 < 1.3e-3. For z from N(0, 1) that is 3.7e-4 rms where rounding dz itself
// is 1.3e-3 (together 4 to 5% more than dz's rounding alone); but it is absolute, so that it
// exceeds dz's rounding where the slope is small: gelu at z = -1 4.0e-4 against 1.3e-4, at -5
// 5% of a slope of 7e-6, next to its zero at -0.75 more than the slope.
//
// The products of the backward pass run in one launch:
//   dx = d W       A = d K-major, B = W MN-major
//   dW = d^T x     both MN-major
// Nothing is transposed in memory, and the tiles of both products share the
// waves: the longer ones first, the workers taking tiles in turn, so that one
// product's last wave is filled by the other's tiles (T = 4096, 2I = 2816, H =
// 2048: 88 tiles of 64 K steps and 128 of 44 on 74 pairs take 172 steps; one
// after the other, 128 + 88).
//
// Tiles: a pair (cta_group::2) computes 256 x kBN, a single CTA 128 x kBN; the
// gated form takes kBN/2 gate and kBN/2 up rows of B for one tile (in a pair
// the leader stages the gate rows, the peer the up rows), so one TMEM lane
// holds both halves of each of its outputs. K runs in steps of 64 through a
// TMA ring of 128-byte-swizzled tiles; two accumulator buffers in TMEM let the
// epilogue of a tile overlap the next tile's MMAs. Ragged edges are TMA's:
// loads fill zeros past the tensor, stores clip.
//
// Warps: 0 TMA producer, 1 MMA issuer, then 8 or 16 epilogue warps (two or four
// per TMEM lane quadrant, taking 32 columns in turn, through 2 KB staging buffers
// and TMA tile stores). Accumulation is fp32 in TMEM; bias,
// activation and residual are applied in fp32 before the one rounding.
//
// Every wait is bounded; a CTA whose wait gave up writes NaN into its tiles.
#include <algorithm>

#include "dense_core.cuh"

namespace moe {
namespace {

constexpr int kBK = 64;
constexpr int kBox = 32 * 64;  // a staging buffer: 32 rows of 64 bytes
constexpr int kStaging = 16 * kBox;
constexpr int kGroupM = 8;  // row blocks that are walked together along the columns (their A and B tiles meet in L2)

enum Mode { kModeGated, kModeLinear, kModeBackward };

// Epilogue warps, each with its share of the staging buffers. The linear form's
// longer epilogue (bias, activation, residual, z) takes sixteen: its part after
// the last tile is exposed (2050 x 2048 -> 4104 with all of it, sustained: 44.7 us
// against 47.0 with eight; the gated form 46.2 against 45.0).
template <int kMode>
struct Epilogue {
  static constexpr int kWarps = kMode == kModeLinear ? 16 : 8;
  static constexpr int kThreads = 64 + 32 * kWarps;
  static constexpr int kParts = kWarps / 4;  // warps of a TMEM lane quadrant
  static constexpr int kBufs = 16 / kWarps;  // staging buffers of a warp
};

// One product: out [M, N] over num_kb K steps, in m_tiles x n_tiles tiles.
struct Product {
  int M, N, num_kb, m_tiles, n_tiles;
  int a_mn;  // the A operand is MN-major (backward mode)
  __nv_bfloat16* out;
};

struct GemmParams {
  Product prod[2];  // the second only in backward mode
  int first_tiles, full, tiles;  // tiles of the first product; whole tiles of both; with the half ones
  int act, stall;                // stall (failure tests): the last CTA of a tile issues no loads
  void* save;                    // linear: bf16 z [M, N]; gated: fp32 [M, 2N]; or null
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
  unsigned long long timeout_ns;
};

// Tensor maps of the products' operands and outputs; save: z, or g and u.
struct GemmMaps {
  CUtensorMap a[2], b[2], y[2], save[2];
};

template <bool kPair, int kBN>
struct Tile {
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kBRows = kBN / kCtas;  // rows of B in one CTA
  static constexpr int kA = kTileM * kBK * 2;
  static constexpr int kB = kBRows * kBK * 2;
  static constexpr int kStage = kA + kB;
  static constexpr int kStages = 196608 / kStage < 8 ? 196608 / kStage : 8;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStage + kStaging + (2 * kStages + 5) * 8 + 16;
};

struct Coord {
  int prob, m, x, nb;  // product, row block, first output column, MMA N of the tile
};
// Entry `i` of the list: the first `full` are whole tiles, then the two halves
// (kBN / 2 columns) of each of the rest.
template <int kMode, int kBN>
__device__ __forceinline__ Coord tile_coord(const GemmParams& p, int i) {
  constexpr int kOutN = kMode == kModeGated ? kBN / 2 : kBN;
  Coord c;
  const bool half = i >= p.full;
  int tile = half ? p.full + (i - p.full) / 2 : i;
  c.prob = kMode == kModeBackward && tile >= p.first_tiles ? 1 : 0;
  if (c.prob) tile -= p.first_tiles;
  const int m_tiles = p.prod[c.prob].m_tiles;
  const int per = kGroupM * p.prod[c.prob].n_tiles;
  const int g = tile / per;
  const int gm = min(kGroupM, m_tiles - g * kGroupM);
  const int r = tile - g * per;
  const int n = r / gm;
  c.m = g * kGroupM + (r - n * gm);
  c.nb = half ? kBN / 2 : kBN;
  c.x = n * kOutN + (half ? ((i - p.full) & 1) * (kOutN / 2) : 0);
  return c;
}

// The warp's staging buffers and the TMA stores out of them.
template <int kBufs>
struct Stager {
  uint8_t* base;
  int buf;
  int lane;
  // a buffer whose last store has been read out
  __device__ __forceinline__ uint32_t take() {
    if (lane == 0) bulk_wait_group_read<kBufs - 1>();
    __syncwarp();
    return smem_u32(base + buf * kBox);
  }
  __device__ __forceinline__ void store(const CUtensorMap* map, int x, int y, bool in) {
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
      if (in) tma_store_2d(map, base + buf * kBox, x, y);
      bulk_commit_group();
    }
    if (kBufs > 1) buf ^= 1;
  }
  // 32 fp32 columns as two boxes of 16
  __device__ __forceinline__ void store_f32(const CUtensorMap* map, const float (&v)[32], int x, int y, int N,
                                            bool in) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t sb = take();
#pragma unroll
      for (int i = 0; i < 4; ++i)
        st_shared_v4(sb + sw64_offset(lane, i), __float_as_uint(v[16 * h + 4 * i]),
                     __float_as_uint(v[16 * h + 4 * i + 1]), __float_as_uint(v[16 * h + 4 * i + 2]),
                     __float_as_uint(v[16 * h + 4 * i + 3]));
      store(map, x + 16 * h, y, in && x + 16 * h < N);
    }
  }
  __device__ __forceinline__ void store_bf16(const CUtensorMap* map, const float (&v)[32], int x, int y, bool in) {
    const uint32_t sb = take();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      st_shared_v4(sb + sw64_offset(lane, i), pack_bf16x2(v[8 * i], v[8 * i + 1]),
                   pack_bf16x2(v[8 * i + 2], v[8 * i + 3]), pack_bf16x2(v[8 * i + 4], v[8 * i + 5]),
                   pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
    store(map, x, y, in);
  }
};

__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld32(addr, r);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

template <bool kPair, int kBN, int kMode>
__global__ void __launch_bounds__(Epilogue<kMode>::kThreads, 1)
    dense_gemm_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmParams p) {
  using TL = Tile<kPair, kBN>;
  constexpr bool kGated = kMode == kModeGated;
  constexpr bool kBmn = kMode == kModeBackward;
  constexpr int kStages = TL::kStages;
  constexpr int kEpiWarps = Epilogue<kMode>::kWarps, kParts = Epilogue<kMode>::kParts;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * TL::kA;
  uint8_t* sY = sB + kStages * TL::kB;
  uint64_t* full = reinterpret_cast<uint64_t*>(sY + kStaging);  // used in the leader
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;  // [2]
  uint64_t* tempty = tfull + 2;       // [2] used in the leader
  uint64_t* drain = tempty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_status = reinterpret_cast<int*>(s_tmem + 2);  // the bounded waits record here; NaN outputs tell the caller

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kPair ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kEpiWarps * TL::kCtas);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    *s_status = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&maps.a[0]);
    prefetch_tensormap(&maps.b[0]);
    prefetch_tensormap(&maps.y[0]);
  }
  if (warp == 1) {
    if (kPair) {
      tmem_alloc_pair(s_tmem, 2 * kBN);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(s_tmem, 2 * kBN);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();  // both CTAs' barriers exist before any cross-CTA arrival
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  pdl_wait();  // the previous kernel on the stream has completed; its writes are visible
  pdl_trigger();
  const int total = p.tiles;
  const int worker = blockIdx.x / TL::kCtas, nworkers = gridDim.x / TL::kCtas;

  int next = 0;  // where the producer stops: the ring's next stage, its phase
  uint32_t next_ph = 0;
  if (warp == 0) {
    if (!p.stall || rank + 1 < TL::kCtas) {
      // ---------------- TMA producer ----------------
      const bool one = elect_one();
      int stage = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = worker; ok && tile < total; tile += nworkers) {
        const Coord c = tile_coord<kMode, kBN>(p, tile);
        const int num_kb = p.prod[c.prob].num_kb;
        const bool a_mn = kMode == kModeBackward && p.prod[c.prob].a_mn;
        const CUtensorMap* tmA = &maps.a[c.prob];
        const CUtensorMap* tmB = &maps.b[c.prob];
        const int up_row = p.prod[0].N;  // gated: the first up row of B
        const int m0 = (c.m * TL::kCtas + rank) * kTileM;
        const int rows64 = c.nb / TL::kCtas / 64;  // boxes of B in this CTA
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!warp_wait(&empty[stage], ph ^ 1, s_abort, s_status, p.timeout_ns)) {
            ok = false;
            break;
          }
          if (one) {
            if (leader)
              mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(TL::kCtas * TL::kA + c.nb * kBK * 2));
            auto load = [&](uint8_t* dst, const CUtensorMap* map, int x, int y) {
              if (kPair)
                tma_load_2d_pair(dst, map, leader_addr(&full[stage]), x, y);
              else
                tma_load_2d(dst, map, &full[stage], x, y);
            };
            uint8_t* a = sA + stage * TL::kA;
            uint8_t* b = sB + stage * TL::kB;
            const int k0 = kb * kBK;
            if (a_mn) {
              load(a, tmA, m0, k0);
              load(a + 8192, tmA, m0 + 64, k0);
            } else {
              load(a, tmA, k0, m0);
            }
            // B in boxes of 64 of its rows (columns of the output)
#pragma unroll
            for (int j = 0; j < TL::kBRows / 64; ++j) {
              if (j >= rows64) break;
              if (kGated) {
                const int row = kPair ? c.x + rank * up_row + 64 * j
                                      : (j < rows64 / 2 ? c.x + 64 * j : c.x + up_row + 64 * (j - rows64 / 2));
                load(b + j * 8192, tmB, k0, row);
              } else if (kBmn) {
                load(b + j * 8192, tmB, c.x + rank * (c.nb / 2) + 64 * j, k0);
              } else {
                load(b + j * 8192, tmB, k0, c.x + rank * (c.nb / 2) + 64 * j);
              }
            }
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            ph ^= 1;
          }
        }
      }
      next = stage;
      next_ph = ph;
    }
  } else if (warp == 1) {
    if (leader) {
      // ---------------- MMA issuer ----------------
      const bool one = elect_one();
      int stage = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      for (int tile = worker; ok && tile < total; tile += nworkers) {
        if (!warp_wait(&tempty[acc], aph ^ 1, s_abort, s_status, p.timeout_ns)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kBN);
        const Coord c = tile_coord<kMode, kBN>(p, tile);
        const int num_kb = p.prod[c.prob].num_kb;
        const bool a_mn = kMode == kModeBackward && p.prod[c.prob].a_mn;
        const uint32_t idesc = idesc_bf16_f32_major(kTileM * TL::kCtas, c.nb, a_mn, kBmn);
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!warp_wait(&full[stage], ph, s_abort, s_status, p.timeout_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (one) {
            const uint32_t a0 = smem_u32(sA + stage * TL::kA);
            const uint32_t b0 = smem_u32(sB + stage * TL::kB);
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) {
              const uint64_t da = a_mn ? sdesc_mnmajor_sw128(a0 + k * 2048) : sdesc_kmajor_sw128(a0 + k * 32);
              const uint64_t db = kBmn ? sdesc_mnmajor_sw128(b0 + k * 2048) : sdesc_kmajor_sw128(b0 + k * 32);
              if (kPair)
                umma_bf16_pair(d, da, db, idesc, (kb | k) != 0 ? 1u : 0u);
              else
                umma_bf16(d, da, db, idesc, (kb | k) != 0 ? 1u : 0u);
            }
            if (kPair)
              umma_commit_pair_mc(&empty[stage], 0x3);
            else
              umma_commit(&empty[stage]);
            if (kb == num_kb - 1) {
              if (kPair)
                umma_commit_pair_mc(&tfull[acc], 0x3);
              else
                umma_commit(&tfull[acc]);
            }
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        acc ^= 1;
        if (acc == 0) aph ^= 1;
      }
      if (one) {
        if (kPair)
          umma_commit_pair(drain);
        else
          umma_commit(drain);
        int never = 0;
        mbar_wait_bounded(drain, 0, &never, s_status, p.timeout_ns);
      }
    }
  } else {
    // ---------------- epilogue (own 128 rows) ----------------
    // the warps of a lane quadrant take blocks of 32 output columns in turn
    const int quad = warp & 3, part = (warp - 2) >> 2;
    constexpr int kBufs = Epilogue<kMode>::kBufs;
    Stager<kBufs> st{sY + (warp - 2) * kBufs * kBox, 0, lane};
    int acc = 0;
    uint32_t aph = 0;
    int tile = worker;
    for (; tile < total; tile += nworkers) {
      const Coord co = tile_coord<kMode, kBN>(p, tile);
      const int outn = kGated ? co.nb / 2 : co.nb;  // output columns of the tile
      const int M = p.prod[co.prob].M, N = p.prod[co.prob].N;
      const CUtensorMap* tmY = &maps.y[co.prob];
      const int y0 = (co.m * TL::kCtas + rank) * kTileM + quad * 32;
      const bool rows = y0 < M;
      const bool mine = y0 + lane < M;
      // the residual of the first columns is on its way while the tile's MMAs run
      const __nv_bfloat16* res =
          kMode == kModeLinear && p.residual != nullptr && mine ? p.residual + static_cast<size_t>(y0 + lane) * N
                                                                : nullptr;
      uint4 rv[4];
      auto load_res = [&](int x) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          rv[i] = res != nullptr && x + 8 * i < N ? *reinterpret_cast<const uint4*>(res + x + 8 * i)
                                                    : make_uint4(0u, 0u, 0u, 0u);
      };
      if (kMode == kModeLinear) load_res(co.x + 32 * part);
      const bool got = mbar_wait_bounded(&tfull[acc], aph, s_abort, s_status, p.timeout_ns);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(acc * kBN);
#pragma unroll 1
      for (int c = 32 * part; c < outn; c += 32 * kParts) {
        const int x = co.x + c;
        float v[32];
        if (kGated) {
          float u[32];
          tmem_load32(tb + c, v);
          tmem_load32(tb + outn + c, u);
          if (p.save != nullptr) {
            st.store_f32(&maps.save[0], v, x, y0, N, rows);
            st.store_f32(&maps.save[1], u, x, y0, N, rows);
          }
          with_act<false>(p.act, [&](auto tag) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              act2<decltype(tag)::value>(v[i], v[i + 1]);
              v[i] *= u[i];
              v[i + 1] *= u[i + 1];
            }
          });
        } else if (kMode == kModeBackward) {
          tmem_load32(tb + c, v);
        } else {
          tmem_load32(tb + c, v);
          if (p.bias != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (x + 8 * i >= N) continue;
              const uint4 b = __ldg(reinterpret_cast<const uint4*>(p.bias + x + 8 * i));
              const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                v[8 * i + 2 * q] += bf16_lo(w[q]);
                v[8 * i + 2 * q + 1] += bf16_hi(w[q]);
              }
            }
          }
          if (p.save != nullptr) st.store_bf16(&maps.save[0], v, x, y0, rows && x < N);
          if (p.act != kActNone) {
            with_act<false>(p.act, [&](auto tag) {
#pragma unroll
              for (int i = 0; i < 32; i += 2) act2<decltype(tag)::value>(v[i], v[i + 1]);
            });
          }
          if (p.residual != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t w[4] = {rv[i].x, rv[i].y, rv[i].z, rv[i].w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                v[8 * i + 2 * q] += bf16_lo(w[q]);
                v[8 * i + 2 * q + 1] += bf16_hi(w[q]);
              }
            }
            if (c + 32 * kParts < outn) load_res(x + 32 * kParts);
          }
        }
        st.store_bf16(tmY, v, x, y0, rows && x < N);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kPair)
          mbar_arrive_cluster(leader_addr(&tempty[acc]));
        else
          mbar_arrive(&tempty[acc]);
      }
      acc ^= 1;
      if (acc == 0) aph ^= 1;
    }
    // a wait gave up (never in normal operation): mark what this warp did not compute
    for (; tile < total; tile += nworkers) {
      const Coord co = tile_coord<kMode, kBN>(p, tile);
      const int outn = kGated ? co.nb / 2 : co.nb;
      const Product& pr = p.prod[co.prob];
      const int y = (co.m * TL::kCtas + rank) * kTileM + quad * 32 + lane;
      if (y >= pr.M) continue;
      const __nv_bfloat16 nan = __ushort_as_bfloat16(0x7FC0);
      for (int c = 32 * part; c < outn; c += 32 * kParts)
        for (int x = co.x + c; x < min(co.x + c + 32, pr.N); ++x) {
          const size_t at = static_cast<size_t>(y) * pr.N + x;
          pr.out[at] = nan;
          if (kMode == kModeBackward || p.save == nullptr) continue;
          if (kGated) {
            float* gu = static_cast<float*>(p.save) + static_cast<size_t>(y) * pr.N + at;
            gu[0] = gu[pr.N] = __bfloat162float(nan);
          } else {
            static_cast<__nv_bfloat16*>(p.save)[at] = nan;
          }
        }
    }
    if (lane == 0) bulk_wait_group<0>();  // every store of this warp has landed
  }

  const bool gave_up = __syncthreads_or(*s_abort) != 0;
  if (kPair) cluster_sync();  // neither CTA frees TMEM while the pair still uses it
  if (warp == 1) {
    tc_fence_after();
    if (kPair)
      tmem_dealloc_pair(tmem_base, 2 * kBN);
    else
      tmem_dealloc(tmem_base, 2 * kBN);
  }
  if (gave_up) {
    // A wait gave up (never in normal operation), perhaps in a role that waited for loads
    // after the producer had issued its last: no load is issued any more, and those on
    // their way land before the shared memory is given back. In a pair they are counted in
    // the leader. A CTA that did not give up has seen all of both CTAs' loads and may have
    // ended (threads that have do not count in the barrier).
    if (leader && threadIdx.x == 0) drain_loads(full, kStages, next, next_ph, s_status);
    __syncwarp();
    if (kPair) cluster_sync();
  }
}

// The tiles of a last round that would leave half of the workers idle are
// computed in halves of 128 columns, twice as many workers at two thirds of a
// tile's time.
bool halve_last(long long tiles, int workers) {
  const long long rest = tiles % workers;
  return rest > 0 && 2 * rest <= workers;
}

template <bool kPair, int kBN, int kMode>
cudaError_t launch_t(const DenseGemm* g, int n, int num_sms, cudaStream_t st) {
  using TL = Tile<kPair, kBN>;
  constexpr bool kGated = kMode == kModeGated;
  constexpr int kOutN = kGated ? kBN / 2 : kBN;
  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  GemmParams p{};
  GemmMaps maps;
  long long tiles = 0;
  for (int i = 0; i < n; ++i) {
    Product& q = p.prod[i];
    q.M = g[i].M;
    q.N = g[i].N;
    q.num_kb = (g[i].K + kBK - 1) / kBK;
    q.m_tiles = (q.M + kTileM * TL::kCtas - 1) / (kTileM * TL::kCtas);
    q.n_tiles = (q.N + kOutN - 1) / kOutN;
    q.a_mn = g[i].order == kLinearTN;
    q.out = static_cast<__nv_bfloat16*>(g[i].out);
    tiles += static_cast<long long>(q.m_tiles) * q.n_tiles;
    if (tiles >= (1ll << 31)) return cudaErrorInvalidValue;
    if (i == 0) p.first_tiles = static_cast<int>(tiles);
    bool ok = q.a_mn ? encode_tensor_map_2d(&maps.a[i], bf16, 2, g[i].a, g[i].M, g[i].K, 64, kBK)
                     : encode_tensor_map_2d(&maps.a[i], bf16, 2, g[i].a, g[i].K, g[i].M, kBK, kTileM);
    ok = ok && (kMode == kModeBackward
                    ? encode_tensor_map_2d(&maps.b[i], bf16, 2, g[i].b, g[i].N, g[i].K, 64, kBK)
                    : encode_tensor_map_2d(&maps.b[i], bf16, 2, g[i].b, g[i].K,
                                           kGated ? 2 * static_cast<uint64_t>(g[i].N) : g[i].N, kBK, 64));
    ok = ok && encode_tensor_map_2d(&maps.y[i], bf16, 2, g[i].out, g[i].N, g[i].M, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
    if (!ok) return cudaErrorInvalidValue;
  }
  if (n == 1) {
    maps.a[1] = maps.a[0];
    maps.b[1] = maps.b[0];
    maps.y[1] = maps.y[0];
  }
  p.act = g->act;
  p.save = g->save;
  p.stall = stall_gate_up_loads();
  p.bias = static_cast<const __nv_bfloat16*>(g->bias);
  p.residual = static_cast<const __nv_bfloat16*>(g->residual);
  p.timeout_ns = wait_limit_ns();
  maps.save[0] = maps.save[1] = maps.y[0];
  if (p.save != nullptr) {
    for (int i = 0; i < (kGated ? 2 : 1); ++i) {
      const bool encoded =
          kGated ? encode_tensor_map_2d_ld(&maps.save[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
                                           static_cast<float*>(g->save) + static_cast<size_t>(i) * g->N, g->N, g->M,
                                           2 * static_cast<uint64_t>(g->N), 16, 32, CU_TENSOR_MAP_SWIZZLE_64B)
                 : encode_tensor_map_2d(&maps.save[i], bf16, 2, g->save, g->N, g->M, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
      if (!encoded) return cudaErrorInvalidValue;
    }
  }

  auto kernel = dense_gemm_kernel<kPair, kBN, kMode>;
  static unsigned long long done = 0;
  cudaError_t err = ensure_max_smem(reinterpret_cast<const void*>(kernel), &done);
  if (err != cudaSuccess) return err;
  int workers = num_sms / TL::kCtas;
  if (kPair) {
    // every pair of the persistent grid must be resident at once
    const int maxc =
        max_active_clusters(reinterpret_cast<const void*>(kernel), 2, Epilogue<kMode>::kThreads, TL::kSmem);
    if (maxc > 0) workers = std::min(workers, maxc);
  }
  p.full = p.tiles = static_cast<int>(tiles);
  if (kBN == 256 && halve_last(tiles, workers)) {
    p.full -= p.tiles % workers;
    p.tiles += p.tiles % workers;
  }
  workers = std::min(workers, p.tiles);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::max(1, workers) * TL::kCtas));
  cfg.blockDim = dim3(Epilogue<kMode>::kThreads);
  cfg.dynamicSmemBytes = TL::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = TL::kCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kPair ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

// Tile choice: the shape with the least estimated time (K steps x a step + a
// tile's overhead, for the worker with the most tiles). Measured on B200 with
// all SMs at work, a K step of 64 takes 0.34-0.38 us for 256 x 256 on a pair and
// 0.40-0.45 for 128 x 256 (a third more bytes through shared memory), but still
// 0.26-0.29 at 128 columns: there the issuing warp's own path (wait, four MMAs,
// commit: 0.20) and the bytes through shared memory, the same for half the
// products, pace it. So the narrow tiles only pay where they save a wave. The
// sum has 4.2 us for the launch, the first loads and the last tile's end, and two
// thirds of the weights' time from HBM (off by 8% over the sweep of the few-token
// form).
struct Shape {
  int best;
  double us;
};
Shape choose_shape(const DenseGemm* g, int n, int num_sms) {
  const bool gated = g->order == kGatedNT;
  auto cost = [&](int rows, int cols, int workers, double per_step) {
    const int outn = gated ? cols / 2 : cols;
    long long tiles[2] = {0, 0};
    double each[2] = {0, 0};
    for (int i = 0; i < n; ++i) tiles[i] = ((g[i].M + rows - 1ll) / rows) * ((g[i].N + outn - 1ll) / outn);
    if (tiles[0] + tiles[1] <= workers) per_step = cols == 128 ? 0.145 : 0.28;  // one round: nothing shared is full
    for (int i = 0; i < n; ++i) each[i] = (g[i].K + kBK - 1ll) / kBK * per_step + 1.8;
    // worker w has the tiles w, w + workers, ... of the list: the most loaded is
    // worker 0, or the one at which the first product's last round ends
    const long long all = (tiles[0] + tiles[1] + workers - 1) / workers;
    const long long full = std::min(all, (tiles[0] + workers - 1) / workers);
    const double halved = cols == 256 && halve_last(tiles[0] + tiles[1], workers) ? 0.3 * each[n - 1] : 0.0;
    return full * each[0] + (all - full) * each[1] - halved;
  };
  const double c[4] = {cost(256, 256, num_sms / 2, 0.347), cost(256, 128, num_sms / 2, 0.270),
                       cost(128, 256, num_sms, 0.410), cost(128, 128, num_sms, 0.260)};
  Shape s{0, 0};
  for (int i = 1; i < 4; ++i)
    if (c[i] < c[s.best]) s.best = i;
  const double bytes = 2.0 * g->K * (static_cast<double>(g->N) * (gated ? 2 : 1) + (n == 2 ? g->M : 0));
  s.us = 4.2 + c[s.best] + 0.67 * bytes / 6.0e6;
  return s;
}

template <int kMode>
cudaError_t launch_mode(const DenseGemm* g, int n, int num_sms, cudaStream_t st) {
  const int best = choose_shape(g, n, num_sms).best;
  switch (best) {
    case 0:
      return launch_t<true, 256, kMode>(g, n, num_sms, st);
    case 1:
      return launch_t<true, 128, kMode>(g, n, num_sms, st);
    case 2:
      return launch_t<false, 256, kMode>(g, n, num_sms, st);
    default:
      return launch_t<false, 128, kMode>(g, n, num_sms, st);
  }
}

}  // namespace

cudaError_t launch_dense_gemm(const DenseGemm& g, int num_sms, cudaStream_t st) {
  switch (g.order) {
    case kGatedNT:
      return launch_mode<kModeGated>(&g, 1, num_sms, st);
    case kLinearNT:
      return launch_mode<kModeLinear>(&g, 1, num_sms, st);
    default:
      return launch_mode<kModeBackward>(&g, 1, num_sms, st);
  }
}

double dense_gemm_us(const DenseGemm& g, int num_sms) { return choose_shape(&g, 1, num_sms).us; }
double dense_gemm_backward_us(const DenseGemm& dx, const DenseGemm& dw, int num_sms) {
  const DenseGemm g[2] = {dx.K >= dw.K ? dx : dw, dx.K >= dw.K ? dw : dx};
  return choose_shape(g, 2, num_sms).us;
}

cudaError_t launch_dense_gemm_backward(const DenseGemm& dx, const DenseGemm& dw, int num_sms, cudaStream_t st) {
  const DenseGemm g[2] = {dx.K >= dw.K ? dx : dw, dx.K >= dw.K ? dw : dx};  // the longer tiles first
  return launch_mode<kModeBackward>(g, 2, num_sms, st);
}

}  // namespace moe
