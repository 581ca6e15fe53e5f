// BF16 matrix products of a prompt-encoder layer on tcgen05 tensor cores
// (sm_100a), fp32 accumulation in TMEM, and their single-token forms:
//
//   Linear           y  = act(a w^T + b) + res                      MM_LINEAR
//   gate | up        h  = act(x gate^T) * (x up^T)                  MM_GATE
//   its backward     dh = dy down;  dg = dh u act'(g);
//                    du = dh act(g);  h = act(g) u                  MM_DGATE
//   input gradient   dx = dg gate + du up                           MM_LINEAR, two segments of K
//   weight gradients dgate = dg^T x, dup = du^T x, ddown = dy^T h   MM_LINEAR, three products in one launch
//
// Every product is D[M, N] = sum_k A(m, k) B(n, k).  An operand whose rows are
// contiguous in k is K-major; one whose rows are contiguous in m (or n) is
// MN-major, which is how a gradient reads a weight or an activation without a
// transposed copy: TMA brings 64 x 64 boxes with the 128-byte swizzle and the
// instruction descriptor's major bit says how the tensor core walks them.
//
// Warp roles in a 320-thread CTA (one per SM, persistent over tiles): warp 0
// TMA producer, warp 1 TMEM allocator and MMA issuer, warps 2..9 epilogue
// (warp w reads TMEM lanes 32 (w % 4) .. + 31; two warps share a lane quarter
// and alternate 32-column chunks).  The accumulator is double-buffered in
// TMEM, so the epilogue of a tile overlaps the MMAs of the next.  With PAIR
// two CTAs share a 256 x BN tile (cta_group::2): each loads 128 rows of A and
// half the rows of B.  MM_GATE takes half of the B rows from each weight, so
// a tile holds BN / 2 gate columns next to the same up columns and the
// product never leaves the registers; in a pair, each CTA loads one weight.
#include <string.h>

#include <atomic>

#include "qi_common.cuh"
#include "qi_internal.h"
#include "qi_tc.cuh"

namespace qi {

enum MmEpilogue { MM_LINEAR = 0, MM_GATE = 1, MM_DGATE = 2 };

constexpr int MM_THREADS = 320;
constexpr int MM_EPI_WARPS = 8;
constexpr int MM_MAX_PROB = 3;

struct MmMaps {
  CUtensorMap a[MM_MAX_PROB], b[MM_MAX_PROB];
};

struct MmParams {
  int n_prob;                  // products of this launch
  int M[MM_MAX_PROB], N[MM_MAX_PROB];   // N: output columns
  int num_kb[MM_MAX_PROB];     // 64-element K blocks of one segment
  int tiles_end[MM_MAX_PROB];  // running number of tiles
  int group_m[MM_MAX_PROB];    // tile order (tile_coords)
  int segs;                    // 2: operands a[0], b[0], then a[1], b[1], into one sum
  uint16_t* y[MM_MAX_PROB];
  int ldy[MM_MAX_PROB];
  int vec;                     // rows of y and res may be accessed 16 bytes at a time
  const uint16_t* bias;
  const uint16_t* res;
  int ld_res;
  int act;
  uint16_t* gu;                // MM_GATE: optional output, MM_DGATE: input, [M, 2F]
  uint16_t* dg;                // MM_DGATE outputs [M, F]
  uint16_t* du;
  uint16_t* h;
  int* status;
};

template <bool PAIR, int BN>
struct MmCfg {
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_ROWS = PAIR ? BN / 2 : BN;
  static constexpr int B_BYTES = B_ROWS * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN == 32 ? 10 : (BN == 64 ? 8 : 6);
  static constexpr int TMEM_COLS = 2 * BN;
  static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + 256;
  static_assert(2 * STAGES + 6 <= 32, "barrier area");
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

// ---------------------------------------------------------------- activations

// 1 / (1 + e^-x): hardware base-2 exponential and a fast divide (relative
// error about 1e-6, far below the bf16 rounding of what it feeds).
__device__ __forceinline__ float logistic_f(float x) {
  return __fdividef(1.0f, 1.0f + ex2_approx(-1.4426950408889634f * x));
}

__device__ __forceinline__ float act_f(float x, int act) {
  if (act == ACT_SILU) return x * logistic_f(x);
  if (act == ACT_GELU_TANH) return gelu_tanh_f(x);
  return x;
}

// act(x) and act'(x).  SiLU: x s, s (1 + x (1 - s)) with s = logistic(x).
// GELU-tanh, written x s with s = logistic(2z), z = k0 (x + k1 x^3):
// act' = s + x s (1 - s) 2 k0 (1 + 3 k1 x^2).
__device__ __forceinline__ void act_grad_f(float x, int act, float& a, float& da) {
  if (act == ACT_SILU) {
    const float s = logistic_f(x);
    a = x * s;
    da = s * fmaf(x, 1.0f - s, 1.0f);
  } else {
    const float k0 = 0.7978845608028654f, k1 = 0.044715f;
    const float x2 = x * x;
    const float s = logistic_f(2.0f * k0 * fmaf(k1 * x, x2, x));
    a = x * s;
    da = fmaf(x * s * (1.0f - s), 2.0f * k0 * fmaf(3.0f * k1, x2, 1.0f), s);
  }
}

// ---------------------------------------------------------------- row access

// 32 bf16 values (16 packed words) to dst; ncols < 32 at the right edge.
// Without vec (rows not 16-byte aligned) and in a group of 8 columns that the
// edge cuts, one value at a time.
__device__ __forceinline__ void store_row32(uint16_t* dst, const uint32_t (&pk)[16], int ncols,
                                            bool vec) {
  if (vec && ncols == 32) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      reinterpret_cast<uint4*>(dst)[j] = make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (2 * i < ncols) dst[2 * i] = static_cast<uint16_t>(pk[i]);
    if (2 * i + 1 < ncols) dst[2 * i + 1] = static_cast<uint16_t>(pk[i] >> 16);
  }
}

__device__ __forceinline__ void load_row32(const uint16_t* src, uint32_t (&pk)[16], int ncols,
                                           bool vec) {
  if (vec && ncols == 32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 v = *(reinterpret_cast<const uint4*>(src) + j);
      pk[4 * j] = v.x;
      pk[4 * j + 1] = v.y;
      pk[4 * j + 2] = v.z;
      pk[4 * j + 3] = v.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t lo = 2 * i < ncols ? src[2 * i] : 0u;
    const uint32_t hi = 2 * i + 1 < ncols ? src[2 * i + 1] : 0u;
    pk[i] = lo | (hi << 16);
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <bool PAIR>
__device__ __forceinline__ void mm_tempty_signal(uint32_t addr) {
  if (PAIR)
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
  else
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(addr) : "memory");
}

// ---------------------------------------------------------------- epilogue

// One accumulator tile: rows m0 .. m0 + 127 of this CTA, output columns from
// n0.  Signals the accumulator buffer free after this warp's last TMEM read.
template <bool PAIR, int BN, int EPI>
__device__ __forceinline__ void mm_epilogue(const MmParams& p, int pr, uint32_t tacc, int m0, int n0,
                                            int quarter, int half, int lane, uint32_t tempty_addr) {
  constexpr int W = EPI == MM_GATE ? BN / 2 : BN;   // output columns of a tile
  constexpr int CH = W / 32;
  const int m = m0 + quarter * 32 + lane;
  const int N = p.N[pr];
  const bool row_ok = m < p.M[pr];
  const bool vec = p.vec != 0;
  const uint32_t t_row = tacc + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
  for (int c = half; c < CH; c += 2) {
    __syncwarp();
    uint32_t r[32];
    tmem_ld32(t_row + c * 32, r);
    uint32_t r2[EPI == MM_GATE ? 32 : 1];
    if constexpr (EPI == MM_GATE) tmem_ld32(t_row + W + c * 32, r2);
    if (c + 2 >= CH) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mm_tempty_signal<PAIR>(tempty_addr);
    }
    const int nb = n0 + c * 32;
    if (!row_ok || nb >= N) continue;
    const int ncols = min(32, N - nb);
    if constexpr (EPI == MM_LINEAR) {
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
      if (p.bias) {
        uint32_t b[16];
        load_row32(p.bias + nb, b, ncols, true);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          v[2 * i] += bf16_lo(b[i]);
          v[2 * i + 1] += bf16_hi(b[i]);
        }
      }
      if (p.act == ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = act_f(v[i], ACT_SILU);
      } else if (p.act == ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = act_f(v[i], ACT_GELU_TANH);
      }
      if (p.res) {
        uint32_t b[16];
        load_row32(p.res + static_cast<size_t>(m) * p.ld_res + nb, b, ncols, vec);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          v[2 * i] += bf16_lo(b[i]);
          v[2 * i + 1] += bf16_hi(b[i]);
        }
      }
      uint32_t pk[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      store_row32(p.y[pr] + static_cast<size_t>(m) * p.ldy[pr] + nb, pk, ncols, vec);
    } else if constexpr (EPI == MM_GATE) {
      // the activation and the product in fp32, rounded once (F % 8 == 0: rows are 16-byte aligned)
      uint32_t pk[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float a0 = act_f(__uint_as_float(r[2 * i]), p.act);
        const float a1 = act_f(__uint_as_float(r[2 * i + 1]), p.act);
        pk[i] = pack_bf16x2(a0 * __uint_as_float(r2[2 * i]), a1 * __uint_as_float(r2[2 * i + 1]));
      }
      store_row32(p.y[0] + static_cast<size_t>(m) * N + nb, pk, ncols, true);
      if (p.gu) {
        uint16_t* row = p.gu + static_cast<size_t>(m) * 2 * N + nb;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          pk[i] = pack_bf16x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        store_row32(row, pk, ncols, true);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          pk[i] = pack_bf16x2(__uint_as_float(r2[2 * i]), __uint_as_float(r2[2 * i + 1]));
        store_row32(row + N, pk, ncols, true);
      }
    } else {
      uint32_t g[16], u[16], h[16];
      const uint16_t* row = p.gu + static_cast<size_t>(m) * 2 * N + nb;
      load_row32(row, g, ncols, true);
      load_row32(row + N, u, ncols, true);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float d0 = __uint_as_float(r[2 * i]), d1 = __uint_as_float(r[2 * i + 1]);
        const float u0 = bf16_lo(u[i]), u1 = bf16_hi(u[i]);
        float a0, a1, e0, e1;
        act_grad_f(bf16_lo(g[i]), p.act, a0, e0);
        act_grad_f(bf16_hi(g[i]), p.act, a1, e1);
        h[i] = pack_bf16x2(a0 * u0, a1 * u1);
        g[i] = pack_bf16x2(d0 * u0 * e0, d1 * u1 * e1);
        u[i] = pack_bf16x2(d0 * a0, d1 * a1);
      }
      const size_t at = static_cast<size_t>(m) * N + nb;
      store_row32(p.dg + at, g, ncols, true);
      store_row32(p.du + at, u, ncols, true);
      if (p.h) store_row32(p.h + at, h, ncols, true);
    }
  }
  if (half >= CH) {   // narrow tiles: no chunk for this warp
    __syncwarp();
    if (lane == 0) mm_tempty_signal<PAIR>(tempty_addr);
  }
}

// Product and tile coordinates of a tile number.
template <bool PAIR, int BN, int EPI>
__device__ __forceinline__ void mm_tile(const MmParams& p, int tile, int& pr, int& mt, int& nt) {
  constexpr int BM = PAIR ? 256 : 128;
  constexpr int W = EPI == MM_GATE ? BN / 2 : BN;
  pr = 0;
  while (pr < p.n_prob - 1 && tile >= p.tiles_end[pr]) ++pr;
  if (pr > 0) tile -= p.tiles_end[pr - 1];
  tile_coords(tile, (p.M[pr] + BM - 1) / BM, p.group_m[pr], (p.N[pr] + W - 1) / W, mt, nt);
}

// ---------------------------------------------------------------- kernel

template <bool PAIR, int BN, bool AMN, bool BMN, int EPI>
__global__ void __launch_bounds__(MM_THREADS, 1)
    mm_kernel(const __grid_constant__ MmMaps maps, const __grid_constant__ MmParams p) {
  using C = MmCfg<PAIR, BN>;
  constexpr int STAGES = C::STAGES;
  constexpr int W = EPI == MM_GATE ? BN / 2 : BN;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * C::A_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE_BYTES);
  uint64_t* full = bars;                     // [STAGES] (pair: even CTA's)
  uint64_t* empty = bars + STAGES;           // [STAGES]
  uint64_t* tfull = bars + 2 * STAGES;       // [2]
  uint64_t* tempty = bars + 2 * STAGES + 2;  // [2] (pair: even CTA's)
  uint64_t* drain = bars + 2 * STAGES + 4;   // MMA drain on the error path
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_rank()) : 0;
  const int worker = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  const int workers = PAIR ? gridDim.x >> 1 : gridDim.x;
  const int num_tiles = p.tiles_end[p.n_prob - 1];

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], (PAIR ? 2 : 1) * MM_EPI_WARPS);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&maps.a[0]);
    prefetch_tmap(&maps.b[0]);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (PAIR) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    // ------------------------------------------------------------ producer (the whole warp, one lane issues)
    {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = worker; tile < num_tiles && ok; tile += workers) {
        int pr, mt, nt;
        mm_tile<PAIR, BN, EPI>(p, tile, pr, mt, nt);
        const int m0 = mt * (PAIR ? 256 : 128) + rank * 128;
        const int num_kb = p.num_kb[pr];
        for (int seg = 0; seg < p.segs && ok; ++seg) {   // segs == 2 only for a single product
          const CUtensorMap* ma = &maps.a[pr + seg];
          const CUtensorMap* mb = &maps.b[EPI == MM_GATE ? rank : pr + seg];
          for (int kb = 0; kb < num_kb; ++kb) {
            if (!mbar_wait_warp(&empty[stage], phase ^ 1u, p.status)) { ok = false; break; }
            const int k = kb * 64;
            uint8_t* da = sA + stage * C::A_BYTES;
            uint8_t* db = sB + stage * C::B_BYTES;
            const uint32_t fb = PAIR ? mapa_shared(smem_u32(&full[stage]), 0) : smem_u32(&full[stage]);
            if (rank == 0) mbar_expect_elect(&full[stage], (PAIR ? 2 : 1) * C::STAGE_BYTES);
            if (AMN) {
#pragma unroll
              for (int i = 0; i < 2; ++i) tma_load_2d_elect<PAIR>(ma, fb, da + i * 8192, m0 + 64 * i, k);
            } else {
              tma_load_2d_elect<PAIR>(ma, fb, da, k, m0);
            }
            if (EPI == MM_GATE) {
              tma_load_2d_elect<PAIR>(mb, fb, db, k, nt * W);
              if (!PAIR) tma_load_2d_elect<PAIR>(&maps.b[1], fb, db + C::B_BYTES / 2, k, nt * W);
            } else if (BMN) {
#pragma unroll
              for (int i = 0; i < C::B_ROWS / 64; ++i)
                tma_load_2d_elect<PAIR>(mb, fb, db + i * 8192, nt * BN + rank * C::B_ROWS + 64 * i, k);
            } else {
              tma_load_2d_elect<PAIR>(mb, fb, db, k, nt * BN + rank * C::B_ROWS);
            }
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          }
        }
      }
      if (!ok) {
        // Error path: the loads in flight must land before the CTA exits.  The
        // CTA that armed the full barriers waits (bounded) on them; the odd CTA
        // of a pair, which cannot, gives its last loads a fixed 200 us.
        if (rank == 0) {
          for (int s = 0; s < STAGES; ++s) {
            const uint32_t par = (s < stage) ? phase : (phase ^ 1u);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&full[s], par) && globaltimer_ns() - t0 < QI_WAIT_NS) {
            }
          }
        } else {
          const uint64_t t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < 200000ull) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (pair: even CTA)
    // The whole warp runs the loop and one elected lane issues: operands that
    // are uniform over a converged warp reach the tensor core's instruction
    // without a move per lane (an MMA issued under a lane test took 54 clocks).
    if (rank == 0) {
      constexpr uint32_t idesc = umma_idesc(false, PAIR ? 256 : 128, BN) | (AMN ? (1u << 15) : 0u) |
                                 (BMN ? (1u << 16) : 0u);
      const uint64_t adesc0 = AMN ? umma_desc_mnmajor_sw128(smem_u32(sA), 8192) : umma_desc_kmajor_sw128(smem_u32(sA));
      const uint64_t bdesc0 = BMN ? umma_desc_mnmajor_sw128(smem_u32(sB), 8192) : umma_desc_kmajor_sw128(smem_u32(sB));
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int tile = worker; tile < num_tiles && ok; tile += workers) {
        int pr, mt, nt;
        mm_tile<PAIR, BN, EPI>(p, tile, pr, mt, nt);
        const int total_kb = p.num_kb[pr] * p.segs;
        const bool free = PAIR ? mbar_wait_cluster(&tempty[acc], acc_phase ^ 1u, p.status)
                               : mbar_wait(&tempty[acc], acc_phase ^ 1u, p.status);
        if (!__all_sync(0xffffffffu, free)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int kb = 0; kb < total_kb; ++kb) {
          if (!mbar_wait_warp(&full[stage], phase, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint64_t adesc = adesc0 + static_cast<uint64_t>(stage * (C::A_BYTES >> 4));
          const uint64_t bdesc = bdesc0 + static_cast<uint64_t>(stage * (C::B_BYTES >> 4));
#pragma unroll
          for (int k = 0; k < 4; ++k) {   // 16 values of K per instruction: 32 bytes of a K-major row, 16 MN-major rows
            const uint64_t ao = static_cast<uint64_t>(k * (AMN ? 2048 : 32)) >> 4;
            const uint64_t bo = static_cast<uint64_t>(k * (BMN ? 2048 : 32)) >> 4;
            umma_f16_elect<PAIR>(d_tmem, adesc + ao, bdesc + bo, idesc, (kb | k) != 0);
          }
          umma_commit_elect<PAIR>(&empty[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        umma_commit_elect<PAIR>(&tfull[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok) {
        // make sure no MMA is still writing TMEM before it is released
        if (PAIR) umma_commit_elect<true>(drain, 0x1);
        else umma_commit_elect<false>(drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < QI_WAIT_NS) {
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int tile = worker; tile < num_tiles; tile += workers) {
      int pr, mt, nt;
      mm_tile<PAIR, BN, EPI>(p, tile, pr, mt, nt);
      const int m0 = mt * (PAIR ? 256 : 128) + rank * 128;
      if (!mbar_wait_warp(&tfull[acc], acc_phase, p.status)) break;
      tc_fence_after();
      const uint32_t te = PAIR ? mapa_shared(smem_u32(&tempty[acc]), 0) : smem_u32(&tempty[acc]);
      mm_epilogue<PAIR, BN, EPI>(p, pr, tmem_base + static_cast<uint32_t>(acc * BN), m0, nt * W,
                                 quarter, half, lane, te);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }

  // Neither CTA of a pair leaves (or frees TMEM) while the other may still read
  // its shared memory, arrive on its barriers, or have MMAs writing its TMEM.
  tc_fence_before();
  if (PAIR) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- few rows
//
// M <= 16 rows: the product is bound by reading the weights once, so the
// weights go straight from memory into the fragments of warp-level MMAs
// (m16n8k16: 16 weight rows against 8 rows of a), with no staging and no
// 128-row tile that would be almost empty.  A thread's fragment of a 32-wide
// step of K is one 16-byte load per row: the four threads of a row take 8
// consecutive k each, and both operands use that same order of k, which a sum
// over k does not notice.  The 8 warps of a CTA share 16 output columns (and,
// with GATE, the same 16 of the second weight) and take 64-wide pieces of K
// in turn; their partial sums are added in shared memory in a fixed order.
constexpr int SK_THREADS = 256;

struct SkinnyParams {
  const uint16_t* a;
  int M, K, N, lda;
  const uint16_t* w;
  const uint16_t* w2;     // GATE: the up weight
  const uint16_t* bias;
  int act;
  const uint16_t* res;
  int ld_res;
  uint16_t* y;
  int ldy;
  uint16_t* gu;           // GATE: optional [M, 2N]
};

template <int NT, bool GATE>
__global__ void __launch_bounds__(SK_THREADS) skinny_kernel(const SkinnyParams p) {
  constexpr int MATS = GATE ? 2 : 1;
  __shared__ float red[SK_THREADS / 32][MATS][NT * 8][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16;
  const int r0 = min(n0 + g, p.N - 1), r1 = min(n0 + g + 8, p.N - 1);   // rows past N: not stored
  float acc[MATS][NT][4];
#pragma unroll
  for (int i = 0; i < MATS; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
  pdl_wait();
  pdl_trigger();
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint16_t* wr[MATS][2];
  wr[0][0] = p.w + static_cast<size_t>(r0) * p.K;
  wr[0][1] = p.w + static_cast<size_t>(r1) * p.K;
  if (GATE) {
    wr[MATS - 1][0] = p.w2 + static_cast<size_t>(r0) * p.K;
    wr[MATS - 1][1] = p.w2 + static_cast<size_t>(r1) * p.K;
  }
  const uint16_t* ar[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) ar[j] = p.a + static_cast<size_t>(min(8 * j + g, p.M - 1)) * p.lda;
#pragma unroll 4
  for (int kb = warp * 64; kb < p.K; kb += SK_THREADS / 32 * 64) {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const int k = kb + 32 * sub + 8 * t;   // K % 8 == 0: a chunk of 8 lies inside or outside
      const bool in = k < p.K;
      uint4 w[MATS][2], x[NT];
#pragma unroll
      for (int i = 0; i < MATS; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) w[i][e] = in ? __ldg(reinterpret_cast<const uint4*>(wr[i][e] + k)) : zero;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        x[j] = in && 8 * j + g < p.M ? *reinterpret_cast<const uint4*>(ar[j] + k) : zero;
#pragma unroll
      for (int i = 0; i < MATS; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma_16816(acc[i][j], w[i][0].x, w[i][1].x, w[i][0].y, w[i][1].y, x[j].x, x[j].y);
          mma_16816(acc[i][j], w[i][0].z, w[i][1].z, w[i][0].w, w[i][1].w, x[j].z, x[j].w);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < MATS; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[warp][i][8 * j + 2 * t + (e & 1)][g + (e & 2) * 4] = acc[i][j][e];
  __syncthreads();
  for (int idx = threadIdx.x; idx < NT * 8 * 16; idx += SK_THREADS) {
    const int r = idx & 15, m = idx >> 4, n = n0 + r;
    if (m >= p.M || n >= p.N) continue;
    float v = 0.f, v2 = 0.f;
#pragma unroll
    for (int s = 0; s < SK_THREADS / 32; ++s) {
      v += red[s][0][m][r];
      if (GATE) v2 += red[s][MATS - 1][m][r];
    }
    if (GATE) {
      if (p.gu) {
        uint16_t* row = p.gu + static_cast<size_t>(m) * 2 * p.N + n;
        row[0] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
        row[p.N] = static_cast<uint16_t>(pack_bf16x2(v2, 0.f));
      }
      v = act_f(v, p.act) * v2;
    } else {
      if (p.bias) v += bf16_bits_to_float(p.bias[n]);
      v = act_f(v, p.act);
      if (p.res) v += bf16_bits_to_float(p.res[static_cast<size_t>(m) * p.ld_res + n]);
    }
    p.y[static_cast<size_t>(m) * p.ldy + n] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
  }
}

// ---------------------------------------------------------------- host side

// Largest dynamic shared memory of a kernel, set once per device.
template <class K>
static bool allow_smem(K kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_release);
  return true;
}

struct MmOperand {
  const void* base;
  int rows, cols, ld;    // row-major [rows, cols]
};

// Operand map: K-major boxes of 64 (k) x box_rows, MN-major boxes of 64 x 64 (k).
static bool mm_map(CUtensorMap* m, const MmOperand& o, bool mn, int box_rows) {
  return make_tmap_2d(m, o.base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<uint64_t>(o.cols),
                      static_cast<uint64_t>(o.rows), static_cast<uint64_t>(o.ld) * 2, 64,
                      static_cast<uint32_t>(mn ? 64 : box_rows));
}

template <bool PAIR, int BN, bool AMN, bool BMN, int EPI>
static int mm_launch(const MmOperand* A, const MmOperand* B, int n_ops_a, int n_ops_b, MmParams p,
                     int num_sms, cudaStream_t st) {
  using C = MmCfg<PAIR, BN>;
  auto kern = mm_kernel<PAIR, BN, AMN, BMN, EPI>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kern, C::SMEM, done)) {
    launch_result();
    return -1;
  }
  MmMaps maps;
  for (int i = 0; i < MM_MAX_PROB; ++i) {
    if (!mm_map(&maps.a[i], A[i < n_ops_a ? i : 0], AMN, 128)) return -2;
    if (!mm_map(&maps.b[i], B[i < n_ops_b ? i : 0], BMN, EPI == MM_GATE ? BN / 2 : C::B_ROWS)) return -2;
  }
  constexpr int BM = PAIR ? 256 : 128;
  constexpr int W = EPI == MM_GATE ? BN / 2 : BN;
  int tiles = 0;
  for (int i = 0; i < p.n_prob; ++i) {
    const int mt = (p.M[i] + BM - 1) / BM;
    tiles += mt * ((p.N[i] + W - 1) / W);
    p.tiles_end[i] = tiles;
    p.group_m[i] = mt < 8 ? mt : 8;
  }
  const int cap = PAIR ? num_sms / 2 : num_sms;
  const int workers = tiles < cap ? tiles : cap;
  launch_pdl(kern, dim3(PAIR ? 2 * workers : workers), dim3(MM_THREADS), C::SMEM, st, PAIR ? 2 : 1,
             maps, p);
  return launch_result();
}

// Tile shape of a launch: the one whose rounds of tiles cost least.  A 64-wide
// K block takes a CTA about 512 clocks in a pair's 256 x 256 tile (the tensor
// pipe) and is bound by the operand bytes an SM can take in (about 64 a clock)
// in the narrower tiles of one CTA.
enum MmShape { MM_PAIR256 = 0, MM_S128 = 1, MM_S64 = 2, MM_S32 = 3 };
static MmShape mm_shape(const MmParams& p, int w_div, int num_sms, int narrowest) {
  static const int bm[4] = {256, 128, 128, 128}, bn[4] = {256, 128, 64, 32};
  static const int clocks[4] = {512, 512, 384, 320};
  long best = 0;
  int pick = 0;
  for (int s = 0; s <= narrowest; ++s) {
    long tiles = 0, kb = 0;
    for (int i = 0; i < p.n_prob; ++i) {
      const int w = bn[s] / w_div;
      tiles += static_cast<long>((p.M[i] + bm[s] - 1) / bm[s]) * ((p.N[i] + w - 1) / w);
      kb = kb > p.num_kb[i] * p.segs ? kb : p.num_kb[i] * p.segs;
    }
    const long cap = s == MM_PAIR256 ? num_sms / 2 : num_sms;
    const long cost = ((tiles + cap - 1) / cap) * kb * clocks[s];
    if (s == 0 || cost < best) {
      best = cost;
      pick = s;
    }
  }
  return static_cast<MmShape>(pick);
}

static MmParams mm_params(int* status) {
  MmParams p;
  memset(&p, 0, sizeof(p));
  p.n_prob = 1;
  p.segs = 1;
  p.vec = 1;
  p.status = status;
  return p;
}

constexpr int SK_MAX_ROWS = 16;

template <bool GATE>
static int launch_skinny(const SkinnyParams& s, cudaStream_t st) {
  const dim3 grid((s.N + 15) / 16);
  if (s.M <= 8) launch_pdl(skinny_kernel<1, GATE>, grid, dim3(SK_THREADS), 0, st, 1, s);
  else launch_pdl(skinny_kernel<2, GATE>, grid, dim3(SK_THREADS), 0, st, 1, s);
  return launch_result();
}

static bool rows16(const void* p, int ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0;
}

int launch_linear_act(const LinearActParams& q, cudaStream_t st) {
  if (q.M <= SK_MAX_ROWS) {
    SkinnyParams s;
    memset(&s, 0, sizeof(s));
    s.a = q.a; s.M = q.M; s.K = q.K; s.N = q.N; s.lda = q.lda;
    s.w = q.w; s.bias = q.bias; s.act = q.act; s.res = q.res; s.ld_res = q.ld_res;
    s.y = q.y; s.ldy = q.ldy;
    return launch_skinny<false>(s, st);
  }
  MmParams p = mm_params(q.status);
  p.M[0] = q.M;
  p.N[0] = q.N;
  p.num_kb[0] = (q.K + 63) / 64;
  p.y[0] = q.y;
  p.ldy[0] = q.ldy;
  p.bias = q.bias;
  p.act = q.act;
  p.res = q.res;
  p.ld_res = q.ld_res;
  p.vec = rows16(q.y, q.ldy) && (!q.res || rows16(q.res, q.ld_res));
  const MmOperand a{q.a, q.M, q.K, q.lda}, b{q.w, q.N, q.K, q.K};
  switch (mm_shape(p, 1, q.num_sms, MM_S32)) {
    case MM_PAIR256: return mm_launch<true, 256, false, false, MM_LINEAR>(&a, &b, 1, 1, p, q.num_sms, st);
    case MM_S128: return mm_launch<false, 128, false, false, MM_LINEAR>(&a, &b, 1, 1, p, q.num_sms, st);
    case MM_S64: return mm_launch<false, 64, false, false, MM_LINEAR>(&a, &b, 1, 1, p, q.num_sms, st);
    case MM_S32: return mm_launch<false, 32, false, false, MM_LINEAR>(&a, &b, 1, 1, p, q.num_sms, st);
  }
  return -1;
}

int launch_gate_up(const GateUpParams& q, cudaStream_t st) {
  if (q.M <= SK_MAX_ROWS) {
    SkinnyParams s;
    memset(&s, 0, sizeof(s));
    s.a = q.x; s.M = q.M; s.K = q.H; s.N = q.F; s.lda = q.ldx;
    s.w = q.gate; s.w2 = q.up; s.act = q.act; s.y = q.h; s.ldy = q.F; s.gu = q.gu;
    return launch_skinny<true>(s, st);
  }
  MmParams p = mm_params(q.status);
  p.M[0] = q.M;
  p.N[0] = q.F;
  p.num_kb[0] = (q.H + 63) / 64;
  p.y[0] = q.h;
  p.act = q.act;
  p.gu = q.gu;
  const MmOperand a{q.x, q.M, q.H, q.ldx};
  const MmOperand b[2] = {{q.gate, q.F, q.H, q.H}, {q.up, q.F, q.H, q.H}};
  switch (mm_shape(p, 2, q.num_sms, MM_S64)) {
    case MM_PAIR256: return mm_launch<true, 256, false, false, MM_GATE>(&a, b, 1, 2, p, q.num_sms, st);
    case MM_S128: return mm_launch<false, 128, false, false, MM_GATE>(&a, b, 1, 2, p, q.num_sms, st);
    case MM_S64: return mm_launch<false, 64, false, false, MM_GATE>(&a, b, 1, 2, p, q.num_sms, st);
    default: return -1;
  }
}

int launch_gated_dh(const GatedBackwardParams& q, cudaStream_t st) {
  MmParams p = mm_params(q.status);
  p.M[0] = q.M;
  p.N[0] = q.F;
  p.num_kb[0] = (q.H + 63) / 64;
  p.act = q.act;
  p.gu = const_cast<uint16_t*>(q.gu);
  p.dg = q.dg;
  p.du = q.du;
  p.h = q.ddown ? q.h : nullptr;
  const MmOperand a{q.dy, q.M, q.H, q.ld_dy}, b{q.down, q.H, q.F, q.F};
  switch (mm_shape(p, 1, q.num_sms, MM_S64)) {
    case MM_PAIR256: return mm_launch<true, 256, false, true, MM_DGATE>(&a, &b, 1, 1, p, q.num_sms, st);
    case MM_S128: return mm_launch<false, 128, false, true, MM_DGATE>(&a, &b, 1, 1, p, q.num_sms, st);
    case MM_S64: return mm_launch<false, 64, false, true, MM_DGATE>(&a, &b, 1, 1, p, q.num_sms, st);
    default: return -1;
  }
}

int launch_gated_dx(const GatedBackwardParams& q, cudaStream_t st) {
  MmParams p = mm_params(q.status);
  p.M[0] = q.M;
  p.N[0] = q.H;
  p.num_kb[0] = (q.F + 63) / 64;
  p.segs = 2;
  p.y[0] = q.dx;
  p.ldy[0] = q.ld_dx;
  const MmOperand a[2] = {{q.dg, q.M, q.F, q.F}, {q.du, q.M, q.F, q.F}};
  const MmOperand b[2] = {{q.gate, q.F, q.H, q.H}, {q.up, q.F, q.H, q.H}};
  switch (mm_shape(p, 1, q.num_sms, MM_S64)) {
    case MM_PAIR256: return mm_launch<true, 256, false, true, MM_LINEAR>(a, b, 2, 2, p, q.num_sms, st);
    case MM_S128: return mm_launch<false, 128, false, true, MM_LINEAR>(a, b, 2, 2, p, q.num_sms, st);
    case MM_S64: return mm_launch<false, 64, false, true, MM_LINEAR>(a, b, 2, 2, p, q.num_sms, st);
    default: return -1;
  }
}

int launch_gated_dw(const GatedBackwardParams& q, cudaStream_t st) {
  MmParams p = mm_params(q.status);
  MmOperand a[MM_MAX_PROB], b[MM_MAX_PROB];
  int n = 0;
  auto add = [&](const MmOperand& A, const MmOperand& B, uint16_t* y) {
    if (!y) return;
    a[n] = A;
    b[n] = B;
    p.M[n] = A.cols;
    p.N[n] = B.cols;
    p.num_kb[n] = (q.M + 63) / 64;
    p.y[n] = y;
    p.ldy[n] = B.cols;
    ++n;
  };
  const MmOperand x{q.x, q.M, q.H, q.ldx};
  add({q.dg, q.M, q.F, q.F}, x, q.dgate);
  add({q.du, q.M, q.F, q.F}, x, q.dup);
  add({q.dy, q.M, q.H, q.ld_dy}, {q.h, q.M, q.F, q.F}, q.ddown);
  if (n == 0) return 0;
  p.n_prob = n;
  switch (mm_shape(p, 1, q.num_sms, MM_S128)) {
    case MM_PAIR256: return mm_launch<true, 256, true, true, MM_LINEAR>(a, b, n, n, p, q.num_sms, st);
    case MM_S128: return mm_launch<false, 128, true, true, MM_LINEAR>(a, b, n, n, p, q.num_sms, st);
    default: return -1;
  }
}

}  // namespace qi
