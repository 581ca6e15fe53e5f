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
// Warp roles in a 320-thread CTA: warp 0 TMA producer, warp 1 TMEM allocator
// and MMA issuer, warps 2..9 epilogue (warp w reads TMEM lanes 32 (w % 4) .. +
// 31; two warps share a lane quarter).  Large products run on persistent CTA
// pairs with 256 x 256 tiles (mm_kernel), or with K shared by a cluster when
// the tiles are few (mm_split_kernel); some hundreds of rows as the narrow
// operand next to 128 rows of the weights (mm_rows_kernel); a few rows on
// warp-level MMAs that stream the weights (skinny_kernel).  MM_GATE takes half
// of the weight rows of a tile from each weight, so a tile holds gate columns
// next to the same up columns and their product never leaves the SM; in a
// pair, each CTA loads one weight.
#include <string.h>

#include <algorithm>
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
  // persistent kernel, boxes of 32 rows x 32 columns: the outputs (MM_DGATE: dg,
  // du, h) and the residual (bf16) or gate | up (fp32)
  CUtensorMap y[MM_MAX_PROB], x;
};

struct MmParams {
  int n_prob;                  // products of this launch
  int M[MM_MAX_PROB], N[MM_MAX_PROB];   // N: output columns
  int num_kb[MM_MAX_PROB];     // 64-element K blocks of one segment
  int tiles_end[MM_MAX_PROB];  // running number of tiles
  int group_m[MM_MAX_PROB];    // tile order (tile_coords)
  int bn;                      // persistent kernel, K-major B: columns of a pair's tile (256, 192 or 128)
  int segs;                    // 2: operands a[0], b[0], then a[1], b[1], into one sum
  uint16_t* y[MM_MAX_PROB];    // MM_DGATE: dg, du and, unless null, h, each [M, F]
  int ldy[MM_MAX_PROB];
  int vec;                     // rows of y and res may be accessed 16 bytes at a time
  const uint16_t* bias;
  const uint16_t* res;
  int ld_res;
  int act;
  float* gu;                   // MM_GATE: optional output, MM_DGATE: input, [M, 2F]
  int* status;
};

constexpr int MM_TILE = 128 * 128;   // bytes of a stage's A or B tile of one CTA: 128 x 64 bf16
constexpr int MM_BN = 256;           // most columns of a pair's tile
constexpr int MM_STAGES = 6;
constexpr int MM_OUT = 32 * 64;      // bytes of an epilogue chunk of 32 rows x 32 bf16 columns
// Persistent kernel: stages of the operands, and chunks of shared memory per
// epilogue warp (an fp32 chunk takes two; MM_DGATE holds gate and up at once).
template <int EPI>
struct MmCfg {
  static constexpr int STAGES = EPI == MM_DGATE ? 5 : MM_STAGES;
  static constexpr int CHUNKS = EPI == MM_DGATE ? 4 : 2;
  static constexpr int SMEM = 1024 + STAGES * 2 * MM_TILE + MM_EPI_WARPS * CHUNKS * MM_OUT + 256;
  static_assert(2 * STAGES + 6 + MM_EPI_WARPS <= 32, "barrier area");
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

// Execution barrier of a cluster that orders no memory, for the end of a kernel
// whose CTAs have no access to each other's shared memory left on its way: every
// remote load has its value, every remote arrival (of a thread or of a commit)
// has been waited for by the CTA it goes to.  (A releasing arrive would wait for
// this CTA's output stores too, 0.3 us.)
__device__ __forceinline__ void cluster_sync_end() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
  __syncwarp();
}

// Before it ends, a producer waits for the commits that free its last stages:
// those of a pair arrive from the other CTA, and where the MMA warp gave up the
// loads may still be on their way.  (They precede the commit that ends the
// sums, so this takes no time.)
__device__ __forceinline__ bool mm_stages_free(uint64_t* empty, int stages, int stage, uint32_t phase, int* status) {
#pragma unroll 1
  for (int i = 0; i < stages; ++i) {
    if (!mbar_wait_warp(&empty[stage], phase ^ 1u, status)) return false;
    if (++stage == stages) { stage = 0; phase ^= 1u; }
  }
  return true;
}

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
// act' = s + x s (1 - s) 2 k0 (1 + 3 k1 x^2); s (1 - s) is 0 long before |x| = 100,
// and x^2 stops there, so that the product is 0 where x^2 would be infinite.
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
    da = fmaf(x * s * (1.0f - s), 2.0f * k0 * fmaf(3.0f * k1, fminf(x2, 1e4f), 1.0f), s);
  }
}

// ---------------------------------------------------------------- row access

// 8 bf16 values (4 packed words) to dst; ncols < 8 at the right edge.  Without
// vec (rows not 16-byte aligned) or at the edge, one value at a time.
__device__ __forceinline__ void store8(uint16_t* dst, const uint32_t (&pk)[4], int ncols, bool vec) {
  if (vec && ncols >= 8) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < ncols) dst[i] = static_cast<uint16_t>(pk[i >> 1] >> (16 * (i & 1)));
}

__device__ __forceinline__ void load8(const uint16_t* src, uint32_t (&pk)[4], int ncols, bool vec) {
  if (vec && ncols >= 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(src);
    pk[0] = v.x;
    pk[1] = v.y;
    pk[2] = v.z;
    pk[3] = v.w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = 2 * i < ncols ? src[2 * i] : 0u;
    const uint32_t hi = 2 * i + 1 < ncols ? src[2 * i + 1] : 0u;
    pk[i] = lo | (hi << 16);
  }
}

// 8 fp32 values, 16-byte aligned.
__device__ __forceinline__ void load8f(const float* src, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 x = reinterpret_cast<const float4*>(src)[i];
    v[4 * i] = x.x;
    v[4 * i + 1] = x.y;
    v[4 * i + 2] = x.z;
    v[4 * i + 3] = x.w;
  }
}
__device__ __forceinline__ void store8f(float* dst, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<float4*>(dst)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// "Accumulator buffer drained", to the even CTA of the pair.
__device__ __forceinline__ void mm_tempty_signal(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// ---------------------------------------------------------------- epilogue

// 8 output columns from their fp32 sums v (MM_GATE: and the up projection's u)
// and inputs: the fused operation, rounded once per output.
//   MM_LINEAR  x residual (with p.res); o0 = act(v + bias) + x
//   MM_GATE    o0 = act(v) u  (v and u themselves are saved in fp32: rounded
//              to bf16 they would double the error of the gradients)
//   MM_DGATE   xg gate, xu up; o0 = dgate, o1 = dup, o2 = act(gate) up
template <int EPI>
__device__ __forceinline__ void mm_math8(const MmParams& p, float (&v)[8], const float (&u)[8], int nb, int ncols,
                                         const uint32_t (&x)[4], const float (&xg)[8], const float (&xu)[8],
                                         uint32_t (&o0)[4], uint32_t (&o1)[4], uint32_t (&o2)[4]) {
  if constexpr (EPI == MM_LINEAR) {
    if (p.bias) {
      uint32_t b[4];
      load8(p.bias + nb, b, ncols, true);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] += bf16_lo(b[i]);
        v[2 * i + 1] += bf16_hi(b[i]);
      }
    }
    if (p.act == ACT_SILU) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act_f(v[i], ACT_SILU);
    } else if (p.act == ACT_GELU_TANH) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act_f(v[i], ACT_GELU_TANH);
    }
    if (p.res) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] += bf16_lo(x[i]);
        v[2 * i + 1] += bf16_hi(x[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o0[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  } else if constexpr (EPI == MM_GATE) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o0[i] = pack_bf16x2(act_f(v[2 * i], p.act) * u[2 * i], act_f(v[2 * i + 1], p.act) * u[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u0 = xu[2 * i], u1 = xu[2 * i + 1];
      float a0, a1, e0, e1;
      act_grad_f(xg[2 * i], p.act, a0, e0);
      act_grad_f(xg[2 * i + 1], p.act, a1, e1);
      o0[i] = pack_bf16x2(v[2 * i] * u0 * e0, v[2 * i + 1] * u1 * e1);
      o1[i] = pack_bf16x2(v[2 * i] * a0, v[2 * i + 1] * a1);
      o2[i] = pack_bf16x2(a0 * u0, a1 * u1);
    }
  }
}

// The same with the thread's own loads and stores: output columns nb .. nb + 7
// of row m.  (Of the gated forms F % 8 == 0: whole 16-byte groups.)
template <int EPI>
__device__ __forceinline__ void mm_out8(const MmParams& p, int pr, int m, int nb, float (&v)[8],
                                        const float (&u)[8]) {
  const int N = p.N[pr], ncols = N - nb;
  if (ncols <= 0) return;
  const bool vec = p.vec != 0;
  uint32_t x[4] = {}, o0[4], o1[4], o2[4];
  float xg[8] = {}, xu[8] = {};
  float* row = EPI == MM_LINEAR ? nullptr : p.gu + static_cast<size_t>(m) * 2 * N + nb;
  if (EPI == MM_LINEAR && p.res) load8(p.res + static_cast<size_t>(m) * p.ld_res + nb, x, ncols, vec);
  if (EPI == MM_DGATE) {
    load8f(row, xg);
    load8f(row + N, xu);
  }
  if (EPI == MM_GATE && p.gu) {
    store8f(row, v);
    store8f(row + N, u);
  }
  mm_math8<EPI>(p, v, u, nb, ncols, x, xg, xu, o0, o1, o2);
  store8(p.y[pr] + static_cast<size_t>(m) * p.ldy[pr] + nb, o0, ncols, vec);
  if (EPI == MM_DGATE) {
    store8(p.y[1] + static_cast<size_t>(m) * N + nb, o1, ncols, true);
    if (p.y[2]) store8(p.y[2] + static_cast<size_t>(m) * N + nb, o2, ncols, true);
  }
}

// An epilogue warp's chunks of shared memory and the barrier of its loads.
struct MmStage {
  uint8_t* buf;
  uint64_t* bar;
  uint32_t phase;
  int turn;        // chunks done; its parity is the one in use where they take turns
  __device__ uint8_t* at(int i) const { return buf + i * MM_OUT; }
};

// Inputs of the 32 x 32 chunk at (row, col) into shared memory, once the stores
// that read it are done.  Gate and up are fp32, which the map counts as pairs
// of 16-bit values.
template <int EPI>
__device__ __forceinline__ void mm_fetch(const MmMaps& maps, MmStage& s, int row, int col, int lane) {
  if (lane == 0) bulk_wait_group_read<EPI == MM_DGATE ? 0 : 1>();
  __syncwarp();
  const uint32_t bar = smem_u32(s.bar);
  mbar_expect_elect(s.bar, EPI == MM_DGATE ? 4 * MM_OUT : MM_OUT);
  if (EPI == MM_DGATE) {
    tma_load_3d_elect(&maps.x, bar, s.at(0), 2 * col, 0, row);
    tma_load_3d_elect(&maps.x, bar, s.at(2), 2 * col, 1, row);
  } else {
    tma_load_3d_elect(&maps.x, bar, s.at(s.turn & 1), col, 0, row);
  }
}

// One accumulator tile of the persistent kernel: rows m0 .. m0 + 127 of this
// CTA, output columns from n0.  Signals the accumulator buffer free after this
// warp's last TMEM read if a later tile takes it (reused): an arrival that
// nobody waits for could reach the even CTA after its exit.  A thread holds one row, so its own accesses would be
// 16 bytes in each of 32 rows, 32 passes of the load/store unit each; instead a
// warp's 32 x 32 chunk goes through shared memory and TMA brings the inputs and
// takes the outputs (TMA keeps to the rows that exist, and to the columns in
// whole groups of 16 bytes).  TMA needs rows that are 16-byte aligned; others
// (p.vec == 0) are read, and they and a chunk that N cuts inside such a group
// are written, by the warp, one value per lane and 32 of a row at a time.
// Swizzles: 16-byte group q of row r of a bf16 chunk lies at q ^ (r / 2 mod 4),
// of an fp32 chunk at q ^ (r mod 8).
template <int EPI>
__device__ __forceinline__ bool mm_epilogue(const MmMaps& maps, const MmParams& p, int pr, uint64_t* tfull,
                                            uint32_t tfull_phase, uint32_t tacc, int m0, int n0, int quarter,
                                            int half, int lane, bool reused, uint32_t tempty_addr, MmStage& s, int W) {
  const int CH = W / 32;   // (W: output columns of a tile)
  const int row0 = m0 + quarter * 32, N = p.N[pr];
  const bool vec = EPI != MM_LINEAR || p.vec;
  const bool rows_in = row0 < p.M[pr];
  const bool has_in = EPI == MM_DGATE || (EPI == MM_LINEAR && p.res && vec);
  const uint32_t t_row = tacc + (static_cast<uint32_t>(quarter * 32) << 16);
  bool fetched = has_in && rows_in && n0 + half * 32 < N;
  if (fetched) mm_fetch<EPI>(maps, s, row0, n0 + half * 32, lane);
  if (!mbar_wait_warp(tfull, tfull_phase, p.status)) {
    if (fetched) {   // the load lands before the CTA exits (bounded)
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(s.bar, s.phase) && globaltimer_ns() - t0 < QI_WAIT_NS) {
      }
    }
    return false;
  }
  tc_fence_after();
#pragma unroll 1
  for (int c = half; c < CH; c += 2) {
    __syncwarp();
    uint32_t r[32];
    tmem_ld32(t_row + c * 32, r);
    uint32_t r2[EPI == MM_GATE ? 32 : 8];
    if constexpr (EPI == MM_GATE) tmem_ld32(t_row + W + c * 32, r2);
    if (c + 2 >= CH) {
      tc_fence_before();
      __syncwarp();
      if (reused && lane == 0) mm_tempty_signal(tempty_addr);
    }
    const int col0 = n0 + c * 32;
    if (!rows_in || col0 >= N) continue;
    float v[8], u[8];
    auto sums = [&](int q) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = __uint_as_float(r[8 * q + i]);
        u[i] = EPI == MM_GATE ? __uint_as_float(r2[8 * q + i]) : 0.f;
      }
    };
    if (has_in) {
      if (!mbar_wait_warp(s.bar, s.phase, p.status)) return false;
      s.phase ^= 1u;
    } else {   // earlier stores have read what is written next
      if (lane == 0) {
        if (EPI == MM_GATE && p.gu) bulk_wait_group_read<0>();
        else bulk_wait_group_read<1>();
      }
      __syncwarp();
    }
    auto group = [&](uint8_t* chunk, int q) {
      return reinterpret_cast<uint4*>(chunk + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4));
    };
    auto put = [&](uint8_t* chunk, int q, const uint32_t (&o)[4]) {
      *group(chunk, q) = make_uint4(o[0], o[1], o[2], o[3]);
    };
    auto group_f = [&](uint8_t* chunk, int q) {
      return reinterpret_cast<uint4*>(chunk + lane * 128 + ((q ^ (lane & 7)) << 4));
    };
    auto send = [&](const CUtensorMap* map, const uint8_t* chunk, int col, int which) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(map, chunk, col, which, row0);
        bulk_commit_group();
      }
    };
    uint32_t x[4] = {}, o0[4], o1[4], o2[4];
    float xg[8] = {}, xu[8] = {};
    if constexpr (EPI == MM_LINEAR) {
      uint8_t* at = s.at(s.turn & 1);
      const int rows = min(32, p.M[pr] - row0);
      const bool col_in = col0 + lane < N;
      auto value = [&](int i) {   // of row i, this lane's column
        return reinterpret_cast<uint16_t*>(at + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4)) + (lane & 7);
      };
      if (!vec && p.res) {
        const uint16_t* src = p.res + static_cast<size_t>(row0) * p.ld_res + col0 + lane;
        uint16_t x16[32];   // (all asked for before the first is used)
#pragma unroll
        for (int i = 0; i < 32; ++i)
          x16[i] = col_in && i < rows ? src[static_cast<size_t>(i) * p.ld_res] : static_cast<uint16_t>(0);
#pragma unroll
        for (int i = 0; i < 32; ++i) *value(i) = x16[i];
        __syncwarp();
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (p.res) {
          const uint4 w = *group(at, q);
          x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
        }
        sums(q);
        mm_math8<EPI>(p, v, u, col0 + q * 8, N - col0 - q * 8, x, xg, xu, o0, o1, o2);
        put(at, q, o0);
      }
      if (vec && (N % 8 == 0 || col0 + 32 <= N)) {
        send(&maps.y[pr], at, col0, 0);
      } else {
        if (lane == 0) bulk_commit_group();   // (one group per chunk, if an empty one, for the waits that count them)
        __syncwarp();
        uint16_t* dst = p.y[pr] + static_cast<size_t>(row0) * p.ldy[pr] + col0 + lane;
        if (col_in)
#pragma unroll 8
          for (int i = 0; i < rows; ++i) dst[static_cast<size_t>(i) * p.ldy[pr]] = *value(i);
        fence_proxy_async_smem();   // read before TMA writes the chunk again
        __syncwarp();
      }
      ++s.turn;
    } else if constexpr (EPI == MM_GATE) {
      uint8_t* at = s.at(p.gu ? 0 : s.turn & 1);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        sums(q);
        mm_math8<EPI>(p, v, u, col0 + q * 8, N - col0 - q * 8, x, xg, xu, o0, o1, o2);
        put(at, q, o0);
      }
      send(&maps.y[0], at, col0, 0);
      ++s.turn;
      if (p.gu) {
        auto save = [&](const uint32_t (&t)[32], int which) {
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q) *group_f(s.at(0), q) = make_uint4(t[4 * q], t[4 * q + 1], t[4 * q + 2], t[4 * q + 3]);
          send(&maps.x, s.at(0), 2 * col0, which);
        };
        save(r, 0);
        save(r2, 1);
      }
    } else {
      uint4 g[8], h[8];   // (all read before any is overwritten: rows of the outputs are shorter)
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        g[q] = *group_f(s.at(0), q);
        h[q] = *group_f(s.at(2), q);
      }
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint4 a = g[2 * q + e], b = h[2 * q + e];
          xg[4 * e] = __uint_as_float(a.x); xg[4 * e + 1] = __uint_as_float(a.y);
          xg[4 * e + 2] = __uint_as_float(a.z); xg[4 * e + 3] = __uint_as_float(a.w);
          xu[4 * e] = __uint_as_float(b.x); xu[4 * e + 1] = __uint_as_float(b.y);
          xu[4 * e + 2] = __uint_as_float(b.z); xu[4 * e + 3] = __uint_as_float(b.w);
        }
        sums(q);
        mm_math8<EPI>(p, v, u, col0 + q * 8, N - col0 - q * 8, x, xg, xu, o0, o1, o2);
        put(s.at(0), q, o0);
        put(s.at(1), q, o1);
        put(s.at(2), q, o2);
      }
      send(&maps.y[0], s.at(0), col0, 0);
      send(&maps.y[1], s.at(1), col0, 0);
      if (p.y[2]) send(&maps.y[2], s.at(2), col0, 0);
    }
    if (has_in && c + 2 < CH && col0 + 64 < N) mm_fetch<EPI>(maps, s, row0, col0 + 64, lane);
  }
  return true;
}

// Product and tile coordinates of a tile number, for tiles of BM rows and W columns.
template <int BM>
__device__ __forceinline__ void mm_tile(const MmParams& p, int tile, int W, int& pr, int& mt, int& nt) {
  pr = 0;
  while (pr < p.n_prob - 1 && tile >= p.tiles_end[pr]) ++pr;
  if (pr > 0) tile -= p.tiles_end[pr - 1];
  tile_coords(tile, (p.M[pr] + BM - 1) / BM, p.group_m[pr], (p.N[pr] + W - 1) / W, mt, nt);
}

// The loads of one K block of a CTA: its 128 rows of A from row m0, and its 128
// rows of B: from row n0, or with MM_GATE 64 or 128 rows of gate and / or up
// (see the kernels).  `bar` counts the bytes.
template <bool PAIR, bool MN>
__device__ __forceinline__ void mm_load(const CUtensorMap* map, uint32_t bar, uint8_t* dst, int k, int row) {
  if (MN) {
#pragma unroll
    for (int i = 0; i < 2; ++i) tma_load_2d_elect<PAIR>(map, bar, dst + i * 8192, row + 64 * i, k);
  } else {
    tma_load_2d_elect<PAIR>(map, bar, dst, k, row);
  }
}

// The four MMAs of a K block: 16 values of K per instruction, 32 bytes of a
// K-major row or 16 MN-major rows.
template <bool PAIR, bool AMN, bool BMN>
__device__ __forceinline__ void mm_block(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool first) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    umma_f16_elect<PAIR>(d_tmem, a + (static_cast<uint64_t>(k * (AMN ? 2048 : 32)) >> 4),
                         b + (static_cast<uint64_t>(k * (BMN ? 2048 : 32)) >> 4), idesc, !first || k > 0);
}

template <bool MN>
__device__ __forceinline__ uint64_t mm_desc(const uint8_t* tile) {
  return MN ? umma_desc_mnmajor_sw128(smem_u32(tile), 8192) : umma_desc_kmajor_sw128(smem_u32(tile));
}

template <bool AMN, bool BMN>
__device__ __forceinline__ uint32_t mm_idesc(int n) {   // of a pair: 256 x n
  return umma_idesc(false, 256, n) | (AMN ? (1u << 15) : 0u) | (BMN ? (1u << 16) : 0u);
}

// ---------------------------------------------------------------- large products
//
// A pair of CTAs (one per SM) shares a 256 x 256 tile (cta_group::2): each
// loads 128 rows of A and 128 rows of B, and the even CTA issues the MMAs for
// both.  Where they fill the last round better, tiles are 192 or 128 columns
// wide.  Persistent over tiles; the accumulator is double-buffered in TMEM, so
// the epilogue of a tile overlaps the MMAs of the next.
template <bool AMN, bool BMN, int EPI>
__global__ void __launch_bounds__(MM_THREADS, 1)
    mm_kernel(const __grid_constant__ MmMaps maps, const __grid_constant__ MmParams p) {
  constexpr int STAGES = MmCfg<EPI>::STAGES;
  const int bn = BMN ? MM_BN : p.bn;   // columns of the accumulator
  const int W = EPI == MM_GATE ? bn / 2 : bn;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * MM_TILE;
  uint8_t* sOut = smem + STAGES * 2 * MM_TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sOut + MM_EPI_WARPS * MmCfg<EPI>::CHUNKS * MM_OUT);
  uint64_t* full = bars;                     // [STAGES] (the even CTA's)
  uint64_t* empty = bars + STAGES;           // [STAGES]
  uint64_t* tfull = bars + 2 * STAGES;       // [2]
  uint64_t* tempty = bars + 2 * STAGES + 2;  // [2] (the even CTA's)
  uint64_t* drain = bars + 2 * STAGES + 4;   // MMA drain on the error path
  uint64_t* xfull = bars + 2 * STAGES + 5;   // [MM_EPI_WARPS] inputs of the epilogue
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(xfull + MM_EPI_WARPS);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int worker = blockIdx.x >> 1, workers = gridDim.x >> 1;
  const int num_tiles = p.tiles_end[p.n_prob - 1];

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * MM_EPI_WARPS);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < MM_EPI_WARPS; ++i) mbar_init(&xfull[i], 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&maps.a[0]);
    prefetch_tmap(&maps.b[EPI == MM_GATE ? rank : 0]);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 2 * MM_BN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  bool ok = true;
  if (warp == 0) {
    // ------------------------------------------------------------ producer (the whole warp, one lane issues)
    int stage = 0;
    uint32_t phase = 0;
    for (int tile = worker; tile < num_tiles && ok; tile += workers) {
      int pr, mt, nt;
      mm_tile<256>(p, tile, W, pr, mt, nt);
      const int m0 = mt * 256 + rank * 128;
      const int n0 = EPI == MM_GATE ? nt * W : nt * bn + rank * (bn / 2);
      const int num_kb = p.num_kb[pr];
      for (int seg = 0; seg < p.segs && ok; ++seg) {   // segs == 2 only for a single product
        const CUtensorMap* ma = &maps.a[pr + seg];
        const CUtensorMap* mb = &maps.b[EPI == MM_GATE ? rank : pr + seg];
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait_warp(&empty[stage], phase ^ 1u, p.status)) { ok = false; break; }
          const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
          if (rank == 0) mbar_expect_elect(&full[stage], static_cast<uint32_t>(2 * MM_TILE + bn * 128));
          mm_load<true, AMN>(ma, fb, sA + stage * MM_TILE, kb * 64, m0);
          mm_load<true, BMN>(mb, fb, sB + stage * MM_TILE, kb * 64, n0);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
    }
    if (ok) ok = mm_stages_free(empty, STAGES, stage, phase, p.status);
    if (!ok) {
      // Error path: the loads in flight must land before the CTA exits.  The
      // even CTA, which armed the full barriers, waits (bounded) on them; the
      // odd one, which cannot, gives its last loads a fixed 200 us.
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
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    // The whole warp runs the loop and one elected lane issues: operands that
    // are uniform over a converged warp reach the tensor core's instruction
    // without a move per lane (an MMA issued under a lane test took 54 clocks).
    if (rank == 0) {
      const uint32_t idesc = mm_idesc<AMN, BMN>(bn);
      const uint64_t adesc = mm_desc<AMN>(sA), bdesc = mm_desc<BMN>(sB);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      for (int tile = worker; tile < num_tiles && ok; tile += workers) {
        int pr, mt, nt;
        mm_tile<256>(p, tile, W, pr, mt, nt);
        const int total_kb = p.num_kb[pr] * p.segs;
        if (!__all_sync(0xffffffffu, mbar_wait_cluster(&tempty[acc], acc_phase ^ 1u, p.status))) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * MM_BN);
        for (int kb = 0; kb < total_kb; ++kb) {
          if (!mbar_wait_warp(&full[stage], phase, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint64_t off = static_cast<uint64_t>(stage * (MM_TILE >> 4));
          mm_block<true, AMN, BMN>(d_tmem, adesc + off, bdesc + off, idesc, kb == 0);
          umma_commit_elect<true>(&empty[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        umma_commit_elect<true>(&tfull[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok) {
        // make sure no MMA is still writing TMEM before it is released
        umma_commit_elect<true>(drain, 0x1);
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
    MmStage stage{sOut + (warp - 2) * MmCfg<EPI>::CHUNKS * MM_OUT, &xfull[warp - 2], 0, 0};
    for (int tile = worker; tile < num_tiles; tile += workers) {
      int pr, mt, nt;
      mm_tile<256>(p, tile, W, pr, mt, nt);
      if (!mm_epilogue<EPI>(maps, p, pr, &tfull[acc], acc_phase, tmem_base + static_cast<uint32_t>(acc * MM_BN),
                            mt * 256 + rank * 128, nt * W, quarter, half, lane, tile + 2 * workers < num_tiles,
                            mapa_shared(smem_u32(&tempty[acc]), 0), stage, W)) {
        ok = false;
        break;
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (lane == 0) bulk_wait_group_read<0>();   // the chunks are read before the CTA leaves
  }

  // Neither CTA of a pair leaves (or frees TMEM) while the other may still read
  // its shared memory, arrive on its barriers, or have MMAs writing its TMEM:
  // the MMA warp has waited for every arrival on tempty, the producers for the
  // last stages.  Behind a wait that ran out arrivals may be left, and the
  // barrier releases them.
  tc_fence_before();
  if (ok) cluster_sync_end();
  else cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * MM_BN);
  }
}

// ---------------------------------------------------------------- middle sizes
//
// Too few 256 x 256 tiles to fill the GPU: K is shared as well.  A cluster of S
// pairs of CTAs computes one tile, each pair over a part of K.  When its MMAs
// are done, a CTA puts its fp32 sums into its shared memory; after a cluster
// barrier every CTA adds up a share of the columns over the S parts' shared
// memory, in the order of K, and runs the epilogue on them.  Nothing goes
// through memory and the result does not depend on timing.
// The sums lie as [groups of 4 columns][128 rows] of float4: the lanes of a
// warp hold consecutive rows and touch 512 contiguous bytes.
// (Sending each share as a bulk copy into its owner's shared memory instead of
// reading it there took 0.7 us longer.)
constexpr int MS_SMEM = 1024 + MM_STAGES * 2 * MM_TILE + 256;
static_assert(128 * MM_BN * 4 <= MM_STAGES * 2 * MM_TILE, "the sums over the stages");

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

template <bool AMN, bool BMN, int EPI>
__global__ void __launch_bounds__(MM_THREADS, 1)
    mm_split_kernel(const __grid_constant__ MmMaps maps, const __grid_constant__ MmParams p, const int S) {
  constexpr int STAGES = MM_STAGES;
  constexpr int W = EPI == MM_GATE ? MM_BN / 2 : MM_BN;   // output columns of a tile
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * MM_TILE;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * 2 * MM_TILE);   // [STAGES] (the even CTA's)
  uint64_t* empty = full + STAGES;                                             // [STAGES]
  uint64_t* tfull = empty + STAGES;
  uint64_t* drain = tfull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t crank = cluster_rank();
  const uint32_t even = crank & ~1u;                // the CTA that issues this one's MMAs
  const int rank = static_cast<int>(crank & 1u);    // half of the tile's rows
  const int part = static_cast<int>(crank >> 1);
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, MM_BN);
    tmem_relinquish_pair();
  }
  int pr, mt, nt;
  mm_tile<256>(p, static_cast<int>(blockIdx.x) / (2 * S), W, pr, mt, nt);
  const int total_kb = p.num_kb[pr] * p.segs;
  const int lo = total_kb * part / S, hi = total_kb * (part + 1) / S;
  const int m0 = mt * 256 + rank * 128;
  const int n0 = EPI == MM_GATE ? nt * W : nt * W + rank * 128;   // first row of B of this CTA
  tc_fence_before();
  cluster_sync_all();   // barriers of both CTAs initialised before any remote arrive
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  bool ok = true;
  if (warp == 0) {
    // ------------------------------------------------------------ producer (the whole warp, one lane issues)
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = lo; kb < hi; ++kb) {
      if (!mbar_wait_warp(&empty[stage], phase ^ 1u, p.status)) { ok = false; break; }
      const int seg = kb >= p.num_kb[pr] ? 1 : 0;   // segs == 2 only for a single product
      const int k = (kb - seg * p.num_kb[pr]) * 64;
      const uint32_t fb = mapa_shared(smem_u32(&full[stage]), even);
      if (rank == 0) mbar_expect_elect(&full[stage], 4 * MM_TILE);
      mm_load<true, AMN>(&maps.a[pr + seg], fb, sA + stage * MM_TILE, k, m0);
      mm_load<true, BMN>(&maps.b[EPI == MM_GATE ? rank : pr + seg], fb, sB + stage * MM_TILE, k, n0);
      if (++stage == STAGES) { stage = 0; phase ^= 1u; }
    }
    if (ok) ok = mm_stages_free(empty, STAGES, stage, phase, p.status);
    if (!ok) {   // the loads in flight must land before the CTA exits (see mm_kernel)
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
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (rank == 0) {
      const uint32_t idesc = mm_idesc<AMN, BMN>(MM_BN);
      const uint64_t adesc = mm_desc<AMN>(sA), bdesc = mm_desc<BMN>(sB);
      const uint16_t both = static_cast<uint16_t>(0x3u << even);
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = lo; kb < hi; ++kb) {
        if (!mbar_wait_warp(&full[stage], phase, p.status)) { ok = false; break; }
        tc_fence_after();
        const uint64_t off = static_cast<uint64_t>(stage * (MM_TILE >> 4));
        mm_block<true, AMN, BMN>(tmem_base, adesc + off, bdesc + off, idesc, kb == lo);
        umma_commit_elect<true>(&empty[stage], both);
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
      if (ok) {
        umma_commit_elect<true>(tfull, both);
      } else {
        umma_commit_elect<true>(drain, static_cast<uint16_t>(0x1u << even));
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < QI_WAIT_NS) {
        }
      }
    }
  } else {
    // ------------------------------------------------------------ this CTA's sums into its shared memory
    // (every MMA of the pair, and so every load, is done with the stages)
    const int quarter = warp & 3, half = (warp - 2) >> 2, row = quarter * 32 + lane;
    float4* sums = reinterpret_cast<float4*>(smem);
    ok = mbar_wait_warp(tfull, 0, p.status);
    tc_fence_after();
    const bool none = lo == hi;   // no K block for this part: TMEM was not written
    if (ok)
#pragma unroll 1
      for (int c = half * (MM_BN / 64); c < (half + 1) * (MM_BN / 64); ++c) {
        uint32_t r[32];
        tmem_ld32(tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + c * 32, r);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          sums[(c * 8 + q) * 128 + row] =
              none ? make_float4(0.f, 0.f, 0.f, 0.f)
                   : make_float4(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]),
                                 __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]));
      }
  }
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, MM_BN);
  }
  if (warp >= 2 && ok) {
    // columns [part W / S, + W / S) of this CTA's rows, 8 of a row at a time; a
    // warp takes 8 rows x 32 columns, so its accesses are whole sectors
    const int ng = W / S / 8;
#pragma unroll 1
    for (int item = threadIdx.x - 64; item < 128 * ng; item += 256) {
      const int c = part * (W / S) + ((item >> 3) & (ng - 1)) * 8;
      const int row = ((item >> 3) / ng) * 8 + (item & 7);
      if (m0 + row >= p.M[pr] || nt * W + c >= p.N[pr]) continue;   // (no load whose value nobody takes)
      const uint32_t mine = smem_u32(smem) + static_cast<uint32_t>(row) * 16;
      float v[8], u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = u[i] = 0.f;
#pragma unroll 2
      for (int s = 0; s < S; ++s) {
        const uint32_t from = mapa_shared(mine, static_cast<uint32_t>(2 * s + rank)) + (c >> 2) * 2048;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 x = ld_cluster4(from + e * 2048);
          v[4 * e] += x.x;
          v[4 * e + 1] += x.y;
          v[4 * e + 2] += x.z;
          v[4 * e + 3] += x.w;
          if (EPI == MM_GATE) {
            const float4 y = ld_cluster4(from + (W / 4 + e) * 2048);   // the up columns, W further on
            u[4 * e] += y.x;
            u[4 * e + 1] += y.y;
            u[4 * e + 2] += y.z;
            u[4 * e + 3] += y.w;
          }
        }
      }
      mm_out8<EPI>(p, pr, m0 + row, nt * W + c, v, u);
    }
  }
  cluster_sync_end();   // no CTA leaves while another may read its sums
}

// ---------------------------------------------------------------- some hundreds of rows
//
// The weights take the 128-row side of the MMA and T rows of a (M, or an equal
// part of it, rounded up to 16) the other one: no tile is half empty, and of
// the shared memory that a K block takes 16 KB are weights on their way, whose
// reading bounds the product.  D[n, m] = sum_k w(n, k) a(m, k): a lane of TMEM is an
// output column, a TMEM column a row of y.  K is shared by a cluster of S CTAs
// as above; a CTA finishes the rows part, part + S, ...
constexpr int MR_MAX_T = 256;
constexpr int MR_MAX_TILES = 2;   // along M: three and more were never faster than 256 x 256 tiles
constexpr int MR_MAX_STAGES = 8;

__host__ __device__ constexpr int mr_stage(int T) { return MM_TILE + T * 128; }
__host__ __device__ constexpr int mr_area(int T, int stages) {
  return stages * mr_stage(T) > 512 * T ? stages * mr_stage(T) : 512 * T;   // the sums lie over the stages
}
static int mr_smem(int T, int stages) { return 1024 + mr_area(T, stages) + 256; }

template <bool WMN, int EPI>
__global__ void __launch_bounds__(MM_THREADS, 2)
    mm_rows_kernel(const __grid_constant__ MmMaps maps, const __grid_constant__ MmParams p, const int S, const int T,
                   const int stages) {
  constexpr int W = EPI == MM_GATE ? 64 : 128;   // output columns of a tile
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + mr_area(T, stages));   // [MR_MAX_STAGES]
  uint64_t* empty = full + MR_MAX_STAGES;                                    // [MR_MAX_STAGES]
  uint64_t* tfull = empty + MR_MAX_STAGES;
  uint64_t* drain = tfull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = S > 1 ? static_cast<int>(cluster_rank()) : 0;
  const uint32_t cols = T <= 64 ? 64 : (T <= 128 ? 128 : 256);
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, cols);
    tmem_relinquish();
  }
  const int tile = static_cast<int>(blockIdx.x) / S, m_tiles = (p.M[0] + T - 1) / T;
  const int n0 = tile / m_tiles * W, m0 = tile % m_tiles * T;
  const int rows = min(T, p.M[0] - m0);
  const int total_kb = p.num_kb[0] * p.segs;
  const int lo = total_kb * part / S, hi = total_kb * (part + 1) / S;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  bool ok = true;
  if (warp == 0) {
    // ------------------------------------------------------------ producer (the whole warp, one lane issues)
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = lo; kb < hi; ++kb) {
      if (!mbar_wait_warp(&empty[stage], phase ^ 1u, p.status)) { ok = false; break; }
      const int seg = kb >= p.num_kb[0] ? 1 : 0;
      const int k = (kb - seg * p.num_kb[0]) * 64;
      const uint32_t fb = smem_u32(&full[stage]);
      uint8_t* dst = smem + stage * mr_stage(T);
      mbar_expect_elect(&full[stage], static_cast<uint32_t>(mr_stage(T)));
      if (EPI == MM_GATE) {
        mm_load<false, false>(&maps.a[0], fb, dst, k, n0);
        mm_load<false, false>(&maps.a[1], fb, dst + MM_TILE / 2, k, n0);
      } else {
        mm_load<false, WMN>(&maps.a[seg], fb, dst, k, n0);
      }
      mm_load<false, false>(&maps.b[seg], fb, dst + MM_TILE, k, m0);
      if (++stage == stages) { stage = 0; phase ^= 1u; }
    }
    if (ok) ok = mm_stages_free(empty, stages, stage, phase, p.status);
    if (!ok) {   // the loads in flight must land before the CTA exits
      for (int s = 0; s < stages; ++s) {
        const uint32_t par = (s < stage) ? phase : (phase ^ 1u);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&full[s], par) && globaltimer_ns() - t0 < QI_WAIT_NS) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc = umma_idesc(false, 128, T) | (WMN ? (1u << 15) : 0u);
    const uint64_t adesc = mm_desc<WMN>(smem), bdesc = mm_desc<false>(smem + MM_TILE);
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = lo; kb < hi; ++kb) {
      if (!mbar_wait_warp(&full[stage], phase, p.status)) { ok = false; break; }
      tc_fence_after();
      const uint64_t off = static_cast<uint64_t>(stage * (mr_stage(T) >> 4));
      mm_block<false, WMN, false>(tmem_base, adesc + off, bdesc + off, idesc, kb == lo);
      umma_commit_elect<false>(&empty[stage]);
      if (++stage == stages) { stage = 0; phase ^= 1u; }
    }
    if (ok) {
      umma_commit_elect<false>(tfull);
    } else {
      umma_commit_elect<false>(drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < QI_WAIT_NS) {
      }
    }
  } else {
    // ------------------------------------------------------------ this CTA's sums into its shared memory: [T][128]
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    float* sums = reinterpret_cast<float*>(smem) + quarter * 32 + lane;
    ok = mbar_wait_warp(tfull, 0, p.status);
    tc_fence_after();
    const bool none = lo == hi;   // no K block for this part: TMEM was not written
    if (ok)
#pragma unroll 1
      for (int c = half * 32; c < T; c += 64) {
        uint32_t r[32];
        tmem_ld32(tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + c, r);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < 16 || c + 16 < T) sums[(c + i) * 128] = none ? 0.f : __uint_as_float(r[i]);
      }
  }
  tc_fence_before();
  if (S > 1) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, cols);
  }
  if (warp >= 2 && ok) {
    // 8 columns of a row at a time, whole rows of the tile per warp
    constexpr int NG = W / 8;
    const uint32_t mine = smem_u32(smem);
#pragma unroll 1
    for (int item = threadIdx.x - 64;; item += 256) {
      const int m = part + S * (item / NG), g = item % NG;
      if (m >= rows) break;
      if (n0 + g * 8 >= p.N[0]) continue;   // (no load whose value nobody takes)
      float v[8], u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = u[i] = 0.f;
#pragma unroll 2
      for (int s = 0; s < S; ++s) {
        const uint32_t from = (S > 1 ? mapa_shared(mine, static_cast<uint32_t>(s)) : mine) +
                              static_cast<uint32_t>(m) * 512 + g * 32;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 x = ld_cluster4(from + e * 16);
          v[4 * e] += x.x;
          v[4 * e + 1] += x.y;
          v[4 * e + 2] += x.z;
          v[4 * e + 3] += x.w;
          if (EPI == MM_GATE) {
            const float4 y = ld_cluster4(from + 256 + e * 16);   // the up columns, 64 further on
            u[4 * e] += y.x;
            u[4 * e + 1] += y.y;
            u[4 * e + 2] += y.z;
            u[4 * e + 3] += y.w;
          }
        }
      }
      mm_out8<EPI>(p, 0, m0 + m, n0 + g * 8, v, u);
    }
  }
  if (S > 1) cluster_sync_end();   // no CTA leaves while another may read its sums
}

// ---------------------------------------------------------------- few rows
//
// A few rows (use_skinny): the product is bound by reading the weights once, so the
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
  float* gu;              // GATE: optional [M, 2N]
};

// 16 bytes of a weight row: read once, not kept in L1.
__device__ __forceinline__ uint4 ld_stream16(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int NT, bool GATE>
__global__ void __launch_bounds__(SK_THREADS, 2) skinny_kernel(const SkinnyParams p) {
  constexpr int MATS = GATE ? 2 : 1;
  constexpr int STEP = SK_THREADS / 32 * 64;
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
  // two batches of loads in turn: one is on its way while the other is multiplied
  struct Batch {
    uint4 w[2][MATS][2], x[2][NT];   // of a 64-wide piece of K
  };
  auto load = [&](Batch& q, int kb) {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const int k = kb + 32 * sub + 8 * t;   // K % 8 == 0: a chunk of 8 lies inside or outside
      const bool in = k < p.K;
#pragma unroll
      for (int i = 0; i < MATS; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) q.w[sub][i][e] = in ? ld_stream16(wr[i][e] + k) : zero;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        q.x[sub][j] = in && 8 * j + g < p.M ? *reinterpret_cast<const uint4*>(ar[j] + k) : zero;
    }
  };
  auto multiply = [&](const Batch& q) {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub)
#pragma unroll
      for (int i = 0; i < MATS; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint4 w0 = q.w[sub][i][0], w1 = q.w[sub][i][1], x = q.x[sub][j];
          mma_16816(acc[i][j], w0.x, w1.x, w0.y, w1.y, x.x, x.y);
          mma_16816(acc[i][j], w0.z, w1.z, w0.w, w1.w, x.z, x.w);
        }
  };
  pdl_wait();
  pdl_trigger();
  {
    Batch q0, q1;
    int kb = warp * 64;
    load(q0, kb);
#pragma unroll 1
    for (; kb < p.K; kb += 2 * STEP) {
      load(q1, kb + STEP);
      multiply(q0);
      load(q0, kb + 2 * STEP);
      multiply(q1);
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
        float* row = p.gu + static_cast<size_t>(m) * 2 * p.N + n;
        row[0] = v;
        row[p.N] = v2;
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

// An attribute of a kernel, set once per device.
template <class K>
static bool set_once(K kern, cudaFuncAttribute attr, int value, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(kern, attr, value) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_release);
  return true;
}
template <class K>
static bool allow_smem(K kern, int bytes, std::atomic<uint64_t>& done) {
  return set_once(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes, done);
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

static MmParams mm_params(int* status) {
  MmParams p;
  memset(&p, 0, sizeof(p));
  p.n_prob = 1;
  p.segs = 1;
  p.vec = 1;
  p.status = status;
  return p;
}

static long mm_count_tiles(MmParams& p, int bm, int w) {
  long tiles = 0;
  for (int i = 0; i < p.n_prob; ++i) {
    const int mt = (p.M[i] + bm - 1) / bm;
    tiles += static_cast<long>(mt) * ((p.N[i] + w - 1) / w);
    p.tiles_end[i] = static_cast<int>(tiles);
    p.group_m[i] = mt < 8 ? mt : 8;
  }
  return tiles;
}

// Clusters of `ctas` CTAs, one CTA per SM, that run at the same time on the
// current device (the SMs of one GPC hold a whole number of clusters: 74, 33 and
// 15 clusters of 2, 4 and 8 on 148 SMs).  Asked once per device, and for every
// kernel with the same shared memory, so that the answer, and with it the order
// of a product's sums, does not depend on which call came first.
template <class K>
static int cluster_places(K kern, int ctas, int num_sms) {
  if (ctas <= 1) return num_sms;
  static std::atomic<int> known[64][4];   // 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return num_sms / ctas;
  const int slot = ctas == 2 ? 0 : (ctas == 4 ? 1 : 2);
  const bool keep = dev < 64;
  int n = keep ? known[dev][slot].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(MM_THREADS, 1, 1);
    cfg.dynamicSmemBytes = MS_SMEM;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = num_sms / ctas;
    }
    if (keep) known[dev][slot].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Kernel of a launch, by estimates in clocks.
// Tiles of 256 rows: rounds of tiles times K blocks times 600 (256 columns: 32
// KB into each SM), 510 (192) or 440 (128), plus what starts and ends a tile (the
// launch, the first loads, the sums' way out): 14000, which the persistent kernel
// pays once, or per round 15000 with shared K, 23000 with the five accesses of
// MM_DGATE, 25000 where y takes single values.  Measured, whole K / parts of K:
// 512 x 4096 x 11008 55 / 38 us; tiles of 256 / 192 / 128 columns: 768 x 4096 x
// 11008 74 / 56 / 89 us, 1000 x 4096 x 11008 70 / 100 / 88.
// mm_rows_kernel: 8000 per round and 9 S T for the exchange, plus the largest of
//   a CTA's K blocks, each its loads' latency (340, or 2000 over the stages) or
//   its bytes at 84 per clock;
//   all CTAs' loads, which L2 gives at 9000 bytes per clock;
//   the weights, which memory gives at 3400.
// Measured, 256 x 256 tiles / this kernel: 64 x 4096 x 4096 16.8 / 11.2 us, 128
// x 22016 x 4096 51 / 39, 333 x 4096 x 4096 19.7 / 15.8; 256 x 6144 x 4096 19.9
// / 20.5, 512 x 6144 x 4096 27.8 / 30.
struct MmShape {
  int bn;       // columns of the persistent kernel's tiles
  bool rows;    // mm_rows_kernel
  int S;        // parts of K (1 and not rows: the persistent kernel)
  int T, stages;
};
template <bool AMN, bool BMN, int EPI>
static bool mm_shape(MmParams p, int num_sms, MmShape* pick) {
  constexpr int W_DIV = EPI == MM_GATE ? 2 : 1;
  static std::atomic<uint64_t> done_p{0};
  auto pair_kern = mm_split_kernel<AMN, BMN, EPI>;
  if (!allow_smem(pair_kern, MS_SMEM, done_p)) return false;
  long kb = 0;
  for (int i = 0; i < p.n_prob; ++i) kb = kb > p.num_kb[i] * p.segs ? kb : p.num_kb[i] * p.segs;
  auto rounds = [](long n, long places) { return (n + places - 1) / places; };
  long best = 0;
  for (int bn = 256; bn >= (BMN ? 256 : 128); bn -= 64) {
    const long cost = rounds(mm_count_tiles(p, 256, bn / W_DIV), num_sms / 2) * kb * (bn == 256 ? 600 : (bn == 192 ? 510 : 440)) + 14000;
    if (best == 0 || cost < best) {
      best = cost;
      *pick = {bn, false, 1, 0, 0};
    }
  }
  const long tiles = mm_count_tiles(p, 256, 256 / W_DIV);
  for (int s = 2; s <= 4; s *= 2) {
    const long cost = rounds(tiles, cluster_places(pair_kern, 2 * s, num_sms)) *
                          (rounds(kb, s) * 600 + (EPI == MM_DGATE ? 23000 : (p.vec ? 15000 : 25000)));
    if (cost < best) {
      best = cost;
      *pick = {256, false, s, 0, 0};
    }
  }
  if constexpr (!AMN) {
    static std::atomic<uint64_t> done_r{0};
    auto kern = mm_rows_kernel<BMN, EPI>;
    if (!allow_smem(kern, 232448, done_r)) return false;
    const int m_tiles = (p.M[0] + MR_MAX_T - 1) / MR_MAX_T;
    if (m_tiles <= MR_MAX_TILES) {
      const int T = ((p.M[0] + m_tiles - 1) / m_tiles + 15) / 16 * 16;
      const long nw = rounds(p.N[0], 128 / W_DIV), n = nw * rounds(p.M[0], T);
      for (int s = 1; s <= 8; s *= 2) {
        // two CTAs per SM when there are more CTAs than SMs and TMEM and shared memory allow it
        const int per_sm = T <= 128 && n * s > num_sms ? 2 : 1;
        const int stages = std::min(MR_MAX_STAGES, ((per_sm == 2 ? 115712 : 232448) - 1280) / mr_stage(T));
        const long r = rounds(n, static_cast<long>(per_sm) * cluster_places(kern, s, num_sms));
        const long block = std::max(mr_stage(T) / 84, std::max(340, 2000 / stages));
        const long cost = r * (8000 + 9 * s * T) + std::max(r * rounds(kb, s) * block,
                                                            std::max(n * kb * mr_stage(T) / 9000, nw * kb * MM_TILE / 3400));
        if (cost < best) {
          best = cost;
          *pick = {0, true, s, T, stages};
        }
      }
    }
  }
  return true;
}

template <bool WMN, int EPI>
static int mm_launch_rows(const MmOperand* A, const MmOperand* B, int n_ops_a, int n_ops_b, MmParams p, MmShape s,
                          cudaStream_t st) {
  MmMaps maps;   // (a: the weights)
  for (int i = 0; i < n_ops_b; ++i)
    if (!mm_map(&maps.a[i], B[i], WMN, EPI == MM_GATE ? 64 : 128)) return -2;
  for (int i = 0; i < n_ops_a; ++i)
    if (!mm_map(&maps.b[i], A[i], false, s.T)) return -2;
  const unsigned tiles = static_cast<unsigned>((p.N[0] + (EPI == MM_GATE ? 63 : 127)) / (EPI == MM_GATE ? 64 : 128) *
                                               ((p.M[0] + s.T - 1) / s.T));
  launch_pdl(mm_rows_kernel<WMN, EPI>, dim3(tiles * s.S), dim3(MM_THREADS), mr_smem(s.T, s.stages), st, s.S, maps, p,
             s.S, s.T, s.stages);
  return launch_result();
}

template <bool AMN, bool BMN, int EPI>
static int mm_launch(const MmOperand* A, const MmOperand* B, int n_ops_a, int n_ops_b, MmParams p,
                     int num_sms, cudaStream_t st) {
  constexpr int W_DIV = EPI == MM_GATE ? 2 : 1;
  MmShape shape;
  if (!mm_shape<AMN, BMN, EPI>(p, num_sms, &shape)) {
    launch_result();
    return -1;
  }
  if constexpr (!AMN)
    if (shape.rows) return mm_launch_rows<BMN, EPI>(A, B, n_ops_a, n_ops_b, p, shape, st);
  MmMaps maps;
  for (int i = 0; i < n_ops_a; ++i)
    if (!mm_map(&maps.a[i], A[i], AMN, 128)) return -2;
  for (int i = 0; i < n_ops_b; ++i)
    if (!mm_map(&maps.b[i], B[i], BMN, shape.bn / 2)) return -2;
  p.bn = shape.bn;
  const long tiles = mm_count_tiles(p, 256, shape.bn / W_DIV);
  if (shape.S > 1) {
    launch_pdl(mm_split_kernel<AMN, BMN, EPI>, dim3(static_cast<unsigned>(tiles) * 2 * shape.S), dim3(MM_THREADS),
               MS_SMEM, st, static_cast<unsigned>(2 * shape.S), maps, p, shape.S);
    return launch_result();
  }
  auto kern = mm_kernel<AMN, BMN, EPI>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kern, MmCfg<EPI>::SMEM, done)) {
    launch_result();
    return -1;
  }
  auto out_map = [](CUtensorMap* m, const void* base, int cols, int rows, int ld) {
    return make_tmap_rows3(m, base, cols, 1, rows, static_cast<uint64_t>(ld) * 2, 32, 1, 32);
  };
  bool ok = true;
  for (int i = 0; i < (EPI == MM_DGATE ? 3 : p.n_prob) && p.vec; ++i) {
    const int pr = EPI == MM_DGATE ? 0 : i;
    if (p.y[i]) ok = ok && out_map(&maps.y[i], p.y[i], p.N[pr], p.M[pr], p.ldy[pr]);
  }
  if (EPI == MM_LINEAR && p.res && p.vec) ok = ok && out_map(&maps.x, p.res, p.N[0], p.M[0], p.ld_res);
  if (EPI != MM_LINEAR && p.gu)
    ok = ok && make_tmap_rows3(&maps.x, p.gu, 2ull * p.N[0], 2, p.M[0], 8ull * p.N[0], 64, 1, 32);
  if (!ok) return -2;
  const int workers = static_cast<int>(tiles < num_sms / 2 ? tiles : num_sms / 2);
  launch_pdl(kern, dim3(2 * workers), dim3(MM_THREADS), MmCfg<EPI>::SMEM, st, 2, maps, p);
  return launch_result();
}

// Whether skinny_kernel runs a product.  It starts and ends 2 us sooner than
// mm_rows_kernel but reads a again in every CTA and pays for rows 9 and up, so:
// up to 8 rows; while all CTAs run at once (two per SM) up to 16, or with short
// K 32.  Measured, this kernel / mm_rows_kernel: 1 x 4096 x 4096 8.4 / 8.8 us,
// 1 x 6144 x 4096 9.7 / 11.2, 16 x 4096 x 4096 9.1 / 9.7, 32 x 1024 x 1024 3.0 /
// 4.8; on the other side 16 x 6144 x 4096 14.6 / 11.6, 32 x 4096 x 4096 12 /
// 10.4.  The gated pair, with two streams per CTA, only while all run at once:
// feed-forward block of 1 x 1024 x 2816 9.0 / 10.2, of 1 x 4096 x 11008 50.5 /
// 47.7, of 8 52.0 / 48.1.  The down projection of a block follows the choice for
// its gate and up: an SM divides its memory anew between L1 and shared memory
// from one of the kernels to the other (52.4 us with one of each).
static bool use_skinny(int M, int N, int K, bool gate, int num_sms) {
  const bool at_once = (N + 15) / 16 <= 2 * num_sms;
  if (M <= 8) return at_once || !gate;
  return at_once && (M <= 16 || (M <= 32 && K <= 1024));
}

template <int NT, bool GATE>
static int launch_skinny_nt(const SkinnyParams& s, cudaStream_t st) {
  // Loads in flight need L1: without this an SM stays divided as the last kernel
  // left it, and a product behind one that uses all of it as shared memory (1 x
  // 4096 x 11008, 17 us) took 40 us.
  static std::atomic<uint64_t> done{0};
  auto kern = skinny_kernel<NT, GATE>;
  if (!set_once(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 30, done)) {
    launch_result();
    return -1;
  }
  launch_pdl(kern, dim3((s.N + 15) / 16), dim3(SK_THREADS), 0, st, 1, s);
  return launch_result();
}
template <bool GATE>
static int launch_skinny(const SkinnyParams& s, cudaStream_t st) {
  if (s.M <= 8) return launch_skinny_nt<1, GATE>(s, st);
  if (s.M <= 16) return launch_skinny_nt<2, GATE>(s, st);
  if (s.M <= 24) return launch_skinny_nt<3, GATE>(s, st);
  return launch_skinny_nt<4, GATE>(s, st);
}

bool gate_up_on_tiles(int M, int H, int F, int num_sms) { return !use_skinny(M, F, H, true, num_sms); }

static bool rows16(const void* p, int ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0;
}

int launch_linear_act(const LinearActParams& q, cudaStream_t st) {
  if (!q.after_tiles && use_skinny(q.M, q.N, q.K, false, q.num_sms)) {
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
  return mm_launch<false, false, MM_LINEAR>(&a, &b, 1, 1, p, q.num_sms, st);
}

int launch_gate_up(const GateUpParams& q, cudaStream_t st) {
  if (!gate_up_on_tiles(q.M, q.H, q.F, q.num_sms)) {
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
  p.ldy[0] = q.F;
  p.act = q.act;
  p.gu = q.gu;
  const MmOperand a{q.x, q.M, q.H, q.ldx};
  const MmOperand b[2] = {{q.gate, q.F, q.H, q.H}, {q.up, q.F, q.H, q.H}};
  return mm_launch<false, false, MM_GATE>(&a, b, 1, 2, p, q.num_sms, st);
}

int launch_gated_dh(const GatedBackwardParams& q, cudaStream_t st) {
  MmParams p = mm_params(q.status);
  p.M[0] = q.M;
  p.N[0] = q.F;
  p.num_kb[0] = (q.H + 63) / 64;
  p.act = q.act;
  p.gu = const_cast<float*>(q.gu);
  p.y[0] = q.dg;
  p.y[1] = q.du;
  p.y[2] = q.ddown ? q.h : nullptr;
  p.ldy[0] = q.F;
  const MmOperand a{q.dy, q.M, q.H, q.ld_dy}, b{q.down, q.H, q.F, q.F};
  return mm_launch<false, true, MM_DGATE>(&a, &b, 1, 1, p, q.num_sms, st);
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
  return mm_launch<false, true, MM_LINEAR>(a, b, 2, 2, p, q.num_sms, st);
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
  return mm_launch<true, true, MM_LINEAR>(a, b, n, n, p, q.num_sms, st);
}

}  // namespace qi
